"""The key/value cache's C ABI without a GPU: refusals on the host before any device work, sizes."""
import ctypes

import pytest

from chunked_gated_deltanet_gb300 import gdn

vp = ctypes.c_void_p


@pytest.fixture(scope="module")
def lib():
    from chunked_gated_deltanet_gb300 import build
    build.build()
    return gdn.load_library()


def _desc(**kw):
    base = dict(n_q_heads=16, n_kv_heads=2, head_dim=128)
    base.update(kw)
    return gdn.make_attn_desc(**base)


def _cache(**kw):   # addresses that are never dereferenced: every call below is refused first
    f = {n: 0x100000 * (i + 1) for i, n in enumerate(("k", "v", "k_scale", "v_scale", "tail", "state", "table",
                                                      "free_pages", "n_free", "refs"))}
    f.update(n_pages=8, n_slots=4, max_blocks=8)
    f.update(kw)
    return gdn.gdn_kv_cache(**f)


def _map(**kw):
    f = dict(rows=0x2000000, units=0x2100000, counts=0x2200000, max_requests=4, max_units=16)
    f.update(kw)
    return gdn.gdn_kv_map(**f)


def test_description(lib):
    ok = gdn.GDN_OK
    for kw in (dict(), dict(n_q_heads=1, n_kv_heads=1, head_dim=64), dict(head_dim=256, in_dtype=gdn.GDN_FP32)):
        assert gdn.gdn_attn_desc_check(_desc(**kw)) == ok
    for kw in (dict(n_q_heads=15), dict(n_kv_heads=0), dict(n_q_heads=0), dict(head_dim=96), dict(head_dim=512),
               dict(in_dtype=2), dict(n_q_heads=1 << 17)):
        assert gdn.gdn_attn_desc_check(_desc(**kw)) == gdn.GDN_ERR_SHAPE, kw
    for s in (0.0, -1.0, float("nan"), float("inf")):
        assert gdn.gdn_attn_desc_check(_desc(scale=s)) == gdn.GDN_ERR_INVALID_ARG
    assert lib.gdn_attn_desc_check(None) == gdn.GDN_ERR_INVALID_ARG


def test_sizes(lib):
    assert gdn.gdn_kv_max_units(1, 1) == 1
    assert gdn.gdn_kv_max_units(256, 256) == 256
    assert gdn.gdn_kv_max_units(130, 1) == 4            # 130 tokens from offset 63 touch 4 blocks
    assert gdn.gdn_kv_max_units(-1, 1) == 0 and gdn.gdn_kv_max_units(1, 0) == 0
    d = _desc()
    small = gdn.gdn_kv_attention_workspace(d, 64, 1, 1024)
    assert 0 < gdn.gdn_kv_attention_workspace_min(d, 1024) <= small
    assert gdn.gdn_kv_attention_workspace(d, 4096, 1, 40000) > small
    assert gdn.gdn_kv_attention_workspace(d, 1 << 20, 64, 1 << 20) < 9 << 30      # bounded: then several launches
    assert gdn.gdn_kv_attention_workspace(d, -1, 1, 1024) == 0
    assert gdn.gdn_kv_attention_workspace(_desc(head_dim=96), 1, 1, 1024) == 0


def test_refusals(lib):
    E = gdn.GDN_ERR_INVALID_ARG
    d, c, m = _desc(), _cache(), _map()
    p = vp(0x3000000)
    R = ctypes.byref

    def plan(desc=d, cache=c, slots=p, n_new=p, n=2, mp=m, so=None, nf=None):
        return lib.gdn_kv_plan(R(desc), R(cache) if cache else None, slots, n_new, n, R(mp) if mp else None, so, nf, None)

    assert plan(desc=_desc(head_dim=32)) == gdn.GDN_ERR_SHAPE
    assert plan(cache=None) == E and plan(mp=None) == E and plan(slots=None) == E and plan(n_new=None) == E
    assert plan(n=0) == E and plan(n=5) == E            # more requests than the map holds
    assert plan(cache=_cache(refs=None)) == E and plan(cache=_cache(n_free=None)) == E
    assert plan(cache=_cache(state=0x1004)) == E and plan(cache=_cache(n_pages=0)) == E
    assert plan(mp=_map(units=0x2100008)) == E and plan(mp=_map(max_requests=5000)) == E
    assert plan(so=vp(0x4000004)) == E and plan(slots=vp(0x3000002)) == E

    def append(cache=c, mp=m, k=p, v=p, n=8):
        return lib.gdn_kv_append(R(d), R(cache), R(mp), k, v, n, None)

    assert append(k=None) == E and append(v=vp(0x3000008)) == E and append(n=-1) == E
    assert append(cache=_cache(k=None)) == E and append(cache=_cache(tail=0x1008)) == E and append(mp=_map(counts=None)) == E
    assert append(n=0, k=None) == gdn.GDN_OK            # nothing to do, no device work

    def attend(cache=c, q=p, out=p, n=8, max_new=4, max_len=4096, ws=p, ws_bytes=1 << 40):
        return lib.gdn_kv_attention(R(d), R(cache), R(m), q, p, p, out, n, max_new, max_len, ws, ws_bytes, None)

    assert attend(q=None) == E and attend(out=vp(0x3000004)) == E and attend(n=-1) == E
    assert attend(max_new=0) == E and attend(max_len=0) == E and attend(max_len=1 << 40) == E
    assert attend(cache=_cache(v_scale=None)) == E
    assert attend(ws=None, max_new=2, max_len=10000) == gdn.GDN_ERR_WORKSPACE
    assert attend(ws_bytes=100, max_new=2, max_len=10000) == gdn.GDN_ERR_WORKSPACE
    assert b"workspace" in lib.gdn_last_error()
    assert attend(ws=vp(0x3000008), max_new=2, max_len=10000) == gdn.GDN_ERR_WORKSPACE
    assert attend(n=0, q=None) == gdn.GDN_OK

    assert lib.gdn_kv_fork(R(d), R(c), 0, 0, None) == E and lib.gdn_kv_fork(R(d), R(c), 0, 4, None) == E
    assert lib.gdn_kv_fork(R(d), R(c), -1, 1, None) == E
    assert lib.gdn_kv_release(R(d), R(c), 4, None) == E and lib.gdn_kv_release(R(d), None, 0, None) == E
    assert lib.gdn_kv_status(None, None) == E
    assert lib.gdn_kv_cache_init(R(d), R(_cache(v=None)), None) == E


def test_binding_refuses_wrong_arrays():
    import torch
    d = _desc(head_dim=64, n_q_heads=4)
    bf = torch.zeros((3, 2, 64), dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        gdn.KvCache(d, 4, 2, 4, "cpu", k=torch.zeros((4, 2, 64, 32), dtype=torch.int8))
    with pytest.raises(ValueError):
        gdn.KvCache(d, 4, 2, 4, "cpu", pages=bf)
    cache = gdn.KvCache(d, 4, 2, 4, "cpu", state=torch.zeros((2, 2), dtype=torch.int32))
    plan = gdn.KvPlan.new(4, 2, "cpu")
    for k, v in ((bf.float(), bf), (bf[:, :1], bf), (bf, bf[:2])):
        with pytest.raises(ValueError):
            gdn.gdn_kv_append(d, cache, plan, k, v)
    with pytest.raises(ValueError):
        gdn.gdn_kv_plan(d, cache, torch.zeros(2, dtype=torch.int64), torch.zeros(2, dtype=torch.int32), plan)


@pytest.mark.parametrize("dtype", [gdn.GDN_BF16, gdn.GDN_FP32])
@pytest.mark.parametrize("heads,d", [((1, 1), 64), ((3, 1), 256), ((16, 2), 256), ((32, 8), 128), ((64, 64), 64), ((40, 1), 128)])
def test_workspace_sizes_grow_with_every_bound(lib, heads, d, dtype):
    """More tokens, requests or keys never need less, and the smallest workspace that works is never above the full one."""
    desc = gdn.make_attn_desc(*heads, d, dtype)
    tokens, requests, lengths = (1, 2, 17, 300, 5000, 70000), (1, 3, 64), (1, 64, 65, 513, 2049, 8193, 40000, 1000000)
    size = {(t, r, n): gdn.gdn_kv_attention_workspace(desc, t, r, n) for t in tokens for r in requests for n in lengths}
    low = [gdn.gdn_kv_attention_workspace_min(desc, n) for n in lengths]
    assert all(v > 0 for v in size.values()) and low == sorted(low)
    for axis, values in enumerate((tokens, requests, lengths)):
        for key, v in size.items():
            i = values.index(key[axis])
            if i:
                assert v >= size[key[:axis] + (values[i - 1],) + key[axis + 1:]], key
    for (t, r, n), v in size.items():
        assert v >= low[lengths.index(n)]

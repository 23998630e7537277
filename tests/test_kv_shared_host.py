"""Shared-prefix attention, batched forks, compaction and rotary positions without a GPU: refusals on the host, sizes, and
what the binding refuses."""
import ctypes

import pytest
import torch

from chunked_gated_deltanet_gb300 import gdn
from test_kv_binding import DESC, I32, _handles, _rows
from test_kv_host import _cache, _desc, _map, lib   # noqa: F401

vp, R = ctypes.c_void_p, ctypes.byref
E, SHAPE = gdn.GDN_ERR_INVALID_ARG, gdn.GDN_ERR_SHAPE
P = 0x3000000


def _groups(**kw):
    f = dict(groups=0x5000000, starts=0x5100000, max_groups=4, max_units=16)
    f.update(kw)
    return gdn.gdn_kv_group_map(**f)


def test_group_refusals(lib):
    def call(desc=_desc(), cache=_cache(), mp=_map(), bounds=P, n=2, g=_groups()):
        return lib.gdn_kv_group(R(desc), R(cache) if cache else None, R(mp) if mp else None, vp(bounds) if bounds else None, n,
                                R(g) if g else None, None)

    assert call(desc=_desc(head_dim=96)) == SHAPE
    assert call(cache=None) == E and call(mp=None) == E and call(g=None) == E and call(bounds=None) == E
    assert call(n=0) == E and call(n=5) == E and call(bounds=P + 2) == E
    assert call(g=_groups(groups=0x5000008)) == E and call(g=_groups(starts=None)) == E
    assert call(g=_groups(max_units=15)) == E and call(g=_groups(max_groups=0)) == E and call(g=_groups(max_groups=5000)) == E
    assert call(cache=_cache(table=None)) == E


def test_shared_attention_refusals(lib):
    def call(desc=_desc(), cache=_cache(), mp=_map(), g=_groups(), q=P, k=P, v=P, out=P, n=8, max_new=1, max_len=1000,
             max_suffix=1000, ws=P, ws_bytes=1 << 40):
        return lib.gdn_kv_attention_shared(R(desc), R(cache) if cache else None, R(mp) if mp else None, R(g) if g else None,
                                           *(vp(x) if x else None for x in (q, k, v, out)), n, max_new, max_len, max_suffix,
                                           vp(ws) if ws else None, ws_bytes, None)

    assert call(desc=_desc(in_dtype=3)) == SHAPE
    assert call(cache=None) == E and call(mp=None) == E and call(g=None) == E
    assert call(cache=_cache(k=None)) == E and call(g=_groups(starts=0x5100002)) == E
    for name in "q k v out".split():
        assert call(**{name: None}) == E and call(**{name: P + 8}) == E
    assert call(n=-1) == E and call(n=1 << 28) == E          # 2^28 rows of 16 heads
    assert call(max_new=0) == E and call(max_len=0) == E and call(max_suffix=0) == E
    assert call(max_len=1 << 31) == E and call(max_suffix=1 << 31) == E
    assert call(max_len=(1 << 31) - 1, max_new=8) == E         # more segments than a launch can have
    need = gdn.gdn_kv_shared_workspace(_desc(), 8, 1000, 1000)
    assert call(ws=None) == gdn.GDN_ERR_WORKSPACE and call(ws=P + 8) == gdn.GDN_ERR_WORKSPACE
    assert call(ws_bytes=600) == gdn.GDN_ERR_WORKSPACE and need > 600
    assert call(n=0) == gdn.GDN_OK


def test_shared_workspace_grows_with_every_bound(lib):
    for d in (_desc(), _desc(head_dim=256, n_q_heads=64), _desc(in_dtype=gdn.GDN_FP32, n_q_heads=2, n_kv_heads=1)):
        last = 0
        for rows in (1, 2, 7, 64, 1000, 20000):
            x = gdn.gdn_kv_shared_workspace(d, rows, 40000, 700)
            assert x >= last
            last = x
            assert gdn.gdn_kv_shared_workspace(d, rows, 80000, 700) >= x and gdn.gdn_kv_shared_workspace(d, rows, 40000, 9000) >= x
    assert gdn.gdn_kv_shared_workspace(_desc(), -1, 10, 10) == 0 and gdn.gdn_kv_shared_workspace(_desc(), 1, 0, 10) == 0
    assert gdn.gdn_kv_shared_workspace(_desc(head_dim=96), 1, 10, 10) == 0


def test_fork_batch_refusals(lib):
    def call(desc=_desc(), cache=_cache(), src=P, dst=P, n=2):
        return lib.gdn_kv_fork_batch(R(desc), R(cache) if cache else None, vp(src) if src else None, vp(dst) if dst else None, n, None)

    assert call(desc=_desc(head_dim=32)) == SHAPE and call(cache=_cache(n_slots=(1 << 20) + 1)) == SHAPE
    assert call(cache=None) == E and call(src=None) == E and call(dst=None) == E and call(src=P + 1) == E
    assert call(n=-1) == E and call(n=4097) == E and call(cache=_cache(tail=None)) == E and call(cache=_cache(refs=None)) == E
    assert call(n=0) == gdn.GDN_OK


def test_compact_refusals(lib):
    def call(desc=_desc(), cache=_cache(), outs=(None,) * 4, n=8, counts=P, ws=P, ws_bytes=1 << 20):
        return lib.gdn_kv_compact(R(desc), R(cache) if cache else None, *(vp(x) if x else None for x in outs), n,
                                  vp(counts) if counts else None, vp(ws) if ws else None, ws_bytes, None)

    assert call(desc=_desc(head_dim=32)) == SHAPE
    assert call(cache=None) == E and call(cache=_cache(v=None)) == E and call(cache=_cache(free_pages=None)) == E
    assert call(n=0) == E and call(counts=None) == E and call(outs=(P + 2, None, None, None)) == E
    assert gdn.gdn_kv_compact_workspace(8) == 96 and gdn.gdn_kv_compact_workspace(0) == 0
    assert call(ws=None) == gdn.GDN_ERR_WORKSPACE and call(ws_bytes=95) == gdn.GDN_ERR_WORKSPACE


def test_rope_descriptions(lib):
    for kw in (dict(rotary_dim=16), dict(rotary_dim=256, layout=gdn.GDN_ROPE_INTERLEAVED),
               dict(rotary_dim=64, scaling=gdn.GDN_ROPE_PARTS, factor=4.0, original_len=4096)):
        assert gdn.gdn_rope_desc_check(gdn.make_rope_desc(**kw)) == gdn.GDN_OK
    for kw in (dict(rotary_dim=8), dict(rotary_dim=24), dict(rotary_dim=272), dict(rotary_dim=0), dict(rotary_dim=64, layout=2),
               dict(rotary_dim=64, scaling=3)):
        assert gdn.gdn_rope_desc_check(gdn.make_rope_desc(**kw)) == SHAPE, kw
    nan, inf = float("nan"), float("inf")
    for kw in (dict(base=0.5), dict(base=nan), dict(base=inf), dict(scaling=1, factor=0.5), dict(scaling=1, factor=inf),
               dict(scaling=2, factor=2.0, original_len=0), dict(scaling=2, factor=2.0, beta_fast=1.0), dict(magnitude=0.0),
               dict(magnitude=inf), dict(eps=-1.0), dict(eps=nan), dict(scaling=2, factor=2.0, beta_slow=nan)):
        assert gdn.gdn_rope_desc_check(gdn.make_rope_desc(64, **kw)) == E, kw
    assert lib.gdn_rope_desc_check(None) == E
    assert lib.gdn_rope_table(R(gdn.make_rope_desc(64)), None, None) == E
    assert lib.gdn_rope_table(R(gdn.make_rope_desc(24)), vp(P), None) == SHAPE


def test_rope_refusals(lib):
    base = dict(desc=_desc(), rope=gdn.make_rope_desc(64), table=P, positions=P, q=0x10000000, qs=2048, k=0x20000000, ks=256,
                v=None, vs=0, qw=None, kw=None, qo=0x30000000, ko=0x40000000, vo=None, n=4)

    def call(**kw):
        f = dict(base, **kw)
        p = {x: vp(f[x]) if f[x] else None for x in ("table", "positions", "q", "k", "v", "qw", "kw", "qo", "ko", "vo")}
        return lib.gdn_rope(R(f["desc"]), R(f["rope"]), p["table"], p["positions"], p["q"], f["qs"], p["k"], f["ks"], p["v"],
                            f["vs"], p["qw"], p["kw"], p["qo"], p["ko"], p["vo"], f["n"], None)

    assert call(n=0) == gdn.GDN_OK
    assert call(desc=_desc(head_dim=96)) == SHAPE and call(rope=gdn.make_rope_desc(144)) == SHAPE   # past the head
    for name in ("table", "positions", "q", "k", "qo", "ko"):
        assert call(**{name: None}) == E and call(**{name: base[name] + 2}) == E
    assert call(n=-1) == E and call(n=1 << 31) == E
    assert call(v=P) == E and call(vo=P) == E and call(v=0x50000000, vs=255, vo=0x60000000) == E
    assert call(qs=2040) == E and call(qs=2052) == E and call(ks=128) == E and call(qw=P + 4) == E and call(kw=P + 8) == E
    # an output over an input that it does not replace, over another row's, and over another output
    assert call(qo=base["k"]) == E and call(qo=base["q"] + 4096) == E and call(qo=base["q"], qs=4096) == E
    assert call(ko=base["qo"] + 1024) == E


def test_positions_refusals(lib):
    m = _map()
    assert lib.gdn_kv_positions(None, 4, vp(P), None) == E and lib.gdn_kv_positions(R(m), 4, None, None) == E
    assert lib.gdn_kv_positions(R(m), -1, vp(P), None) == E and lib.gdn_kv_positions(R(m), 0, vp(P), None) == gdn.GDN_OK
    assert lib.gdn_kv_positions(R(_map(units=None)), 4, vp(P), None) == E


def test_the_binding_refuses_host_memory_and_other_shapes():
    cache, plan = _handles()
    groups = gdn.KvGroups(torch.zeros((2, 4), dtype=I32), torch.zeros(8, dtype=I32))
    two, q, k = torch.zeros(2, dtype=I32), _rows(1, 4), _rows(1, 2)
    ws = torch.zeros(64, dtype=torch.uint8)
    rope = gdn.make_rope_desc(64)
    table, pos = torch.zeros(32, dtype=torch.int64), torch.zeros(1, dtype=I32)
    for call in (lambda: gdn.gdn_kv_group(DESC, cache, plan, two, groups),
                 lambda: gdn.gdn_kv_attention_shared(DESC, cache, plan, groups, q, k, k, q, ws, 1, 64, 64),
                 lambda: gdn.gdn_kv_fork_batch(DESC, cache, two, two), lambda: gdn.gdn_kv_compact(DESC, cache, ws, torch.zeros(3, dtype=I32)),
                 lambda: gdn.gdn_rope_table(rope, table), lambda: gdn.gdn_kv_positions(plan, pos),
                 lambda: gdn.gdn_rope(DESC, rope, table, pos, q, k, q, k)):
        with pytest.raises(ValueError, match="GPU memory"):
            call()
    wide = gdn.make_attn_desc(8, 8, 64)
    for call in (lambda: gdn.gdn_kv_group(wide, cache, plan, two, groups), lambda: gdn.gdn_kv_fork_batch(wide, cache, two, two),
                 lambda: gdn.gdn_kv_compact(wide, cache, ws, two)):
        with pytest.raises(ValueError, match="description"):
            call()
    with pytest.raises(ValueError, match="groups must be"):
        gdn.KvGroups(torch.zeros((2, 3), dtype=I32), torch.zeros(8, dtype=I32))
    with pytest.raises(ValueError, match="dst must be"):
        gdn.gdn_kv_fork_batch(DESC, cache, two, torch.zeros(3, dtype=I32))
    with pytest.raises(ValueError, match="table must be"):
        gdn.gdn_rope_table(rope, torch.zeros(16, dtype=torch.int64))

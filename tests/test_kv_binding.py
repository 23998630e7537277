"""What the Python binding of the key/value cache refuses before it hands a pointer to the library."""
import pytest
import torch

from chunked_gated_deltanet_gb300 import gdn

I32 = torch.int32
DESC = gdn.make_attn_desc(4, 2, 64)


def _handles(device="cpu", desc=DESC):
    z = lambda *s, dtype=I32: torch.zeros(s, dtype=dtype, device=device)   # noqa: E731
    cache = gdn.KvCache(desc, 4, 2, 4, device, k=z(4, desc.n_kv_heads, 64, 64, dtype=torch.int8), state=z(2, 2), table=z(2, 4),
                        free=z(4), n_free=z(1), refs=z(4))
    return cache, gdn.KvPlan(z(3), z(8, 8), z(2))


def _rows(n, heads, device="cpu"):
    return torch.zeros((n, heads, 64), dtype=torch.bfloat16, device=device)


def test_host_memory_is_refused():
    cache, plan = _handles()
    one, q, k = torch.ones(1, dtype=I32), _rows(1, 4), _rows(1, 2)
    for call in (lambda: gdn.gdn_kv_plan(DESC, cache, one, one, plan), lambda: gdn.gdn_kv_append(DESC, cache, plan, k, k),
                 lambda: gdn.gdn_kv_attention(DESC, cache, plan, q, k, k, q, None, 1, 64), lambda: gdn.gdn_kv_fork(DESC, cache, 0, 1),
                 lambda: gdn.gdn_kv_release(DESC, cache, 0), lambda: gdn.gdn_kv_status(plan), lambda: gdn.gdn_kv_cache_init(DESC, cache)):
        with pytest.raises(ValueError, match="GPU memory"):
            call()


def test_another_description_is_refused():
    cache, plan = _handles()
    one, q = torch.ones(1, dtype=I32), _rows(1, 8)
    wide = gdn.make_attn_desc(8, 8, 64)      # more heads than the cache's pages have
    for call in (lambda: gdn.gdn_kv_plan(wide, cache, one, one, plan), lambda: gdn.gdn_kv_append(wide, cache, plan, q, q),
                 lambda: gdn.gdn_kv_attention(wide, cache, plan, q, q, q, q, None, 1, 64), lambda: gdn.gdn_kv_fork(wide, cache, 0, 1),
                 lambda: gdn.gdn_kv_release(wide, cache, 0), lambda: gdn.gdn_kv_cache_init(wide, cache)):
        with pytest.raises(ValueError, match="description"):
            call()


@pytest.mark.gpu
def test_wrong_plan_outputs_are_refused(cuda_device):
    """state_out and n_free_out are written at slot indices: their shapes and types, and where the tensors live."""
    cache, plan = _handles(cuda_device)
    one = torch.ones(1, dtype=I32, device=cuda_device)
    z = lambda *s, dtype=I32: torch.zeros(s, dtype=dtype, device=cuda_device)   # noqa: E731
    for kw in (dict(state_out=z(1, 2)), dict(state_out=z(2, 2, dtype=torch.int16)), dict(state_out=z(4)), dict(n_free_out=z(0)),
               dict(n_free_out=z(1, dtype=torch.int64)), dict(state_out=z(2, 2).cpu()), dict(n_free_out=z(1).cpu())):
        with pytest.raises(ValueError):
            gdn.gdn_kv_plan(DESC, cache, one, one, plan, **kw)
    with pytest.raises(ValueError):
        gdn.gdn_kv_plan(DESC, cache, one.cpu(), one, plan)
    k = _rows(1, 2, cuda_device)
    for a, b in ((k.cpu(), k), (k, k.cpu())):
        with pytest.raises(ValueError):
            gdn.gdn_kv_append(DESC, cache, plan, a, b)
    q = _rows(1, 4, cuda_device)
    for a, out, ws in ((q.cpu(), q, None), (q, q.cpu(), None), (q, q, torch.zeros(64, dtype=torch.uint8))):
        with pytest.raises(ValueError):
            gdn.gdn_kv_attention(DESC, cache, plan, a, k, k, out, ws, 1, 64)
    same = gdn.make_attn_desc(4, 2, 64)      # another object of the same description
    out_state, n_free = z(2, 2), z(1)
    gdn.gdn_kv_plan(same, cache, one, one, plan, state_out=out_state, n_free_out=n_free)
    assert gdn.gdn_kv_status(plan) == gdn.GDN_OK and out_state.tolist() == [[0, 0], [1, 0]]

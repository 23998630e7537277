"""Attention of requests that share their first blocks, against the plain model (bounds: kv_shared_ref.py)."""
import numpy as np
import pytest
import torch

from chunked_gated_deltanet_gb300 import gdn
from kv_shared_ref import Shared

pytestmark = pytest.mark.gpu

BF, F32 = gdn.GDN_BF16, gdn.GDN_FP32
HEADS = [(1, 1), (4, 2), (6, 2), (16, 1), (24, 1)]   # query heads per key/value head: 1, 2, 3, 16, 24
both = pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "fp32"])


@both
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("heads", HEADS, ids=lambda h: f"{h[0]}q{h[1]}kv")
def test_forks_match_the_definition(cuda_device, heads, d, dtype):
    """Tokens and prompts of forks in one group, from a prefix that ends inside a block; then forks that have gone apart."""
    m = Shared(heads, d, dtype, n_slots=5, seed=heads[0] + d)
    m.step([2], [200], check=False)
    m.fork(2, 0, 1, 4)
    m.shared_step([0, 2, 1, 4], [1, 1, 1, 1], [0, 4])
    m.shared_step([1, 0, 4], [70, 1, 3], [0, 3])            # slot 1 fills a block of its own
    m.shared_step([4, 0, 1, 2], [1, 1, 1, 1], [0, 4])       # still three shared blocks
    m.shared_step([0, 1], [130, 65], [0, 2], q_size=3.0)
    m.check_contents()


@both
def test_groups_of_every_kind(cuda_device, dtype):
    """Two families, a request in no group before and after them, a group of one request, a request without new tokens,
    an empty group, one whose requests share nothing, and room for more groups."""
    m = Shared((8, 2), 128, dtype, n_pages=80, n_slots=10, seed=5)
    m.step([0, 5, 8, 9], [140, 300, 77, 64], check=False)
    m.fork(0, 1, 2)
    m.fork(5, 6, 7, 3)
    m.shared_step([8, 0, 1, 2, 5, 6, 7, 9, 4, 3], [2, 1, 3, 0, 1, 9, 1, 5, 7, 2], [1, 4, 4, 7, 8, 9], max_groups=9)
    m.shared_step([8, 9, 0], [1, 1, 1], [0, 3])               # no block alike
    m.shared_step([2, 1], [1, 1], [0, 1, 2])                  # two groups of one request each
    m.shared_step([1, 2], [0, 0], [0, 2])                     # nothing new at all
    m.check_contents()


@pytest.mark.parametrize("heads,d,dtype", [((8, 2), 128, BF), ((2, 2), 64, BF), ((8, 1), 256, BF), ((4, 2), 64, F32)])
def test_long_prefixes_are_cut_and_joined(cuda_device, heads, d, dtype):
    """A prefix of many pieces with sharp weights, own keys of several segments, tokens and prompts."""
    m = Shared(heads, d, dtype, n_pages=400, n_slots=4, max_blocks=140, seed=3)
    m.step([0], [4090], check=False)
    m.fork(0, 1, 2)
    m.step([1], [700 if dtype == BF else 1100], check=False)
    m.step([2], [4200], check=False)
    m.shared_step([0, 1, 2], [1, 1, 1], [0, 3], q_size=4.0)
    m.shared_step([2, 0, 1], [3, 20, 40], [0, 3], q_size=3.0)
    m.shared_step([0, 1], [1, 1], [0, 2], q_size=4.0, max_len=8800, max_suffix=800 if dtype == BF else 1200)
    m.check_contents()


@pytest.mark.parametrize("d", [64, 128, 256])
def test_row_tiles(cuda_device, d):
    """Rows of a group that fill one, two and more row tiles and leave the last one ragged."""
    m = Shared((3, 1), d, BF, n_pages=200, n_slots=30, max_blocks=20, seed=4)
    m.step([0], [330], check=False)
    m.fork(0, *range(1, 30))
    for k, new in ((29, 1), (30, 3), (5, 51), (4, 77), (2, 258)):   # 87, 270, 765, 924, 1,548 rows
        m.shared_step(list(range(k)), [new] * k, [0, k], rows_check=[0, 1, k - 1])


@pytest.mark.parametrize("heads,new", [((4, 1), 1), ((6, 1), 1), ((8, 1), 1), ((12, 1), 1), ((16, 1), 1), ((5, 1), 3), ((2, 2), 8)],
                         ids=lambda x: f"{x[0]}q{x[1]}kv" if isinstance(x, tuple) else f"{x}new")
@pytest.mark.parametrize("d", [64, 128, 256])
def test_row_tiles_of_tokens(cuda_device, d, heads, new):
    """Single tokens and a few: three groups over prefixes of many segments, whose tiles of 8 or 16 rows end inside a request."""
    m = Shared(heads, d, BF, n_pages=300, n_slots=20, max_blocks=50, seed=7)
    m.step([0, 7, 14], [2600, 1000, 70], check=False)
    m.fork(0, *range(1, 7))
    m.fork(7, *range(8, 14))
    m.fork(14, *range(15, 20))
    m.step([3, 9, 16], [300, 64, 1], check=False)
    m.shared_step(list(range(20)), [new] * 20, [0, 7, 14, 20], q_size=3.0)
    m.shared_step([3, 0, 1, 8, 9], [new, 1, new, 1, new], [0, 3, 5])
    m.check_contents()


@both
@pytest.mark.parametrize("heads", [(8, 2), (24, 1)], ids=["few", "many"])
def test_as_the_unshared_attention(cuda_device, heads, dtype):
    """The same plan through both calls: equal within twice the bounds, and the same bits twice."""
    m = Shared(heads, 128, dtype, n_pages=100, n_slots=6, seed=8)
    m.step([0], [500], check=False)
    m.fork(0, 1, 2, 3, 4)
    n = 5
    out = m.shared_step([0, 1, 2, 3, 4], [1] * n, [0, n], max_new=1)
    assert torch.isfinite(out).all()
    plan, groups = m.last
    q, k, v = (m.draw(n, h).to(m.dev) for h in (m.hq, m.hkv, m.hkv))
    a, b, c = (torch.empty_like(q) for _ in range(3))
    ws = gdn.kv_attention_workspace(m.desc, n, n, 600, m.dev)
    gdn.gdn_kv_attention(m.desc, m.cache, plan, q, k, v, a, ws, 1, 600)
    ws = gdn.kv_shared_workspace(m.desc, n, 600, 600, m.dev)
    for o in (b, c):
        gdn.gdn_kv_attention_shared(m.desc, m.cache, plan, groups, q, k, v, o, ws, 1, 600, 600)
    assert torch.equal(b, c)
    # weights and values are of size 1: two results of 2^-8 relative (bf16) and sums of 500 terms (fp32)
    tol = 2 * 2.0 ** -8 if dtype == BF else 2 * 500 * 2.0 ** -24
    assert float((a.float() - b.float()).abs().max()) <= tol * max(1.0, float(a.float().abs().max()))


@both
@pytest.mark.parametrize("n", [1, 40])
@pytest.mark.parametrize("ratio", [12, 30, 80], ids=lambda r: f"2^{r}")
@pytest.mark.parametrize("sizes", [[0, 0, 1, 1, 1, 1], [1, 1, 0, 0, 0, 0], [0, 1, 0, 1, 1, 0], [0, 0, 0, 0, 0, 1], [1, 1, 1, 1, 1, 0]],
                         ids=["grows", "falls", "alternates", "last large", "last small"])
def test_shared_blocks_of_unequal_values(cuda_device, sizes, ratio, n, dtype):
    """Values of shared blocks (and of the open one) that are 2^ratio apart, in one column of the large ones only, so that
    every other column is the small ones' alone; a block of zeros between."""
    m = Shared((4, 2), 128, dtype, n_slots=4, seed=22)
    v = m.draw(384, 2)
    for b, big in enumerate([*sizes[:3], 2, *sizes[3:5]]):
        rows = v[64 * b:64 * b + 64]
        if big:
            keep = rows[:, :, 3].clone()
            rows.zero_()
            rows[:, :, 3] = keep * (2.0 ** ratio if big == 1 else 0.0)
    m.step([0], [384], check=False, data=(m.draw(384, 4), m.draw(384, 2), v))
    m.fork(0, 1, 2)
    own = m.draw(3 * n, 2)
    if sizes[5]:
        own[:, :, 3] *= 2.0 ** ratio
    m.shared_step([0, 1, 2], [n] * 3, [0, 3], data=(m.draw(3 * n, 4, 2.0), m.draw(3 * n, 2), own))


@both
def test_empty_sessions(cuda_device, dtype):
    """First tokens and prompts of slots that hold nothing, alone in a group and beside one another."""
    m = Shared((4, 2), 64, dtype, n_slots=5, seed=4)
    q, k, v = m.draw(2, 4), m.draw(2, 2), m.draw(2, 2)
    out = m.shared_step([0, 3], [1, 1], [0, 2], data=(q, k, v))
    assert torch.equal(out.cpu(), v.repeat_interleave(2, 1))       # each sees itself alone
    m.shared_step([1, 2, 0], [70, 64, 63], [0, 2, 3])
    m.check_contents()


def test_more_groups_than_a_warp_looks_at(cuda_device):
    m = Shared((2, 1), 64, BF, n_pages=400, n_slots=90, max_blocks=8, seed=12)
    sources, dst = list(range(0, 80, 2)), list(range(1, 80, 2))
    m.step(sources, [60 + 5 * i for i in range(40)], check=False)
    gdn.gdn_kv_fork_batch(m.desc, m.cache, m.i32(sources), m.i32(dst))
    for s, t in zip(sources, dst):
        m.slots[t] = m.slots[s].copy()
    m.shared_step(list(range(80)), [1] * 80, list(range(0, 81, 2)))
    m.shared_step(list(range(80)), [1 + i % 3 for i in range(80)], list(range(0, 81, 2)))
    m.check_contents()


@both
def test_shared_pages_past_two_gigabytes(cuda_device, dtype):
    n_pages = 2 ** 31 // (8 * 64 * 256) + 40
    m = Shared((8, 8), 256, dtype, n_pages=n_pages, n_slots=3, max_blocks=8)
    m.cache.free.copy_(torch.arange(n_pages, dtype=torch.int32, device=cuda_device))
    m.step([0], [140], check=False)
    m.fork(0, 1, 2)
    m.shared_step([0, 1, 2], [1, 1, 70], [0, 3])
    assert int(m.cache.table[1, 0]) * 8 * 64 * 256 > 2 ** 31


@pytest.mark.parametrize("heads,dtype", [((8, 2), BF), ((24, 1), BF), ((4, 2), F32)])
def test_fewer_rows_than_the_plan(cuda_device, heads, dtype):
    """Arrays that end before the plan does: the units past them are left out (the launch may not even look at them), the
    others right."""
    m = Shared(heads, 128, dtype, n_slots=5, seed=3)
    m.step([0], [200], check=False)
    m.fork(0, 1, 2)
    n = 3
    plan = gdn.KvPlan.new(n, n, m.dev)
    groups = gdn.KvGroups.new(plan, 1)
    gdn.gdn_kv_plan(m.desc, m.cache, m.i32([0, 1, 2]), m.i32([1] * n), plan)
    q, k, v = m.draw(2, m.hq), m.draw(2, m.hkv), m.draw(2, m.hkv)
    qd, kd, vd = (t.to(m.dev) for t in (q, k, v))
    gdn.gdn_kv_append(m.desc, m.cache, plan, kd, vd)
    gdn.gdn_kv_group(m.desc, m.cache, plan, m.i32([0, n]), groups)
    out = torch.full_like(qd, float("nan"))
    ws = gdn.kv_shared_workspace(m.desc, 2, 300, 300, m.dev)
    ws.fill_(255)
    gdn.gdn_kv_attention_shared(m.desc, m.cache, plan, groups, qd, kd, vd, out, ws, 1, 300, 300)
    gdn.gdn_device_status()                                        # says so, or not
    for i in (0, 1):
        m.slots[i].k.append(k[i].float().numpy())
        m.slots[i].v.append(v[i].float().numpy())
        ref, bound = m.attention(i, 200, q[i:i + 1].double().numpy())
        assert (np.abs(out[i:i + 1].double().cpu().numpy() - ref) <= bound).all()


@both
def test_what_is_not_finite_keeps_to_its_rows(cuda_device, dtype):
    """A query that is not finite, and keys and values that are not in a fork's own block, reach the other rows in no way."""
    for new in (1, 40):
        m = Shared((4, 2), 64, dtype, n_slots=4, seed=6)
        m.step([0], [150], check=False)
        m.fork(0, 1, 2)
        n = 3 * new
        q, k, v = m.draw(n, 4), m.draw(n, 2), m.draw(n, 2)
        q[new, 1] = float("nan")                      # request 1
        k[new, 0], v[new, 1] = float("inf"), float("nan")
        m.shared_step([0, 1, 2], [new] * 3, [0, 3], data=(q, k, v), rows_check=[0, 2])


def test_sizes_below_the_batch_are_reported(cuda_device):
    """A request past max_suffix is left out, its rows as they were, and the others are right."""
    m = Shared((4, 2), 128, BF, n_slots=4, seed=2)
    m.step([0], [130], check=False)
    m.fork(0, 1, 2)
    m.step([1], [140], check=False)
    before = [len(m.slots[s].k) for s in (0, 1, 2)]
    data = (m.draw(3, 4), m.draw(3, 2), m.draw(3, 2))
    out = m.shared_step([0, 1, 2], [1, 1, 1], [0, 3], data=data, max_suffix=64, check=False, fill=7.0)
    assert gdn.gdn_device_status() == gdn.GDN_ERR_INVALID_ARG
    assert (out[1] == 7).all()
    for i, s in ((0, 0), (2, 2)):
        ref, bound = m.attention(s, before[i], data[0][i:i + 1].double().numpy())
        assert (np.abs(out[i:i + 1].double().cpu().numpy() - ref) <= bound).all()


def test_bounds_out_of_order_share_nothing(cuda_device):
    m = Shared((4, 2), 64, BF, n_slots=4, seed=2)
    m.step([0], [130], check=False)
    m.fork(0, 1, 2)
    before = len(m.slots[0].k)
    data = (m.draw(3, 4), m.draw(3, 2), m.draw(3, 2))
    for bounds in ([2, 0], [-1, 3], [0, 9], [0, 2, 1, 3], [0, 9, 3]):
        for s in (0, 1, 2):
            del m.slots[s].k[before:], m.slots[s].v[before:]
        m.cache.state[:3, 0] = before
        out = m.shared_step([0, 1, 2], [1, 1, 1], bounds, data=data, check=False)
        assert gdn.gdn_device_status() == gdn.GDN_ERR_INVALID_ARG
        assert not m.last[1].groups[:, 3].any() and not m.last[1].starts[:3].any()
        for i in range(3):
            ref, bound = m.attention(i, before, data[0][i:i + 1].double().numpy())
            assert (np.abs(out[i:i + 1].double().cpu().numpy() - ref) <= bound).all()


def test_a_plan_that_did_not_fit_has_no_groups(cuda_device):
    m = Shared((4, 2), 64, BF, n_pages=4, n_slots=3, max_blocks=4, seed=2)
    m.step([0], [130], check=False)
    m.fork(0, 1)
    plan = gdn.KvPlan.new(600, 2, m.dev)
    groups = gdn.KvGroups.new(plan, 1)
    gdn.gdn_kv_plan(m.desc, m.cache, m.i32([0, 1]), m.i32([300, 300]), plan)
    gdn.gdn_kv_group(m.desc, m.cache, plan, m.i32([0, 2]), groups)
    q, k = m.draw(600, 4).to(m.dev), m.draw(600, 2).to(m.dev)
    out = torch.full_like(q, 7)
    gdn.gdn_kv_attention_shared(m.desc, m.cache, plan, groups, q, k, k, out, gdn.kv_shared_workspace(m.desc, 600, 600, 600, m.dev),
                                300, 600, 600)
    assert gdn.gdn_kv_status(plan) == gdn.GDN_ERR_CAPACITY
    assert (out == 7).all() and not groups.groups.any()
    assert gdn.gdn_device_status() == gdn.GDN_OK


def test_another_stream(cuda_device):
    m = Shared((8, 2), 128, BF, n_slots=4, seed=9)
    m.step([0], [260], check=False)
    m.fork(0, 1, 2)
    torch.cuda.synchronize()
    m.shared_step([0, 1, 2], [1, 2, 1], [0, 3], stream=torch.cuda.Stream())


@pytest.mark.parametrize("heads,d,dtype,new", [((16, 2), 256, BF, 1), ((16, 2), 128, BF, 40), ((4, 2), 64, F32, 5), ((8, 8), 64, BF, 1)],
                         ids=["few", "many", "fp32", "together"])
def test_calls_on_one_workspace_in_a_row(cuda_device, heads, d, dtype, new):
    """Own keys run beside the shared blocks, joins after both: two batches in turn on one workspace, eager and in a graph, give
    the bits that each gives alone, whichever part takes longer."""
    m = Shared(heads, d, dtype, n_pages=400, n_slots=8, max_blocks=140, seed=2)
    m.step([0, 4], [6000, 200], check=False)
    m.fork(0, 1, 2, 3)
    m.fork(4, 5, 6, 7)
    m.step([2], [900], check=False)          # one short own part and one long one
    m.step([6], [2500], check=False)         # own keys longer than what is shared
    calls, alone = [], []
    for slots in ([0, 1, 2, 3], [4, 5, 6, 7]):
        n = 4 * new
        plan = gdn.KvPlan.new(n, 4, m.dev)
        groups = gdn.KvGroups.new(plan, 1)
        q, k, v = (m.draw(n, h).to(m.dev) for h in (m.hq, m.hkv, m.hkv))
        gdn.gdn_kv_plan(m.desc, m.cache, m.i32(slots), m.i32([new] * 4), plan)
        gdn.gdn_kv_append(m.desc, m.cache, plan, k, v)
        gdn.gdn_kv_group(m.desc, m.cache, plan, m.i32([0, 4]), groups)
        calls.append((plan, groups, q, k, v))
    ws = gdn.kv_shared_workspace(m.desc, 4 * new, 7000, 2800, m.dev)

    def attend(i, out):
        plan, groups, q, k, v = calls[i]
        gdn.gdn_kv_attention_shared(m.desc, m.cache, plan, groups, q, k, v, out, ws, new, 7000, 2800)

    outs = [torch.empty_like(calls[0][2]) for _ in range(24)]
    for i in range(2):
        ws.fill_(255)
        attend(i, outs[i])
        torch.cuda.synchronize()
        alone.append(outs[i].clone())
        assert not outs[i].isnan().any()
    for first in (0, 1):
        ws.fill_(255)
        for j, out in enumerate(outs):
            out.fill_(float("nan")) if j % 5 == 0 else None
            attend((j + first) % 2, out)
        for j, out in enumerate(outs):
            assert torch.equal(out, alone[(j + first) % 2])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for j, out in enumerate(outs):
            attend(j % 2, out)
    for _ in range(3):
        ws.fill_(255)
        for out in outs:
            out.zero_()
        graph.replay()
        for j, out in enumerate(outs):
            assert torch.equal(out, alone[j % 2])
    assert gdn.gdn_device_status() == gdn.GDN_OK


def test_a_captured_step_replays(cuda_device):
    """Batched forks, then plan, append, grouping and attention of their tokens from one graph; each replay advances the
    slots, over the end of a block."""
    m = Shared((8, 2), 128, BF, n_pages=60, n_slots=5, seed=1)
    m.step([0], [185], check=False)
    n, steps = 4, 10
    slots = [1, 2, 3, 4]
    src, dst, ones, bounds = m.i32([0] * n), m.i32(slots), m.i32([1] * n), m.i32([0, n])
    plan = gdn.KvPlan.new(n, n, m.dev)
    groups = gdn.KvGroups.new(plan, 1)
    ws = gdn.kv_shared_workspace(m.desc, n, 256, 128, m.dev)
    q, k, v = (torch.zeros((n, h, 128), dtype=torch.bfloat16, device=m.dev) for h in (8, 2, 2))
    out = torch.zeros_like(q)

    def step():
        gdn.gdn_kv_plan(m.desc, m.cache, dst, ones, plan)
        gdn.gdn_kv_append(m.desc, m.cache, plan, k, v)
        gdn.gdn_kv_group(m.desc, m.cache, plan, bounds, groups)
        gdn.gdn_kv_attention_shared(m.desc, m.cache, plan, groups, q, k, v, out, ws, 1, 256, 128)

    gdn.gdn_kv_fork_batch(m.desc, m.cache, src, dst)
    step()                                                    # sets every kernel's attributes before the capture
    torch.cuda.synchronize()
    fork, graph = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(fork):
        gdn.gdn_kv_fork_batch(m.desc, m.cache, src, dst)
    with torch.cuda.graph(graph):
        step()
    fork.replay()
    for s in slots:
        m.slots[s] = m.slots[0].copy()
    for _ in range(steps):
        x = m.draw(n, 8), m.draw(n, 2), m.draw(n, 2)
        for t, y in zip((q, k, v), x):
            t.copy_(y)
        before = len(m.slots[1].k)
        graph.replay()
        got = out.double().cpu().numpy()
        for i, s in enumerate(slots):
            m.slots[s].k.append(x[1][i].float().numpy())
            m.slots[s].v.append(x[2][i].float().numpy())
            ref, bound = m.attention(s, before, x[0][i:i + 1].double().numpy())
            assert (np.abs(got[i:i + 1] - ref) <= bound).all()
    assert gdn.gdn_device_status() == gdn.GDN_OK
    m.check_contents()


@pytest.mark.parametrize("heads,d,dtype,new", [((8, 1), 256, BF, 1), ((16, 1), 128, BF, 3), ((4, 2), 64, F32, 2), ((8, 2), 128, BF, 1)],
                         ids=["few", "many", "fp32", "together"])
def test_a_captured_step_with_other_batches(cuda_device, heads, d, dtype, new):
    """One graph of plan, append, grouping and attention replayed for two families in turn, whose slots, shared blocks and
    lengths differ: every launch reads what the replay's own plan and grouping wrote."""
    m = Shared(heads, d, dtype, n_pages=120, n_slots=8, max_blocks=30, seed=6)
    m.step([0, 4], [700, 130], check=False)
    m.fork(0, 1, 2, 3)
    m.fork(4, 5, 6, 7)
    m.step([2, 7], [100, 200], check=False)
    families = [[0, 1, 2, 3], [4, 7, 5, 6]]
    n = 4 * new
    dst, bounds, news = m.i32(families[0]), m.i32([0, 4]), m.i32([new] * 4)
    plan = gdn.KvPlan.new(n, 4, m.dev)
    groups = gdn.KvGroups.new(plan, 1)
    ws = gdn.kv_shared_workspace(m.desc, n, 1000, 400, m.dev)
    q, k, v = (m.draw(n, h).to(m.dev) for h in (m.hq, m.hkv, m.hkv))
    out = torch.zeros_like(q)

    def step():
        gdn.gdn_kv_plan(m.desc, m.cache, dst, news, plan)
        gdn.gdn_kv_append(m.desc, m.cache, plan, k, v)
        gdn.gdn_kv_group(m.desc, m.cache, plan, bounds, groups)
        gdn.gdn_kv_attention_shared(m.desc, m.cache, plan, groups, q, k, v, out, ws, new, 1000, 400)

    def advance(replay, slots):
        x = m.draw(n, m.hq), m.draw(n, m.hkv), m.draw(n, m.hkv)
        for t, y in zip((q, k, v), x):
            t.copy_(y)
        dst.copy_(torch.tensor(slots, dtype=torch.int32))
        before = [len(m.slots[s].k) for s in slots]
        replay()
        got = out.double().cpu().numpy()
        for i, s in enumerate(slots):
            rows = slice(i * new, (i + 1) * new)
            m.slots[s].k += list(x[1][rows].float().numpy())
            m.slots[s].v += list(x[2][rows].float().numpy())
            ref, bound = m.attention(s, before[i], x[0][rows].double().numpy())
            assert (np.abs(got[rows] - ref) <= bound).all(), (s, before[i])

    advance(step, families[0])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for j in range(12):
        advance(graph.replay, families[(j + 1) % 2])
    assert gdn.gdn_device_status() == gdn.GDN_OK
    m.check_contents()


@pytest.mark.parametrize("d", [128, 256])
def test_wait_timeout_is_reported_and_context_survives(cuda_device, d):
    m = Shared((48, 2), d, BF, n_slots=4, seed=9)
    m.step([0], [260], check=False)
    m.fork(0, 1, 2)
    torch.cuda.synchronize()
    gdn.gdn_debug_inject_wait_timeout(3, 2000)
    try:
        m.shared_step([0, 1, 2], [1, 1, 1], [0, 3], check=False)
        assert gdn.gdn_device_status() == gdn.GDN_ERR_TIMEOUT
    finally:
        gdn.gdn_debug_inject_wait_timeout(0)
    m.shared_step([0, 1, 2], [1, 2, 1], [0, 3])

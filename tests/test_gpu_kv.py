"""The paged 8-bit key/value cache and its attention on the GPU, against the plain model of kv_ref.py (its docstring
derives the bounds)."""
import numpy as np
import pytest
import torch

from chunked_gated_deltanet_gb300 import gdn
from kv_ref import B, Model

pytestmark = pytest.mark.gpu

BF, F32 = gdn.GDN_BF16, gdn.GDN_FP32
HEADS = [(1, 1), (4, 4), (4, 2), (6, 2), (8, 1), (16, 1), (24, 1)]   # query heads per key/value head: 1, 1, 2, 3, 8, 16, 24


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("heads", HEADS, ids=lambda h: f"{h[0]}q{h[1]}kv")
def test_steps_match_the_definition(cuda_device, heads, d, dtype):
    """Prompts, single tokens, empty requests and blocks that close at their first and last token, over several steps."""
    m = Model(heads, d, dtype, seed=heads[0] + d)
    m.step([3, 0, 1], [1, 64, 130])
    m.step([0, 1, 2, 3], [1, 1, 0, 62])
    m.step([3, 2], [1, 63])           # slot 3 closes a block with one token
    m.step([2, 3, 0], [1, 1, 1])
    m.step([1, 4], [70, 200])
    m.step([1, 2, 0, 4, 3], [1, 2, 3, 4, 1])
    m.check_contents()


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "fp32"])
def test_one_token_session(cuda_device, dtype):
    """The first token sees itself alone: its output is its own value."""
    m = Model((4, 2), 128, dtype)
    q, k, v = m.draw(1, 4), m.draw(1, 2), m.draw(1, 2)
    out = m.step([2], [1], data=(q, k, v))
    assert torch.equal(out.cpu(), v.repeat_interleave(2, 1))


@pytest.mark.parametrize("heads,d,dtype", [((8, 2), 128, BF), ((2, 2), 64, BF), ((8, 1), 256, BF), ((4, 2), 64, F32)])
def test_segments_are_joined(cuda_device, heads, d, dtype):
    """Contexts past one segment (512 keys for few rows, 4,096 for many), with sharp weights, and through a workspace
    that holds the partial results of a single unit at a time."""
    m = Model(heads, d, dtype, n_pages=80, n_slots=2, max_blocks=80, seed=3)
    m.step([0], [4090], check=False)
    m.step([0], [9], q_size=4.0)               # many rows or few, by the head count; a block closes at 4,096
    m.step([0], [1], q_size=4.0)
    m.ws_bytes = gdn.gdn_kv_attention_workspace_min(m.desc, 4400)
    m.step([0, 1], [200, 30], q_size=3.0)
    m.step([1, 0], [1, 1], q_size=3.0)
    m.check_contents()


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_contents_do_not_depend_on_the_split(cuda_device, d, dtype):
    """One call or many: the same pages, scales and open rows, bit for bit; prompt rows bit for bit as well."""
    g = torch.Generator().manual_seed(9)
    dt = torch.bfloat16 if dtype == BF else torch.float32
    n = 333
    q, k, v = (torch.randn((n, h, d), generator=g).to(dt) for h in (12, 2, 2))
    outs, models = [], []
    for cuts in ([0, n], [0, 100, 200, n], [0, 64, 128, 131, 256, n]):
        m = Model((12, 2), d, dtype)
        outs.append(torch.cat([m.step([1], [b - a], check=False, data=(q[a:b], k[a:b], v[a:b]), max_new=64)
                               for a, b in zip(cuts, cuts[1:])]))
        m.check_contents()
        models.append(m)
    for o, m in zip(outs[1:], models[1:]):
        assert torch.equal(o, outs[0])


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "fp32"])
def test_a_row_does_not_depend_on_the_batch(cuda_device, dtype):
    """A session alone and beside others gives the same bits, for prompts and for single tokens."""
    g = torch.Generator().manual_seed(4)
    dt = torch.bfloat16 if dtype == BF else torch.float32
    mk = lambda n, h: torch.randn((n, h, 128), generator=g).to(dt)   # noqa: E731
    a, b = Model((8, 2), 128, dtype), Model((8, 2), 128, dtype)
    for new in (150, 1):
        mine, other = [mk(new, h) for h in (8, 2, 2)], [mk(new + 37 * (new > 1), h) for h in (8, 2, 2)]
        n2 = other[0].shape[0]
        alone = a.step([2], [new], check=False, data=mine)
        both = b.step([4, 2], [n2, new], check=False, data=[torch.cat([y, x]) for x, y in zip(mine, other)])
        assert torch.equal(alone, both[n2:])


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "fp32"])
def test_values_that_are_not_finite_in_every_part_of_the_block(cuda_device, dtype):
    """Few rows: infinities and NaN among the own block's values reach the rows that see them, once each, and no other."""
    m = Model((4, 2), 128, dtype)
    n = 63
    q, k, v = m.draw(n, 4), m.draw(n, 2), m.draw(n, 2)
    clean = v.clone()
    for key, col, x in ((3, 5, "inf"), (20, 5, "inf"), (37, 5, "inf"), (50, 9, "-inf"), (21, 7, "nan"), (60, 70, "inf"), (62, 100, "inf")):
        v[key, 0, col], clean[key, 0, col] = float(x), 0.0
    m.step([1], [61], check=False, data=(q[:61], k[:61], clean[:61]))
    m.step([0], [61], check=False, data=(q[:61], k[:61], v[:61]))
    out = m.step([0], [2], check=False, data=(q[61:], k[61:], v[61:])).double().cpu().numpy()
    m.slots[1].k += [x.float().numpy() for x in k[61:]]
    m.slots[1].v += [x.float().numpy() for x in clean[61:]]
    ref, bound = m.attention(1, 61, q[61:].double().numpy())
    for row in range(2):
        want = {5: np.inf, 9: -np.inf, 7: np.nan, 70: np.inf, **({100: np.inf} if row else {})}
        for h in range(4):
            for c in range(128):
                if h < 2 and c in want:
                    assert np.array_equal(out[row, h, c], want[c], equal_nan=True), (row, h, c)
                else:
                    assert abs(out[row, h, c] - ref[row, h, c]) <= bound[row, h, c], (row, h, c)


@pytest.mark.parametrize("n", [2, 200], ids=["few", "many"])
@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "fp32"])
def test_a_query_that_is_not_finite_keeps_to_its_row(cuda_device, dtype, n):
    """NaN and infinities in some heads of a token's query: the other rows are as without them, zero and tiny ones too."""
    m = Model((4, 2), 128, dtype)
    m.step([1], [150], check=False)
    q, k, v = m.draw(n, 4), m.draw(n, 2), m.draw(n, 2)
    q[n - 1, 0, 3], q[0, 3, 0], q[0, 1, 127] = float("nan"), float("inf"), float("-inf")
    q[0, 0], q[n - 1, 2] = 0.0, q[n - 1, 2] * 2.0 ** -100
    out = m.step([1], [n], check=False, data=(q, k, v)).double().cpu().numpy()
    bad = {(n - 1, 0), (0, 3), (0, 1)}
    for t in (0, n - 1):
        clean = q[t:t + 1].clone()
        for row, head in bad:
            if row == t:
                clean[0, head] = 0.0
        ref, bound = m.attention(1, 150 + t, clean.double().numpy())
        for head in range(4):
            if (t, head) in bad:
                assert np.isnan(out[t, head]).all(), (t, head)
            else:
                assert (np.abs(out[t, head] - ref[0, head]) <= bound[0, head]).all(), (t, head)


def test_segments_of_every_length(cuda_device):
    """33,000 keys and as many rows as make each rule of the segments hold (32 blocks, 48, growing to 256, 128), through a
    workspace of the smallest size; the first and last rows of each call."""
    m = Model((16, 2), 64, BF, n_pages=580, n_slots=1, max_blocks=580, seed=12)
    m.ws_bytes = gdn.gdn_kv_attention_workspace_min(m.desc, 580 * B)
    m.step([0], [33000], check=False, max_len=580 * B)
    for n in (40, 200, 700, 3000):
        start = len(m.slots[0].k)
        q, k, v = m.draw(n, 16, 3.0), m.draw(n, 2), m.draw(n, 2)
        out = m.step([0], [n], check=False, data=(q, k, v), max_len=580 * B).double().cpu().numpy()
        for a in (0, n - 2):
            ref, bound = m.attention(0, start + a, q[a:a + 2].double().numpy())
            assert (np.abs(out[a:a + 2] - ref) <= bound).all(), (n, a)


@pytest.mark.parametrize("d", [64, 256])
def test_a_long_context_does_not_depend_on_the_batch(cuda_device, d):
    """As above past one segment: with the same max_new, the bits of a session alone."""
    g = torch.Generator().manual_seed(6)
    mk = lambda n, h: torch.randn((n, h, d), generator=g).to(torch.bfloat16)   # noqa: E731
    a, b = (Model((8, 2), d, BF, n_pages=140, max_blocks=70) for _ in range(2))
    for new in (3500, 20, 1):
        mine, other = [mk(new, h) for h in (8, 2, 2)], [mk(new, h) for h in (8, 2, 2)]
        alone = a.step([2], [new], check=False, data=mine)
        both = b.step([4, 2], [new, new], check=False, data=[torch.cat([y, x]) for x, y in zip(mine, other)])
        assert torch.equal(alone, both[new:])


@pytest.mark.parametrize("heads,d,new", [((3, 1), 256, 105), ((4, 2), 64, 169), ((8, 2), 128, 1), ((32, 8), 128, 30)])
def test_the_workspace_takes_one_launch(cuda_device, heads, d, new):
    """The workspace of a batch's tokens, requests and longest context holds its partial results, whatever max_new."""
    m = Model(heads, d, BF, max_blocks=600)
    gdn.gdn_timing_begin(100)
    m.step([0, 3, 4], [new] * 3, check=False, max_len=38000)
    assert gdn.gdn_timing_end()["kv_attention"][1] == 1


@pytest.mark.parametrize("few", [True, False], ids=["token", "prompt"])
@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "fp32"])
def test_unused_memory_is_not_read_into_results(cuda_device, dtype, few):
    """Pages, scales, tails and rows that no key lies in hold NaN patterns; a later token's NaN and infinite key and value
    in the same block do not reach earlier rows."""
    m = Model((8, 2), 128, dtype, n_pages=12, max_blocks=12)
    m.cache.k_scale.fill_(float("nan"))
    m.cache.v_scale.fill_(float("nan"))
    m.cache.tail.fill_(float("nan"))
    m.cache.k.fill_(-128)
    m.step([1], [70])
    m.step([1], [1])
    if few:
        m.step([1, 0], [1, 1])
        return
    n = 40
    q, k, v = m.draw(n, 8), m.draw(n, 2), m.draw(n, 2)
    k[30], v[31, 0, 5], v[32, 0, 7], v[33, 1, 0] = float("nan"), float("inf"), float("nan"), float("-inf")
    out = m.step([2], [n], check=False, data=(q, k, v))
    ref, bound = m.attention(2, 0, q[:30].double().numpy())
    assert (np.abs(out[:30].double().cpu().numpy() - ref) <= bound).all()
    assert torch.isnan(out[30:]).all()          # a NaN key makes every weight of the row NaN


def test_forks_share_pages_and_diverge(cuda_device):
    m = Model((8, 2), 128, BF)
    m.step([0], [200])
    before = int(m.cache.n_free.item())
    gdn.gdn_kv_fork(m.desc, m.cache, 0, 1)
    gdn.gdn_kv_fork(m.desc, m.cache, 0, 3)
    m.slots[1], m.slots[3] = m.slots[0].copy(), m.slots[0].copy()
    assert int(m.cache.n_free.item()) == before
    m.check_contents()
    m.step([1, 0, 3], [60, 1, 20])
    m.step([3, 1, 0], [1, 1, 1])
    m.check_contents()
    gdn.gdn_kv_fork(m.desc, m.cache, 1, 0)       # restore over a slot that holds pages of its own
    m.slots[0] = m.slots[1].copy()
    m.check_contents()
    for s in (3, 0, 1):
        gdn.gdn_kv_release(m.desc, m.cache, s)
        m.slots[s].k, m.slots[s].v = [], []
        m.check_contents()
    assert int(m.cache.n_free.item()) == m.cache.n_pages
    m.step([1], [130])
    m.check_contents()


def test_a_batch_that_does_not_fit_changes_nothing(cuda_device):
    m = Model((4, 2), 64, BF, n_pages=4, n_slots=3, max_blocks=3)
    m.step([0], [150])
    names = ("state", "table", "n_free", "refs", "free", "tail", "k")
    plan = gdn.KvPlan.new(1000, 3)

    def refused(slots, new, p=plan):
        bits = lambda n: getattr(m.cache, n).view(torch.uint8)   # noqa: E731  (unused rows may hold NaN patterns)
        kept = {n: bits(n).clone() for n in names}
        gdn.gdn_kv_plan(m.desc, m.cache, m.i32(slots), m.i32(new), p)
        assert gdn.gdn_kv_status(p) == gdn.GDN_ERR_CAPACITY
        n = max(sum(x for x in new if x > 0), 1)
        q, k = torch.ones((n, 4, 64), dtype=torch.bfloat16, device="cuda"), torch.ones((n, 2, 64), dtype=torch.bfloat16, device="cuda")
        out = torch.full_like(q, 7.0)
        gdn.gdn_kv_append(m.desc, m.cache, p, k, k)
        gdn.gdn_kv_attention(m.desc, m.cache, p, q, k, k, out, None, 64, 64)
        assert gdn.gdn_device_status() == gdn.GDN_OK and (out == 7.0).all()
        for n in names:
            assert torch.equal(kept[n], bits(n)), n

    refused([1, 0], [64, 128])                            # 3 pages of 2
    refused([0], [106])                                   # past max_blocks
    refused([3], [1])                                     # no such slot
    refused([-1], [1])
    refused([0, 1], [1, -1])
    refused([0, 1], [60, 64], gdn.KvPlan.new(1, 2))       # more units than the map holds
    m.step([0, 1], [1, 1])
    m.check_contents()


def test_bounds_smaller_than_the_batch_are_reported(cuda_device):
    """max_new or max_len below the plan's: the units outside are left out and the device status says so."""
    m = Model((4, 2), 64, BF)
    m.step([0], [600])
    q, k = m.draw(30, 4).cuda(), m.draw(30, 2).cuda()
    plan = gdn.KvPlan.new(30, 1)
    gdn.gdn_kv_plan(m.desc, m.cache, m.i32([0]), m.i32([30]), plan)
    ws = gdn.kv_attention_workspace(m.desc, 30, 1, 1000)
    for max_new, max_len, rows in ((3, 1000, 30), (30, 1000, 20)):
        out = torch.full_like(q, 7.0)
        gdn.gdn_kv_attention(m.desc, m.cache, plan, q[:rows].contiguous(), k[:rows].contiguous(), k[:rows].contiguous(),
                             out[:rows], ws, max_new, max_len)
        assert gdn.gdn_device_status() == gdn.GDN_ERR_INVALID_ARG
        assert gdn.gdn_device_status() == gdn.GDN_OK


def test_all_zero_blocks(cuda_device):
    m = Model((4, 2), 64, BF)
    z = lambda n, h: torch.zeros((n, h, 64), dtype=torch.bfloat16)   # noqa: E731
    m.step([0], [64], data=(m.draw(64, 4), z(64, 2), z(64, 2)))
    m.step([0], [3])
    m.check_contents()


@pytest.mark.parametrize("size", [1e-30, 1e30], ids=["tiny", "huge"])
@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "fp32"])
def test_scales_at_the_ends_of_the_range(cuda_device, dtype, size):
    """Values far from 1: the scales carry them (queries the other way, so that the scores stay ordinary)."""
    m = Model((4, 2), 64, dtype)
    f = lambda n, h, s: (torch.randn((n, h, 64), generator=m.gen) * s).to(torch.bfloat16 if dtype == BF else torch.float32)   # noqa: E731
    m.step([0], [100], data=(f(100, 4, 1 / size), f(100, 2, size), f(100, 2, size)))
    m.step([0], [1], data=(f(1, 4, 1 / size), f(1, 2, size), f(1, 2, size)))
    m.check_contents()


def test_a_captured_step_replays(cuda_device):
    """Plan, append and attention of single tokens in one CUDA graph: every replay advances the slots."""
    eager, graphed = Model((8, 2), 128, BF, seed=5), Model((8, 2), 128, BF, seed=5)
    for m in (eager, graphed):
        m.step([0, 1], [126, 63])
    slots, ones = graphed.i32([1, 0]), graphed.i32([1, 1])
    plan = gdn.KvPlan.new(2, 2)
    q, k, v = (torch.zeros((2, h, 128), dtype=torch.bfloat16, device="cuda") for h in (8, 2, 2))
    out = torch.empty_like(q)
    ws = gdn.kv_attention_workspace(graphed.desc, 2, 2, 1024)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        gdn.gdn_kv_plan(graphed.desc, graphed.cache, slots, ones, plan)
        gdn.gdn_kv_append(graphed.desc, graphed.cache, plan, k, v)
        gdn.gdn_kv_attention(graphed.desc, graphed.cache, plan, q, k, v, out, ws, 1, 1024)
    for _ in range(5):
        data = [eager.draw(2, h) for h in (8, 2, 2)]
        want = eager.step([1, 0], [1, 1], data=data, max_len=1024)
        for dst, src in zip((q, k, v), data):
            dst.copy_(src)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)
    graphed.slots = eager.slots
    graphed.check_contents()


def test_other_streams(cuda_device):
    """The calls run on the stream that they are given."""
    a, b = Model((8, 2), 128, BF, seed=6), Model((8, 2), 128, BF, seed=6)
    side = torch.cuda.Stream()
    for new in (100, 1):
        data = [a.draw(new, h) for h in (8, 2, 2)]
        want = a.step([0], [new], data=data)
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            got = b.step([0], [new], data=data)
        side.synchronize()
        assert torch.equal(got, want)


@pytest.mark.parametrize("d", [64, 128, 256])
def test_wait_timeout_is_reported_and_context_survives(cuda_device, d):
    """The tcgen05 attention's waits are bounded: with its first key tile never announced they run out, the status says
    so, and the next call is right."""
    m = Model((8, 2), d, BF, seed=8)
    gdn.gdn_debug_inject_wait_timeout(3, 2000)
    try:
        q, k = m.draw(300, 8).cuda(), m.draw(300, 2).cuda()
        plan, out = gdn.KvPlan.new(300, 1), torch.zeros_like(q)
        gdn.gdn_kv_plan(m.desc, m.cache, m.i32([4]), m.i32([300]), plan)
        gdn.gdn_kv_append(m.desc, m.cache, plan, k, k)
        gdn.gdn_kv_attention(m.desc, m.cache, plan, q, k, k, out, None, 300, 300)
        status = gdn.gdn_device_status()
    finally:
        gdn.gdn_debug_inject_wait_timeout(0)
    assert status == gdn.GDN_ERR_TIMEOUT
    assert gdn.gdn_device_status() == gdn.GDN_OK
    m.step([1], [200])


def test_many_sessions_share_the_gpu(cuda_device):
    """So many (session, head) chains of tokens that a CTA takes several segments of one: the bits of a few sessions alone."""
    n, heads, d = 40, (64, 64), 64
    m, one = (Model(heads, d, BF, n_pages=40 * 75, n_slots=n, max_blocks=80, seed=2) for _ in range(2))
    lens = [4700 if i % 3 == 0 else 64 * i + 5 for i in range(n)]
    g = torch.Generator(device="cuda").manual_seed(1)
    mk = lambda k, h: torch.randn((k, h, d), generator=g, device="cuda").to(torch.bfloat16)   # noqa: E731

    def run(model, slots, new, q, k, v, max_len):
        plan = gdn.KvPlan.new(sum(new), len(slots))
        gdn.gdn_kv_plan(model.desc, model.cache, model.i32(slots), model.i32(new), plan)
        gdn.gdn_kv_append(model.desc, model.cache, plan, k, v)
        out = torch.full((sum(new), heads[0], d), 7.0, dtype=torch.bfloat16, device="cuda")
        if q is not None:
            ws = gdn.kv_attention_workspace(model.desc, sum(new), len(slots), max_len)
            gdn.gdn_kv_attention(model.desc, model.cache, plan, q, k, v, out, ws, max(new), max_len)
        assert gdn.gdn_kv_status(plan) == gdn.GDN_OK and gdn.gdn_device_status() == gdn.GDN_OK
        return out

    k, v = mk(sum(lens), 64), mk(sum(lens), 64)
    run(m, list(range(n)), lens, None, k, v, 5000)
    row = 0
    for i in (0, 1, 39):
        row = sum(lens[:i])
        run(one, [i], [lens[i]], None, k[row:row + lens[i]].contiguous(), v[row:row + lens[i]].contiguous(), 5000)
    q, k, v = mk(n, 64), mk(n, 64), mk(n, 64)
    out = run(m, list(range(n)), [1] * n, q, k, v, 5000)
    assert torch.isfinite(out).all()
    for i in (0, 1, 39):
        assert torch.equal(run(one, [i], [1], *(t[i:i + 1].contiguous() for t in (q, k, v)), 5000)[0], out[i])


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "fp32"])
def test_pages_past_two_gigabytes(cuda_device, dtype):
    """A pool of more than 2^31 bytes of keys whose last pages are handed out first: append, prompt and single tokens."""
    n_pages = 2 ** 31 // (8 * 64 * 256) + 40
    m = Model((8, 8), 256, dtype, n_pages=n_pages, n_slots=2, max_blocks=16)
    m.cache.free.copy_(torch.arange(n_pages, dtype=torch.int32, device=cuda_device))
    m.step([1, 0], [130, 70])
    m.step([0, 1], [1, 1])
    m.step([1], [70])
    assert int(m.cache.table[1, 0]) * 8 * 64 * 256 > 2 ** 31


def test_the_example_serves_a_conversation(cuda_device):
    """The hybrid block of examples/: prompt turns, a fork and graph replays equal to eager steps."""
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.abspath(__file__)), "..", "examples", "hybrid_session.py")
    spec = importlib.util.spec_from_file_location("hybrid_session", path)
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    diff, _ = example.run(turn=192, branches=3, steps=70, device=cuda_device)
    assert diff == 0.0

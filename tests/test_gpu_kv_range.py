"""Attention over the 8-bit cache where its values, weights or queries are of very unequal size, against the bounds of
kv_bounds.py."""
import pytest
import torch

from chunked_gated_deltanet_gb300 import gdn
from kv_bounds import Bounded
from kv_ref import TORCH

pytestmark = pytest.mark.gpu

BF, F32 = gdn.GDN_BF16, gdn.GDN_FP32
DTYPES = pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "fp32"])
FORMS = pytest.mark.parametrize("n", [2, 40], ids=["few", "many"])
DIMS = pytest.mark.parametrize("d", [64, 128, 256])


def fill(m, k, v):
    """The keys and values of slot 0, without a look at the outputs."""
    q = torch.zeros((k.shape[0], m.hq, m.d), dtype=k.dtype)
    m.step([0], [k.shape[0]], check=False, data=(q, k, v))


@FORMS
@DIMS
@pytest.mark.parametrize("zeros", [1, 12], ids=["one zero block", "twelve"])
def test_small_values_after_blocks_of_zeros(cuda_device, d, n, zeros):
    """A prefix whose values are all zero has no scale of its own to hold the others to."""
    m = Bounded((8, 2), d, BF, seed=21)
    a, b = 64 * zeros, 300
    v = m.draw(a + b, 2, 1e-6)
    v[:a] = 0
    fill(m, m.draw(a + b, 2), v)
    m.step([0], [n], q_size=2.0, data=(m.draw(n, 8, 2.0), m.draw(n, 2), m.draw(n, 2, 1e-6)))
    m.check_contents()


PATTERNS = {"grows": [0, 0, 1, 1, 1, 1], "falls": [1, 1, 0, 0, 0, 0], "alternates": [0, 1, 0, 1, 1, 0],
            "one large": [0, 0, 0, 1, 0, 0], "last large": [0, 0, 0, 0, 0, 1], "last small": [1, 1, 1, 1, 1, 0]}


@FORMS
@DTYPES
@pytest.mark.parametrize("ratio", [12, 20, 30, 80], ids=lambda r: f"2^{r}")
@pytest.mark.parametrize("pattern", PATTERNS)
def test_blocks_of_unequal_values(cuda_device, pattern, ratio, dtype, n):
    """Values of blocks (and of the open block) that are 2^ratio apart, in one column of the large ones only, so that every
    other column is the small ones' alone."""
    m = Bounded((4, 2), 128, dtype, seed=22)
    sizes = PATTERNS[pattern]
    v = m.draw(320, 2)
    for b, big in enumerate(sizes[:5]):
        rows = v[64 * b:64 * b + 64]
        if big:
            keep = rows[:, :, 3].clone()
            rows.zero_()
            rows[:, :, 3] = keep * 2.0 ** ratio
    fill(m, m.draw(320, 2), v)
    own = m.draw(n, 2)
    if sizes[5]:
        own[:, :, 3] *= 2.0 ** ratio
    m.step([0], [n], data=(m.draw(n, 4, 2.0), m.draw(n, 2), own))


@FORMS
@DIMS
def test_an_own_block_far_from_the_cache(cuda_device, d, n):
    """Values near the ends of the range: the cache's tiny and the open block's huge, and the other way round."""
    for cached, own in ((1e-12, 1e12), (1e12, 1e-12)):
        m = Bounded((8, 2), d, BF, seed=23)
        fill(m, m.draw(200, 2), m.draw(200, 2, cached))
        m.step([0], [n], data=(m.draw(n, 8, 2.0), m.draw(n, 2), m.draw(n, 2, own)))


@FORMS
@DIMS
@pytest.mark.parametrize("lead", [6.0, 14.0], ids=["e^6", "e^14"])
def test_a_first_token_that_takes_the_weight(cuda_device, d, n, lead):
    """An attention sink: the first key has e^lead times the weight of the others and a value of zero, so that the output
    is what the small weights sum to."""
    m = Bounded((4, 1), d, BF, seed=24)
    q = m.draw(n, 4, 0.3)
    q[:, :, 0] = 1.0
    k, v = m.draw(500, 1, 0.3), m.draw(500, 1)
    k[:, :, 0] = 0.0
    k[0] = 0.0
    k[0, :, 0] = lead * d ** 0.5
    v[0] = 0.0
    fill(m, k, v)
    m.step([0], [n], data=(q, m.draw(n, 1, 0.3), m.draw(n, 1)))


@FORMS
@DIMS
@pytest.mark.parametrize("mean", [3.0, 10.0])
@pytest.mark.parametrize("channel", [1.0, 30.0], ids=["even keys", "one large channel"])
def test_queries_with_a_common_offset(cuda_device, d, n, mean, channel):
    """Queries whose sum is far from zero, over complete blocks and the open one, with keys of one size and with a channel
    that sets the blocks' scales."""
    m = Bounded((8, 2), d, BF, seed=25)
    k = m.draw(400, 2)
    k[:, :, 5] *= channel
    fill(m, k, m.draw(400, 2))
    q = m.draw(n, 8) + mean
    if channel > 1:
        q[:, :, 5] = m.draw(n, 8)[:, :, 5]
    own = m.draw(n, 2)
    own[:, :, 5] *= channel
    m.step([0], [n], data=(q.to(TORCH[BF]), own, m.draw(n, 2)))


@DTYPES
@pytest.mark.parametrize("heads", [(4, 4), (8, 1), (16, 1)], ids=lambda h: f"{h[0]}q{h[1]}kv")
@DIMS
def test_ordinary_rows_keep_the_stated_bounds(cuda_device, d, heads, dtype):
    """Sharp and flat rows, prompts and single tokens, within the bounds of the arithmetic that the library states."""
    m = Bounded(heads, d, dtype, seed=26)
    m.step([0, 1], [200, 45], q_size=3.0)
    m.step([0, 1], [1, 30], q_size=1.0)
    m.step([1, 0], [1, 1], q_size=4.0)


@pytest.mark.parametrize("heads", [(2, 2), (12, 2)], ids=lambda h: f"{h[0]}q{h[1]}kv")
@DIMS
def test_unequal_values_do_not_depend_on_the_split(cuda_device, d, heads):
    """Rows of the many-row form are the same bits however the session was cut into calls, blocks of any size beside and
    after theirs."""
    g = torch.Generator().manual_seed(27)
    n = 450
    q, k, v = (torch.randn((n, h, d), generator=g).to(torch.bfloat16) for h in (heads[0], 2, 2))
    for b, e in enumerate((0, 25, -10, 3, 40, -30, 0, 20)):
        v[64 * b:64 * b + 64] *= 2.0 ** e
    v[64:128, :, 1:] = 0
    v[320:384] = 0
    outs = []
    for cuts in ([0, n], [0, 100, 200, n], [0, 64, 128, 150, 256, 300, n]):
        m = Bounded(heads, d, BF)
        outs.append(torch.cat([m.step([1], [b - a], check=False, data=(q[a:b], k[a:b], v[a:b]))
                               for a, b in zip(cuts, cuts[1:])]))
        m.check_contents()
    for o in outs[1:]:
        assert torch.equal(o, outs[0])


@DTYPES
@pytest.mark.parametrize("heads,n", [((4, 2), 3), ((4, 2), 90), ((2, 2), 200)], ids=["few", "many", "many, one head a group"])
def test_a_length_past_max_len_is_reported(cuda_device, heads, n, dtype):
    """max_len below a slot's length, inside the last segment too: the blocks' rows past it are left out and the status says
    so; the rows of the blocks before it, and those of the other request, are there."""
    m = Bounded(heads, 64, dtype)
    m.step([0, 1], [600, 30])
    q, k = m.draw(2 * n, heads[0]).to(cuda_device), m.draw(2 * n, 2).to(cuda_device)
    plan = gdn.KvPlan.new(2 * n, 2)
    gdn.gdn_kv_plan(m.desc, m.cache, m.i32([0, 1]), m.i32([n, n]), plan)
    gdn.gdn_kv_append(m.desc, m.cache, plan, k, k)
    assert gdn.gdn_device_status() == gdn.GDN_OK
    ws = gdn.kv_attention_workspace(m.desc, 2 * n, 2, 600 + n)

    def attend(max_len):
        out = torch.full_like(q, 7.0)
        gdn.gdn_kv_attention(m.desc, m.cache, plan, q, k, k, out, ws, n, max_len)
        return out, gdn.gdn_device_status()

    want, status = attend(600 + n)
    assert status == gdn.GDN_OK and not (want == 7.0).all(2).any()
    for short in (599 + n, 599 + n // 2, 300):
        out, status = attend(short)
        assert status == gdn.GDN_ERR_INVALID_ARG and gdn.gdn_device_status() == gdn.GDN_OK
        assert torch.equal(out[n:], want[n:])
        kept = sum(min(n, b + 64 - 600) - max(0, b - 600) for b in range(576, 600 + n, 64) if min(b + 64, 600 + n) <= short)
        assert torch.equal(out[:kept], want[:kept]) and (out[kept:n] == 7.0).all()


@pytest.mark.parametrize("max_new", [64, 40])
@pytest.mark.parametrize("d", [64, 256])
def test_rows_past_max_new_are_right_or_left_out(cuda_device, d, max_new):
    """A request of more than max_new tokens, over several segments, with blocks that share a tile: a row is what it is with
    the right bound, or untouched and reported."""
    m = Bounded((2, 2), d, BF, n_pages=80, n_slots=1, max_blocks=80)
    m.step([0], [4480 + 30], check=False)
    n = 200
    q, k = m.draw(n, 2).to(cuda_device), m.draw(n, 2).to(cuda_device)
    plan = gdn.KvPlan.new(n, 1)
    gdn.gdn_kv_plan(m.desc, m.cache, m.i32([0]), m.i32([n]), plan)
    gdn.gdn_kv_append(m.desc, m.cache, plan, k, k)
    ws = gdn.kv_attention_workspace(m.desc, n, 1, 5000)
    outs = []
    for bound in (n, max_new):
        ws.fill_(0xFF)     # NaN in what no segment writes
        out = torch.full_like(q, 7.0)
        gdn.gdn_kv_attention(m.desc, m.cache, plan, q, k, k, out, ws, bound, 5000)
        outs.append((out, gdn.gdn_device_status()))
    (want, ok), (out, status) = outs
    assert ok == gdn.GDN_OK and torch.isfinite(want).all()
    right, untouched = (out == want).all(2).all(1), (out == 7.0).all(2).all(1)
    assert (right | untouched).all()
    assert status == (gdn.GDN_ERR_INVALID_ARG if untouched.any() else gdn.GDN_OK)


def test_many_heads_and_tokens_in_the_few_row_form(cuda_device):
    """4,096 heads and 16 tokens over two segments, 65,536 rows to join for one block: every head as it is beside 7 others."""
    H, n, ctx = 4096, 16, 530
    g = torch.Generator(device=cuda_device).manual_seed(31)
    mk = lambda k: torch.randn((k, H, 64), generator=g, device=cuda_device)   # noqa: E731
    k0, q, k, v = mk(ctx), mk(n), mk(n), mk(n)

    def run(h0, heads):
        desc = gdn.make_attn_desc(heads, heads, 64, F32)
        cache, plan = gdn.KvCache(desc, 9, 1, 9, cuda_device), gdn.KvPlan.new(ctx, 1)
        cut = lambda t: t[:, h0:h0 + heads].contiguous()   # noqa: E731
        one = lambda c: torch.tensor([c], dtype=torch.int32, device=cuda_device)   # noqa: E731
        gdn.gdn_kv_plan(desc, cache, one(0), one(ctx), plan)
        gdn.gdn_kv_append(desc, cache, plan, cut(k0), cut(k0))
        gdn.gdn_kv_plan(desc, cache, one(0), one(n), plan)
        gdn.gdn_kv_append(desc, cache, plan, cut(k), cut(v))
        out = torch.zeros((n, heads, 64), device=cuda_device)
        ws = gdn.kv_attention_workspace(desc, n, 1, ctx + n)
        gdn.gdn_kv_attention(desc, cache, plan, cut(q), cut(k), cut(v), out, ws, n, ctx + n)
        assert gdn.gdn_kv_status(plan) == gdn.GDN_OK and gdn.gdn_device_status() == gdn.GDN_OK
        return out

    out = run(0, H)
    for h0 in (0, 2040, H - 8):
        assert torch.equal(out[:, h0:h0 + 8], run(h0, 8))


@DTYPES
@pytest.mark.parametrize("heads,d", [((8, 2), 128), ((2, 2), 64), ((8, 1), 256)], ids=["8q2kv-128", "2q2kv-64", "8q1kv-256"])
def test_segments_of_unequal_values_are_joined(cuda_device, heads, d, dtype):
    """Contexts over several segments whose blocks' values are of any size from 2^-30 to 2^30, some zero: few rows and many."""
    m = Bounded(heads, d, dtype, n_pages=80, n_slots=1, max_blocks=80, seed=28)
    ctx = 4410
    v = m.draw(ctx, heads[1])
    e = torch.randint(-30, 31, (ctx // 64 + 1,), generator=m.gen)
    v = (v.float() * 2.0 ** e.repeat_interleave(64)[:ctx, None, None]).to(v.dtype)
    v[640:1280] = 0
    fill(m, m.draw(ctx, heads[1]), v)
    for n in (2, 70):
        m.step([0], [n], data=(m.draw(n, heads[0], 2.0), m.draw(n, heads[1]), m.draw(n, heads[1], 2.0 ** int(e[n % 64]))))

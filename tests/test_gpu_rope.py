"""Rotary positions with the per-head norm, against the formula in 64 bits.

Bound of an element, with (a, b) its pair after the norm and m the magnitude: the angle in half turns is rounded to fp32
(2^-24, so pi 2^-24 of the angle) after a truncation of 2^-31, cos and sin are off by 2^-23 more, their products and sum by
three roundings: (3.2 + 2 + 3) 2^-24 < 2^-20 of m (|a| + |b|). The norm: a sum of d squares, 16 in a row and 5 joined, a mean,
a root, a division and two products, (21 / 2 + 6) 2^-24 < 2^-19 of each. bf16 adds half a step, 2^-8 of the result."""
import math

import numpy as np
import pytest
import torch

from chunked_gated_deltanet_gb300 import gdn
from kv_ref import Model, TORCH

pytestmark = pytest.mark.gpu

BF, F32 = gdn.GDN_BF16, gdn.GDN_FP32
HALF, INTER = gdn.GDN_ROPE_HALF, gdn.GDN_ROPE_INTERLEAVED
both = pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "fp32"])


def paces(r):
    f = [math.exp(-2 * i / r.rotary_dim * math.log(r.base)) for i in range(r.rotary_dim // 2)]
    if r.scaling == gdn.GDN_ROPE_LINEAR:
        f = [x / r.factor for x in f]
    elif r.scaling == gdn.GDN_ROPE_PARTS:
        keep = [min(1.0, max(0.0, (r.original_len * x / (2 * math.pi) - r.beta_slow) / (r.beta_fast - r.beta_slow))) for x in f]
        f = [c * x + (1 - c) * x / r.factor for c, x in zip(keep, f)]
    return np.array(f)


def turned(x, pos, r, weight, dtype):
    """x fp64 [n][heads][d] -> the rows turned, and their bound."""
    rd, h = r.rotary_dim, r.rotary_dim // 2
    e = np.zeros_like(x)
    if weight is not None:
        x = x / np.sqrt((x * x).mean(2, keepdims=True) + r.eps) * weight
        e = 2.0 ** -19 * np.abs(x)
    angle = np.asarray(pos, np.float64)[:, None, None] * paces(r)
    cos, sin = np.cos(angle) * r.magnitude, np.sin(angle) * r.magnitude
    one, two = (slice(0, h), slice(h, rd)) if r.layout == HALF else (slice(0, rd, 2), slice(1, rd, 2))
    a, b = x[..., one], x[..., two]
    y = x.copy()
    y[..., one], y[..., two] = a * cos - b * sin, a * sin + b * cos
    both_ = (np.abs(a) + np.abs(b)) * r.magnitude
    turn = 2.0 ** -20 * both_ + (e[..., one] + e[..., two]) * r.magnitude
    e[..., one] = e[..., two] = turn
    if dtype == BF:
        e = e + 2.0 ** -8 * (np.abs(y) + e)
    return y, e


def check(got, ref, bound):
    err = np.abs(got.double().cpu().numpy() - ref)
    assert (err <= bound + 1e-30).all(), float((err / (bound + 1e-30)).max())


def run(heads, d, dtype, r, pos, norm=True, with_v=True, packed=True, seed=0, in_place=False):
    hq, hkv = heads
    n = len(pos)
    gen = torch.Generator().manual_seed(seed)
    draw = lambda *s: torch.randn(s, generator=gen).to(TORCH[dtype]).cuda()   # noqa: E731
    if packed:
        q, k, v = draw(n, hq + 2 * hkv, d).split([hq, hkv, hkv], 1)
    else:
        q, k, v = draw(n, hq, d), draw(n, hkv, d), draw(n, hkv, d)
    wq, wk = (1 + 0.3 * draw(d), 1 + 0.3 * draw(d)) if norm else (None, None)
    refs = [turned(x.double().cpu().numpy(), pos, r, None if w is None else w.double().cpu().numpy(), dtype)
            for x, w in ((q, wq), (k, wk))]
    v_was = v.clone()
    outs = (q, k, v) if in_place else tuple(torch.full(x.shape, 7, dtype=x.dtype, device="cuda") for x in (q, k, v))
    desc = gdn.make_attn_desc(hq, hkv, d, dtype)
    table = gdn.rope_table(r)
    positions = torch.tensor(pos, dtype=torch.int32, device="cuda")
    gdn.gdn_rope(desc, r, table, positions, q, k, outs[0], outs[1], v if with_v else None, outs[2] if with_v else None, wq, wk)
    for o, (ref, bound) in zip(outs, refs):
        check(o, ref, bound)
    assert torch.equal(outs[2], v_was) if with_v else (outs[2] == (v_was if in_place else 7)).all()
    return outs


@both
@pytest.mark.parametrize("layout", [HALF, INTER], ids=["half", "interleaved"])
@pytest.mark.parametrize("d,rd", [(64, 64), (64, 16), (128, 128), (128, 48), (256, 64), (256, 256), (256, 176)])
def test_layouts_and_parts_of_the_head(cuda_device, d, rd, layout, dtype):
    pos = [0, 1, 2, 63, 64, 41802, 1000003]
    for heads in ((1, 1), (6, 2), (16, 8)):
        for norm in (True, False):
            run(heads, d, dtype, gdn.make_rope_desc(rd, layout, 1e4), pos, norm=norm, packed=norm, seed=rd)


@pytest.mark.parametrize("kw", [dict(scaling=gdn.GDN_ROPE_LINEAR, factor=8.0),
                                dict(scaling=gdn.GDN_ROPE_PARTS, factor=16.0, original_len=4096, magnitude=0.1 * math.log(16) + 1),
                                dict(scaling=gdn.GDN_ROPE_PARTS, factor=4.0, original_len=32768, beta_fast=8.0, beta_slow=0.5),
                                dict(base=1.0), dict(base=1e7), dict(magnitude=0.25)])
def test_scalings(cuda_device, kw):
    for layout in (HALF, INTER):
        run((4, 2), 128, F32, gdn.make_rope_desc(96, layout, **kw), [0, 5, 4096, 131072, 999999], norm=False)


def test_far_positions(cuda_device):
    """Angles at the largest positions: p 2^-53 turns of the table's double precision, 2 pi 2^-22 of an angle at 2^31."""
    r = gdn.make_rope_desc(64, HALF, 1e4)
    pos = [2 ** 31 - 1, 2 ** 30 + 12345, 2 ** 24 + 1]
    x = torch.zeros((3, 2, 64), device="cuda")
    x[:, :, :32] = 1.0
    desc = gdn.make_attn_desc(2, 2, 64, F32)
    out, k = torch.empty_like(x), torch.empty_like(x)
    gdn.gdn_rope(desc, r, gdn.rope_table(r), torch.tensor(pos, dtype=torch.int32, device="cuda"), x, x.clone(), out, k)
    # the angle modulo a turn, from rational arithmetic
    from fractions import Fraction
    turn = Fraction("6.28318530717958647692528676655900576839433879875021")
    want = np.zeros((3, 2, 64))
    for i, p in enumerate(pos):
        for j in range(32):
            f = Fraction(math.exp(-2 * j / 64 * math.log(1e4))) if j else Fraction(1)
            t = float((p * f / turn) % 1) * 2 * math.pi
            want[i, :, j], want[i, :, 32 + j] = math.cos(t), math.sin(t)
    # the reference's own pace is off by 2^-52 and more of exp, as the table's: 4 times p 2^-53 of a turn
    bound = np.array([2.0 ** -20 + 4 * p * 2.0 ** -53 * 2 * math.pi for p in pos])[:, None, None]
    assert (np.abs(out.double().cpu().numpy() - want) <= bound).all()


@both
@pytest.mark.parametrize("n", [1, 2, 7, 300, 5000])
def test_rows_of_every_number(cuda_device, n, dtype):
    """From one row, whose heads go to many warps, to many rows."""
    rs = np.random.RandomState(n)
    run((10, 2), 128, dtype, gdn.make_rope_desc(64, HALF, 5e5), rs.randint(0, 200000, n).tolist(), seed=n)


@both
def test_in_place(cuda_device, dtype):
    for layout in (HALF, INTER):
        run((4, 2), 256, dtype, gdn.make_rope_desc(64, layout), [3, 100, 70000], packed=False, in_place=True)


def test_negative_positions_leave_rows(cuda_device):
    desc, r = gdn.make_attn_desc(4, 2, 64, BF), gdn.make_rope_desc(64)
    q, k = (torch.randn((3, h, 64), device="cuda").bfloat16() for h in (4, 2))
    qo, ko = torch.full_like(q, 7), torch.full_like(k, 7)
    gdn.gdn_rope(desc, r, gdn.rope_table(r), torch.tensor([0, -1, 0], dtype=torch.int32, device="cuda"), q, k, qo, ko)
    assert torch.equal(qo[[0, 2]], q[[0, 2]]) and (qo[1] == 7).all() and (ko[1] == 7).all()


def test_a_norm_of_one_side(cuda_device):
    """Weights for the queries alone: the keys are turned as they came."""
    desc, r = gdn.make_attn_desc(4, 2, 128, F32), gdn.make_rope_desc(128)
    q, k = torch.randn((5, 4, 128), device="cuda"), torch.randn((5, 2, 128), device="cuda")
    w = torch.rand(128, device="cuda")
    pos = [9, 8, 7, 6, 1 << 20]
    p = torch.tensor(pos, dtype=torch.int32, device="cuda")
    for a, b in ((w, None), (None, w)):
        qo, ko = torch.empty_like(q), torch.empty_like(k)
        gdn.gdn_rope(desc, r, gdn.rope_table(r), p, q, k, qo, ko, q_weight=a, k_weight=b)
        for x, y, wt in ((q, qo, a), (k, ko, b)):
            check(y, *turned(x.double().cpu().numpy(), pos, r, None if wt is None else wt.double().cpu().numpy(), F32))


def test_rows_that_are_not_finite_keep_to_themselves(cuda_device):
    desc, r = gdn.make_attn_desc(2, 1, 64, BF), gdn.make_rope_desc(32)
    q, k, w = torch.ones((3, 2, 64), device="cuda").bfloat16(), torch.ones((3, 1, 64), device="cuda").bfloat16(), torch.ones(64, device="cuda").bfloat16()
    q[1, 0, 5] = float("nan")
    qo, ko = torch.empty_like(q), torch.empty_like(k)
    gdn.gdn_rope(desc, r, gdn.rope_table(r), torch.tensor([1, 2, 3], dtype=torch.int32, device="cuda"), q, k, qo, ko, q_weight=w, k_weight=w)
    assert qo[1, 0].isnan().all() and qo[[0, 2]].isfinite().all() and qo[1, 1].isfinite().all() and ko.isfinite().all()


def test_positions_of_a_plan(cuda_device):
    """Rows of prompts and single tokens, and rows past the plan's."""
    m = Model((2, 1), 64, BF, n_slots=5, max_blocks=16, seed=1)
    m.step([0, 1, 4], [130, 63, 1], check=False)
    slots, new = [1, 3, 0, 2, 4], [1, 70, 200, 0, 66]
    plan = gdn.KvPlan.new(sum(new), 5, m.dev)
    gdn.gdn_kv_plan(m.desc, m.cache, m.i32(slots), m.i32(new), plan)
    got = torch.full((sum(new) + 3,), 7, dtype=torch.int32, device=m.dev)
    gdn.gdn_kv_positions(plan, got)
    want = [p for s, k in zip(slots, new) for p in range(len(m.slots[s].k), len(m.slots[s].k) + k)] + [-1] * 3
    assert got.tolist() == want
    gdn.gdn_kv_plan(m.desc, m.cache, m.i32(slots), m.i32([0, 0, 10 ** 6, 0, 0]), plan)     # does not fit: no rows
    gdn.gdn_kv_positions(plan, got)
    assert (got == -1).all()


def test_scores_depend_on_distances(cuda_device):
    """Turned queries and keys of one distance have one product, wherever they stand."""
    desc, r = gdn.make_attn_desc(1, 1, 128, F32), gdn.make_rope_desc(128, base=1e6)
    q, k = torch.randn((1, 1, 128), device="cuda"), torch.randn((1, 1, 128), device="cuda")
    starts = [0, 1, 777, 123456, 16000000]
    pos = torch.tensor([s + 40 for s in starts], dtype=torch.int32, device="cuda")
    base = torch.tensor(starts, dtype=torch.int32, device="cuda")
    n = len(starts)
    qq, kk = q.expand(n, 1, 128).contiguous(), k.expand(n, 1, 128).contiguous()
    qo, ko, x = (torch.empty_like(qq) for _ in range(3))
    table = gdn.rope_table(r)
    gdn.gdn_rope(desc, r, table, pos, qq, kk, qo, x)
    gdn.gdn_rope(desc, r, table, base, qq, kk, x, ko)
    s = (qo.double() * ko.double()).sum((1, 2))
    # each side's elements are off by 2^-20 (|a| + |b|): twice 2 sqrt(2) 2^-20 |q| |k| of the product
    tol = 2 * 2 * math.sqrt(2) * 2.0 ** -20 * float(q.norm() * k.norm())
    assert float((s - s[0]).abs().max()) <= 2 * tol


def test_on_another_stream_and_captured(cuda_device):
    desc, r = gdn.make_attn_desc(4, 2, 128, BF), gdn.make_rope_desc(64, INTER)
    q, k = torch.randn((9, 4, 128), device="cuda").bfloat16(), torch.randn((9, 2, 128), device="cuda").bfloat16()
    table, pos = gdn.rope_table(r), torch.arange(9, dtype=torch.int32, device="cuda") * 1000
    want = [torch.empty_like(q), torch.empty_like(k)]
    gdn.gdn_rope(desc, r, table, pos, q, k, *want)
    torch.cuda.synchronize()
    side, got = torch.cuda.Stream(), [torch.empty_like(q), torch.empty_like(k)]
    gdn.gdn_rope(desc, r, table, pos, q, k, *got, stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        gdn.gdn_rope(desc, r, table, pos, q, k, *got)
    pos += 1
    graph.replay()
    gdn.gdn_rope(desc, r, table, pos, q, k, *want)
    assert all(torch.equal(a, b) for a, b in zip(got, want))

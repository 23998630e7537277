// Rotary positions of queries and keys, with the per-head norm before them, and the rows' way out of a q/k/v product into
// contiguous arrays (declared in include/gdn.h).
//
// The mathematics, per row at position p and head: y = x w / sqrt(mean(x^2) + eps) where weights are given, else x; then
// for each pair i of the first rotary_dim elements ((i, i + rotary_dim / 2), or (2 i, 2 i + 1)) with angle a = p f_i
//   (y_0, y_1) -> magnitude (y_0 cos a - y_1 sin a, y_0 sin a + y_1 cos a),
// the other elements as they are. fp32 from the loaded values to the one rounding at the end.
//
// The angle is a whole number of 2^-64 turns: f_i / 2 pi as a 64-bit fraction (the table), times p modulo 2^64: one 64-bit
// product, without an error of its own at any position. Its upper 32 bits in units of half turns are what sincospi takes, in
// [-1, 1), rounded to fp32. Two errors are left: the table's, as it is made in fp64 (a power, two quotients, some 2^-50.2 of
// f_i / 2 pi <= 0.16 at worst), about p 2^-53 turns; and the fp32 argument's, 2^-26 turns whatever p is.
#include <cmath>

#include "common.cuh"
#include "gdn.h"
#include "host.h"

#include <algorithm>

using namespace gdn_host;

namespace gdn {

__global__ void rope_table_kernel(const gdn_rope_desc r, unsigned long long *table) {
    grid_dep_wait();
    grid_dep_launch();
    const int i = blockIdx.x * blockDim.x + threadIdx.x, half = r.rotary_dim / 2;
    if (i >= half) return;
    constexpr double kTurn = 6.283185307179586476925;
    double f = pow((double)r.base, -(double)i / half);
    if (r.scaling == GDN_ROPE_LINEAR) {
        f /= (double)r.factor;
    } else if (r.scaling == GDN_ROPE_PARTS) {
        const double turns = r.original_len * f / kTurn;
        const double keep = fmin(fmax((turns - (double)r.beta_slow) / ((double)r.beta_fast - (double)r.beta_slow), 0.0), 1.0);
        f = keep * f + (1.0 - keep) * (f / (double)r.factor);
    }
    const double turns = f / kTurn;
    table[i] = __double2ull_rn((turns - floor(turns)) * 18446744073709551616.0);
}

template <typename T> struct RopeVec;   // 16 bytes
template <> struct RopeVec<float> {
    static constexpr int N = 4;
    static __device__ __forceinline__ void get(const uint4 &u, float *f) {
        f[0] = __uint_as_float(u.x); f[1] = __uint_as_float(u.y); f[2] = __uint_as_float(u.z); f[3] = __uint_as_float(u.w);
    }
    static __device__ __forceinline__ uint4 put(const float *f) {
        return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
    }
};
template <> struct RopeVec<__nv_bfloat16> {
    static constexpr int N = 8;
    static __device__ __forceinline__ void get(const uint4 &u, float *f) {
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f[2 * i] = __uint_as_float(w[i] << 16);
            f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
    }
    static __device__ __forceinline__ uint4 put(const float *f) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __nv_bfloat162 p = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
            w[i] = *reinterpret_cast<const uint32_t *>(&p);
        }
        return make_uint4(w[0], w[1], w[2], w[3]);
    }
};

struct RopeArgs {
    const void *q, *k, *v;
    int64_t q_stride, k_stride, v_stride;   // elements between rows
    const void *q_weight, *k_weight;
    void *q_out, *k_out, *v_out;
    const int32_t *positions;
    const unsigned long long *table;
    int64_t n_rows;
    int Hq, Hkv, heads;                     // heads: Hq + Hkv, + Hkv with values
    int rotary_dim, interleaved;
    float magnitude, eps;
    int splits;                             // warps of a row
};

// A warp per row and share of its heads, LPH lanes a head, two 16-byte vectors a lane: the two that a lane's pairs lie in
// where it rotates (i and i + rotary_dim / 2: one of each half; neighbours: two in a row), any other two where not. So a
// lane's angles are the same for all heads of the row; the lanes of a column in the warp's HPW heads share them out, one
// sincospi a pair and row (all of them in every lane: 194 us on the case below).
// Bound: HBM, every element in and out once: 47,880 rows of 32 + 8 + 8 heads of 128, 186 us, 6.3 TB/s; 24,000 such rows in fp32
// 179 us, 6.6 TB/s, with the norm or without. One pass of heads at a time: with two under way it takes 215 us, with 5 CTAs an SM
// in place of 4 199, with 3 218. One row: 6 us in a graph, its heads over as many warps as they fill (three dependent reads:
// position, table, elements).
template <typename InT, int D>
__global__ void __launch_bounds__(256) rope_kernel(const RopeArgs a) {
    using V = RopeVec<InT>;
    constexpr int N = V::N, LPH = D / (2 * N), HPW = 32 / LPH;
    grid_dep_wait();
    grid_dep_launch();
    const int64_t task = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
    const int64_t row = task / a.splits;
    if (row >= a.n_rows) return;
    const int share = (int)(task - row * a.splits);
    const int pos = a.positions[row];
    if (pos < 0) return;
    const int lane = threadIdx.x & 31, t = lane % LPH, rot = a.rotary_dim / (2 * N);
    const bool turns = t < rot;
    // the lane's two vectors, in elements
    const int c0 = turns ? (a.interleaved ? 2 * t * N : t * N) : 2 * t * N;
    const int c1 = turns && !a.interleaved ? c0 + a.rotary_dim / 2 : c0 + N;
    // the lanes of a pair's column in the HPW heads share out its N angles
    constexpr int kOwn = N / HPW;
    float cs[N], sn[N], own_cs[kOwn], own_sn[kOwn];
#pragma unroll
    for (int i = 0; i < kOwn; ++i) {
        own_cs[i] = own_sn[i] = 0.f;
        if (turns) {
            const unsigned long long phase = (unsigned long long)pos * a.table[t * N + lane / LPH * kOwn + i];
            sincospif((float)(int)(phase >> 32) * 0x1p-31f, &own_sn[i], &own_cs[i]);
        }
    }
#pragma unroll
    for (int i = 0; i < N; ++i) {
        cs[i] = __shfl_sync(0xffffffffu, own_cs[i % kOwn], i / kOwn * LPH + t) * a.magnitude;
        sn[i] = __shfl_sync(0xffffffffu, own_sn[i % kOwn], i / kOwn * LPH + t) * a.magnitude;
    }
    const int step = HPW * a.splits;
#pragma unroll 1
    for (int h0 = share * HPW; h0 < a.heads; h0 += step) {
        const int h = h0 + lane / LPH;
        const bool live = h < a.heads;
        const int kind = h < a.Hq ? 0 : h < a.Hq + a.Hkv ? 1 : 2;
        const int hh = kind == 0 ? h : kind == 1 ? h - a.Hq : h - a.Hq - a.Hkv;
        const InT *src = static_cast<const InT *>(kind == 0 ? a.q : kind == 1 ? a.k : a.v) +
                         row * (kind == 0 ? a.q_stride : kind == 1 ? a.k_stride : a.v_stride) + hh * D;
        InT *dst = static_cast<InT *>(kind == 0 ? a.q_out : kind == 1 ? a.k_out : a.v_out) +
                   (row * (kind == 0 ? a.Hq : a.Hkv) + hh) * D;
        uint4 w0 = make_uint4(0, 0, 0, 0), w1 = w0;
        if (live) {
            w0 = *reinterpret_cast<const uint4 *>(src + c0);
            w1 = *reinterpret_cast<const uint4 *>(src + c1);
        }
        float x[2 * N];
        V::get(w0, x);
        V::get(w1, x + N);
        const InT *weight = static_cast<const InT *>(kind == 0 ? a.q_weight : kind == 1 ? a.k_weight : nullptr);
        if (a.q_weight || a.k_weight) {
            float sum = 0.f;
#pragma unroll
            for (int i = 0; i < 2 * N; ++i) sum = fmaf(x[i], x[i], sum);
#pragma unroll
            for (int o = 1; o < LPH; o <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
            if (weight) {
                const float r = 1.f / sqrtf(sum * (1.f / D) + a.eps);
                float w[2 * N];
                V::get(__ldg(reinterpret_cast<const uint4 *>(weight + c0)), w);
                V::get(__ldg(reinterpret_cast<const uint4 *>(weight + c1)), w + N);
#pragma unroll
                for (int i = 0; i < 2 * N; ++i) x[i] = x[i] * r * w[i];
            }
        }
        if (turns && kind < 2) {
            float y[2 * N];
            if (a.interleaved) {
#pragma unroll
                for (int i = 0; i < N; ++i) {
                    y[2 * i] = x[2 * i] * cs[i] - x[2 * i + 1] * sn[i];
                    y[2 * i + 1] = x[2 * i] * sn[i] + x[2 * i + 1] * cs[i];
                }
            } else {
#pragma unroll
                for (int i = 0; i < N; ++i) {
                    y[i] = x[i] * cs[i] - x[N + i] * sn[i];
                    y[N + i] = x[i] * sn[i] + x[N + i] * cs[i];
                }
            }
#pragma unroll
            for (int i = 0; i < 2 * N; ++i) x[i] = y[i];
        }
        if (live) {
            *reinterpret_cast<uint4 *>(dst + c0) = kind == 2 || (!weight && !turns) ? w0 : V::put(x);
            *reinterpret_cast<uint4 *>(dst + c1) = kind == 2 || (!weight && !turns) ? w1 : V::put(x + N);
        }
    }
}

// Position of each packed row of a plan, -1 of a row in no unit: the unit by bisection, as units are in row order.
__global__ void __launch_bounds__(256) kv_positions_kernel(const int32_t *units, const int32_t *counts, int max_units, int64_t n_rows,
                                                           int32_t *positions) {
    grid_dep_wait();
    grid_dep_launch();
    const int64_t row = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (row >= n_rows) return;
    int lo = 0, hi = min(counts[0], max_units);
    while (lo < hi) {   // the first unit after the row
        const int mid = (lo + hi) >> 1;
        if (units[8 * (int64_t)mid + 5] <= row) lo = mid + 1;
        else hi = mid;
    }
    int pos = -1;
    if (lo > 0) {
        const int32_t *u = units + 8 * (int64_t)(lo - 1);
        const int64_t off = row - u[5];
        if (off >= 0 && off < u[4]) pos = u[1] * kBlock + u[3] + (int)off;
    }
    positions[row] = pos;
}

template <typename InT, int D>
cudaError_t launch_rope(const RopeArgs &a, cudaStream_t st) {
    const int64_t ctas = (a.n_rows * a.splits + 7) / 8;
    const cudaError_t e = gdn_launch_pdl(rope_kernel<InT, D>, dim3((unsigned)ctas), 256, 0, st, a);
    return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace gdn

namespace {

gdn_status check_rope(const gdn_rope_desc *r) {
    if (!r) return fail(GDN_ERR_INVALID_ARG, "rotary description is NULL");
    if (r->rotary_dim < 16 || r->rotary_dim > 256 || r->rotary_dim % 16 != 0)
        return fail(GDN_ERR_SHAPE, "rotary_dim must be a multiple of 16 in [16, 256] (got %d)", r->rotary_dim);
    if (r->layout != GDN_ROPE_HALF && r->layout != GDN_ROPE_INTERLEAVED)
        return fail(GDN_ERR_SHAPE, "layout must be GDN_ROPE_HALF or GDN_ROPE_INTERLEAVED (got %d)", r->layout);
    if (!(r->base >= 1.f) || !std::isfinite(r->base)) return fail(GDN_ERR_INVALID_ARG, "base must be finite and >= 1");
    if (r->scaling != GDN_ROPE_NONE && r->scaling != GDN_ROPE_LINEAR && r->scaling != GDN_ROPE_PARTS)
        return fail(GDN_ERR_SHAPE, "scaling must be GDN_ROPE_NONE, GDN_ROPE_LINEAR or GDN_ROPE_PARTS (got %d)", r->scaling);
    if (r->scaling != GDN_ROPE_NONE && (!(r->factor >= 1.f) || !std::isfinite(r->factor)))
        return fail(GDN_ERR_INVALID_ARG, "factor must be finite and >= 1");
    if (r->scaling == GDN_ROPE_PARTS &&
        (r->original_len < 1 || !(r->beta_slow >= 0.f) || !(r->beta_fast > r->beta_slow) || !std::isfinite(r->beta_fast)))
        return fail(GDN_ERR_INVALID_ARG, "original_len must be >= 1 and 0 <= beta_slow < beta_fast");
    if (!(r->magnitude > 0.f) || !std::isfinite(r->magnitude)) return fail(GDN_ERR_INVALID_ARG, "magnitude must be finite and > 0");
    if (!(r->eps >= 0.f) || !std::isfinite(r->eps)) return fail(GDN_ERR_INVALID_ARG, "eps must be finite and >= 0");
    return GDN_OK;
}

bool aligned_to(const void *p, uintptr_t n) { return p && (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

}  // namespace

GDN_API gdn_status gdn_rope_desc_check(const gdn_rope_desc *r) { return check_rope(r); }

GDN_API gdn_status gdn_rope_table(const gdn_rope_desc *r, uint64_t *table, gdn_stream_t stream) {
    const gdn_status st = check_rope(r);
    if (st != GDN_OK) return st;
    if (!aligned_to(table, 16)) return fail(GDN_ERR_INVALID_ARG, "table must be non-NULL and 16-byte aligned");
    const cudaError_t e = launch_k(K_ROPE, (cudaStream_t)stream, [&] {
        const cudaError_t l = gdn_launch_pdl(gdn::rope_table_kernel, dim3(1), 128, 0, (cudaStream_t)stream, *r,
                                             reinterpret_cast<unsigned long long *>(table));
        return l != cudaSuccess ? l : cudaGetLastError();
    });
    return e != cudaSuccess ? cuda_fail(e, "rotary table kernel") : GDN_OK;
}

GDN_API gdn_status gdn_kv_positions(const gdn_kv_map *m, int64_t n_rows, int32_t *positions, gdn_stream_t stream) {
    if (!m || !aligned_to(m->units, 16) || !aligned_to(m->counts, 4) || m->max_units < 1)
        return fail(GDN_ERR_INVALID_ARG, "map: units (16-byte aligned) and counts must be non-NULL, max_units >= 1");
    if (n_rows < 0 || n_rows > INT32_MAX) return fail(GDN_ERR_INVALID_ARG, "n_rows out of range (%lld)", (long long)n_rows);
    if (n_rows == 0) return GDN_OK;
    if (!aligned_to(positions, 4)) return fail(GDN_ERR_INVALID_ARG, "positions must be non-NULL");
    const cudaError_t e = launch_k(K_ROPE, (cudaStream_t)stream, [&] {
        const cudaError_t l = gdn_launch_pdl(gdn::kv_positions_kernel, dim3((unsigned)((n_rows + 255) / 256)), 256, 0,
                                             (cudaStream_t)stream, m->units, m->counts, m->max_units, n_rows, positions);
        return l != cudaSuccess ? l : cudaGetLastError();
    });
    return e != cudaSuccess ? cuda_fail(e, "positions kernel") : GDN_OK;
}

GDN_API gdn_status gdn_rope(const gdn_attn_desc *d, const gdn_rope_desc *r, const uint64_t *table, const int32_t *positions,
                            const void *q, int64_t q_stride, const void *k, int64_t k_stride, const void *v, int64_t v_stride,
                            const void *q_weight, const void *k_weight, void *q_out, void *k_out, void *v_out, int64_t n_rows,
                            gdn_stream_t stream) {
    gdn_status st = gdn_attn_desc_check(d);
    if (st != GDN_OK || (st = check_rope(r)) != GDN_OK) return st;
    if (r->rotary_dim > d->head_dim) return fail(GDN_ERR_SHAPE, "rotary_dim %d is above head_dim %d", r->rotary_dim, d->head_dim);
    if (n_rows < 0 || n_rows > INT32_MAX) return fail(GDN_ERR_INVALID_ARG, "n_rows out of range (%lld)", (long long)n_rows);
    if (n_rows == 0) return GDN_OK;
    if (!aligned_to(table, 16) || !aligned_to(positions, 4))
        return fail(GDN_ERR_INVALID_ARG, "table (16-byte aligned) and positions must be non-NULL");
    if (!aligned_to(q, 16) || !aligned_to(k, 16) || !aligned_to(q_out, 16) || !aligned_to(k_out, 16))
        return fail(GDN_ERR_INVALID_ARG, "q, k, q_out and k_out must be non-NULL and 16-byte aligned");
    if ((v != nullptr) != (v_out != nullptr) || (v && (!aligned_to(v, 16) || !aligned_to(v_out, 16))))
        return fail(GDN_ERR_INVALID_ARG, "v and v_out must be given together, 16-byte aligned");
    if ((q_weight && !aligned_to(q_weight, 16)) || (k_weight && !aligned_to(k_weight, 16)))
        return fail(GDN_ERR_INVALID_ARG, "q_weight and k_weight must be 16-byte aligned");
    const int64_t vec = d->in_dtype == GDN_BF16 ? 8 : 4, wq = (int64_t)d->n_q_heads * d->head_dim, wk = (int64_t)d->n_kv_heads * d->head_dim;
    if (q_stride < wq || k_stride < wk || (v && v_stride < wk) || q_stride % vec || k_stride % vec || (v && v_stride % vec))
        return fail(GDN_ERR_INVALID_ARG, "strides must be a row's heads at least and a multiple of 16 bytes (q %lld, k %lld, v %lld)",
                    (long long)q_stride, (long long)k_stride, (long long)v_stride);
    // an output may be its own input, row by row; no other overlap
    const int64_t e = d->in_dtype == GDN_BF16 ? 2 : 4;
    struct Span { const char *lo, *hi; int64_t stride; } in[3], out[3];
    auto span = [&](const void *p, int64_t stride, int64_t width) {
        const char *lo = static_cast<const char *>(p);
        return Span{lo, p ? lo + ((n_rows - 1) * stride + width) * e : lo, stride};
    };
    in[0] = span(q, q_stride, wq); in[1] = span(k, k_stride, wk); in[2] = span(v, v_stride, wk);
    out[0] = span(q_out, wq, wq); out[1] = span(k_out, wk, wk); out[2] = span(v_out, wk, wk);
    for (int o = 0; o < 3; ++o)
        for (int i = 0; i < 3; ++i) {
            const bool same = o == i && out[o].lo == in[i].lo && (n_rows == 1 || out[o].stride == in[i].stride);
            if (!same && out[o].lo < in[i].hi && in[i].lo < out[o].hi)
                return fail(GDN_ERR_INVALID_ARG, "an output overlaps an input that it does not replace row by row");
            if (o < i && out[o].lo < out[i].hi && out[i].lo < out[o].hi)
                return fail(GDN_ERR_INVALID_ARG, "two outputs overlap");
        }
    gdn::RopeArgs a = {};
    a.q = q; a.k = k; a.v = v;
    a.q_stride = q_stride; a.k_stride = k_stride; a.v_stride = v_stride;
    a.q_weight = q_weight; a.k_weight = k_weight;
    a.q_out = q_out; a.k_out = k_out; a.v_out = v_out;
    a.positions = positions;
    a.table = reinterpret_cast<const unsigned long long *>(table);
    a.n_rows = n_rows;
    a.Hq = d->n_q_heads; a.Hkv = d->n_kv_heads;
    a.heads = a.Hq + a.Hkv * (v ? 2 : 1);
    a.rotary_dim = r->rotary_dim; a.interleaved = r->layout == GDN_ROPE_INTERLEAVED;
    a.magnitude = r->magnitude; a.eps = r->eps;
    int sms = 1;
    cudaError_t ce = gdn_sm_count(&sms);
    if (ce != cudaSuccess) return cuda_fail(ce, "SM count");
    // warps of a row: more while the rows alone are fewer than 32 warps an SM
    const int per_warp = 32 / (d->head_dim / (2 * (int)vec)), passes = (a.heads + per_warp - 1) / per_warp;
    a.splits = (int)std::min<int64_t>(passes, std::max<int64_t>(1, 32LL * sms / n_rows));
    cudaStream_t cst = (cudaStream_t)stream;
    ce = launch_k(K_ROPE, cst, [&] {
        using bf = __nv_bfloat16;
        if (d->in_dtype == GDN_BF16)
            return d->head_dim == 64 ? gdn::launch_rope<bf, 64>(a, cst) : d->head_dim == 128 ? gdn::launch_rope<bf, 128>(a, cst)
                                                                                             : gdn::launch_rope<bf, 256>(a, cst);
        return d->head_dim == 64 ? gdn::launch_rope<float, 64>(a, cst) : d->head_dim == 128 ? gdn::launch_rope<float, 128>(a, cst)
                                                                                            : gdn::launch_rope<float, 256>(a, cst);
    });
    return ce != cudaSuccess ? cuda_fail(ce, "rotary kernel") : GDN_OK;
}

// Attention of requests that share their first blocks (forks of a session): the groups of a plan, the launches of the two
// parts (shared blocks for all rows of a group, each request's own keys) and their join.
//
// Softmax over a row's keys as that over two sets of them: each part leaves (O, m, l) of its segments, O the sum of
// 2^{x - m} v and l that of 2^{x - m} over its keys, and the row is sum 2^{m_s - M} O_s / sum 2^{m_s - M} l_s with M the
// largest m_s, in the order of s: the shared blocks' segments, then the own ones.
#include "kv_attn_prompt.cuh"
#include "kv_attn_simt.cuh"
#include "kv_attn_token.cuh"

namespace gdn {

constexpr int kGroupThreads = 1024;

// Groups of a plan, a CTA each: requests [bounds[g], bounds[g + 1]) -> {first row, rows, slot of its first unit, shared blocks}.
// Shared: the blocks that every request's table names alike and that lie before every request's first new token; none of a
// group without units. starts: the shared blocks of each unit's group, 0 of a unit in none.
// Bound: latency, a chain of dependent reads (bounds, rows, units by bisection, tables).
__global__ void __launch_bounds__(kGroupThreads) kv_group_kernel(const KvCache c, const int32_t *rows, const int32_t *units,
                                                                 const int32_t *counts, int max_requests, int max_units,
                                                                 const int32_t *bounds, int n_groups, int32_t *groups,
                                                                 int32_t *starts, unsigned *err) {
    grid_dep_wait();
    grid_dep_launch();
    __shared__ int common;
    const int g = blockIdx.x, t = threadIdx.x, warp = t >> 5, lane = t & 31;
    if (g >= n_groups) {   // a record that this call leaves empty
        if (t == 0) reinterpret_cast<int4 *>(groups)[g] = make_int4(0, 0, 0, 0);
        return;
    }
    const int n_units = min(counts[0], max_units);
    const int b0 = bounds[g], b1 = bounds[g + 1];
    if (t == 0) common = INT32_MAX;
    int row0 = 0, row1 = 0;
    const bool in = n_units > 0 && b0 >= 0 && b0 <= b1 && b1 <= max_requests;
    if (in) {
        row0 = rows[b0];
        row1 = rows[b1];
    }
    bool ok = n_units == 0 || (in && row0 >= 0 && row0 <= row1);
    if (!ok) row0 = row1 = 0;
    // the first unit at or after a row: units are in row order
    auto unit_at = [&](int row) {
        int lo = 0, hi = n_units;
        while (lo < hi) {
            const int mid = (lo + hi) >> 1;
            if (units[8 * (int64_t)mid + 5] < row) lo = mid + 1;
            else hi = mid;
        }
        return lo;
    };
    const int u0 = unit_at(row0), u1 = max(unit_at(row1), u0);
    __syncthreads();
    int slot = 0;
    if (u1 > u0) {
        slot = units[8 * (int64_t)u0];
        int first = INT32_MAX;
        for (int i = u0 + t; i < u1; i += kGroupThreads) first = min(first, units[8 * (int64_t)i + 1]);
        first = __reduce_min_sync(0xffffffffu, first);
        if (lane == 0) atomicMin(&common, first);
        __syncthreads();
        const int most = min(common, c.max_blocks);
        ok = ok && (unsigned)slot < (unsigned)c.n_slots && most >= 0;
        if (ok) {
            const int32_t *mine = c.table + (int64_t)slot * c.max_blocks;
            int upto = most;   // of this lane
            for (int i = u0 + 1 + warp; i < u1; i += kGroupThreads / 32) {
                const int s = units[8 * (int64_t)i];
                if (s == units[8 * (int64_t)(i - 1)] || s == slot) continue;   // a request's first unit stands for it
                if ((unsigned)s >= (unsigned)c.n_slots) {
                    upto = 0;
                    continue;
                }
                const int32_t *theirs = c.table + (int64_t)s * c.max_blocks;
#pragma unroll 4
                for (int b = lane; b < upto; b += 32)
                    if (theirs[b] != mine[b]) upto = b;
            }
            upto = __reduce_min_sync(0xffffffffu, upto);
            if (lane == 0) atomicMin(&common, upto);
        }
        __syncthreads();
    }
    const int shared = ok && u1 > u0 ? min(common, c.max_blocks) : 0;
    if (t == 0) {
        reinterpret_cast<int4 *>(groups)[g] = make_int4(row0, row1 - row0, slot, shared);
        if (!ok) atomicOr(err, kErrKvBounds);
    }
    // units before the first group's and after the last one's are in none
    const int from = g == 0 ? 0 : u0, to = g == n_groups - 1 ? n_units : u1;
    for (int i = from + t; i < to; i += kGroupThreads) starts[i] = i >= u0 && i < u1 ? shared : 0;
}

// Every row of a unit: the segments of its group's shared blocks, then its own ones. A warp per (token, query head).
template <typename InT, int D>
__global__ void __launch_bounds__(256) kv_shared_join_kernel(const KvAttn a) {
    grid_dep_wait();
    grid_dep_launch();
    const int ui = a.unit0 + blockIdx.x;
    if (ui >= a.counts[0]) return;
    const KvUnit u = kv_load_unit(a.units, ui);
    const int start = a.starts[ui];
    if (!kv_suffix_unit_ok(a, u, start)) return;
    const int pre = (start + a.pre_blocks - 1) / a.pre_blocks, n = pre + u.block / a.seg_blocks - start / a.seg_blocks + 1;
    constexpr int W = D == 64 ? 2 : 4, N = D / (32 * W);
    const int lane = threadIdx.x & 31;
    for (int64_t r = blockIdx.y * 8 + (threadIdx.x >> 5); r < (int64_t)u.count * a.Hq; r += gridDim.y * 8) {
        const int64_t row = (int64_t)u.row * a.Hq + r;
        auto at = [&](int s) { return (s < pre ? s : a.n_pre + s - pre) * a.part_rows + row; };
        float M = -INFINITY;
        for (int s = lane; s < n; s += 32) M = fmaxf(M, a.part_ml[at(s)].x);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
        const float base = M == -INFINITY ? 0.f : M;
        float o[N][W], l = 0.f;
#pragma unroll
        for (int j = 0; j < N; ++j)
#pragma unroll
            for (int k = 0; k < W; ++k) o[j][k] = 0.f;
#pragma unroll 4
        for (int s = 0; s < n; ++s) {
            const float2 ml = a.part_ml[at(s)];
            const float f = exp2f(ml.x - base);
            l = fmaf(f, ml.y, l);
            const float *src = a.part_o + at(s) * D;
#pragma unroll
            for (int j = 0; j < N; ++j) {
                float v[W];
                if constexpr (W == 4) *reinterpret_cast<float4 *>(v) = *reinterpret_cast<const float4 *>(src + W * (lane + 32 * j));
                else *reinterpret_cast<float2 *>(v) = *reinterpret_cast<const float2 *>(src + W * (lane + 32 * j));
#pragma unroll
                for (int k = 0; k < W; ++k) o[j][k] = fmaf(f, v[k], o[j][k]);
            }
        }
        const float inv = l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l);   // no key: zero; NaN stays
        InT *dst = static_cast<InT *>(a.out) + row * D;
#pragma unroll
        for (int j = 0; j < N; ++j)
#pragma unroll
            for (int k = 0; k < W; ++k) dst[W * (lane + 32 * j) + k] = from_f<InT>(o[j][k] * inv);
    }
}

template <int PART>
cudaError_t launch_simt_part(const KvAttn &a, int d, int n, int rows_max, cudaStream_t st) {
    if (d == 64) return launch_simt_many<64, PART>(a, n, rows_max, st);
    if (d == 128) return launch_simt_many<128, PART>(a, n, rows_max, st);
    return launch_simt_many<256, PART>(a, n, rows_max, st);
}

template <typename InT>
cudaError_t launch_shared_join(const KvAttn &a, int d, int unit_bound, cudaStream_t st) {
    const dim3 grid((unsigned)unit_bound, (unsigned)std::min((a.tok_stride * a.Hq + 7) / 8, 64));
    if (d == 64) return gdn_launch_pdl(kv_shared_join_kernel<InT, 64>, grid, 256, 0, st, a);
    if (d == 128) return gdn_launch_pdl(kv_shared_join_kernel<InT, 128>, grid, 256, 0, st, a);
    return gdn_launch_pdl(kv_shared_join_kernel<InT, 256>, grid, 256, 0, st, a);
}

}  // namespace gdn

cudaError_t gdn_launch_kv_group(const gdn::KvCache &c, const int32_t *rows, const int32_t *units, const int32_t *counts,
                                int max_requests, int max_units, const int32_t *bounds, int n_groups, int max_groups,
                                int32_t *groups, int32_t *starts, unsigned *err, cudaStream_t st) {
    const cudaError_t e = gdn_launch_pdl(gdn::kv_group_kernel, (unsigned)max_groups, gdn::kGroupThreads, 0, st, c, rows, units, counts,
                                         max_requests, max_units, bounds, n_groups, groups, starts, err);
    return e != cudaSuccess ? e : cudaGetLastError();
}

cudaError_t gdn_launch_kv_suffix(const gdn::KvAttn &a, int d, int bf16, int unit_bound, int rows_max, int few, cudaStream_t st) {
    using namespace gdn;
    const cudaError_t e = !bf16 ? launch_simt_part<kKvSuffix>(a, d, unit_bound, rows_max, st)
                          : few ? launch_token_part<kKvSuffix>(a, d, unit_bound, rows_max, st)
                                : launch_prompt_part<kKvSuffix>(a, d, unit_bound, st);
    return e != cudaSuccess ? e : cudaGetLastError();
}

cudaError_t gdn_launch_kv_shared(const gdn::KvAttn &a, int d, int bf16, int tile_bound, cudaStream_t st) {
    using namespace gdn;
    const cudaError_t e = bf16 ? launch_prompt_part<kKvShared>(a, d, tile_bound, st) : launch_simt_part<kKvShared>(a, d, tile_bound, 0, st);
    return e != cudaSuccess ? e : cudaGetLastError();
}

cudaError_t gdn_launch_kv_shared_join(const gdn::KvAttn &a, int d, int bf16, int unit_bound, cudaStream_t st) {
    using namespace gdn;
    const cudaError_t e = bf16 ? launch_shared_join<__nv_bfloat16>(a, d, unit_bound, st) : launch_shared_join<float>(a, d, unit_bound, st);
    return e != cudaSuccess ? e : cudaGetLastError();
}

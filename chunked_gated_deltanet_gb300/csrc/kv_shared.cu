// Attention of requests that share their first blocks (forks of a session): the groups of a plan, the launches of the two
// parts (shared blocks for all rows of a group, each request's own keys) and their join.
//
// Softmax over a row's keys as that over two sets of them: each part leaves (O, m, l) of its segments, O the sum of
// 2^{x - m} v and l that of 2^{x - m} over its keys, and the row is sum 2^{m_s - M} O_s / sum 2^{m_s - M} l_s with M the
// largest m_s, in the order of s: the shared blocks' segments, then the own ones.
//
// The parts run in the kernels of kv_attn_prompt.cuh, kv_attn_token.cuh and kv_attn_simt.cuh, each built for its part (KvPart),
// so that the shared blocks' loop has no mask and no raw block in it: 8,000 x 16 rows over 37,760 shared keys (d = 128) take
// 1.71 ms, 1.45 PFLOP/s, where the same loop with the raw blocks' code beside it reaches 1.18. A row's group stands in consecutive
// packed rows, so a tile of it is filled across requests. Single tokens of small families take both parts in one launch
// (kv_attn_token.cuh); kv_api.cu has the rule.
#include "kv_attn_prompt.cuh"
#include "kv_attn_simt.cuh"
#include "kv_attn_token.cuh"

#include <cooperative_groups.h>

namespace gdn {

namespace cg = cooperative_groups;

constexpr int kGroupThreads = 512, kGroupCluster = 8;

// Groups of a plan, a cluster each: requests [bounds[g], bounds[g + 1]) -> {first row, rows, slot of its first unit, shared
// blocks}. Shared: the blocks that every request's table names alike and that lie before every request's first new token;
// none of a group without units. starts: the shared blocks of each unit's group, 0 of a unit in none.
// Every CTA finds the group's units (one pass over the plan's, which are in row order) and compares its share of the table
// entries; the least difference is the first CTA's. Bound: latency, four dependent reads (bounds, rows, units, tables): 6 us, 9 us
// for 64 requests of 653 blocks.
__global__ void __launch_bounds__(kGroupThreads) kv_group_kernel(const KvCache c, const int32_t *rows, const int32_t *units,
                                                                 const int32_t *counts, int max_requests, int max_units,
                                                                 const int32_t *bounds, int n_groups, int32_t *groups,
                                                                 int32_t *starts, unsigned *err) {
    grid_dep_wait();
    grid_dep_launch();
    __shared__ int slots[kKvMaxRequests], n_slots, before0, before1, first, common;
    cg::cluster_group cl = cg::this_cluster();
    const int n_cl = (int)cl.num_blocks(), rank = (int)cl.block_rank(), g = blockIdx.x / n_cl, t = threadIdx.x;
    if (g >= n_groups) {   // a record that this call leaves empty
        if (rank == 0 && t == 0) reinterpret_cast<int4 *>(groups)[g] = make_int4(0, 0, 0, 0);
        return;
    }
    const int n_units = min(counts[0], max_units);
    if (t == 0) {
        n_slots = before0 = before1 = 0;
        first = common = INT32_MAX;
    }
    // the bounds of all groups, requests and rows: one out of order or range and none shares anything, as groups could overlap
    bool bad = false;
    for (int i = t; n_units > 0 && i < n_groups; i += kGroupThreads) {
        const int from = bounds[i], to = bounds[i + 1];
        bad = bad || from < 0 || from > to || to > max_requests || rows[max(min(from, max_requests), 0)] < 0 ||
              rows[max(min(from, max_requests), 0)] > rows[max(min(to, max_requests), 0)];
    }
    int row0 = 0, row1 = 0;
    if (n_units > 0) {
        row0 = rows[max(min(bounds[g], max_requests), 0)];
        row1 = rows[max(min(bounds[g + 1], max_requests), 0)];
    }
    bool ok = __syncthreads_or(bad) == 0;
    if (!ok) row0 = row1 = 0;
    // the group's units: those before its first row and before its end, the first block of any, a slot per request
    int n0 = 0, n1 = 0, low = INT32_MAX;
    for (int i = t; i < n_units; i += kGroupThreads) {
        const KvUnit u = kv_load_unit(units, i);
        n0 += u.row < row0;
        n1 += u.row < row1;
        if (u.row < row0 || u.row >= row1) continue;
        low = min(low, u.block);
        if (i == 0 || u.row == row0 || units[8 * (int64_t)(i - 1)] != u.slot) {   // a request's first unit stands for it
            const int k = atomicAdd(&n_slots, 1);
            if (k < kKvMaxRequests) slots[k] = u.slot;
        }
    }
    n0 = __reduce_add_sync(0xffffffffu, n0);
    n1 = __reduce_add_sync(0xffffffffu, n1);
    low = __reduce_min_sync(0xffffffffu, low);
    if ((t & 31) == 0) {
        atomicAdd(&before0, n0);
        atomicAdd(&before1, n1);
        atomicMin(&first, low);
    }
    __syncthreads();
    const int u0 = before0, u1 = before1, n = min(n_slots, kKvMaxRequests);
    const int slot = u1 > u0 ? units[8 * (int64_t)u0] : 0;
    const int most = min(first, c.max_blocks);
    ok = ok && (u1 == u0 || ((unsigned)slot < (unsigned)c.n_slots && most >= 0));
    int upto = u1 > u0 && ok ? most : 0;
    if (n > 1 && upto > 0) {
        const int32_t *mine = c.table + (int64_t)slot * c.max_blocks;
        // a warp takes 128 blocks of a request at a time: four loads of either table a lane
        const int warps = n_cl * (kGroupThreads / 32), chunks = (most + 127) / 128, lane = t & 31;
        int r = 0, c0 = rank * (kGroupThreads / 32) + (t >> 5);
        for (;; c0 += warps) {
            while (r < n && c0 >= chunks) {
                c0 -= chunks;
                ++r;
            }
            if (r >= n) break;
            const int s = slots[r];
            if ((unsigned)s >= (unsigned)c.n_slots) {
                upto = 0;
                continue;
            }
            const int32_t *theirs = c.table + (int64_t)s * c.max_blocks;
            int x[4], y[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int b = 128 * c0 + 32 * i + lane;
                x[i] = b < most ? mine[b] : 0;
                y[i] = b < most ? theirs[b] : 0;
            }
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (x[i] != y[i]) upto = min(upto, 128 * c0 + 32 * i + lane);
        }
    }
    upto = __reduce_min_sync(0xffffffffu, upto);
    cl.sync();   // the first CTA's minimum is set up
    if ((t & 31) == 0) atomicMin(cl.map_shared_rank(&common, 0), upto);
    cl.sync();
    const int shared = *cl.map_shared_rank(&common, 0);
    if (rank == 0 && t == 0) {
        reinterpret_cast<int4 *>(groups)[g] = make_int4(row0, row1 - row0, slot, shared);
        if (!ok) atomicOr(err, kErrKvBounds);
    }
    // units before the first group's and after the last one's are in none
    const int from = g == 0 ? 0 : u0, to = g == n_groups - 1 ? n_units : u1;
    for (int i = from + rank * kGroupThreads + t; i < to; i += n_cl * kGroupThreads) starts[i] = i >= u0 && i < u1 ? shared : 0;
    cl.sync();   // the first CTA's minimum is read
}

// Every row of a unit: the segments of its group's shared blocks, then its own ones. W warps of a CTA to a (token, query
// head), each every W-th segment; their sums are added in order. Few rows have many segments and leave room for more warps
// (launch_shared_join), many rows few (128,000 rows of 4 or 5, d = 128: 58 us, 4.9 TB/s).
template <typename InT, int D, int W>
__global__ void __launch_bounds__(256) kv_shared_join_kernel(const KvAttn a) {
    grid_dep_wait();
    grid_dep_launch();
    const int ui = blockIdx.x;
    const KvUnit u = kv_load_unit(a.units, ui);   // inside the map whatever the count
    const int start = a.starts[ui], cut = a.cut ? *a.cut : a.pre_blocks;
    if (ui >= a.counts[0] || !kv_suffix_unit_ok(a, u, start)) return;
    const int pre = (start + cut - 1) / cut, n = pre + kv_own_segs(a, u.block, start);
    constexpr int V = D == 64 ? 2 : 4, N = D / (32 * V), B = W == 8 ? 4 : 2;   // B segments loaded together
    __shared__ float so[W > 1 ? 8 : 1][D], sl[W > 1 ? 8 : 1];   // a warp's sums, W > 1
    const int t = threadIdx.x, warp = t >> 5, lane = t & 31, mine = warp % W;
    const int n_row = u.count * a.Hq;
    for (int r0 = blockIdx.y * (8 / W); r0 < n_row; r0 += gridDim.y * (8 / W)) {   // 8 / W rows, the same passes in every warp
        const int r = r0 + warp / W;
        const bool live = r < n_row;
        if (W == 1 && !live) break;
        const int64_t row = (int64_t)u.row * a.Hq + (live ? r : r0);
        auto at = [&](int s) { return (s < pre ? s : a.n_pre + s - pre) * a.part_rows + row; };
        float2 ml[B];
        float v[B][N][V];
        auto load = [&](int s0) {
#pragma unroll
            for (int i = 0; i < B; ++i) {
                const int s = s0 + W * i;
                ml[i] = make_float2(-INFINITY, 0.f);
                if (s < n) ml[i] = a.part_ml[at(s)];
#pragma unroll
                for (int j = 0; j < N; ++j) {
#pragma unroll
                    for (int k = 0; k < V; ++k) v[i][j][k] = 0.f;
                    if (s >= n) continue;
                    const float *src = a.part_o + at(s) * D + V * (lane + 32 * j);
                    if constexpr (V == 4) *reinterpret_cast<float4 *>(v[i][j]) = *reinterpret_cast<const float4 *>(src);
                    else *reinterpret_cast<float2 *>(v[i][j]) = *reinterpret_cast<const float2 *>(src);
                }
            }
        };
        load(mine);
        float M = -INFINITY;
        for (int s = lane; s < n; s += 32) M = fmaxf(M, a.part_ml[at(s)].x);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
        const float base = M == -INFINITY ? 0.f : M;
        float o[N][V], l = 0.f;
#pragma unroll
        for (int j = 0; j < N; ++j)
#pragma unroll
            for (int k = 0; k < V; ++k) o[j][k] = 0.f;
#pragma unroll 1
        for (int s0 = mine; s0 < n; s0 += W * B) {
            if (s0 != mine) load(s0);
#pragma unroll
            for (int i = 0; i < B; ++i) {
                const float f = exp2f(ml[i].x - base);   // 0 for a segment that is not there
                l = fmaf(f, ml[i].y, l);
#pragma unroll
                for (int j = 0; j < N; ++j)
#pragma unroll
                    for (int k = 0; k < V; ++k) o[j][k] = fmaf(f, v[i][j][k], o[j][k]);
            }
        }
        InT *dst = static_cast<InT *>(a.out) + row * D;
        if constexpr (W == 1) {
            const float inv = l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l);   // no key: zero; NaN stays
#pragma unroll
            for (int j = 0; j < N; ++j)
#pragma unroll
                for (int k = 0; k < V; ++k) dst[V * (lane + 32 * j) + k] = from_f<InT>(o[j][k] * inv);
        } else {
            __syncthreads();   // the rows before are read
#pragma unroll
            for (int j = 0; j < N; ++j)
#pragma unroll
                for (int k = 0; k < V; ++k) so[warp][V * (lane + 32 * j) + k] = o[j][k];
            if (lane == 0) sl[warp] = l;
            __syncthreads();
            if (!live) continue;
            const int w0 = warp - mine;   // the row's first warp
            float L = 0.f;
#pragma unroll
            for (int w = 0; w < W; ++w) L += sl[w0 + w];
            const float inv = L > 0.f ? 1.f / L : (L == 0.f ? 0.f : L);
            for (int c = 32 * mine + lane; c < D; c += 32 * W) {
                float x = 0.f;
#pragma unroll
                for (int w = 0; w < W; ++w) x += so[w0 + w][c];
                dst[c] = from_f<InT>(x * inv);
            }
        }
    }
}

template <int PART>
cudaError_t launch_simt_part(const KvAttn &a, int d, int n, int rows_max, cudaStream_t st) {
    if (d == 64) return launch_simt_many<64, PART>(a, n, rows_max, st);
    if (d == 128) return launch_simt_many<128, PART>(a, n, rows_max, st);
    return launch_simt_many<256, PART>(a, n, rows_max, st);
}

template <typename InT, int D, int W>
cudaError_t launch_join_warps(const KvAttn &a, int unit_bound, int most, cudaStream_t st) {   // most: CTAs of a unit
    const int per_unit = (a.tok_stride * a.Hq * W + 7) / 8;
    return gdn_launch_pdl(kv_shared_join_kernel<InT, D, W>, dim3((unsigned)unit_bound, (unsigned)std::min(per_unit, most)), 256, 0, st, a);
}
// As many warps a row as one wave of CTAs has room for, about: 128 rows of 4 segments (d = 128) with 8 warps 6 us, with 4 8; 1,024
// of 22 (d = 256) 12 and 10; 1,984 of 3 to 9 (d = 128) 12 and 10, with 2 8. Beyond, a warp a row, CTAs of several rows: 128,000
// rows with up to 48 CTAs a unit 61, with 64 63, with 128 74. (Event times, 2 us above the kernels'.)
template <typename InT, int D>
cudaError_t launch_shared_join(const KvAttn &a, int unit_bound, cudaStream_t st) {
    if (a.part_rows <= 512) return launch_join_warps<InT, D, 8>(a, unit_bound, 4096, st);
    if (a.part_rows <= 8 * kSharedSms) return launch_join_warps<InT, D, 4>(a, unit_bound, 4096, st);
    if (a.part_rows <= 4096) return launch_join_warps<InT, D, 2>(a, unit_bound, 4096, st);
    return launch_join_warps<InT, D, 1>(a, unit_bound, 48, st);
}

}  // namespace gdn

cudaError_t gdn_launch_kv_group(const gdn::KvCache &c, const int32_t *rows, const int32_t *units, const int32_t *counts,
                                int max_requests, int max_units, const int32_t *bounds, int n_groups, int max_groups,
                                int32_t *groups, int32_t *starts, unsigned *err, cudaStream_t st) {
    using namespace gdn;
    // a cluster to a group while they fit the SMs at once, a CTA otherwise
    const unsigned n_cl = max_groups * kGroupCluster <= 304 ? kGroupCluster : 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)max_groups * n_cl);
    cfg.blockDim = dim3(kGroupThreads);
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = n_cl;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kv_group_kernel, c, rows, units, counts, max_requests, max_units, bounds, n_groups,
                                             groups, starts, err);
    return e != cudaSuccess ? e : cudaGetLastError();
}

cudaError_t gdn_launch_kv_suffix(const gdn::KvAttn &a, int d, int bf16, int unit_bound, int rows_max, cudaStream_t st) {
    using namespace gdn;
    const cudaError_t e = bf16 ? launch_prompt_part<kKvSuffix>(a, d, unit_bound, st) : launch_simt_part<kKvSuffix>(a, d, unit_bound, rows_max, st);
    return e != cudaSuccess ? e : cudaGetLastError();
}

cudaError_t gdn_launch_kv_few(const gdn::KvAttn &a, int d, int unit_bound, int tiles, int rows_max, cudaStream_t st) {
    return gdn::launch_token_part<gdn::kKvFew>(a, d, unit_bound + tiles, rows_max, st);
}

cudaError_t gdn_launch_kv_shared(const gdn::KvAttn &a, int d, int bf16, int n_pieces, cudaStream_t st) {
    using namespace gdn;
    const cudaError_t e = bf16 ? launch_prompt_part<kKvShared>(a, d, n_pieces, st) : launch_simt_part<kKvShared>(a, d, n_pieces, 0, st);
    return e != cudaSuccess ? e : cudaGetLastError();
}

cudaError_t gdn_launch_kv_shared_join(const gdn::KvAttn &a, int d, int bf16, int unit_bound, cudaStream_t st) {
    using namespace gdn;
    using bf = __nv_bfloat16;
    cudaError_t e;
    if (d == 64) e = bf16 ? launch_shared_join<bf, 64>(a, unit_bound, st) : launch_shared_join<float, 64>(a, unit_bound, st);
    else if (d == 128) e = bf16 ? launch_shared_join<bf, 128>(a, unit_bound, st) : launch_shared_join<float, 128>(a, unit_bound, st);
    else e = bf16 ? launch_shared_join<bf, 256>(a, unit_bound, st) : launch_shared_join<float, 256>(a, unit_bound, st);
    return e != cudaSuccess ? e : cudaGetLastError();
}

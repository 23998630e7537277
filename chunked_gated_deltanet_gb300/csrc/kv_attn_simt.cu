// Attention over the paged 8-bit key/value cache in fp32 arithmetic, and the join of the segments' partial results.
//
// Per query row (token at position p, query head), with the block b = p / 64:
//   s_j = scale q . k_j over the blocks 0 .. b-1 (8 bits: k_j = k_scale[block] * int8) and block b's keys j <= p as they came,
//   out = sum_j exp(s_j - max) v_j / sum_j exp(s_j - max).
// One pass over the keys in position order, a 64-key block at a time, with the running maximum m and sum l in the
// log2 domain (the scale carries log2 e). Keys are cut into segments at absolute positions; each segment starts afresh
// and leaves (O, m, l), and the join adds the segments in order. What a row computes so depends on its position and
// the cache alone, not on the other rows of the call.
#include "kv.cuh"

#include <algorithm>

namespace gdn {

template <typename T> __device__ __forceinline__ T from_f(float x);
template <> __device__ __forceinline__ float from_f<float>(float x) { return x; }
template <> __device__ __forceinline__ __nv_bfloat16 from_f<__nv_bfloat16>(float x) { return __float2bfloat16_rn(x); }

// 64 rows of an 8-bit page as floats into shared memory (row stride LD); page values are exact in fp32.
template <int D, int LD>
__device__ __forceinline__ void load_page(float *dst, const int8_t *src) {
#pragma unroll
    for (int i = 0; i < D / 64; ++i) {
        const int e = threadIdx.x + 256 * i, r = e / (D / 16), c = (e % (D / 16)) * 16;
        const uint4 w = *reinterpret_cast<const uint4 *>(src + r * D + c);
        const uint32_t x[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            float4 f;
            f.x = (float)(int8_t)(x[j] & 0xff);
            f.y = (float)(int8_t)((x[j] >> 8) & 0xff);
            f.z = (float)(int8_t)((x[j] >> 16) & 0xff);
            f.w = (float)(int8_t)(x[j] >> 24);
            *reinterpret_cast<float4 *>(dst + r * LD + c + 4 * j) = f;
        }
    }
}

// The open block's rows as they came: offsets below u.first from the tail, the unit's own from the new rows, none after.
template <typename InT, int D, int LD>
__device__ __forceinline__ void load_raw(float *dst, const KvUnit &u, const InT *tail, const InT *x, int Hkv, int h) {
    for (int e = threadIdx.x; e < kKvBlock * D / 4; e += 256) {
        const int r = e / (D / 4), c = (e % (D / 4)) * 4, o = r - u.first;
        const InT *s = o < 0 ? tail + r * D + c : (o < u.count ? x + ((int64_t)(u.row + o) * Hkv + h) * D + c : nullptr);
        float4 f = make_float4(0.f, 0.f, 0.f, 0.f);
        if (s) f = make_float4(to_f(s[0]), to_f(s[1]), to_f(s[2]), to_f(s[3]));
        *reinterpret_cast<float4 *>(dst + r * LD + c) = f;
    }
}

// CTA (unit x row tile, kv head, segment), 256 threads, R rows. R = 64: thread (ty, tx) holds 4 rows, 4 keys of the
// scores and D / 16 columns of the output. R = 8 (few rows): a warp per row, 2 keys and D / 32 columns per lane.
template <typename InT, int D, int R>
struct SimtPlan {
    static constexpr int LD = D + 4, PLD = kKvBlock + 4;   // 16-byte rows that start 4 banks apart
    static constexpr size_t kBytes = (size_t)(R * LD + kKvBlock * LD + R * PLD) * sizeof(float);
    static constexpr int RT = R == 64 ? 4 : 1;             // rows per thread
    static constexpr int KT = R == 64 ? 4 : 2;             // keys per thread
    static constexpr int CT = R == 64 ? D / 16 : D / 32;   // output columns per thread
};

template <typename InT, int D, int R>
__global__ void __launch_bounds__(256) kv_attn_simt_kernel(const KvAttn a, int row_tiles) {
    using P = SimtPlan<InT, D, R>;
    constexpr int LD = P::LD, PLD = P::PLD, RT = P::RT, KT = P::KT, CT = P::CT;
    grid_dep_wait();
    grid_dep_launch();
    const int ui = a.unit0 + blockIdx.x / row_tiles, rt = blockIdx.x % row_tiles, h = blockIdx.y, seg = blockIdx.z;
    if (ui >= a.counts[0]) return;
    const KvUnit u = kv_load_unit(a.units, ui);
    const int last_seg = u.block / a.seg_blocks;
    if (!kv_unit_ok(u, a.c, a.n_rows) || u.count > a.max_new || last_seg >= a.n_seg) {
        if (threadIdx.x == 0) atomicOr(a.err, kErrKvBounds);
        return;
    }
    const int n_row = u.count * a.G, r0 = rt * R;
    if (r0 >= n_row || seg > last_seg) return;

    extern __shared__ __align__(16) unsigned char simt_smem[];
    float *Q = reinterpret_cast<float *>(simt_smem), *KV = Q + R * LD, *Pm = KV + kKvBlock * LD;
    const int t = threadIdx.x;
    const InT *q = static_cast<const InT *>(a.q);
    for (int e = t; e < R * D / 4; e += 256) {
        const int r = e / (D / 4), c = (e % (D / 4)) * 4;
        float4 f = make_float4(0.f, 0.f, 0.f, 0.f);
        if (r0 + r < n_row) {
            const InT *s = q + ((int64_t)(u.row + (r0 + r) / a.G) * a.Hq + h * a.G + (r0 + r) % a.G) * D + c;
            f = make_float4(to_f(s[0]), to_f(s[1]), to_f(s[2]), to_f(s[3]));
        }
        *reinterpret_cast<float4 *>(Q + r * LD + c) = f;
    }
    const int ty = R == 64 ? t >> 4 : t >> 5, tx = R == 64 ? t & 15 : t & 31;
    constexpr int TX = R == 64 ? 16 : 32;
    float o[RT][CT], m[RT], l[RT];
    int limit[RT];   // the last offset of its own block that a row sees
#pragma unroll
    for (int i = 0; i < RT; ++i) {
        m[i] = -INFINITY;
        l[i] = 0.f;
        limit[i] = u.first + (r0 + ty * RT + i) / a.G;
#pragma unroll
        for (int j = 0; j < CT; ++j) o[i][j] = 0.f;
    }
    const int b0 = seg * a.seg_blocks, b1 = min(u.block, b0 + a.seg_blocks);
    const int n_blk = b1 - b0 + (seg == last_seg ? 1 : 0);
    const int64_t Hkv = a.Hkv;
    for (int i = 0; i < n_blk; ++i) {
        const bool raw = b0 + i == u.block;
        int64_t ph = 0;
        float ks = 1.f, vs = 1.f;
        if (!raw) {
            const int page = a.c.table[(int64_t)u.slot * a.c.max_blocks + b0 + i];
            if ((unsigned)page >= (unsigned)a.c.n_pages) {
                if (t == 0) atomicOr(a.err, kErrKvBounds);
                continue;   // the same page number in every thread
            }
            ph = (int64_t)page * Hkv + h;
            ks = a.c.k_scale[ph];
            vs = a.c.v_scale[ph];
        }
        const InT *tail = static_cast<const InT *>(a.c.tail) + kv_tail_offset(u.slot, u.src, 0, h, a.Hkv, D);
        __syncthreads();   // the block before is done with KV and Pm (the first time: Q is written)
        if (raw) load_raw<InT, D, LD>(KV, u, tail, static_cast<const InT *>(a.k_new), a.Hkv, h);
        else load_page<D, LD>(KV, a.c.k + ph * kKvBlock * D);
        __syncthreads();
        float s[RT][KT];
#pragma unroll
        for (int x = 0; x < RT; ++x)
#pragma unroll
            for (int y = 0; y < KT; ++y) s[x][y] = 0.f;
#pragma unroll 4
        for (int c = 0; c < D; c += 4) {
            float4 qf[RT], kf[KT];
#pragma unroll
            for (int x = 0; x < RT; ++x) qf[x] = *reinterpret_cast<const float4 *>(Q + (ty * RT + x) * LD + c);
#pragma unroll
            for (int y = 0; y < KT; ++y) kf[y] = *reinterpret_cast<const float4 *>(KV + (tx + TX * y) * LD + c);
#pragma unroll
            for (int x = 0; x < RT; ++x)
#pragma unroll
                for (int y = 0; y < KT; ++y) {
                    s[x][y] = fmaf(qf[x].x, kf[y].x, s[x][y]);
                    s[x][y] = fmaf(qf[x].y, kf[y].y, s[x][y]);
                    s[x][y] = fmaf(qf[x].z, kf[y].z, s[x][y]);
                    s[x][y] = fmaf(qf[x].w, kf[y].w, s[x][y]);
                }
        }
        const float c = a.scale_log2 * ks;
#pragma unroll
        for (int x = 0; x < RT; ++x) {
            float mb = -INFINITY;
#pragma unroll
            for (int y = 0; y < KT; ++y) {
                s[x][y] = raw && tx + TX * y > limit[x] ? -INFINITY : s[x][y] * c;
                mb = fmaxf(mb, s[x][y]);
            }
#pragma unroll
            for (int w = TX / 2; w > 0; w >>= 1) mb = fmaxf(mb, __shfl_xor_sync(0xffffffffu, mb, w));
            const float mn = fmaxf(m[x], mb), base = mn == -INFINITY ? 0.f : mn;
            const float corr = exp2f(m[x] - base);
            float sum = 0.f;
#pragma unroll
            for (int y = 0; y < KT; ++y) {
                const float p = exp2f(s[x][y] - base);
                sum += p;
                Pm[(ty * RT + x) * PLD + tx + TX * y] = p * vs;
            }
#pragma unroll
            for (int w = TX / 2; w > 0; w >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, w);
            m[x] = mn;
            l[x] = l[x] * corr + sum;
#pragma unroll
            for (int j = 0; j < CT; ++j) o[x][j] *= corr;
        }
        __syncthreads();   // K is read, P is written
        if (raw) load_raw<InT, D, LD>(KV, u, tail + (int64_t)a.Hkv * kKvBlock * D, static_cast<const InT *>(a.v_new), a.Hkv, h);
        else load_page<D, LD>(KV, a.c.v + ph * kKvBlock * D);
        __syncthreads();
        // a key that the mask took has weight zero; it adds nothing whatever its value (a NaN or an infinity after
        // the row's position does not reach the row)
#pragma unroll 2
        for (int k = 0; k < kKvBlock; k += 4) {
            float4 pf[RT];
#pragma unroll
            for (int x = 0; x < RT; ++x) pf[x] = *reinterpret_cast<const float4 *>(Pm + (ty * RT + x) * PLD + k);
#pragma unroll
            for (int kk = 0; kk < 4; ++kk) {
                float v[CT];
                if constexpr (R == 64) {
#pragma unroll
                    for (int j = 0; j < CT / 4; ++j) {
                        const float4 f = *reinterpret_cast<const float4 *>(KV + (k + kk) * LD + 4 * tx + 64 * j);
                        v[4 * j] = f.x; v[4 * j + 1] = f.y; v[4 * j + 2] = f.z; v[4 * j + 3] = f.w;
                    }
                } else {
#pragma unroll
                    for (int j = 0; j < CT / 2; ++j) {
                        const float2 f = *reinterpret_cast<const float2 *>(KV + (k + kk) * LD + 2 * tx + 64 * j);
                        v[2 * j] = f.x; v[2 * j + 1] = f.y;
                    }
                }
#pragma unroll
                for (int x = 0; x < RT; ++x) {
                    const float p = kk == 0 ? pf[x].x : kk == 1 ? pf[x].y : kk == 2 ? pf[x].z : pf[x].w;
                    if (raw && p == 0.f) continue;
#pragma unroll
                    for (int j = 0; j < CT; ++j) o[x][j] = fmaf(p, v[j], o[x][j]);
                }
            }
        }
    }
    // one segment: the result; several: the partial one (column j of a thread: 4 tx + 64 (j / 4) + j % 4, or the pairs)
    constexpr int W = R == 64 ? 4 : 2;
#pragma unroll
    for (int x = 0; x < RT; ++x) {
        const int r = r0 + ty * RT + x;
        if (r >= n_row) continue;
        const int head = h * a.G + r % a.G;
        if (last_seg == 0) {
            const float inv = l[x] > 0.f ? 1.f / l[x] : (l[x] == 0.f ? 0.f : l[x]);   // no key: zero; NaN stays
            InT *dst = static_cast<InT *>(a.out) + ((int64_t)(u.row + r / a.G) * a.Hq + head) * D;
#pragma unroll
            for (int j = 0; j < CT; ++j) dst[W * tx + 64 * (j / W) + j % W] = from_f<InT>(o[x][j] * inv);
        } else {
            const int64_t pr = kv_part_row(a, ui, seg, r / a.G, head);
            float *dst = a.part_o + pr * D;
#pragma unroll
            for (int j = 0; j < CT; ++j) dst[W * tx + 64 * (j / W) + j % W] = o[x][j];
            if (tx == 0) a.part_ml[pr] = make_float2(m[x], l[x]);
        }
    }
}

// Rows of a unit with more than one segment: out = sum_s 2^{m_s - M} O_s / sum_s 2^{m_s - M} l_s, s in order.
// A warp per (token, query head); lane c / 4 of every 128 columns holds column c .. c + 3 (d = 64: two per lane).
template <typename InT, int D>
__global__ void __launch_bounds__(256) kv_join_kernel(const KvAttn a) {
    grid_dep_wait();
    grid_dep_launch();
    const int ui = a.unit0 + blockIdx.x;
    if (ui >= a.counts[0]) return;
    const KvUnit u = kv_load_unit(a.units, ui);
    const int n_seg = u.block / a.seg_blocks + 1;
    if (!kv_unit_ok(u, a.c, a.n_rows) || u.count > a.max_new || n_seg > a.n_seg || n_seg == 1) return;
    constexpr int W = D == 64 ? 2 : 4, N = D / (32 * W);
    const int lane = threadIdx.x & 31;
    const int64_t stride = a.part_rows;
    for (int64_t r = blockIdx.y * 8 + (threadIdx.x >> 5); r < (int64_t)u.count * a.Hq; r += gridDim.y * 8) {
        const int64_t row = (int64_t)u.row * a.Hq + r, pr = kv_part_row(a, ui, 0, 0, 0) + r;
        float M = -INFINITY;
        for (int s = 0; s < n_seg; ++s) M = fmaxf(M, a.part_ml[s * stride + pr].x);
        const float base = M == -INFINITY ? 0.f : M;
        float o[N][W], l = 0.f;
#pragma unroll
        for (int j = 0; j < N; ++j)
#pragma unroll
            for (int k = 0; k < W; ++k) o[j][k] = 0.f;
#pragma unroll 2
        for (int s = 0; s < n_seg; ++s) {
            const float2 ml = a.part_ml[s * stride + pr];
            const float f = exp2f(ml.x - base);
            l = fmaf(f, ml.y, l);
            const float *src = a.part_o + (s * stride + pr) * D;
#pragma unroll
            for (int j = 0; j < N; ++j) {
                float v[W];
                if constexpr (W == 4) *reinterpret_cast<float4 *>(v) = *reinterpret_cast<const float4 *>(src + W * (lane + 32 * j));
                else *reinterpret_cast<float2 *>(v) = *reinterpret_cast<const float2 *>(src + W * (lane + 32 * j));
#pragma unroll
                for (int k = 0; k < W; ++k) o[j][k] = fmaf(f, v[k], o[j][k]);
            }
        }
        const float inv = l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l);
        InT *dst = static_cast<InT *>(a.out) + row * D;
#pragma unroll
        for (int j = 0; j < N; ++j)
#pragma unroll
            for (int k = 0; k < W; ++k) dst[W * (lane + 32 * j) + k] = from_f<InT>(o[j][k] * inv);
    }
}

// The same for the few-row form, whose rows have many segments: a CTA per (token, query head), warp w taking segments
// w, w + 8, ... and the eight sums added in order.
template <typename InT, int D>
__global__ void __launch_bounds__(256) kv_join_few_kernel(const KvAttn a) {
    grid_dep_wait();
    grid_dep_launch();
    const int ui = a.unit0 + blockIdx.x, r = blockIdx.y;
    const KvUnit u = kv_load_unit(a.units, ui);
    if (ui >= a.counts[0]) return;
    const int n_seg = u.block / a.seg_blocks + 1;
    if (!kv_unit_ok(u, a.c, a.n_rows) || u.count > a.max_new || n_seg > a.n_seg || n_seg == 1 || r >= u.count * a.Hq) return;
    constexpr int W = D == 64 ? 2 : 4, N = D / (32 * W);
    __shared__ float so[8][D], sl[8];
    const int t = threadIdx.x, warp = t >> 5, lane = t & 31;
    const int64_t stride = a.part_rows, pr = kv_part_row(a, ui, 0, 0, 0) + r;
    float M = -INFINITY;
    for (int s = lane; s < n_seg; s += 32) M = fmaxf(M, a.part_ml[s * stride + pr].x);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
    const float base = M == -INFINITY ? 0.f : M;
    float o[N][W], l = 0.f;
#pragma unroll
    for (int j = 0; j < N; ++j)
#pragma unroll
        for (int k = 0; k < W; ++k) o[j][k] = 0.f;
#pragma unroll 4
    for (int s = warp; s < n_seg; s += 8) {
        const float2 ml = a.part_ml[s * stride + pr];
        const float f = exp2f(ml.x - base);
        l = fmaf(f, ml.y, l);
        const float *src = a.part_o + (s * stride + pr) * D;
#pragma unroll
        for (int j = 0; j < N; ++j) {
            float v[W];
            if constexpr (W == 4) *reinterpret_cast<float4 *>(v) = *reinterpret_cast<const float4 *>(src + W * (lane + 32 * j));
            else *reinterpret_cast<float2 *>(v) = *reinterpret_cast<const float2 *>(src + W * (lane + 32 * j));
#pragma unroll
            for (int k = 0; k < W; ++k) o[j][k] = fmaf(f, v[k], o[j][k]);
        }
    }
#pragma unroll
    for (int j = 0; j < N; ++j)
#pragma unroll
        for (int k = 0; k < W; ++k) so[warp][W * (lane + 32 * j) + k] = o[j][k];
    if (lane == 0) sl[warp] = l;
    __syncthreads();
    if (t >= D) return;
    float x = 0.f, L = 0.f;
#pragma unroll
    for (int w = 0; w < 8; ++w) {
        x += so[w][t];
        L += sl[w];
    }
    const float inv = L > 0.f ? 1.f / L : (L == 0.f ? 0.f : L);
    static_cast<InT *>(a.out)[((int64_t)u.row * a.Hq + r) * D + t] = from_f<InT>(x * inv);
}

template <typename InT, int D, int R>
cudaError_t launch_simt(const KvAttn &a, int unit_bound, int rows_max, cudaStream_t st) {
    using P = SimtPlan<InT, D, R>;
    if (P::kBytes > 48 * 1024) {
        const cudaError_t e = cudaFuncSetAttribute(kv_attn_simt_kernel<InT, D, R>,
                                                   cudaFuncAttributeMaxDynamicSharedMemorySize, (int)P::kBytes);
        if (e != cudaSuccess) return e;
    }
    const int row_tiles = (rows_max + R - 1) / R;
    const dim3 grid((unsigned)((int64_t)unit_bound * row_tiles), (unsigned)a.Hkv, (unsigned)a.n_seg);
    const cudaError_t e = gdn_launch_pdl(kv_attn_simt_kernel<InT, D, R>, grid, 256, P::kBytes, st, a, row_tiles);
    return e != cudaSuccess ? e : cudaGetLastError();
}

template <typename InT>
cudaError_t launch_simt_d(const KvAttn &a, int d, int unit_bound, int rows_max, int few, cudaStream_t st) {
    // few rows: tiles of 8 (a warp each), so that a single token's heads do not leave most of a 64-row tile idle
    if (d == 64) return few ? launch_simt<InT, 64, 8>(a, unit_bound, rows_max, st) : launch_simt<InT, 64, 64>(a, unit_bound, rows_max, st);
    if (d == 128) return few ? launch_simt<InT, 128, 8>(a, unit_bound, rows_max, st) : launch_simt<InT, 128, 64>(a, unit_bound, rows_max, st);
    return few ? launch_simt<InT, 256, 8>(a, unit_bound, rows_max, st) : launch_simt<InT, 256, 64>(a, unit_bound, rows_max, st);
}

template <typename InT, int D>
cudaError_t launch_join(const KvAttn &a, int unit_bound, int few, cudaStream_t st) {
    const int per_unit = a.tok_stride * a.Hq;
    if (few) {
        const cudaError_t e = gdn_launch_pdl(kv_join_few_kernel<InT, D>, dim3((unsigned)unit_bound, (unsigned)per_unit), 256, 0, st, a);
        return e != cudaSuccess ? e : cudaGetLastError();
    }
    const dim3 grid((unsigned)unit_bound, (unsigned)std::min((per_unit + 7) / 8, 64));
    const cudaError_t e = gdn_launch_pdl(kv_join_kernel<InT, D>, grid, 256, 0, st, a);
    return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace gdn

cudaError_t gdn_launch_kv_attn_simt(const gdn::KvAttn &a, int d, int unit_bound, int rows_max, int few, cudaStream_t st) {
    return gdn::launch_simt_d<float>(a, d, unit_bound, rows_max, few, st);
}

cudaError_t gdn_launch_kv_join(const gdn::KvAttn &a, int d, int bf16, int unit_bound, int few, cudaStream_t st) {
    using namespace gdn;
    using bf = __nv_bfloat16;
    if (d == 64) return bf16 ? launch_join<bf, 64>(a, unit_bound, few, st) : launch_join<float, 64>(a, unit_bound, few, st);
    if (d == 128) return bf16 ? launch_join<bf, 128>(a, unit_bound, few, st) : launch_join<float, 128>(a, unit_bound, few, st);
    return bf16 ? launch_join<bf, 256>(a, unit_bound, few, st) : launch_join<float, 256>(a, unit_bound, few, st);
}

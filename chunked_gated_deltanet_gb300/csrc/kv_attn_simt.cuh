// Attention over the paged 8-bit key/value cache in fp32 arithmetic, and the join of the segments' partial results.
//
// Per query row (token at position p, query head), with the block b = p / 64:
//   s_j = scale q . k_j over the blocks 0 .. b-1 (8 bits: k_j = k_scale[block] * int8) and block b's keys j <= p as they came,
//   out = sum_j exp(s_j - max) v_j / sum_j exp(s_j - max).
// One pass over the keys in position order, a 64-key block at a time, with the running maximum m and sum l in the
// log2 domain (the scale carries log2 e). Keys are cut into segments at absolute positions; each segment starts afresh
// and leaves (O, m, l), and the join adds the segments in order. What a row computes so depends on its position and
// the cache alone, not on the other rows of the call.
#pragma once

#include "kv_shared_piece.cuh"

#include <algorithm>
#include <type_traits>

namespace gdn {

// 16 int8 as floats: a byte b ^ 0x80 under 0x4B0000 reads 2^23 + 128 + b.
__device__ __forceinline__ void i8_to_f(const uint4 &u, float (&f)[16]) {
    const uint32_t w[4] = {u.x ^ 0x80808080u, u.y ^ 0x80808080u, u.z ^ 0x80808080u, u.w ^ 0x80808080u};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[4 * i] = __uint_as_float(__byte_perm(w[i], 0x4B000000u, 0x7440)) - 8388736.f;
        f[4 * i + 1] = __uint_as_float(__byte_perm(w[i], 0x4B000000u, 0x7441)) - 8388736.f;
        f[4 * i + 2] = __uint_as_float(__byte_perm(w[i], 0x4B000000u, 0x7442)) - 8388736.f;
        f[4 * i + 3] = __uint_as_float(__byte_perm(w[i], 0x4B000000u, 0x7443)) - 8388736.f;
    }
}
// 16 floats of a row that may not be there
__device__ __forceinline__ void ld_own16(const float *row, int col, float (&f)[16]) {
#pragma unroll
    for (int i = 0; i < 16; i += 4) {
        const float4 x = row ? *reinterpret_cast<const float4 *>(row + col + i) : make_float4(0.f, 0.f, 0.f, 0.f);
        f[i] = x.x; f[i + 1] = x.y; f[i + 2] = x.z; f[i + 3] = x.w;
    }
}

template <typename T> __device__ __forceinline__ T from_f(float x);
template <> __device__ __forceinline__ float from_f<float>(float x) { return x; }
template <> __device__ __forceinline__ __nv_bfloat16 from_f<__nv_bfloat16>(float x) { return __float2bfloat16_rn(x); }

// 64 rows of an 8-bit page from global memory, and as floats into shared memory (row stride LD; exact).
template <int D>
__device__ __forceinline__ void load_page(uint4 (&w)[D / 64], const int8_t *src) {
#pragma unroll
    for (int i = 0; i < D / 64; ++i) w[i] = __ldg(reinterpret_cast<const uint4 *>(src) + threadIdx.x + 256 * i);
}
template <int D, int LD>
__device__ __forceinline__ void store_page(float *dst, const uint4 (&w)[D / 64]) {
#pragma unroll
    for (int i = 0; i < D / 64; ++i) {
        const int e = threadIdx.x + 256 * i, r = e / (D / 16), c = (e % (D / 16)) * 16;
        float f[16];
        i8_to_f(w[i], f);
#pragma unroll
        for (int j = 0; j < 16; j += 4) *reinterpret_cast<float4 *>(dst + r * LD + c + j) = make_float4(f[j], f[j + 1], f[j + 2], f[j + 3]);
    }
}

// Row `off` of the rows' own block as it came: below u.first from the tail, the unit's own from the new rows, none after.
__device__ __forceinline__ const float *own_row(const KvAttn &a, const KvUnit &u, int kv, int h, int off, int D) {
    if (off < u.first) return static_cast<const float *>(a.c.tail) + kv_tail_offset(u.slot, u.src, kv, h, a.Hkv, D) + (int64_t)off * D;
    if (off < u.first + u.count)
        return static_cast<const float *>(kv ? a.v_new : a.k_new) + ((int64_t)(u.row + off - u.first) * a.Hkv + h) * D;
    return nullptr;
}

template <int D, int LD>
__device__ __forceinline__ void load_own(float *dst, const KvAttn &a, const KvUnit &u, int kv, int h) {
    for (int e = threadIdx.x; e < kKvBlock * D / 4; e += 256) {
        const int r = e / (D / 4), c = (e % (D / 4)) * 4;
        const float *s = own_row(a, u, kv, h, r, D);
        *reinterpret_cast<float4 *>(dst + r * LD + c) = s ? *reinterpret_cast<const float4 *>(s + c) : make_float4(0.f, 0.f, 0.f, 0.f);
    }
}

// Many rows: CTA (unit x tile of 64 rows, kv head, segment), 256 threads; thread (ty, tx) holds 4 rows, 4 keys of the scores
// and D / 16 columns of the output. Bound: the shared-memory reads (eight 16-byte
// ones beside 64 FMAs of a 4 x 4 tile), which halve the FMA rate. A prompt of 2,048 tokens, 2 heads of 64: 46 us with the
// join, 23 TFLOP/s.
template <int D>
struct SimtPlan {
    static constexpr int R = kKvSimtRows, LD = D + 4, PLD = kKvBlock + 4;   // 16-byte rows that start 4 banks apart
    static constexpr size_t kBytes = (size_t)(R * LD + kKvBlock * LD + R * PLD) * sizeof(float);
};

template <int D, int PART = kKvWhole>
__global__ void __launch_bounds__(256) kv_attn_simt_kernel(const KvAttn a, int row_tiles) {
    using P = SimtPlan<D>;
    constexpr int R = P::R, LD = P::LD, PLD = P::PLD, CT = D / 16;
    const KvBeside beside(PART == kKvSuffix);
    int h = blockIdx.y, ui = 0, r0 = 0, seg = blockIdx.z, seg0 = 0, last_seg = 0, start = 0, cut = a.seg_blocks;
    KvUnit u;
    if constexpr (PART == kKvShared) {
        // a group's rows as those of one unit that starts where the shared blocks end: every row sees all of them
        int4 rec;
        if (!kv_shared_piece<R>(a, r0, h, seg, cut, rec)) return;
        if (!kv_group_ok(a, rec)) {
            if (threadIdx.x == 0) atomicOr(a.err, kErrKvBounds);
            return;
        }
        u = {rec.z, rec.w, -1, 0, rec.y, rec.x, 0, 0};
        last_seg = INT32_MAX;   // no segment has a block of the rows' own
    } else {
        ui = a.unit0 + blockIdx.x / row_tiles;
        r0 = blockIdx.x % row_tiles * R;
        if (ui >= a.counts[0]) return;
        u = kv_load_unit(a.units, ui);
        if (PART == kKvSuffix) start = a.starts[ui];   // the first block of the pass
        last_seg = u.block / a.seg_blocks;
        if (!kv_part_unit_ok<PART>(a, u, start)) {
            if (threadIdx.x == 0) atomicOr(a.err, kErrKvBounds);
            return;
        }
        seg0 = kv_part_seg0<PART>(a, start);
        seg += seg0;
        if (seg > last_seg) return;
    }
    const int n_row = u.count * a.G;
    if (r0 >= n_row) return;

    extern __shared__ __align__(16) unsigned char simt_smem[];
    float *Q = reinterpret_cast<float *>(simt_smem), *KV = Q + R * LD, *Pm = KV + kKvBlock * LD;
    const int t = threadIdx.x, ty = t >> 4, tx = t & 15;
    const float *q = static_cast<const float *>(a.q);
    for (int e = t; e < R * D / 4; e += 256) {
        const int r = e / (D / 4), c = (e % (D / 4)) * 4;
        float4 f = make_float4(0.f, 0.f, 0.f, 0.f);
        if (r0 + r < n_row)
            f = *reinterpret_cast<const float4 *>(q + ((int64_t)(u.row + (r0 + r) / a.G) * a.Hq + h * a.G + (r0 + r) % a.G) * D + c);
        *reinterpret_cast<float4 *>(Q + r * LD + c) = f;
    }
    float o[4][CT], m[4], l[4];
    int limit[4];   // the last offset of its own block that a row sees
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        m[i] = -INFINITY;
        l[i] = 0.f;
        limit[i] = u.first + (r0 + ty * 4 + i) / a.G;
#pragma unroll
        for (int j = 0; j < CT; ++j) o[i][j] = 0.f;
    }
    // scores of the block in KV and their weights into Pm; then the block's values in KV
    auto scores = [&](auto raw_c, float ks, float vs) {
        constexpr bool raw = decltype(raw_c)::value;
        float s[4][4];
#pragma unroll
        for (int x = 0; x < 4; ++x)
#pragma unroll
            for (int y = 0; y < 4; ++y) s[x][y] = 0.f;
#pragma unroll 4
        for (int c = 0; c < D; c += 4) {
            float4 qf[4], kf[4];
#pragma unroll
            for (int x = 0; x < 4; ++x) qf[x] = *reinterpret_cast<const float4 *>(Q + (ty * 4 + x) * LD + c);
#pragma unroll
            for (int y = 0; y < 4; ++y) kf[y] = *reinterpret_cast<const float4 *>(KV + (tx + 16 * y) * LD + c);
#pragma unroll
            for (int x = 0; x < 4; ++x)
#pragma unroll
                for (int y = 0; y < 4; ++y) {
                    s[x][y] = fmaf(qf[x].x, kf[y].x, s[x][y]);
                    s[x][y] = fmaf(qf[x].y, kf[y].y, s[x][y]);
                    s[x][y] = fmaf(qf[x].z, kf[y].z, s[x][y]);
                    s[x][y] = fmaf(qf[x].w, kf[y].w, s[x][y]);
                }
        }
        const float c = a.scale_log2 * ks;
#pragma unroll
        for (int x = 0; x < 4; ++x) {
            float mb = -INFINITY;
#pragma unroll
            for (int y = 0; y < 4; ++y) {
                s[x][y] = raw && tx + 16 * y > limit[x] ? -INFINITY : s[x][y] * c;
                mb = fmaxf(mb, s[x][y]);
            }
#pragma unroll
            for (int w = 8; w > 0; w >>= 1) mb = fmaxf(mb, __shfl_xor_sync(0xffffffffu, mb, w));
            const float mn = fmaxf(m[x], mb), base = mn == -INFINITY ? 0.f : mn;
            const float corr = exp2f(m[x] - base);
            float sum = 0.f;
#pragma unroll
            for (int y = 0; y < 4; ++y) {
                const float p = exp2f(s[x][y] - base);
                sum += p;
                Pm[(ty * 4 + x) * PLD + tx + 16 * y] = p * vs;
            }
#pragma unroll
            for (int w = 8; w > 0; w >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, w);
            m[x] = mn;
            l[x] = l[x] * corr + sum;
#pragma unroll
            for (int j = 0; j < CT; ++j) o[x][j] *= corr;
        }
    };
    auto values = [&](auto raw_c) {
        constexpr bool raw = decltype(raw_c)::value;
        // a key that the mask took has weight zero; it adds nothing whatever its value (a NaN or an infinity after
        // the row's position does not reach the row)
#pragma unroll 2
        for (int k = 0; k < kKvBlock; k += 4) {
            float4 pf[4];
#pragma unroll
            for (int x = 0; x < 4; ++x) pf[x] = *reinterpret_cast<const float4 *>(Pm + (ty * 4 + x) * PLD + k);
#pragma unroll
            for (int kk = 0; kk < 4; ++kk) {
                float v[CT];
#pragma unroll
                for (int j = 0; j < CT / 4; ++j) {
                    const float4 f = *reinterpret_cast<const float4 *>(KV + (k + kk) * LD + 4 * tx + 64 * j);
                    v[4 * j] = f.x; v[4 * j + 1] = f.y; v[4 * j + 2] = f.z; v[4 * j + 3] = f.w;
                }
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    const float p = kk == 0 ? pf[x].x : kk == 1 ? pf[x].y : kk == 2 ? pf[x].z : pf[x].w;
                    if (raw && p == 0.f) continue;
#pragma unroll
                    for (int j = 0; j < CT; ++j) o[x][j] = fmaf(p, v[j], o[x][j]);
                }
            }
        }
    };
    const int b0 = max(seg * cut, start), b1 = min(u.block, (seg + 1) * cut);
    const int32_t *table = a.c.table + (int64_t)u.slot * a.c.max_blocks;
    // the head's part of block b's page, the page in bounds whatever the table holds (the result is reported as invalid then)
    auto part_of = [&](int b) {
        int page = table[b];
        if ((unsigned)page >= (unsigned)a.c.n_pages) {
            if (t == 0) atomicOr(a.err, kErrKvBounds);
            page = 0;
        }
        return (int64_t)page * a.Hkv + h;
    };
    // keys are loaded a block ahead, values while the scores are computed
    uint4 kw[D / 64], vw[D / 64];
    int64_t ph = b0 < b1 ? part_of(b0) : 0;
    if (b0 < b1) load_page<D>(kw, a.c.k + ph * kKvBlock * D);
#pragma unroll 1
    for (int b = b0; b < b1; ++b) {
        const float ks = a.c.k_scale[ph], vs = a.c.v_scale[ph];
        __syncthreads();   // the block before is done with KV and Pm (the first time: Q is written)
        store_page<D, LD>(KV, kw);
        load_page<D>(vw, a.c.v + ph * kKvBlock * D);
        __syncthreads();
        if (b + 1 < b1) {
            ph = part_of(b + 1);
            load_page<D>(kw, a.c.k + ph * kKvBlock * D);
        }
        scores(std::false_type{}, ks, vs);
        __syncthreads();   // K is read, P is written
        store_page<D, LD>(KV, vw);
        __syncthreads();
        values(std::false_type{});
    }
    if (seg == last_seg) {
        __syncthreads();
        load_own<D, LD>(KV, a, u, 0, h);
        __syncthreads();
        scores(std::true_type{}, 1.f, 1.f);
        __syncthreads();
        load_own<D, LD>(KV, a, u, 1, h);
        __syncthreads();
        values(std::true_type{});
    }
    // one segment: the result; several: the partial one (columns 4 tx + 64 j ..)
#pragma unroll
    for (int x = 0; x < 4; ++x) {
        const int r = r0 + ty * 4 + x;
        if (r >= n_row) continue;
        const int head = h * a.G + r % a.G;
        const bool one = PART == kKvWhole && last_seg == 0;
        const float inv = !one ? 1.f : l[x] > 0.f ? 1.f / l[x] : (l[x] == 0.f ? 0.f : l[x]);   // no key: zero; NaN stays
        float *dst;
        if (one) {
            dst = static_cast<float *>(a.out) + ((int64_t)(u.row + r / a.G) * a.Hq + head) * D;
        } else {
            const int64_t pr = PART == kKvWhole ? kv_part_row(a, ui, seg, r / a.G, head)
                                                : kv_shared_part_row(a, PART == kKvShared ? seg : a.n_pre + seg - seg0, u.row + r / a.G, head);
            dst = a.part_o + pr * D;
            if (tx == 0) a.part_ml[pr] = make_float2(m[x], l[x]);
        }
#pragma unroll
        for (int j = 0; j < CT; j += 4)
            *reinterpret_cast<float4 *>(dst + 4 * tx + 16 * j) = make_float4(o[x][j] * inv, o[x][j + 1] * inv, o[x][j + 2] * inv, o[x][j + 3] * inv);
    }
}

template <int D, int PART = kKvWhole>
cudaError_t launch_simt_many(const KvAttn &a, int n, int rows_max, cudaStream_t st) {   // n: units, or the most pieces (kKvShared)
    using P = SimtPlan<D>;
    const cudaError_t e = cudaFuncSetAttribute(kv_attn_simt_kernel<D, PART>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)P::kBytes);
    if (e != cudaSuccess) return e;
    const int row_tiles = PART == kKvShared ? 1 : (rows_max + P::R - 1) / P::R;
    const dim3 grid = PART == kKvShared ? kv_shared_grid(a, n) : dim3((unsigned)((int64_t)n * row_tiles), (unsigned)a.Hkv, (unsigned)a.n_seg);
    return gdn_launch_pdl(kv_attn_simt_kernel<D, PART>, grid, 256, P::kBytes, st, a, row_tiles);
}

}  // namespace gdn

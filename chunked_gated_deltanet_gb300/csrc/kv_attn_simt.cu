// Attention over the 8-bit cache in fp32 arithmetic (many rows: kv_attn_simt.cuh; few rows here), and the join of the
// segments' partial results.
#include "kv_attn_simt.cuh"

namespace gdn {

// Few rows (a single token's heads): CTA (unit x tile of RT rows, kv head, segment), 4 warps, every fourth block each.
//   scores   lane (g, t) = (lane / 4, lane % 4): 16 values of key 8 i + g at columns 16 t + 64 j, times RT rows' q from
//            shared memory, added over t;
//   output   lane (r, c): 16 columns 16 c of the keys = r modulo the rows a warp reads at once, added over r at the end.
// The warps' results are added in order. Bound: the latency of a few dependent reads, then HBM.
// 16 tokens over 100 to 4,096 keys (8/8 heads of 64): 12 us with the join, 1.7 TB/s.
template <int D, int RT>
__global__ void __launch_bounds__(128) kv_attn_few_simt_kernel(const KvAttn a, int row_tiles) {
    constexpr int J = D / 64, LPR = D / 16, KPR = 32 / LPR;   // 16-column chunks of a lane; lanes of a value row, rows at once
    grid_dep_wait();
    grid_dep_launch();
    const int ui = a.unit0 + blockIdx.x / row_tiles, r0 = blockIdx.x % row_tiles * RT, h = blockIdx.y, seg = blockIdx.z;
    const KvUnit u = kv_load_unit(a.units, ui);   // inside the map whatever the count
    if (ui >= a.counts[0]) return;
    const int last_seg = u.block / a.seg_blocks, n_row = u.count * a.G;
    if (!kv_attn_unit_ok(a, u)) {
        if (threadIdx.x == 0) atomicOr(a.err, kErrKvBounds);
        return;
    }
    if (r0 >= n_row || seg > last_seg) return;
    __shared__ __align__(16) float sq[RT][D], sp[4][RT][kKvBlock], so[4][RT][D], sm[4][RT], sl[4][RT];
    const int t = threadIdx.x, warp = t >> 5, lane = t & 31, g = lane >> 2, tq = lane & 3, vr = lane / LPR, vc = lane % LPR;
    for (int e = t; e < RT * D / 4; e += 128) {
        const int r = r0 + e / (D / 4), c = e % (D / 4) * 4;
        float4 f = make_float4(0.f, 0.f, 0.f, 0.f);
        if (r < n_row)
            f = *reinterpret_cast<const float4 *>(static_cast<const float *>(a.q) + ((int64_t)(u.row + r / a.G) * a.Hq + h * a.G + r % a.G) * D + c);
        *reinterpret_cast<float4 *>(&sq[e / (D / 4)][c]) = f;
    }
    __syncthreads();
    float o[RT][16], m[RT], l[RT];
#pragma unroll
    for (int x = 0; x < RT; ++x) {
        m[x] = -INFINITY;
        l[x] = 0.f;
#pragma unroll
        for (int j = 0; j < 16; ++j) o[x][j] = 0.f;
    }
    // complete blocks, then 16 keys a warp of the rows' own, the first by the warp whose turn it is (one warp for all of them
    // would be the longest part of a short context)
    const int own0 = 16 * ((warp - u.block) & 3);
    auto block_step = [&](auto raw_c, int b) {
        constexpr bool raw = decltype(raw_c)::value;
        int64_t ph = 0;
        float c = a.scale_log2, vs = 1.f;
        if constexpr (!raw) {
            int page = a.c.table[(int64_t)u.slot * a.c.max_blocks + b];
            if ((unsigned)page >= (unsigned)a.c.n_pages) {
                if (lane == 0) atomicOr(a.err, kErrKvBounds);
                page = 0;   // in bounds; the result is reported as invalid
            }
            ph = (int64_t)page * a.Hkv + h;
            c *= a.c.k_scale[ph];
            vs = a.c.v_scale[ph];
        }
        const int8_t *kp = a.c.k + ph * (kKvBlock * D) + g * D + 16 * tq, *vp = a.c.v + ph * (kKvBlock * D) + vr * D + 16 * vc;
        float s[RT][8];   // keys 8 i + g
#pragma unroll
        for (int i = 0; i < 8; ++i) {
#pragma unroll
            for (int x = 0; x < RT; ++x) s[x][i] = 0.f;
            if (raw && 16 * (i / 2) != own0) continue;
#pragma unroll
            for (int j = 0; j < J; ++j) {
                float f[16];
                if constexpr (!raw) i8_to_f(__ldg(reinterpret_cast<const uint4 *>(kp + 8 * i * D + 64 * j)), f);
                else ld_own16(own_row(a, u, 0, h, 8 * i + g, D), 64 * j + 16 * tq, f);
#pragma unroll
                for (int x = 0; x < RT; ++x)
#pragma unroll
                    for (int k = 0; k < 16; k += 4) {
                        const float4 qf = *reinterpret_cast<const float4 *>(&sq[x][64 * j + 16 * tq + k]);
                        s[x][i] = fmaf(qf.x, f[k], s[x][i]);
                        s[x][i] = fmaf(qf.y, f[k + 1], s[x][i]);
                        s[x][i] = fmaf(qf.z, f[k + 2], s[x][i]);
                        s[x][i] = fmaf(qf.w, f[k + 3], s[x][i]);
                    }
            }
        }
        __syncwarp();   // the block before is done with sp
#pragma unroll
        for (int x = 0; x < RT; ++x) {
            const int limit = raw ? u.first + (r0 + x) / a.G : kKvBlock;
            float mb = -INFINITY;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                s[x][i] += __shfl_xor_sync(0xffffffffu, s[x][i], 1);
                s[x][i] += __shfl_xor_sync(0xffffffffu, s[x][i], 2);
                s[x][i] = 8 * i + g > limit || (raw && 16 * (i / 2) != own0) ? -INFINITY : s[x][i] * c;
                mb = fmaxf(mb, s[x][i]);
            }
#pragma unroll
            for (int w = 4; w < 32; w <<= 1) mb = fmaxf(mb, __shfl_xor_sync(0xffffffffu, mb, w));
            const float mn = fmaxf(m[x], mb), base = mn == -INFINITY ? 0.f : mn;
            const float corr = exp2f(m[x] - base);
            float sum = 0.f;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float p = exp2f(s[x][i] - base);
                sum += p;
                if (tq == 0) sp[warp][x][8 * i + g] = p * vs;
            }
#pragma unroll
            for (int w = 4; w < 32; w <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, w);
            m[x] = mn;
            l[x] = l[x] * corr + sum;
#pragma unroll
            for (int j = 0; j < 16; ++j) o[x][j] *= corr;
        }
        __syncwarp();
        const int k1 = raw ? own0 + 16 : kKvBlock;
#pragma unroll 4
        for (int k = raw ? own0 : 0; k < k1; k += KPR) {
            float f[16];
            if constexpr (!raw) i8_to_f(__ldg(reinterpret_cast<const uint4 *>(vp + k * D)), f);
            else ld_own16(own_row(a, u, 1, h, k + vr, D), 16 * vc, f);
#pragma unroll
            for (int x = 0; x < RT; ++x) {
                const float p = sp[warp][x][k + vr];
                if (raw && p == 0.f) continue;   // masked: nothing, whatever the value
#pragma unroll
                for (int j = 0; j < 16; ++j) o[x][j] = fmaf(p, f[j], o[x][j]);
            }
        }
    };
    const int b0 = seg * a.seg_blocks, b1 = min(u.block, b0 + a.seg_blocks);
    for (int b = b0 + warp; b < b1; b += 4) block_step(std::false_type{}, b);
    if (seg == last_seg && own0 < u.first + u.count) block_step(std::true_type{}, u.block);
#pragma unroll
    for (int x = 0; x < RT; ++x) {
#pragma unroll
        for (int j = 0; j < 16; ++j) {
#pragma unroll
            for (int w = LPR; w < 32; w <<= 1) o[x][j] += __shfl_xor_sync(0xffffffffu, o[x][j], w);
            if (vr == 0) so[warp][x][16 * vc + j] = o[x][j];
        }
        if (lane == 0) {
            sm[warp][x] = m[x];
            sl[warp][x] = l[x];
        }
    }
    __syncthreads();
    for (int e = t; e < RT * D; e += 128) {
        const int x = e / D, col = e % D, r = r0 + x;
        if (r >= n_row) break;
        const float M = fmaxf(fmaxf(sm[0][x], sm[1][x]), fmaxf(sm[2][x], sm[3][x])), base = M == -INFINITY ? 0.f : M;
        float y = 0.f, L = 0.f;
#pragma unroll
        for (int w = 0; w < 4; ++w) {
            const float f = exp2f(sm[w][x] - base);
            y = fmaf(f, so[w][x][col], y);
            L = fmaf(f, sl[w][x], L);
        }
        const int head = h * a.G + r % a.G;
        if (last_seg == 0) {
            const float inv = L > 0.f ? 1.f / L : (L == 0.f ? 0.f : L);
            static_cast<float *>(a.out)[((int64_t)(u.row + r / a.G) * a.Hq + head) * D + col] = y * inv;
        } else {
            const int64_t pr = kv_part_row(a, ui, seg, r / a.G, head);
            a.part_o[pr * D + col] = y;
            if (col == 0) a.part_ml[pr] = make_float2(M, L);
        }
    }
}

// Rows of a unit with more than one segment: out = sum_s 2^{m_s - M} O_s / sum_s 2^{m_s - M} l_s, s in order.
// A warp per (token, query head); lane c / 4 of every 128 columns holds column c .. c + 3 (d = 64: two per lane).
// Bound: HBM latency; 64,000 rows of 6 segments, d = 128: 43 us, 4.3 TB/s (four segments' loads in flight: 47).
template <typename InT, int D>
__global__ void __launch_bounds__(256) kv_join_kernel(const KvAttn a) {
    grid_dep_wait();
    grid_dep_launch();
    const int ui = a.unit0 + blockIdx.x;
    if (ui >= a.counts[0]) return;
    const KvUnit u = kv_load_unit(a.units, ui);
    const int n_seg = kv_seg_of(a, u.block) + 1;
    if (!kv_attn_unit_ok(a, u) || n_seg == 1) return;
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

// The same for the few-row form, whose rows have many segments: a CTA per (token, query head) and unit, units innermost,
// warp w taking segments w, w + 8, ... and the eight sums added in order.
template <typename InT, int D, int B>
__global__ void __launch_bounds__(256) kv_join_few_kernel(const KvAttn a, int n_units) {
    grid_dep_wait();
    grid_dep_launch();
    const int r = blockIdx.x / n_units, ui = a.unit0 + blockIdx.x % n_units;
    const KvUnit u = kv_load_unit(a.units, ui);
    if (ui >= a.counts[0]) return;
    const int n_seg = u.block / a.seg_blocks + 1;
    if (!kv_attn_unit_ok(a, u) || n_seg == 1 || r >= u.count * a.Hq) return;
    constexpr int W = D == 64 ? 2 : 4, N = D / (32 * W);
    __shared__ float so[8][D], sl[8];
    const int t = threadIdx.x, warp = t >> 5, lane = t & 31;
    const int64_t stride = a.part_rows, pr = kv_part_row(a, ui, 0, 0, 0) + r;
    // B of the warp's segments at a time, the first before the maximum is known: one latency for all of them
    float2 ml[B];
    float v[B][N][W];
    auto load = [&](int s0) {
#pragma unroll
        for (int i = 0; i < B; ++i) {
            const int s = s0 + 8 * i;
            ml[i] = make_float2(-INFINITY, 0.f);
            if (s < n_seg) ml[i] = a.part_ml[s * stride + pr];
            const float *src = a.part_o + (s * stride + pr) * D;
#pragma unroll
            for (int j = 0; j < N; ++j) {
#pragma unroll
                for (int k = 0; k < W; ++k) v[i][j][k] = 0.f;
                if (s >= n_seg) continue;
                if constexpr (W == 4) *reinterpret_cast<float4 *>(v[i][j]) = *reinterpret_cast<const float4 *>(src + W * (lane + 32 * j));
                else *reinterpret_cast<float2 *>(v[i][j]) = *reinterpret_cast<const float2 *>(src + W * (lane + 32 * j));
            }
        }
    };
    load(warp);
    float M = -INFINITY;
#pragma unroll 4
    for (int s = lane; s < n_seg; s += 32) M = fmaxf(M, a.part_ml[s * stride + pr].x);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
    const float base = M == -INFINITY ? 0.f : M;
    float o[N][W], l = 0.f;
#pragma unroll
    for (int j = 0; j < N; ++j)
#pragma unroll
        for (int k = 0; k < W; ++k) o[j][k] = 0.f;
#pragma unroll 1
    for (int s0 = warp; s0 < n_seg; s0 += 8 * B) {
        if (s0 != warp) load(s0);
#pragma unroll
        for (int i = 0; i < B; ++i) {
            const float f = exp2f(ml[i].x - base);   // 0 for a segment that is not there
            l = fmaf(f, ml[i].y, l);
#pragma unroll
            for (int j = 0; j < N; ++j)
#pragma unroll
                for (int k = 0; k < W; ++k) o[j][k] = fmaf(f, v[i][j][k], o[j][k]);
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

template <int D>
cudaError_t launch_simt(const KvAttn &a, int unit_bound, int rows_max, int few, cudaStream_t st) {
    cudaError_t e;
    if (few) {
        // rows per CTA: what there is, up to 4 (16 columns each in registers)
        const int rt = rows_max == 1 ? 1 : rows_max == 2 ? 2 : 4, row_tiles = (rows_max + rt - 1) / rt;
        const dim3 grid((unsigned)((int64_t)unit_bound * row_tiles), (unsigned)a.Hkv, (unsigned)a.n_seg);
        e = rt == 1 ? gdn_launch_pdl(kv_attn_few_simt_kernel<D, 1>, grid, 128, 0, st, a, row_tiles)
            : rt == 2 ? gdn_launch_pdl(kv_attn_few_simt_kernel<D, 2>, grid, 128, 0, st, a, row_tiles)
                      : gdn_launch_pdl(kv_attn_few_simt_kernel<D, 4>, grid, 128, 0, st, a, row_tiles);
    } else {
        e = launch_simt_many<D>(a, unit_bound, rows_max, st);
    }
    return e != cudaSuccess ? e : cudaGetLastError();
}

template <typename InT, int D>
cudaError_t launch_join(const KvAttn &a, int unit_bound, int few, cudaStream_t st) {
    const int per_unit = a.tok_stride * a.Hq;
    if (few) {
        // loads under way against CTAs on an SM, with the attention: 82 segments of 16 rows, d = 256, 23.3 us with eight and
        // 24.7 with two; 8 segments of 2,048 rows, d = 128, 112.9 and 109.8
        const unsigned grid = (unsigned)((int64_t)unit_bound * per_unit);   // rows of the workspace: far below 2^31
        const cudaError_t e = a.n_seg > 32 ? gdn_launch_pdl(kv_join_few_kernel<InT, D, 8>, grid, 256, 0, st, a, unit_bound)
                                           : gdn_launch_pdl(kv_join_few_kernel<InT, D, 2>, grid, 256, 0, st, a, unit_bound);
        return e != cudaSuccess ? e : cudaGetLastError();
    }
    const dim3 grid((unsigned)unit_bound, (unsigned)std::min((per_unit + 7) / 8, 64));
    const cudaError_t e = gdn_launch_pdl(kv_join_kernel<InT, D>, grid, 256, 0, st, a);
    return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace gdn

cudaError_t gdn_launch_kv_attn_simt(const gdn::KvAttn &a, int d, int unit_bound, int rows_max, int few, cudaStream_t st) {
    if (d == 64) return gdn::launch_simt<64>(a, unit_bound, rows_max, few, st);
    if (d == 128) return gdn::launch_simt<128>(a, unit_bound, rows_max, few, st);
    return gdn::launch_simt<256>(a, unit_bound, rows_max, few, st);
}

cudaError_t gdn_launch_kv_join(const gdn::KvAttn &a, int d, int bf16, int unit_bound, int few, cudaStream_t st) {
    using namespace gdn;
    using bf = __nv_bfloat16;
    if (d == 64) return bf16 ? launch_join<bf, 64>(a, unit_bound, few, st) : launch_join<float, 64>(a, unit_bound, few, st);
    if (d == 128) return bf16 ? launch_join<bf, 128>(a, unit_bound, few, st) : launch_join<float, 128>(a, unit_bound, few, st);
    return bf16 ? launch_join<bf, 256>(a, unit_bound, few, st) : launch_join<float, 256>(a, unit_bound, few, st);
}

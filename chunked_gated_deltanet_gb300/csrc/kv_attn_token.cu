// Attention of few query rows (single tokens, short continuations) over the paged 8-bit key/value cache, bf16 inputs.
//
// The mathematics is that of kv_attn_prompt.cu (weights with the value scale in the running exponent, fp16; the row's own
// block in two bf16 products), on warp-level MMAs: with up to 16 rows the work is reading the cache, 2 d bytes a key and
// head against 4 d flops a row, and tcgen05's 128 rows would be empty.
//
// CTA (unit, kv head, segment of 8 blocks), 4 warps, two blocks each in position order. A warp reads its keys and values
// from global memory straight into the fragments of the products, without shared memory: the order of the reduction
// index of a product is free as long as both operands share it, so
//   S = q K^T     m16n8k16, A = q (rows), B = 8 keys; lane (g, t) = (lane / 4, lane % 4) reads 16 bytes of key 8 a + g at
//                 columns 64 j + 16 t: four k-steps of four columns each;
//   O += P V      A = P in the score fragments' own layout; lane (g, t) reads d / 8 bytes at column g d / 8 of the four keys
//                 that its weights belong to: byte i of them is n-tile i, so O's column n of n-tile i is n d / 8 + i.
// Units of UK keys are loaded one ahead. The four warps' results are added in order in shared memory.
// Bound: HBM.
#include "kv_attn.cuh"
#include "umma.cuh"

#include <algorithm>

namespace gdn {

constexpr int kTokenWarps = 4, kTokenBlocks = 2;   // blocks of a warp: kTokenWarps * kTokenBlocks = the segment's

__device__ __forceinline__ void mma_f16(float (&d)[4], const uint32_t (&a)[4], const uint32_t (&b)[2]) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
        "{%0,%1,%2,%3};\n"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b[0]), "r"(b[1]));
}

template <int D, int R>
struct TokenPlan {
    static constexpr int UK = D == 256 ? 16 : 32;   // keys of a unit: 64 registers of loads in flight at most
    static constexpr int NA = UK / 8;               // key n-tiles
    static constexpr int J = D / 64;                // 16-byte chunks of a key row per lane
    static constexpr int W = D / 32;                // 32-bit words of a value row per lane
    static constexpr int NO = D / 8;                // output n-tiles
    static constexpr int RF = R / 8;                // row halves of a fragment in use
    static constexpr size_t kBytes = kTokenWarps * R * (D + 2) * sizeof(float);
};

// N 32-bit words from global memory (N = 2 or a multiple of 4)
template <int N>
__device__ __forceinline__ void ld_words(uint32_t (&w)[N], const void *p) {
    if constexpr (N == 2) {
        const uint2 x = __ldg(static_cast<const uint2 *>(p));
        w[0] = x.x; w[1] = x.y;
    } else {
#pragma unroll
        for (int i = 0; i < N / 4; ++i) {
            const uint4 x = __ldg(static_cast<const uint4 *>(p) + i);
            w[4 * i] = x.x; w[4 * i + 1] = x.y; w[4 * i + 2] = x.z; w[4 * i + 3] = x.w;
        }
    }
}

template <int D, int R>
__global__ void __launch_bounds__(32 * kTokenWarps) kv_attn_token_kernel(const KvAttn a) {
    using P = TokenPlan<D, R>;
    using bf = __nv_bfloat16;
    constexpr int UK = P::UK, NA = P::NA, J = P::J, W = P::W, NO = P::NO, RF = P::RF;
    grid_dep_wait();
    grid_dep_launch();
    const int ui = a.unit0 + blockIdx.x, h = blockIdx.y, seg = blockIdx.z;
    if (ui >= a.counts[0]) return;
    const KvUnit u = kv_load_unit(a.units, ui);
    const int last_seg = u.block / a.seg_blocks;
    const int n_row = u.count * a.G;
    if (!kv_unit_ok(u, a.c, a.n_rows) || u.count > a.max_new || last_seg >= a.n_seg || n_row > R) {
        if (threadIdx.x == 0) atomicOr(a.err, kErrKvBounds);
        return;
    }
    if (seg > last_seg) return;
    const int t = threadIdx.x, warp = t >> 5, lane = t & 31, g = lane >> 2, tq = lane & 3;
    const int32_t *table = a.c.table + (int64_t)u.slot * a.c.max_blocks;

    // this warp's 8-bit blocks [w0, w1), and whether its last block is the row's own
    const int w0 = seg * a.seg_blocks + kTokenBlocks * warp, w1 = min(u.block, w0 + kTokenBlocks);
    const int n_unit = max(w1 - w0, 0) * (kKvBlock / UK);
    const bool raw_here = w0 <= u.block && u.block < w0 + kTokenBlocks;
    int page[kTokenBlocks];
    float c8[kTokenBlocks], lv[kTokenBlocks], iv[kTokenBlocks];
#pragma unroll
    for (int i = 0; i < kTokenBlocks; ++i) {
        page[i] = 0;
        c8[i] = lv[i] = 0.f;
        iv[i] = 1.f;
        if (w0 + i < w1) {
            const int pg = table[w0 + i];
            if ((unsigned)pg < (unsigned)a.c.n_pages) {
                page[i] = pg;
                c8[i] = a.scale_log2 * a.c.k_scale[(int64_t)pg * a.Hkv + h];
            } else if (lane == 0) {
                atomicOr(a.err, kErrKvBounds);   // page 0 is read instead; the result is reported as invalid
            }
        }
    }

    uint32_t kb[NA][J][4], vb[UK / 16][4][W];
    auto load_k = [&](int n) {
        const int blk = n / (kKvBlock / UK), k0 = n % (kKvBlock / UK) * UK;
        const int8_t *src = a.c.k + ((int64_t)(blk == 0 ? page[0] : page[1]) * a.Hkv + h) * (kKvBlock * D) + (k0 + g) * D + 16 * tq;
#pragma unroll
        for (int x = 0; x < NA; ++x)
#pragma unroll
            for (int j = 0; j < J; ++j) ld_words(kb[x][j], src + 8 * x * D + 64 * j);
    };
    auto load_v = [&](int n) {
        const int blk = n / (kKvBlock / UK), k0 = n % (kKvBlock / UK) * UK;
        const int8_t *src = a.c.v + ((int64_t)(blk == 0 ? page[0] : page[1]) * a.Hkv + h) * (kKvBlock * D) + (k0 + 2 * tq) * D + g * NO;
#pragma unroll
        for (int x = 0; x < UK / 16; ++x)
#pragma unroll
            for (int y = 0; y < 4; ++y) ld_words(vb[x][y], src + (16 * x + (y & 1) + 8 * (y >> 1)) * D);
    };
    if (n_unit > 0) {
        load_k(0);
        load_v(0);
    }
    // value scales (and, while the loads are under way, the queries)
#pragma unroll
    for (int i = 0; i < kTokenBlocks; ++i)
        if (w0 + i < w1) {
            lv[i] = kv_log2_vscale(a, table, w0 + i, h, 9);
            iv[i] = ex2(-lv[i]);
        }
    const float lraw = raw_here ? kv_log2_vscale(a, table, u.block - 1, h, 9) : 0.f;
    uint32_t qa[J][4][2 * RF];   // per k-step: columns 0, 1 and 2, 3 of the lane's four, rows g (and g + 8)
    const bf *q = static_cast<const bf *>(a.q);
#pragma unroll
    for (int f = 0; f < RF; ++f) {
        const int r = g + 8 * f;
        const bf *src = q + ((int64_t)(u.row + r / a.G) * a.Hq + h * a.G + r % a.G) * D + 16 * tq;
#pragma unroll
        for (int j = 0; j < J; ++j) {
            uint32_t w[8] = {0, 0, 0, 0, 0, 0, 0, 0};
            if (r < n_row) ld_words(w, src + 64 * j);
#pragma unroll
            for (int s = 0; s < 4; ++s) {
                qa[j][s][f] = w[2 * s];
                qa[j][s][RF + f] = w[2 * s + 1];
            }
        }
    }

    float o[NO][2 * RF], m[RF], l[RF], dead[2] = {0.f, 0.f};
#pragma unroll
    for (int i = 0; i < NO; ++i)
#pragma unroll
        for (int f = 0; f < 2 * RF; ++f) o[i][f] = 0.f;
#pragma unroll
    for (int f = 0; f < RF; ++f) {
        m[f] = -INFINITY;
        l[f] = 0.f;
    }
    // One product on fragments whose rows 8..15 may be absent (R = 8): their accumulators stay zero and are shared.
    auto mma_rows = [&](float *acc, const uint32_t *x, const uint32_t (&b)[2], bool half) {
        float d4[4] = {acc[0], acc[1], RF == 2 ? acc[2] : dead[0], RF == 2 ? acc[3] : dead[1]};
        const uint32_t a4[4] = {x[0], RF == 2 ? x[1] : 0u, x[RF], RF == 2 ? x[3] : 0u};
        if (half) mma_f16(d4, a4, b);
        else mma_bf16(d4, a4, b);
        acc[0] = d4[0];
        acc[1] = d4[1];
        if (RF == 2) {
            acc[2] = d4[2];
            acc[3] = d4[3];
        }
    };
    // Scores -> weights of a unit: the running maximum (of c s + lv) and sum, O rescaled; s holds the weights after.
    auto softmax = [&](float (&s)[NA][2 * RF], float c, float lvs, float ivs, bool raw) {
#pragma unroll
        for (int f = 0; f < RF; ++f) {
            float top = -INFINITY;
#pragma unroll
            for (int x = 0; x < NA; ++x) top = fmaxf(top, fmaxf(s[x][2 * f], s[x][2 * f + 1]));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
            if (top > -INFINITY) top = top * c + lvs;
            const float mn = fmaxf(m[f], top), base = mn == -INFINITY ? 0.f : mn;
            const float corr = ex2(m[f] - base);
            m[f] = mn;
            const float add = raw ? -base : lvs - base;
            float sum = 0.f;
#pragma unroll
            for (int x = 0; x < NA; ++x)
#pragma unroll
                for (int y = 0; y < 2; ++y) {
                    const float p = ex2(fmaf(s[x][2 * f + y], c, add));
                    s[x][2 * f + y] = p;
                    sum += p;
                }
            sum += __shfl_xor_sync(0xffffffffu, sum, 1);
            sum += __shfl_xor_sync(0xffffffffu, sum, 2);
            l[f] = fmaf(sum, ivs, l[f] * corr);
            if (corr != 1.f) {
#pragma unroll
                for (int i = 0; i < NO; ++i) {
                    o[i][2 * f] *= corr;
                    o[i][2 * f + 1] *= corr;
                }
            }
        }
    };

    for (int n = 0; n < n_unit; ++n) {
        const bool first = n < kKvBlock / UK;
        float s[NA][2 * RF];
#pragma unroll
        for (int x = 0; x < NA; ++x) {
#pragma unroll
            for (int f = 0; f < 2 * RF; ++f) s[x][f] = 0.f;
#pragma unroll
            for (int j = 0; j < J; ++j)
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const uint2 b2 = i8_to_bf16x4(kb[x][j][k]);
                    const uint32_t b[2] = {b2.x, b2.y};
                    mma_rows(s[x], qa[j][k], b, false);
                }
        }
        if (n + 1 < n_unit) load_k(n + 1);
        softmax(s, first ? c8[0] : c8[1], first ? lv[0] : lv[1], first ? iv[0] : iv[1], false);
#pragma unroll
        for (int x = 0; x < UK / 16; ++x) {
            uint32_t pa[2 * RF];   // rows g (g + 8) of the first and of the second 8 keys
#pragma unroll
            for (int f = 0; f < RF; ++f) {
                pa[f] = f2_to_h2(s[2 * x][2 * f], s[2 * x][2 * f + 1]);
                pa[RF + f] = f2_to_h2(s[2 * x + 1][2 * f], s[2 * x + 1][2 * f + 1]);
            }
#pragma unroll
            for (int w = 0; w < W; ++w) {
                const uint32_t off = 0x64806480u;
                uint32_t e[2][4];   // per key pair, byte i of both keys as fp16
#pragma unroll
                for (int y = 0; y < 2; ++y) {
                    const uint32_t x0 = vb[x][2 * y][w] ^ 0x80808080u, x1 = vb[x][2 * y + 1][w] ^ 0x80808080u;
                    const uint32_t lo = __byte_perm(x0, x1, 0x5140), hi = __byte_perm(x0, x1, 0x7362);
                    const uint32_t v[4] = {__byte_perm(lo, 0x64646464u, 0x4140), __byte_perm(lo, 0x64646464u, 0x4342),
                                           __byte_perm(hi, 0x64646464u, 0x4140), __byte_perm(hi, 0x64646464u, 0x4342)};
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const __half2 d2 = __hsub2(*reinterpret_cast<const __half2 *>(&v[i]), *reinterpret_cast<const __half2 *>(&off));
                        e[y][i] = *reinterpret_cast<const uint32_t *>(&d2);
                    }
                }
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const uint32_t b[2] = {e[0][i], e[1][i]};
                    mma_rows(o[4 * w + i], pa, b, true);
                }
            }
        }
        if (n + 1 < n_unit) load_v(n + 1);
    }

    // the row's own block as it came: 16 keys at a time
    bool odd_value = false;
    if (raw_here) {
        const bf *tail = static_cast<const bf *>(a.c.tail);
        auto raw_row = [&](int kv, int off) -> const bf * {
            if (off < u.first) return tail + kv_tail_offset(u.slot, u.src, kv, h, a.Hkv, D) + (int64_t)off * D;
            if (off < u.first + u.count)
                return static_cast<const bf *>(kv ? a.v_new : a.k_new) + ((int64_t)(u.row + off - u.first) * a.Hkv + h) * D;
            return nullptr;
        };
        const int n_key = u.first + u.count;
        for (int k0 = 0; k0 < n_key; k0 += 16) {
            float s[NA][2 * RF];
#pragma unroll
            for (int x = 0; x < NA; ++x)
#pragma unroll
                for (int f = 0; f < 2 * RF; ++f) s[x][f] = x < 2 ? 0.f : -INFINITY;
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                const bf *src = raw_row(0, k0 + 8 * x + g);
#pragma unroll
                for (int j = 0; j < J; ++j) {
                    uint32_t w[8] = {0, 0, 0, 0, 0, 0, 0, 0};
                    if (src) ld_words(w, src + 64 * j + 16 * tq);
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const uint32_t b[2] = {w[2 * k], w[2 * k + 1]};
                        mma_rows(s[x], qa[j][k], b, false);
                    }
                }
#pragma unroll
                for (int f = 0; f < RF; ++f)
#pragma unroll
                    for (int y = 0; y < 2; ++y)
                        if (k0 + 8 * x + 2 * tq + y > u.first + (g + 8 * f) / a.G) s[x][2 * f + y] = -INFINITY;
            }
            softmax(s, a.scale_log2, lraw, 1.f, true);
            uint32_t ph[2 * RF], pl[2 * RF];
#pragma unroll
            for (int f = 0; f < RF; ++f)
#pragma unroll
                for (int x = 0; x < 2; ++x) split_bf16x2(s[x][2 * f], s[x][2 * f + 1], ph[x * RF + f], pl[x * RF + f]);
#pragma unroll
            for (int i = 0; i < NO / 8; ++i) {   // eight columns of the four keys
                uint32_t v[4][4];
#pragma unroll
                for (int y = 0; y < 4; ++y) {
                    const bf *src = raw_row(1, k0 + 2 * tq + (y & 1) + 8 * (y >> 1));
                    v[y][0] = v[y][1] = v[y][2] = v[y][3] = 0;
                    if (src) ld_words(v[y], src + g * NO + 8 * i);
                    // a value that is not finite would reach rows that do not see it (0 * inf): left out here, and added
                    // by the rows that do at the end
#pragma unroll
                    for (int w = 0; w < 4; ++w) {
                        if ((v[y][w] & 0x7F80u) == 0x7F80u) { v[y][w] &= 0xFFFF0000u; odd_value = true; }
                        if ((v[y][w] & 0x7F800000u) == 0x7F800000u) { v[y][w] &= 0xFFFFu; odd_value = true; }
                    }
                }
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    const uint32_t sel = k & 1 ? 0x7632 : 0x5410;
                    const uint32_t b[2] = {__byte_perm(v[0][k / 2], v[1][k / 2], sel), __byte_perm(v[2][k / 2], v[3][k / 2], sel)};
                    mma_rows(o[8 * i + k], ph, b, false);
                    mma_rows(o[8 * i + k], pl, b, false);
                }
            }
        }
        if (__any_sync(0xffffffffu, odd_value)) {
#pragma unroll
            for (int f = 0; f < RF; ++f) {
                const int r = g + 8 * f, n_see = r < n_row ? u.first + r / a.G + 1 : 0;
#pragma unroll 1
                for (int k = 0; k < n_see; ++k) {
                    const bf *src = raw_row(1, k) + 2 * tq * NO;
#pragma unroll
                    for (int i = 0; i < NO; ++i)
#pragma unroll
                        for (int y = 0; y < 2; ++y) {
                            const float x = to_f(src[y * NO + i]);
                            if (!(fabsf(x) <= 3.4e38f)) o[i][2 * f + y] += x;
                        }
                }
            }
        }
    }

    // the warps' results, added in order
    extern __shared__ __align__(16) float token_smem[];
    float *so = token_smem + warp * R * D, *sml = token_smem + kTokenWarps * R * D;
#pragma unroll
    for (int f = 0; f < RF; ++f) {
        float *dst = so + (g + 8 * f) * D + 2 * tq * NO;
#pragma unroll
        for (int y = 0; y < 2; ++y)
#pragma unroll
            for (int i = 0; i < NO; i += 4)
                *reinterpret_cast<float4 *>(dst + y * NO + i) =
                    make_float4(o[i][2 * f + y], o[i + 1][2 * f + y], o[i + 2][2 * f + y], o[i + 3][2 * f + y]);
        if (tq == 0) {
            sml[2 * (warp * R + g + 8 * f)] = m[f];
            sml[2 * (warp * R + g + 8 * f) + 1] = l[f];
        }
    }
    __syncthreads();
    for (int e = t; e < n_row * (D / 4); e += 32 * kTokenWarps) {
        const int r = e / (D / 4), col = (e % (D / 4)) * 4;
        float M = -INFINITY;
#pragma unroll
        for (int w = 0; w < kTokenWarps; ++w) M = fmaxf(M, sml[2 * (w * R + r)]);
        const float base = M == -INFINITY ? 0.f : M;
        float L = 0.f;
        float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int w = 0; w < kTokenWarps; ++w) {
            const float f = ex2(sml[2 * (w * R + r)] - base);
            const float4 y = *reinterpret_cast<const float4 *>(token_smem + (w * R + r) * D + col);
            L = fmaf(f, sml[2 * (w * R + r) + 1], L);
            x.x = fmaf(f, y.x, x.x); x.y = fmaf(f, y.y, x.y);
            x.z = fmaf(f, y.z, x.z); x.w = fmaf(f, y.w, x.w);
        }
        const int tok = r / a.G, head = h * a.G + r % a.G;
        if (last_seg == 0) {
            const float inv = L > 0.f ? 1.f / L : (L == 0.f ? 0.f : L);   // no key: zero; NaN stays
            const __nv_bfloat162 p0 = __floats2bfloat162_rn(x.x * inv, x.y * inv), p1 = __floats2bfloat162_rn(x.z * inv, x.w * inv);
            *reinterpret_cast<uint2 *>(static_cast<bf *>(a.out) + ((int64_t)(u.row + tok) * a.Hq + head) * D + col) =
                make_uint2(*reinterpret_cast<const uint32_t *>(&p0), *reinterpret_cast<const uint32_t *>(&p1));
        } else {
            const int64_t pr = kv_part_row(a, ui, seg, tok, head);
            *reinterpret_cast<float4 *>(a.part_o + pr * D + col) = x;
            if (col == 0) a.part_ml[pr] = make_float2(M, L);
        }
    }
}

template <int D, int R>
cudaError_t launch_token(const KvAttn &a, int n_units, cudaStream_t st) {
    using P = TokenPlan<D, R>;
    if (P::kBytes > 48 * 1024) {
        const cudaError_t e = cudaFuncSetAttribute(kv_attn_token_kernel<D, R>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)P::kBytes);
        if (e != cudaSuccess) return e;
    }
    const dim3 grid((unsigned)n_units, (unsigned)a.Hkv, (unsigned)a.n_seg);
    const cudaError_t e = gdn_launch_pdl(kv_attn_token_kernel<D, R>, grid, 32 * kTokenWarps, P::kBytes, st, a);
    return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace gdn

cudaError_t gdn_launch_kv_attn_token(const gdn::KvAttn &a, int d, int n_units, int rows_max, cudaStream_t st) {
    using namespace gdn;
    const bool r8 = rows_max <= 8;   // half the accumulators and query fragments
    if (d == 64) return r8 ? launch_token<64, 8>(a, n_units, st) : launch_token<64, 16>(a, n_units, st);
    if (d == 128) return r8 ? launch_token<128, 8>(a, n_units, st) : launch_token<128, 16>(a, n_units, st);
    return r8 ? launch_token<256, 8>(a, n_units, st) : launch_token<256, 16>(a, n_units, st);
}

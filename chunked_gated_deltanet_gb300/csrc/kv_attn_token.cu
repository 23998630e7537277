// Attention of few query rows (single tokens, short continuations) over the paged 8-bit key/value cache, bf16 inputs.
//
// The mathematics is that of kv_attn_prompt.cu (keys in fp16 against rows scaled by a power of two, weights
// in fp16 with the value scale over the unit of the warp's O, the largest so far at 2^15; the row's own block in two bf16 products), on warp-level MMAs: with
// up to 16 rows the work is reading the cache, 2 d bytes a key and head against 4 d flops a row, and tcgen05's 128 rows
// would be empty.
//
// CTA (unit, kv head, every Z-th segment), 4 warps, every fourth block each. A warp reads its keys and values from global
// memory straight into the fragments of the products, without shared memory: the order of the reduction index of a
// product is free as long as both operands share it, so
//   S^T = K q^T    m16n8k16, A = 16 keys, B = 8 rows; lane (g, t) = (lane / 4, lane % 4) reads 16 bytes of keys g and g + 8
//                  at columns 64 j + 16 t: four k-steps of four columns each; q's fragments lie in shared memory;
//   O^T += V^T P^T A = V^T, B = P^T: the scores' fragments, transposed 8 x 8 at a time (movmatrix); lane (g, t) reads d / 8
//                  bytes at column g d / 8 of the four keys that its weights belong to, and bytes 2 i, 2 i + 1 of them are
//                  m-tile i: rows g and g + 8 of it are columns g d / 8 + 2 i, + 1.
// With the rows as the narrow side (8 or 16) no accumulator and no product is spent on rows that are not there.
// Units of UK keys are loaded one ahead, across blocks and segments too. The four warps' results are added in order in shared memory
// and leave as the segment's partial result (or the result, where there is one segment only).
// Bound: HBM. 64 tokens over 500 to 16,384 keys (32/8 heads of 128): 107 us, 5.2 TB/s read; the registers hold one unit of
// loads ahead at 12 warps an SM. One token over 41,802 keys (16/2 heads of 256): 22 us, latency and the join's launch.
#include "kv_attn.cuh"

#include <algorithm>

namespace gdn {

constexpr int kTokenWarps = 4;   // warp w takes blocks w, w + 4, ... of a segment

__device__ __forceinline__ void mma_f16(float (&d)[4], const uint32_t (&a)[4], const uint32_t (&b)[2]) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
        "{%0,%1,%2,%3};\n"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b[0]), "r"(b[1]));
}

// The 8 x 8 matrix of 16-bit elements whose row g is lanes 4 g .. 4 g + 3's pairs, transposed.
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;\n" : "=r"(y) : "r"(x));
    return y;
}

template <int D, int R>
struct TokenPlan {
    static constexpr int UK = D == 256 ? 16 : 32;   // keys of a unit: 16 or 32 registers of loads each for keys and values
    static constexpr int NA = UK / 16;              // key m-tiles
    static constexpr int J = D / 64;                // 16-byte chunks of a key row per lane
    static constexpr int W = D / 32;                // 32-bit words of a value row per lane
    static constexpr int NO = D / 8;                // output columns of a lane
    static constexpr int NT = R / 8;                // row n-tiles
    static constexpr int NU = kKvBlock / UK;        // units of a block
    static constexpr size_t kSo = 0, kMl = kTokenWarps * R * D * sizeof(float), kQf = kMl + kTokenWarps * R * 8,
                            kQr = kQf + 4 * J * 32 * 2 * NT * 4, kBytes = kQr + R * 4;
    // CTAs on an SM: as many as the accumulators and loads leave registers for
    static constexpr int kCtas = D * R <= 1024 ? 3 : 2;
};

// N 32-bit words from global memory (N = 2 or a multiple of 4)
template <int N>
__device__ __forceinline__ void ld_words(uint32_t *w, const void *p) {
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

constexpr float kTokenLift = 15.f;   // log2 of a row's largest weight: fp16 keeps the 11 bits of those down to 2^-29 of it

// Scores of 16 N keys -> weights: exponents c s + add, the running maximum and sum (of the lane's keys, without the value
// scale, 1 / ivs; added over the lanes at the end), O rescaled.
template <int N, int NT, int NO>
__device__ __forceinline__ void token_softmax(float (&s)[N][NT][4], const float (&c)[NT][2], const float (&add)[NT][2], float ivs,
                                              float (&m)[NT][2], float (&l)[NT][2], float (&o)[NO / 2][NT][4]) {
#pragma unroll
    for (int f = 0; f < NT; ++f) {
        float corr[2];
#pragma unroll
        for (int y = 0; y < 2; ++y) {
            float top = -INFINITY;
#pragma unroll
            for (int x = 0; x < N; ++x) top = fmaxf(top, fmaxf(s[x][f][y], s[x][f][2 + y]));
#pragma unroll
            for (int w = 4; w < 32; w <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, w));
            if (top > -INFINITY) top = fmaf(top, c[f][y], add[f][y] - kTokenLift);
            const float mn = fmaxf(m[f][y], top), base = mn == -INFINITY ? 0.f : mn;
            corr[y] = ex2(m[f][y] - base);
            m[f][y] = mn;
            const float off = add[f][y] - base;
            float sum = 0.f;
#pragma unroll
            for (int x = 0; x < N; ++x)
#pragma unroll
                for (int k = y; k < 4; k += 2) {
                    const float p = ex2(fmaf(s[x][f][k], c[f][y], off));
                    s[x][f][k] = p;
                    sum += p;
                }
            l[f][y] = fmaf(sum, ivs, l[f][y] * corr[y]);
        }
        if (__any_sync(0xffffffffu, corr[0] != 1.f || corr[1] != 1.f)) {
#pragma unroll
            for (int i = 0; i < NO / 2; ++i)
#pragma unroll
                for (int k = 0; k < 4; ++k) o[i][f][k] *= corr[k & 1];
        }
    }
}

template <int D, int R>
__global__ void __launch_bounds__(32 * kTokenWarps, TokenPlan<D, R>::kCtas) kv_attn_token_kernel(const KvAttn a) {
    using P = TokenPlan<D, R>;
    using bf = __nv_bfloat16;
    constexpr int UK = P::UK, NA = P::NA, J = P::J, W = P::W, NO = P::NO, NT = P::NT, NU = P::NU;
    constexpr int VB = NO < 16 ? NO : 16;   // bytes of a value row that a lane reads at once
    auto col = [](int g, int i) { return i / VB * (8 * VB) + g * VB + i % VB; };   // column i of lane group g
    grid_dep_wait();
    grid_dep_launch();
    const int ui = a.unit0 + blockIdx.x, h = blockIdx.y;
    const KvUnit u = kv_load_unit(a.units, ui);   // inside the map whatever the count
    if (ui >= a.counts[0]) return;
    const int last_seg = u.block / a.seg_blocks;
    const int n_row = u.count * a.G;
    if (!kv_attn_unit_ok(a, u) || n_row > R) {
        if (threadIdx.x == 0) atomicOr(a.err, kErrKvBounds);
        return;
    }
    if ((int)blockIdx.z > last_seg) return;
    extern __shared__ __align__(16) unsigned char token_smem[];
    float *so = reinterpret_cast<float *>(token_smem + P::kSo);
    float2 *sml = reinterpret_cast<float2 *>(token_smem + P::kMl);
    float *sqr = reinterpret_cast<float *>(token_smem + P::kQr);
    uint32_t *sqf = reinterpret_cast<uint32_t *>(token_smem + P::kQf);
    const int t = threadIdx.x, warp = t >> 5, lane = t & 31, g = lane >> 2, tq = lane & 3;
    const int32_t *table = a.c.table + (int64_t)u.slot * a.c.max_blocks;

    // page of an 8-bit block (-1: it is none of the pass's)
    auto page_of = [&](int b) {
        if (b >= u.block) return -1;
        const int pg = table[b];
        if ((unsigned)pg < (unsigned)a.c.n_pages) return pg;
        if (lane == 0) atomicOr(a.err, kErrKvBounds);
        return 0;   // in bounds; the result is reported as invalid
    };
    uint32_t kb[NA][2][J][4], vb[NA][4][W];
    auto load_k = [&](int page, int n) {
        const int8_t *src = a.c.k + ((int64_t)page * a.Hkv + h) * (kKvBlock * D) + (n * UK + g) * D + 16 * tq;
#pragma unroll
        for (int x = 0; x < 2 * NA; ++x)
#pragma unroll
            for (int j = 0; j < J; ++j) ld_words<4>(kb[x / 2][x % 2][j], src + 8 * x * D + 64 * j);
    };
    auto load_v = [&](int page, int n) {
        const int8_t *src = a.c.v + ((int64_t)page * a.Hkv + h) * (kKvBlock * D) + (n * UK + 2 * tq) * D + g * VB;
#pragma unroll
        for (int x = 0; x < NA; ++x)
#pragma unroll
            for (int y = 0; y < 4; ++y)
#pragma unroll
                for (int i = 0; i < W; i += VB / 4) ld_words<VB / 4>(&vb[x][y][i], src + (16 * x + (y & 1) + 8 * (y >> 1)) * D + 8 * 4 * i);
    };
    int blk = blockIdx.z * a.seg_blocks + warp, page = page_of(blk);
    if (page >= 0) {
        load_k(page, 0);
        load_v(page, 0);
    }
    // q's fragments, by warp 0: per k-step the lane's columns 0, 1 and 2, 3 of rows g (and g + 8), scaled, in fp16
    const bf *q = static_cast<const bf *>(a.q);
    auto q_row = [&](int r) { return q + ((int64_t)(u.row + r / a.G) * a.Hq + h * a.G + r % a.G) * D + 16 * tq; };
    if (warp == 0) {
#pragma unroll
        for (int f = 0; f < NT; ++f) {
            const int r = g + 8 * f;
            uint4 w[J][2];
            float top = 0.f, back;
#pragma unroll
            for (int j = 0; j < J; ++j)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    w[j][i] = make_uint4(0, 0, 0, 0);
                    if (r < n_row) w[j][i] = __ldg(reinterpret_cast<const uint4 *>(q_row(r) + 64 * j + 8 * i));
                }
#pragma unroll
            for (int j = 0; j < J; ++j)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    float x[8];
                    b8_to_f(w[j][i], x);
#pragma unroll
                    for (int k = 0; k < 8; ++k) top = fmaxf(top, fabsf(x[k]));
                }
#pragma unroll
            for (int o = 1; o < 4; o <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
            const float up = pow2_to_2_15(top, back);
            if (tq == 0) sqr[r] = back;
#pragma unroll
            for (int j = 0; j < J; ++j)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    float x[8];
                    b8_to_f(w[j][i], x);
#pragma unroll
                    for (int k = 0; k < 8; ++k) x[k] *= up;
                    const uint4 y = f8_to_h8(x);
                    uint32_t *dst = sqf + ((4 * j + 2 * i) * 32 + lane) * 2 * NT + 2 * f;
                    dst[0] = y.x;
                    dst[1] = y.y;
                    dst[64 * NT] = y.z;
                    dst[64 * NT + 1] = y.w;
                }
        }
    }
    __syncthreads();
    float qr[NT][2];   // of the lane's rows, 8 f + 2 tq + y
#pragma unroll
    for (int f = 0; f < NT; ++f)
#pragma unroll
        for (int y = 0; y < 2; ++y) qr[f][y] = sqr[8 * f + 2 * tq + y];

    float o[NO / 2][NT][4], m[NT][2], l[NT][2];   // o: columns g NO + 2 i (+ 1 in [2], [3]) of the lane's two rows
    float lref = 0.f;                             // O is in units of 2^lref
    // the rows' own block, at the end of the last segment: as it came, 16 keys a warp, the first by the warp whose turn it is
    // (one warp for all of them would be the longest part of a short context)
    const int own0 = 16 * ((warp - u.block) & 3);
    static_assert(kTokenWarps == 4, "16 keys each");
    auto own_block = [&] {
        bool odd_value = false;
        const bf *tail = static_cast<const bf *>(a.c.tail);
        auto raw_row = [&](int kv, int off) -> const bf * {
            if (off < u.first) return tail + kv_tail_offset(u.slot, u.src, kv, h, a.Hkv, D) + (int64_t)off * D;
            if (off < u.first + u.count)
                return static_cast<const bf *>(kv ? a.v_new : a.k_new) + ((int64_t)(u.row + off - u.first) * a.Hkv + h) * D;
            return nullptr;
        };
        // these values are their own: the unit becomes 1
        const float move = pow2_of(lref);
        lref = 0.f;
#pragma unroll
        for (int i = 0; i < NO / 2; ++i)
#pragma unroll
            for (int f = 0; f < NT; ++f)
#pragma unroll
                for (int k = 0; k < 4; ++k) o[i][f][k] *= move;
        float c[NT][2], add[NT][2];
#pragma unroll
        for (int f = 0; f < NT; ++f)
#pragma unroll
            for (int y = 0; y < 2; ++y) {
                c[f][y] = a.scale_log2;
                add[f][y] = 0.f;
            }
        const int k0 = own0;
        float s[1][NT][4];
#pragma unroll
        for (int f = 0; f < NT; ++f)
#pragma unroll
            for (int k = 0; k < 4; ++k) s[0][f][k] = 0.f;
        const bf *key[2] = {raw_row(0, k0 + g), raw_row(0, k0 + 8 + g)};
#pragma unroll 1
        for (int j = 0; j < J; ++j) {
            uint32_t w[2][8], qw[NT][8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                w[0][i] = w[1][i] = 0;
#pragma unroll
                for (int f = 0; f < NT; ++f) qw[f][i] = 0;
            }
#pragma unroll
            for (int x = 0; x < 2; ++x)
                if (key[x]) ld_words<8>(w[x], key[x] + 64 * j + 16 * tq);
#pragma unroll
            for (int f = 0; f < NT; ++f)
                if (g + 8 * f < n_row) ld_words<8>(qw[f], q_row(g + 8 * f) + 64 * j);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const uint32_t ka[4] = {w[0][2 * k], w[1][2 * k], w[0][2 * k + 1], w[1][2 * k + 1]};
#pragma unroll
                for (int f = 0; f < NT; ++f) {
                    const uint32_t b[2] = {qw[f][2 * k], qw[f][2 * k + 1]};
                    mma_bf16(s[0][f], ka, b);
                }
            }
        }
#pragma unroll
        for (int f = 0; f < NT; ++f)
#pragma unroll
            for (int k = 0; k < 4; ++k)
                if (k0 + g + 8 * (k >> 1) > u.first + (8 * f + 2 * tq + (k & 1)) / a.G) s[0][f][k] = -INFINITY;
        token_softmax<1, NT, NO>(s, c, add, 1.f, m, l, o);
        uint32_t ph[NT][2], pl[NT][2];   // weights of keys g and g + 8, rows 2 tq, 2 tq + 1; transposed
#pragma unroll
        for (int f = 0; f < NT; ++f)
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                split_bf16x2(s[0][f][2 * x], s[0][f][2 * x + 1], ph[f][x], pl[f][x]);
                ph[f][x] = transpose8(ph[f][x]);
                pl[f][x] = transpose8(pl[f][x]);
            }
        const bf *val[4];
#pragma unroll
        for (int y = 0; y < 4; ++y) val[y] = raw_row(1, k0 + 2 * tq + (y & 1) + 8 * (y >> 1));
#pragma unroll
        for (int i = 0; i < NO / 8; ++i) {   // eight columns of the four keys
            uint32_t v[4][4];
#pragma unroll
            for (int y = 0; y < 4; ++y) {
                uint4 x = make_uint4(0, 0, 0, 0);
                if (val[y]) x = __ldg(reinterpret_cast<const uint4 *>(val[y] + col(g, 8 * i)));
                // a value that is not finite would reach rows that do not see it (0 * inf): left out here, and
                // added by the rows that do at the end
                odd_value |= drop_not_finite(x);
                v[y][0] = x.x; v[y][1] = x.y; v[y][2] = x.z; v[y][3] = x.w;
            }
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const uint32_t va[4] = {__byte_perm(v[0][k], v[1][k], 0x5410), __byte_perm(v[0][k], v[1][k], 0x7632),
                                        __byte_perm(v[2][k], v[3][k], 0x5410), __byte_perm(v[2][k], v[3][k], 0x7632)};
#pragma unroll
                for (int f = 0; f < NT; ++f) {
                    mma_bf16(o[4 * i + k][f], va, ph[f]);
                    mma_bf16(o[4 * i + k][f], va, pl[f]);
                }
            }
        }
        if (__any_sync(0xffffffffu, odd_value)) {
#pragma unroll
            for (int f = 0; f < NT; ++f)
#pragma unroll
                for (int y = 0; y < 2; ++y) {
                    const int r = 8 * f + 2 * tq + y, n_see = r < n_row ? min(k0 + 16, u.first + r / a.G + 1) : 0;
#pragma unroll 1
                    for (int k = k0; k < n_see; ++k) {
                        const bf *src = raw_row(1, k);
#pragma unroll
                        for (int i = 0; i < NO; ++i) {
                            const float x = to_f(src[col(g, i)]);
                            if (!(fabsf(x) <= 3.4e38f)) o[i / 2][f][2 * (i & 1) + y] += x;
                        }
                    }
                }
        }
    };
    // the warps' results of a segment, added in order (a warp without a key of it has none: weight 0)
    auto merge = [&](int seg) {
        const float unit = pow2_of(lref);
#pragma unroll
        for (int f = 0; f < NT; ++f)
#pragma unroll
            for (int y = 0; y < 2; ++y) {
                const int r = 8 * f + 2 * tq + y;
                float *dst = so + (warp * R + r) * D;
#pragma unroll
                for (int i = 0; i < NO / 2; i += 2)
                    *reinterpret_cast<float4 *>(dst + col(g, 2 * i)) =
                        make_float4(o[i][f][y] * unit, o[i][f][2 + y] * unit, o[i + 1][f][y] * unit, o[i + 1][f][2 + y] * unit);
                float sum = l[f][y];
#pragma unroll
                for (int w = 4; w < 32; w <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, w);
                if (g == 0) sml[warp * R + r] = make_float2(m[f][y], sum);
            }
        __syncthreads();
        for (int e = t; e < n_row * (D / 4); e += 32 * kTokenWarps) {
            const int r = e / (D / 4), col = (e % (D / 4)) * 4;
            float M = -INFINITY;
            for (int w = 0; w < kTokenWarps; ++w) M = fmaxf(M, sml[w * R + r].x);
            const float base = M == -INFINITY ? 0.f : M;
            float L = 0.f;
            float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
            for (int w = 0; w < kTokenWarps; ++w) {
                const float2 ml = sml[w * R + r];
                const float f = ex2(ml.x - base);
                const float4 y = *reinterpret_cast<const float4 *>(so + (w * R + r) * D + col);
                L = fmaf(f, ml.y, L);
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
        __syncthreads();   // read before the next segment's results
    };

    for (int seg = blockIdx.z;;) {
        lref = 0.f;
#pragma unroll
        for (int f = 0; f < NT; ++f) {
            m[f][0] = m[f][1] = -INFINITY;
            l[f][0] = l[f][1] = 0.f;
#pragma unroll
            for (int i = 0; i < NO / 2; ++i)
#pragma unroll
                for (int k = 0; k < 4; ++k) o[i][f][k] = 0.f;
        }
        const int seg_end = (seg + 1) * a.seg_blocks, next_seg = seg + gridDim.z;
#pragma unroll 1
        for (; blk < min(seg_end, u.block); blk += kTokenWarps) {
            const int next = page_of(blk + kTokenWarps < seg_end ? blk + kTokenWarps : next_seg * a.seg_blocks + warp);
            const int64_t ph = (int64_t)page * a.Hkv + h;
            const float ks = a.scale_log2 * a.c.k_scale[ph], vs = a.c.v_scale[ph];
            float move = 1.f;
            const float dv = kv_unit(kv_log2_scale(vs), lref, move), ivs = ex2(-dv);
            if (move != 1.f) {
#pragma unroll
                for (int i = 0; i < NO / 2; ++i)
#pragma unroll
                    for (int f = 0; f < NT; ++f)
#pragma unroll
                        for (int k = 0; k < 4; ++k) o[i][f][k] *= move;
            }
            float c[NT][2], add[NT][2];
#pragma unroll
            for (int f = 0; f < NT; ++f)
#pragma unroll
                for (int y = 0; y < 2; ++y) {
                    c[f][y] = ks * qr[f][y];
                    add[f][y] = dv;
                }
#pragma unroll 1
            for (int n = 0; n < NU; ++n) {
                float s[NA][NT][4];
#pragma unroll
                for (int x = 0; x < NA; ++x)
#pragma unroll
                    for (int f = 0; f < NT; ++f)
#pragma unroll
                        for (int k = 0; k < 4; ++k) s[x][f][k] = 0.f;
#pragma unroll
                for (int j = 0; j < J; ++j)
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        uint32_t b[NT][2];
                        const uint32_t *src = sqf + ((4 * j + k) * 32 + lane) * 2 * NT;
#pragma unroll
                        for (int f = 0; f < NT; ++f) {
                            b[f][0] = src[2 * f];
                            b[f][1] = src[2 * f + 1];
                        }
#pragma unroll
                        for (int x = 0; x < NA; ++x) {
                            const uint2 lo = i8_to_f16x4(kb[x][0][j][k]), hi = i8_to_f16x4(kb[x][1][j][k]);
                            const uint32_t ka[4] = {lo.x, hi.x, lo.y, hi.y};
#pragma unroll
                            for (int f = 0; f < NT; ++f) mma_f16(s[x][f], ka, b[f]);
                        }
                    }
                const int pn = n + 1 < NU ? page : next;
                if (pn >= 0) load_k(pn, (n + 1) % NU);
                token_softmax<NA, NT, NO>(s, c, add, ivs, m, l, o);
#pragma unroll
                for (int x = 0; x < NA; ++x) {
                    uint32_t pb[NT][2];
#pragma unroll
                    for (int f = 0; f < NT; ++f)
#pragma unroll
                        for (int y = 0; y < 2; ++y) pb[f][y] = transpose8(f2_to_h2(s[x][f][2 * y], s[x][f][2 * y + 1]));
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
                        for (int i = 0; i < 2; ++i) {
                            const uint32_t va[4] = {e[0][2 * i], e[0][2 * i + 1], e[1][2 * i], e[1][2 * i + 1]};
#pragma unroll
                            for (int f = 0; f < NT; ++f) mma_f16(o[2 * w + i][f], va, pb[f]);
                        }
                    }
                }
                if (pn >= 0) load_v(pn, (n + 1) % NU);
            }
            page = next;
        }
        // nothing is loaded ahead past the last segment (told apart here, so that no register is kept for it)
        if (seg == last_seg) {
            if (own0 < u.first + u.count) own_block();
            merge(seg);
            return;
        }
        merge(seg);
        if (next_seg > last_seg) return;
        seg = next_seg;
        blk = seg * a.seg_blocks + warp;
    }
}

template <int D, int R>
cudaError_t launch_token(const KvAttn &a, int n_units, cudaStream_t st) {
    using P = TokenPlan<D, R>;
    if (P::kBytes > 48 * 1024) {
        const cudaError_t e = cudaFuncSetAttribute(kv_attn_token_kernel<D, R>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)P::kBytes);
        if (e != cudaSuccess) return e;
    }
    // CTAs per (unit, kv head): one per segment while that leaves the GPU unfilled, else about 16 per SM in all, so that few
    // of a ragged batch's start to find no segment left
    int sms = 1;
    cudaError_t e = gdn_sm_count(&sms);
    if (e != cudaSuccess) return e;
    const int64_t chains = (int64_t)n_units * a.Hkv, z = (16LL * sms + chains - 1) / chains;
    const dim3 grid((unsigned)n_units, (unsigned)a.Hkv, (unsigned)std::min<int64_t>(a.n_seg, z));
    e = gdn_launch_pdl(kv_attn_token_kernel<D, R>, grid, 32 * kTokenWarps, P::kBytes, st, a);
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

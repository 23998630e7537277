// Attention of many query rows over the paged 8-bit key/value cache on the 5th-generation tensor core (bf16 inputs).
//
// The mathematics is that of kv_attn_simt.cu; here the two products of a step of 128 keys are tcgen05 MMAs:
//   S = Q K^T     128 rows x 128 keys, K = d: both operands bf16 in shared memory. An int8 key is exact in bf16, so S is
//                 exact up to fp32 accumulation; the block's scale and the softmax scale multiply S afterwards.
//   O += P V      128 rows x d, K = 64 keys: P in TMEM as the A operand, V in shared memory. An 8-bit block: V int8 -> fp16
//                 (exact), P = 2^{c s + log2 vs - m} with the block's value scale vs in the weight and m the running
//                 maximum of exactly that exponent, so P <= 2^8 whatever the scales, and fp16 rounds it by 2^-11 of its
//                 size (2^-25 absolute below 2^-14, where a key adds next to nothing). The row's own block as it came: V
//                 bf16, P in two bf16 products, its upper and lower 8 bits: a row with few keys has nothing to average a
//                 rounding out. The sum l takes the unrounded weights, 2^{c s - m}.
//
// CTA: one row tile of R = 256 rows (two MMA tiles of 128; d = 256: one tile) of one kv head, over one segment of keys.
// Rows are the (token, query head of the group) pairs of a span: consecutive blocks of one request, aligned to `span`
// blocks, so that 64 span G >= R where it can be. Warp roles:
//   softmax   a warpgroup per MMA tile, one row per thread: TMEM scores -> weights -> TMEM P, running maximum and sum
//   convert   4 warps (d = 256: 8): pages from global memory, int8 -> bf16 in registers, into the operand layout
//   MMA       one thread issues every product
// With two tiles the tensor core works on one tile while the other's softmax runs; with one tile the two score buffers
// take alternate steps.
//
// The running maximum m only moves when a half step (64 keys, one block) exceeds it by 8 (log2 domain): weights stay
// below 2^8, and O is rescaled (by the softmax warps, after the products before it) only then. Every decision is a row's
// own and every block is one softmax step, so a row's bits do not depend on the rows beside it.
// Bound: tensor pipe; per 128 keys and 128 rows the MMAs take 4 * 128 * 128 * d / 8192 cycles (1,024 for d = 128).
#include "kv_attn.cuh"
#include "umma.cuh"

#include <algorithm>
#include <type_traits>

namespace gdn {

// D[tmem] (+)= A[tmem] * B[smem], one K-step of 16 16-bit elements; A: lane = row, a column holds two K elements.
__device__ __forceinline__ void umma_bf16_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t bdesc, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(d_tmem),
        "r"(a_tmem), "l"(bdesc), "r"(idesc), "r"(accumulate)
        : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};\n" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]),
        "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;\n" ::: "memory"); }
// named barrier `id` over n threads (whole warps)
__device__ __forceinline__ void kv_named_barrier(int id, int n) { asm volatile("bar.sync %0, %1;\n" ::"r"(id), "r"(n) : "memory"); }

template <int D>
struct PromptPlan {
    static constexpr int NQ = D == 256 ? 1 : 2;              // MMA tiles of 128 rows
    static constexpr int R = 128 * NQ;
    static constexpr int NB = D == 256 ? 1 : 2;              // K and V buffers of 128 keys each
    static constexpr int CW = D == 256 ? 8 : 4;              // convert warps
    static constexpr int NT = 128 * NQ + 32 * CW + 32;
    static constexpr int kConvert0 = 128 * NQ, kMma = NT - 32;   // first thread of the roles
    static constexpr uint32_t kTile = 128 * D * 2;           // bytes of a 128 x D bf16 operand
    static constexpr uint32_t kQ = 0, kK = NQ * kTile, kV = kK + NB * kTile, kHalf = kV + NB * kTile;
    static constexpr int kMaxHalves = 64 + 4;                // int8 blocks of a segment and raw blocks of a span
    static constexpr uint32_t kBar = kHalf + ((kMaxHalves + 2) * 16 + 15) / 16 * 16;
    // barriers: kfull[NB], kfree[NB], vfull[NB], vfree[NB], sfull[2], pready[2][2], pvdone[NQ][2], drain
    static constexpr int bKFull = 0, bKFree = NB, bVFull = 2 * NB, bVFree = 3 * NB, bS = 4 * NB, bP = bS + 2, bPV = bP + 4,
                         bDrain = bPV + 2 * NQ, kNBar = bDrain + 1;
    static constexpr uint32_t kSlot = kBar + kNBar * 8;
    static constexpr uint32_t kBad = kSlot + 16;             // per raw block of the span: it has a value that is not finite
    static constexpr uint32_t kBytes = kBad + 16;
    static constexpr uint32_t kO = 256;                      // TMEM columns: scores [0, 256), outputs from here
    static constexpr uint32_t kTmemCols = 512;
    static constexpr int kVec = D / 64;                      // 64-column groups
    static constexpr int kLoads = 16 * kVec / CW;            // 16-byte loads of a convert thread per 128-key tile
    static_assert(kBytes <= 227 * 1024, "shared memory");
    static_assert(kLoads * CW == 16 * kVec, "convert split");
};

// A half step's block: its page, c = scale log2(e) k_scale, log2 of the value scale in the exponent that m is the maximum
// of, and the factor of its weights in the sum (1 / v_scale). A raw block counts with the value scale of the block before
// it (so that m compares like with like), but its weights are of the values themselves.
struct HalfInfo {
    int page;
    float c, lvs, ivs;
};


template <int D>
__global__ void __launch_bounds__(PromptPlan<D>::NT, 1) kv_attn_prompt_kernel(const KvAttn a, int row_tiles, int span, int n_units) {
    using P = PromptPlan<D>;
    using bf = __nv_bfloat16;
    constexpr int NB = P::NB;
    grid_dep_wait();
    grid_dep_launch();
    // later units (longer contexts) first: a causal launch then ends on its short ones
    const int ui = a.unit0 + n_units - 1 - (int)(blockIdx.x / row_tiles), rt = blockIdx.x % row_tiles, h = blockIdx.y, seg = blockIdx.z;
    const int unit1 = min(a.unit0 + n_units, a.counts[0]);
    if (ui >= unit1) return;
    const KvUnit u = kv_load_unit(a.units, ui);
    bool ok = kv_unit_ok(u, a.c, a.n_rows) && u.count <= a.max_new && u.block / a.seg_blocks < a.n_seg;
    // the span's first unit works for all of it
    if (ok && ui > a.unit0 && u.block % span != 0) {
        const KvUnit w = kv_load_unit(a.units, ui - 1);
        if (w.slot == u.slot && w.block == u.block - 1) return;
    }
    int n_tok = u.count;
    for (int i = 1; ok && i < span && ui + i < unit1 && (u.block + i) % span != 0; ++i) {
        const KvUnit w = kv_load_unit(a.units, ui + i);
        if (w.slot != u.slot || w.block != u.block + i) break;
        ok = kv_unit_ok(w, a.c, a.n_rows) && w.first == 0 && w.row == u.row + n_tok;
        n_tok += w.count;
    }
    if (!ok || n_tok > a.max_new) {
        if (threadIdx.x == 0) atomicOr(a.err, kErrKvBounds);
        return;
    }
    const int last_seg = u.block / a.seg_blocks;   // a span lies in one segment: span divides seg_blocks
    const int n_row = n_tok * a.G, r0 = rt * P::R;
    if (r0 >= n_row || seg > last_seg) return;

    extern __shared__ __align__(1024) unsigned char sm[];
    uint64_t *bar = reinterpret_cast<uint64_t *>(sm + P::kBar);
    uint32_t *tslot = reinterpret_cast<uint32_t *>(sm + P::kSlot);
    uint32_t *bad_v = reinterpret_cast<uint32_t *>(sm + P::kBad);
    HalfInfo *half = reinterpret_cast<HalfInfo *>(sm + P::kHalf);
    const int t = threadIdx.x, warp = t >> 5, lane = t & 31;
    const int pos0 = u.block * kKvBlock + u.first;
    const int rows_here = min(P::R, n_row - r0);
    const int nt = rows_here > 128 ? 2 : 1;        // MMA tiles in use
    // blocks of this tile's rows, and the halves: 8-bit blocks [c0, c0 + n8), then raw blocks from blo
    const int blo = (pos0 + r0 / a.G) / kKvBlock, bhi = (pos0 + (r0 + rows_here - 1) / a.G) / kKvBlock;
    const int c0 = seg * a.seg_blocks;
    const int n8 = min(bhi - c0, a.seg_blocks);
    const int nh = n8 + (seg == last_seg ? bhi - blo + 1 : 0);
    const int steps = (nh + 1) / 2, n_items = steps * nt;

    if (t == 0) {
        for (int i = 0; i < NB; ++i) {
            mbar_init(&bar[P::bKFull + i], 32 * P::CW);
            mbar_init(&bar[P::bVFull + i], 32 * P::CW);
            mbar_init(&bar[P::bKFree + i], 1);
            mbar_init(&bar[P::bVFree + i], 1);
        }
        for (int i = 0; i < 2; ++i) mbar_init(&bar[P::bS + i], 1);
        for (int i = 0; i < 4; ++i) mbar_init(&bar[P::bP + i], 128);
        for (int i = 0; i < 2 * P::NQ; ++i) mbar_init(&bar[P::bPV + i], 1);
        mbar_init(&bar[P::bDrain], 1);
        mbar_init_fence();
        for (int i = 0; i < 4; ++i) bad_v[i] = 0;
    }
    if (warp == 0) {
        tmem_alloc(tslot, P::kTmemCols);
        tmem_relinquish();
    }
    // pages and scales of the segment's blocks
    const int32_t *table = a.c.table + (int64_t)u.slot * a.c.max_blocks;
    for (int i = t; i < nh; i += P::NT) {
        HalfInfo x = {0, a.scale_log2, 0.f, 1.f};
        if (i < n8) {
            x.page = table[c0 + i];
            x.lvs = kv_log2_vscale(a, table, c0 + i, h);
            x.ivs = ex2(-x.lvs);
            if ((unsigned)x.page < (unsigned)a.c.n_pages) {
                x.c = a.scale_log2 * a.c.k_scale[(int64_t)x.page * a.Hkv + h];
            } else {
                x.page = 0;                        // in bounds; the result is reported as invalid
                x.c = 0.f;
                atomicOr(a.err, kErrKvBounds);
            }
        } else {
            x.lvs = kv_log2_vscale(a, table, blo + i - n8 - 1, h);
        }
        half[i] = x;
    }
    // Q: K-major core matrices (8 rows x 16 bytes), rows past the end zero
    const bf *q = static_cast<const bf *>(a.q);
    for (int e = t; e < nt * 128 * (D / 8); e += P::NT) {
        const int r = e / (D / 8), c = e % (D / 8);
        uint4 w = make_uint4(0, 0, 0, 0);
        if (r < rows_here) {
            const int rr = r0 + r;
            w = *reinterpret_cast<const uint4 *>(q + ((int64_t)(u.row + rr / a.G) * a.Hq + h * a.G + rr % a.G) * D + c * 8);
        }
        *reinterpret_cast<uint4 *>(sm + P::kQ + (r >> 7) * P::kTile + ((r & 127) >> 3) * (D * 16) + c * 128 + (r & 7) * 16) = w;
    }
    fence_proxy_async();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tslot;
    const long long limit = a.wait_limit;
    bool alive = true;

    if (t >= P::kMma) {
        // ---- the issuing thread ----
        if (t == P::kMma) {
            constexpr uint32_t idS = umma_idesc_bf16(128, 128, 0, 0), idO8 = umma_idesc_f16(128, D, 0, 1),
                               idOraw = umma_idesc_bf16(128, D, 0, 1);
            auto issue_s = [&](int i) {
                const int step = i / nt, tile = i - step * nt, slot = step % NB, b = i & 1;
                if (tile == 0 && !mbar_wait_bounded(&bar[P::bKFull + slot], (step / NB) & 1, limit)) return false;
                tc_fence_after();
                const uint64_t dq = umma_smem_desc(sm + P::kQ + tile * P::kTile, 128, D * 16);
                const uint64_t dk = umma_smem_desc(sm + P::kK + slot * P::kTile, 128, D * 16);
#pragma unroll
                for (int k = 0; k < D / 16; ++k) umma_bf16(tmem + 128 * b, dq + 16 * k, dk + 16 * k, idS, k > 0);
                umma_commit(&bar[P::bS + b]);
                if (tile == nt - 1) umma_commit(&bar[P::bKFree + slot]);
                return true;
            };
            alive = issue_s(0) && (n_items < 2 || issue_s(1));
            for (int i = 0; alive && i < n_items; ++i) {
                const int step = i / nt, tile = i - step * nt, slot = step % NB, b = i & 1;
                const int halves = min(2, nh - 2 * step);
                if (tile == 0) alive = mbar_wait_bounded(&bar[P::bVFull + slot], (step / NB) & 1, limit);
                for (int hh = 0; alive && hh < halves; ++hh) {
                    alive = mbar_wait_bounded(&bar[P::bP + 2 * b + hh], (i / 2) & 1, limit);
                    if (!alive) break;
                    tc_fence_after();
                    const bool raw = 2 * step + hh >= n8;
                    const uint32_t idO = raw ? idOraw : idO8;
                    const uint64_t dv = umma_smem_desc(sm + P::kV + slot * P::kTile + hh * (8 * D * 16), D * 16, 128);
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        umma_bf16_ts(tmem + P::kO + tile * D, tmem + 128 * b + 64 * hh + 8 * k, dv + (uint64_t)(2 * D * k), idO,
                                     step > 0 || hh > 0 || k > 0);
                    if (raw) {   // the low parts of the raw block's weights
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            umma_bf16_ts(tmem + P::kO + tile * D, tmem + 128 * b + 64 * hh + 32 + 8 * k, dv + (uint64_t)(2 * D * k),
                                         idO, 1);
                    }
                    umma_commit(&bar[P::bPV + 2 * tile + hh]);
                }
                if (!alive) break;
                if (tile == nt - 1) umma_commit(&bar[P::bVFree + slot]);
                if (i + 2 < n_items) alive = issue_s(i + 2);
            }
            if (!alive) atomicOr(a.err, kErrTimeout);
            umma_commit(&bar[P::bDrain]);
            if (!mbar_wait_bounded(&bar[P::bDrain], 0, limit)) atomicOr(a.err, kErrTimeout);
        }
    } else if (t >= P::kConvert0) {
        // ---- convert warps ----
        const int cw = warp - P::kConvert0 / 32;
        const int kr = lane & 7, ch = lane >> 3;   // key of 8 and 16-byte chunk of 64
        const bf *tail = static_cast<const bf *>(a.c.tail);
        const int n_seq = 2 * steps;               // K(0), K(1), V(0), K(2), V(1), ..., V(steps - 1)
        auto what = [&](int s, int &kv, int &step) {
            if (s == 0) { kv = 0; step = 0; }
            else if (s == n_seq - 1) { kv = 1; step = steps - 1; }
            else { kv = (s + 1) & 1; step = (s + 1) / 2 - kv; }
        };
        // 16-byte loads of tile (kv, step): load i of this warp is 8 keys x 64 columns, number cw + CW i of (half, key group,
        // column group). Both loops are unrolled over the loads only: the roles share the instruction cache.
        uint4 w[P::kLoads];
        auto load8 = [&](int kv, int step) {
            const int8_t *pool = (kv ? a.c.v : a.c.k) + (int64_t)h * (kKvBlock * D) + kr * D + ch * 16;
            const int64_t stride = (int64_t)a.Hkv * (kKvBlock * D);
            const int8_t *base[2];
#pragma unroll
            for (int hh = 0; hh < 2; ++hh) base[hh] = pool + half[min(2 * step + hh, nh - 1)].page * stride;
#pragma unroll
            for (int i = 0; i < P::kLoads; ++i) {
                const int j = cw + P::CW * i, hh = P::CW * i / (8 * P::kVec), kg = j / P::kVec % 8, dg = j % P::kVec;
                w[i] = __ldg(reinterpret_cast<const uint4 *>(base[hh] + kg * (8 * D) + dg * 64));
            }
        };
        auto store8 = [&](auto is_v, unsigned char *dst, int n_half) {
            constexpr bool f16 = decltype(is_v)::value;
#pragma unroll
            for (int i = 0; i < P::kLoads; ++i) {
                const int j = cw + P::CW * i, hh = P::CW * i / (8 * P::kVec), kg = j / P::kVec % 8, dg = j % P::kVec;
                if (hh >= n_half) break;
                uint4 lo, hi;
                if (f16) {
                    const uint2 x0 = i8_to_f16x4(w[i].x), x1 = i8_to_f16x4(w[i].y), x2 = i8_to_f16x4(w[i].z), x3 = i8_to_f16x4(w[i].w);
                    lo = make_uint4(x0.x, x0.y, x1.x, x1.y);
                    hi = make_uint4(x2.x, x2.y, x3.x, x3.y);
                } else {
                    const uint2 x0 = i8_to_bf16x4(w[i].x), x1 = i8_to_bf16x4(w[i].y), x2 = i8_to_bf16x4(w[i].z), x3 = i8_to_bf16x4(w[i].w);
                    lo = make_uint4(x0.x, x0.y, x1.x, x1.y);
                    hi = make_uint4(x2.x, x2.y, x3.x, x3.y);
                }
                unsigned char *o = dst + (hh * 8 + kg) * (D * 16) + (dg * 8 + ch * 2) * 128 + kr * 16;
                *reinterpret_cast<uint4 *>(o) = lo;
                *reinterpret_cast<uint4 *>(o + 128) = hi;
            }
        };
        // a raw block: the tail's rows, then the new ones, zero past the last
        auto store_raw = [&](int kv, int hh, int block, unsigned char *dst) {
#pragma unroll 1
            for (int j = cw; j < 8 * P::kVec; j += P::CW) {
                const int kg = j / P::kVec, dg = j % P::kVec, off = kg * 8 + kr, pos = block * kKvBlock + off;
                const bf *src = nullptr;
                if (pos < pos0) src = tail + kv_tail_offset(u.slot, u.src, kv, h, a.Hkv, D) + (int64_t)off * D;
                else if (pos < pos0 + n_tok)
                    src = static_cast<const bf *>(kv ? a.v_new : a.k_new) + ((int64_t)(u.row + pos - pos0) * a.Hkv + h) * D;
                uint32_t x[8] = {0, 0, 0, 0, 0, 0, 0, 0};
                if (src) {
                    const uint4 *q4 = reinterpret_cast<const uint4 *>(src + dg * 64 + ch * 16);
                    const uint4 y0 = q4[0], y1 = q4[1];
                    x[0] = y0.x; x[1] = y0.y; x[2] = y0.z; x[3] = y0.w;
                    x[4] = y1.x; x[5] = y1.y; x[6] = y1.z; x[7] = y1.w;
                }
                if (kv) {
                    // a value that is not finite would reach rows that do not see it (0 * inf): left out here, and added by
                    // the rows that do at the end
                    bool any = false;
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        if ((x[k] & 0x7F80u) == 0x7F80u) { x[k] &= 0xFFFF0000u; any = true; }
                        if ((x[k] & 0x7F800000u) == 0x7F800000u) { x[k] &= 0xFFFFu; any = true; }
                    }
                    if (any) atomicOr(&bad_v[block - blo], 1u);
                }
                unsigned char *o = dst + (hh * 8 + kg) * (D * 16) + (dg * 8 + ch * 2) * 128 + kr * 16;
                *reinterpret_cast<uint4 *>(o) = make_uint4(x[0], x[1], x[2], x[3]);
                *reinterpret_cast<uint4 *>(o + 128) = make_uint4(x[4], x[5], x[6], x[7]);
            }
        };
        load8(0, 0);
#pragma unroll 1
        for (int s = 0; s < n_seq; ++s) {
            int kv, step;
            what(s, kv, step);
            const int slot = step % NB, n_half = min(max(n8 - 2 * step, 0), 2);
            if (step >= NB) {
                if (!mbar_wait_bounded(&bar[(kv ? P::bVFree : P::bKFree) + slot], (step / NB - 1) & 1, limit)) {
                    alive = false;
                    break;
                }
            }
            unsigned char *dst = sm + (kv ? P::kV : P::kK) + slot * P::kTile;
            if (kv) store8(std::true_type{}, dst, n_half);
            else store8(std::false_type{}, dst, n_half);
            if (s + 1 < n_seq) {   // the next tile's loads are under way while this one is finished and the next slot waited for
                int kv1, step1;
                what(s + 1, kv1, step1);
                load8(kv1, step1);
            }
            for (int hh = n_half; hh < 2 && 2 * step + hh < nh; ++hh) store_raw(kv, hh, blo + 2 * step + hh - n8, dst);
            fence_proxy_async();
            if (s > 0 || a.skip_first_copy != 3) mbar_arrive(&bar[(kv ? P::bVFull : P::bKFull) + slot]);   // 3: the test hook
        }
        if (!alive && lane == 0) atomicOr(a.err, kErrTimeout);
        kv_named_barrier(1, P::kMma);
    } else if (warp / 4 < nt) {
        // ---- softmax warps ----
        const int tile = warp >> 2, r = r0 + t;    // t = 128 tile + row
        const uint32_t lanes = (uint32_t)(32 * (warp & 3)) << 16;
        const int pos = pos0 + r / a.G, blk = pos / kKvBlock, off = pos % kKvBlock;
        const uint32_t o_tm = tmem + lanes + P::kO + tile * D;
        float m = -INFINITY, l = 0.f;
        for (int step = 0; alive && step < steps; ++step) {
            const int i = step * nt + tile, b = i & 1;
            const uint32_t s_tm = tmem + lanes + 128 * b;
            alive = __all_sync(0xffffffffu, mbar_wait_bounded(&bar[P::bS + b], (i / 2) & 1, limit));
            if (!alive) break;
            tc_fence_after();
            const int halves = min(2, nh - 2 * step);
            auto half_step = [&](auto is_raw, int hh) {
                constexpr bool raw = decltype(is_raw)::value;
                const int hi = 2 * step + hh;
                const HalfInfo x = half[hi];
                // keys of the half that the row sees: all or none of an 8-bit block, up to its own offset of its raw block
                const int see = raw ? (blk == blo + hi - n8 ? off + 1 : 0) : (blk > c0 + hi ? kKvBlock : 0);
                float s[64];
                {
                    uint32_t w[4][16];
#pragma unroll
                    for (int j = 0; j < 4; ++j) tmem_ld16_nowait(s_tm + 64 * hh + 16 * j, w[j]);
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        tmem_wait_ld(w[j]);
#pragma unroll
                        for (int k = 0; k < 16; ++k) s[16 * j + k] = __uint_as_float(w[j][k]);
                    }
                }
                if (raw) {
#pragma unroll
                    for (int j = 0; j < 64; ++j) s[j] = j < see ? s[j] : -INFINITY;
                }
                float mx[4] = {s[0], s[1], s[2], s[3]};
#pragma unroll
                for (int j = 4; j < 64; ++j) mx[j & 3] = fmaxf(mx[j & 3], s[j]);
                const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * x.c + x.lvs;
                float f = 1.f;
                if (see > 0 && top > m + 8.f) {    // also the row's first keys (m = -inf)
                    f = ex2(m - top);              // 0 then
                    m = top;
                    l *= f;
                }
                // O is rescaled once the products that are under way on it are done (a row's first keys meet O = 0)
                if ((step > 0 || hh > 0) && __any_sync(0xffffffffu, f != 1.f)) {
                    bool done = true;
                    if (step > 0) done = __all_sync(0xffffffffu, mbar_wait_bounded(&bar[P::bPV + 2 * tile + 1], (step - 1) & 1, limit));
                    if (done && hh == 1)
                        done = __all_sync(0xffffffffu, mbar_wait_bounded(&bar[P::bPV + 2 * tile], step & 1, limit));
                    if (!done) return false;
                    tc_fence_after();
#pragma unroll 1
                    for (int c = 0; c < D; c += 16) {
                        uint32_t w[16];
                        tmem_ld16_nowait(o_tm + c, w);
                        tmem_wait_ld(w);
#pragma unroll
                        for (int k = 0; k < 16; ++k) w[k] = __float_as_uint(__uint_as_float(w[k]) * f);
                        tmem_st16(o_tm + c, w);
                    }
                    tmem_wait_st();
                }
                // the weights (8-bit blocks: times the value scale, which the sum takes out again); none of a block that
                // the row does not see
                const uint64_t cc = f2_pack(x.c, x.c);
                const float add = see == 0 ? -INFINITY : (raw ? 0.f : x.lvs) - (m == -INFINITY ? 0.f : m);
                const uint64_t bb = f2_pack(add, add);
                uint64_t sum[2] = {0, 0};
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    uint32_t w[16], lo[16];
#pragma unroll
                    for (int k = 0; k < 16; ++k) {
                        const int e = 32 * j + 2 * k;
                        float p0, p1;
                        f2_unpack(f2_fma(f2_pack(s[e], s[e + 1]), cc, bb), p0, p1);
                        p0 = ex2(p0);
                        p1 = ex2(p1);
                        sum[k & 1] = f2_add(sum[k & 1], f2_pack(p0, p1));
                        if (raw) {
                            uint32_t x1;
                            split_bf16x2(p0, p1, x1, lo[k]);
                            w[k] = x1;
                        } else {
                            w[k] = f2_to_h2(p0, p1);
                        }
                    }
                    tmem_st16(s_tm + 64 * hh + 16 * j, w);
                    if (raw) tmem_st16(s_tm + 64 * hh + 32 + 16 * j, lo);
                }
                float s0, s1;
                f2_unpack(f2_add(sum[0], sum[1]), s0, s1);
                l = fmaf(s0 + s1, x.ivs, l);
                tmem_wait_st();
                tc_fence_before();
                mbar_arrive(&bar[P::bP + 2 * b + hh]);
                return true;
            };
#pragma unroll 1
            for (int hh = 0; alive && hh < halves; ++hh)
                alive = 2 * step + hh < n8 ? half_step(std::false_type{}, hh) : half_step(std::true_type{}, hh);
        }
        // every product is done, and the convert warps have said what they left out: the rows
        kv_named_barrier(1, P::kMma);
        if (alive) alive = __all_sync(0xffffffffu, mbar_wait_bounded(&bar[P::bDrain], 0, limit));
        if (alive) {
            tc_fence_after();
            const bool live = t < rows_here;
            const int head = h * a.G + r % a.G, tok = r / a.G;
            const bool one = last_seg == 0;
            const float inv = one ? (l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l)) : 1.f;   // no key: zero; NaN stays
            bf *out = static_cast<bf *>(a.out) + ((int64_t)(u.row + tok) * a.Hq + head) * D;
            int64_t pr = 0;
            if (live && !one) {
                pr = kv_part_row(a, ui + blk - u.block, seg, blk == u.block ? tok : off, head);
                a.part_ml[pr] = make_float2(m, l);
            }
            const bool fix = live && seg == last_seg && bad_v[min(max(blk - blo, 0), 3)] != 0;
#pragma unroll 1
            for (int c = 0; c < D; c += 16) {
                uint32_t w[16];
                tmem_ld16_nowait(o_tm + c, w);
                tmem_wait_ld(w);
                float v[16];
#pragma unroll
                for (int k = 0; k < 16; ++k) v[k] = __uint_as_float(w[k]) * inv;
                if (fix) {
                    for (int j = 0; j <= off; ++j) {
                        const int kp = blk * kKvBlock + j;
                        const bf *src = kp < pos0 ? static_cast<const bf *>(a.c.tail) + kv_tail_offset(u.slot, u.src, 1, h, a.Hkv, D) + (int64_t)j * D
                                                  : static_cast<const bf *>(a.v_new) + ((int64_t)(u.row + kp - pos0) * a.Hkv + h) * D;
                        for (int k = 0; k < 16; ++k) {
                            const float y = to_f(src[c + k]);
                            if (!(fabsf(y) <= 3.4e38f)) v[k] += y;
                        }
                    }
                }
                if (!live) continue;
                if (one) {
                    uint32_t o[8];
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        const __nv_bfloat162 x = __floats2bfloat162_rn(v[2 * k], v[2 * k + 1]);
                        o[k] = *reinterpret_cast<const uint32_t *>(&x);
                    }
                    *reinterpret_cast<uint4 *>(out + c) = make_uint4(o[0], o[1], o[2], o[3]);
                    *reinterpret_cast<uint4 *>(out + c + 8) = make_uint4(o[4], o[5], o[6], o[7]);
                } else {
                    float4 *dst = reinterpret_cast<float4 *>(a.part_o + pr * D + c);
#pragma unroll
                    for (int k = 0; k < 4; ++k) dst[k] = make_float4(v[4 * k], v[4 * k + 1], v[4 * k + 2], v[4 * k + 3]);
                }
            }
        } else if (lane == 0) {
            atomicOr(a.err, kErrTimeout);
        }
    } else {
        kv_named_barrier(1, P::kMma);   // the second tile's warps, without rows
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 0) tmem_dealloc(tmem, P::kTmemCols);
}

template <int D>
cudaError_t launch_prompt(const KvAttn &a, int n_units, cudaStream_t st) {
    using P = PromptPlan<D>;
    cudaError_t e = cudaFuncSetAttribute(kv_attn_prompt_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)P::kBytes);
    if (e != cudaSuccess) return e;
    // blocks of a span: enough rows to fill the tile where a block's tokens are too few (G = 1, 2), a power of two <= 4
    int span = 1;
    while (span < 4 && 2 * span * kKvBlock * a.G <= P::R) span *= 2;
    const int64_t rows_max = (int64_t)std::min(span * kKvBlock, a.max_new) * a.G;
    const int row_tiles = (int)((rows_max + P::R - 1) / P::R);
    const dim3 grid((unsigned)((int64_t)n_units * row_tiles), (unsigned)a.Hkv, (unsigned)a.n_seg);
    e = gdn_launch_pdl(kv_attn_prompt_kernel<D>, grid, P::NT, P::kBytes, st, a, row_tiles, span, n_units);
    return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace gdn

cudaError_t gdn_launch_kv_attn_prompt(const gdn::KvAttn &a, int d, int n_units, cudaStream_t st) {
    if (d == 64) return gdn::launch_prompt<64>(a, n_units, st);
    if (d == 128) return gdn::launch_prompt<128>(a, n_units, st);
    return gdn::launch_prompt<256>(a, n_units, st);
}

// Attention of many query rows over the paged 8-bit key/value cache on the 5th-generation tensor core (bf16 inputs).
//
// The mathematics is that of kv_attn_simt.cuh; here the two products of a block of 64 keys are tcgen05 MMAs:
//   S = Q K^T     128 rows x 64 keys, K = d, operands fp16 in shared memory. A row of Q is scaled by a power of two to a
//                 largest element in [2^14, 2^15), which is exact (but for elements 2^-32 of the largest), and taken out
//                 of the scores again. An int8 key is exact in fp16. A key of the row's own block, which is read as it
//                 came, is scaled by a power of two like a row of Q.
//   O += P V      128 rows x d, K = 64 keys: P in TMEM as the A operand, V in shared memory. An 8-bit block: V int8 -> fp16
//                 (exact), P = 2^{c s + dv - m} with the block's value scale over the unit of O, 2^dv (kv_attn.cuh), in
//                 the weight and m 4 below the running maximum of exactly that exponent, so P <= 2^15.5 whatever the
//                 scales, and fp16 rounds it by 2^-11 of its size down to 2^-18 of the segment's largest (2^-25 absolute
//                 below 2^-14): keys beside a first token that takes nearly all of the weight, and whose value is next to
//                 nothing, keep their bits. The row's own block: V bf16, P in two bf16 products, its upper and lower 8
//                 bits: a row with few keys has nothing to average a rounding out. The sum l takes the unrounded weights
//                 without the scale, 2^{c s - m}.
//
// CTA: one row tile of R = 256 rows (two MMA tiles of 128; d = 256: one tile) of one kv head, over one segment of keys.
// Rows are the (token, query head of the group) pairs of a span: consecutive blocks of one request, aligned to `span`
// blocks, so that 64 span G >= R where it can be. Warp roles:
//   softmax   a warpgroup per MMA tile, one row per thread: TMEM scores -> weights -> TMEM P, running maximum and sum
//   keys, values   4 warps each: pages from global memory, int8 -> fp16 in registers, into the operand layout
//   MMA       a warp per MMA tile issues its products
// Each MMA tile has two score buffers of 64 columns, so the next block's scores are computed while a block's weights are
// (N = 64 makes S smem-bound, 48 cycles an MMA against 32, measured; with one 128-column buffer the softmax and the
// tensor core waited for each other, 5,600 against 2,560 cycles per 128 keys of the two tiles). The weights overwrite the
// scores that they came from.
//
// m only moves when a block's weights would pass 2^15.5 (fp16 ends at 2^16): O is rescaled (by the softmax warps, after the
// product before it) only then. Room above m spares moves, room below spares the small weights' bits: with 14 above (and m
// at the maximum) the turn below took 1,066 us, with 11.5 1,095, with 8 1,137, most of the moves being those of sharp rows
// after their first block. Every decision is a row's own and every block is one softmax step, so a row's bits do
// not depend on the rows beside it.
//
// Built for each part (KvPart): whole contexts; a request's own keys past the blocks that its group shares, from the first of
// them on; and a group's shared blocks (kv_shared_piece.cuh), where rows are the group's, in tiles that go across its requests,
// no row has a mask and no block is raw, and the loop is that much shorter.
//
// Bound: the softmax warps' issue slots and the tensor core about evenly, 1,700 cycles for a block of 64 keys and two row
// tiles (1,900 with a segment's start and end), of which the products are 1,280: the scores' 768, as their MMAs of 64 keys
// take 48 cycles each, and the values' 512. 4,000 x 16 rows over 37,802 keys (d = 128): 1.10 ms, 1.18 PFLOP/s, tensor pipe
// 51 %; 290 x 16 rows over 41,802 keys (d = 256): 217 us, 0.92 PFLOP/s; the same turn with d = 64: 0.93 ms.
// Shared blocks: 8,000 x 16 rows over 37,760 keys (d = 128) 1.71 ms, 1.45 PFLOP/s, tensor pipe 59 %; 64 x 16 rows over 41,792
// keys (d = 256, 35 blocks a CTA) 50 us, 0.88 PFLOP/s, a quarter of it start and end. Tried there and slower: two threads a row
// (a block's cost is not its elements'), persistent CTAs that walk a list of pieces (2.0 ms: the issuing warps' waits grow).
#pragma once

#include "kv_attn.cuh"
#include "kv_shared_piece.cuh"

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

// mbarriers by 32-bit shared-memory address, waits bounded by `limit` polls.
__device__ __forceinline__ bool bar_test(uint32_t bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n selp.u32 %0, 1, 0, p;\n}\n"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    return ok != 0;
}
__device__ __forceinline__ bool bar_wait(uint32_t bar, uint32_t parity, int limit) {
    for (int i = 0; i < limit; ++i)
        if (bar_test(bar, parity)) return true;
    return false;
}
// Three barriers tested together, their latencies overlapping.
__device__ __forceinline__ bool bar_wait3(uint32_t b0, uint32_t p0, uint32_t b1, uint32_t p1, uint32_t b2, uint32_t p2, int limit) {
    for (int i = 0; i < limit; ++i) {
        const bool x = bar_test(b0, p0), y = bar_test(b1, p1), z = bar_test(b2, p2);
        if (x && y && z) return true;
    }
    return false;
}
// One arrival per warp and one polling lane: an arrival or a test by 32 lanes is 32 passes through the shared-memory
// pipe, which the MMA operands and the score loads fill already.
__device__ __forceinline__ void warp_arrive(uint32_t bar) {
    __syncwarp();
    if ((threadIdx.x & 31) == 0) asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];\n" ::"r"(bar) : "memory");
}
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, int limit) {
    bool ok = true;
    if ((threadIdx.x & 31) == 0) ok = bar_wait(bar, parity, limit);
    ok = __all_sync(0xffffffffu, ok);
    __syncwarp();   // what lane 0 has acquired, for the other lanes: a vote alone orders no memory
    return ok;
}
// The same with every lane polling, for waits that are rare.
__device__ __forceinline__ bool lanes_wait(uint32_t bar, uint32_t parity, int limit) {
    return __all_sync(0xffffffffu, bar_wait(bar, parity, limit));
}
__device__ __forceinline__ void bar_commit(uint32_t bar) {   // once the MMAs this thread issued are done
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n" ::"r"(bar) : "memory");
}
// One lane of a converged warp.
__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile("{\n .reg .pred q;\n elect.sync _|q, 0xffffffff;\n selp.u32 %0, 1, 0, q;\n}\n" : "=r"(p));
    return p != 0;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}
constexpr float kLift = 4.f;     // where a row's largest weight stands when m moves, log2
constexpr float kSlack = 11.5f;  // and how much further it may go before m moves again

template <int D>
struct PromptPlan {
    static constexpr int NQ = D == 256 ? 1 : 2;              // MMA tiles of 128 rows
    static constexpr int R = 128 * NQ;
    static constexpr int NS = D == 256 ? 3 : 4;              // key and value slots of 64 keys each
    // One tile leaves TMEM columns for its queries: they are the A operand from there, which spares the shared-memory pipe
    // two thirds of S's reads and the queries' place.
    static constexpr bool kQT = NQ == 1;
    static constexpr int CW = D == 256 ? 8 : 4;              // warps that convert keys, and as many that convert values
    // First thread of the roles. The issuing warps come first: a scheduler that prefers older warps then lets their few
    // instructions through.
    static constexpr int kSoft0 = 128, kKeys0 = kSoft0 + 128 * NQ, kVals0 = kKeys0 + 32 * CW, NT = kVals0 + 32 * CW;
    static constexpr uint32_t kTile = 128 * D * 2;           // bytes of a 128-row query tile
    // A slot's core matrices (8 keys x 16 bytes) lie 144 bytes apart along d and kGroup apart along the keys. With 128 the
    // lanes that write without bank conflicts are 8 keys of one column, whose 16-byte reads of 8 pages' rows take 32 passes
    // of the load pipe; with 144 they are 2 keys of 4 columns, and take 8.
    static constexpr uint32_t kCore = 144, kGroup = D / 8 * kCore;
    static constexpr uint32_t kBlk = 8 * kGroup;             // bytes of a slot
    // queries, key slots, value slots; with the queries in TMEM they pass through the third key and value slots
    static constexpr uint32_t kQ = kQT ? 4 * kBlk : 0, kK = kQT ? 0 : NQ * kTile, kV = kK + (kQT ? 2 : NS) * kBlk,
                              kInfo = kQT ? 6 * kBlk : kV + NS * kBlk;
    __host__ __device__ static constexpr uint32_t key_slot(uint32_t i) { return kK + (kQT && i == 2 ? 4 : i) * kBlk; }
    __host__ __device__ static constexpr uint32_t val_slot(uint32_t i) { return kV + (kQT && i == 2 ? 3 : i) * kBlk; }
    static constexpr int kMaxBlocks = kKvMaxSegBlocks + 4;                // 8-bit blocks of a segment and raw blocks of a span
    static constexpr uint32_t kRow = kInfo + kMaxBlocks * 16;        // float [R]: what takes Q's scaling out
    static constexpr uint32_t kRawK = kRow + R * 4;                  // float [4][64]: the scalings of the raw blocks' keys
    static constexpr uint32_t kBar = kRawK + 4 * 64 * 4;
    // barriers: key and value slots full and free, scores and weights of (tile, buffer), a tile's product before its last,
    // all products, the queries and the blocks' scales, the
    // queries in TMEM
    static constexpr int bKFull = 0, bKFree = NS, bVFull = 2 * NS, bVFree = 3 * NS, bS = 4 * NS, bP = bS + 2 * NQ,
                         bPV = bP + 2 * NQ, bDrain = bPV + NQ, bReady = bDrain + 1, bQ = bReady + 1, kNBar = bQ + 1;
    static constexpr uint32_t kSlot = kBar + (kNBar + 1) / 2 * 16;
    static constexpr uint32_t kBad = kSlot + 16;             // per raw block of the span: it has a value that is not finite
    static constexpr uint32_t kBytes = kBad + 16;
    static constexpr uint32_t kO = 256;                      // TMEM columns: scores [0, 128 NQ), queries from 128, outputs from here
    static constexpr uint32_t kTmemCols = 512;
    static constexpr int kVec = D / 64;                      // 64-column groups
    static constexpr int kLoads = 8 * kVec / CW;             // 16-byte loads of a key or value thread per block
    // Registers: an SM partition's 512 per lane hold 5 of the 20 warps (two tiles) at 96, or 6 of the 24 (one tile) at 80.
    // Then the issuing, key and value warps go down to 64 and the softmax warps up to 144: per partition
    // 64 + 2 x 144 + 2 x 64 = 480 of 480 (two tiles), 64 + 144 + 4 x 64 = 464 of 480 (one tile).
    static_assert(kBytes <= 227 * 1024 && R == kv_prompt_rows(D), "shared memory, rows of a CTA");
};

// A block of the pass: its page, c = scale log2(e) k_scale, and log2 of the value scale (kv_log2_scale; not of a raw block).
struct __align__(16) BlockInfo {
    int page;
    float c, lvs;
};
constexpr float kRawSpan = 16.f;   // how far a raw block's values, whose two-part weights have 8-bit exponents, may be from the unit 1


template <int D, int PART = kKvWhole>
__global__ void __launch_bounds__(PromptPlan<D>::NT, 1) kv_attn_prompt_kernel(const KvAttn a, int row_tiles, int span, int n_units) {
    using P = PromptPlan<D>;
    using bf = __nv_bfloat16;
    constexpr int NS = P::NS;
    const KvBeside beside(PART == kKvSuffix);
    int h = blockIdx.y, ui = 0, rt = 0, seg = 0, n_tok = 0, seg0 = 0, last_seg = 0, r0 = 0, cut = 0;
    KvUnit u;
    if constexpr (PART == kKvShared) {
        // a group's rows as those of one unit that starts where the shared blocks end: every row sees all of them
        int4 rec;
        if (!kv_shared_piece<P::R>(a, r0, h, seg, cut, rec)) return;
        if (!kv_group_ok(a, rec)) {
            if (threadIdx.x == 0) atomicOr(a.err, kErrKvBounds);
            return;
        }
        u = {rec.z, rec.w, -1, 0, rec.y, rec.x, 0, 0};
        n_tok = rec.y;
        last_seg = INT32_MAX;   // no segment has a block of the rows' own
    } else {
        // later units (longer contexts) first: a causal launch then ends on its short ones
        ui = a.unit0 + n_units - 1 - (int)(blockIdx.x / row_tiles);
        rt = blockIdx.x % row_tiles;
        // and of growing segments the longer ones
        seg = a.seg_blocks ? (int)blockIdx.z : a.n_seg - 1 - (int)blockIdx.z;
        u = kv_load_unit(a.units, ui);   // inside the map whatever the count
        const int unit1 = min(a.unit0 + n_units, a.counts[0]);
        if (ui >= unit1) return;
        const int start = PART == kKvSuffix ? a.starts[ui] : 0;   // the first block of the pass
        bool ok = kv_part_unit_ok<PART>(a, u, start);
        // the span's first unit works for all of it (the first of a run of them, where one between is left out)
        if (ok && ui > a.unit0 && u.block % span != 0) {
            const KvUnit w = kv_load_unit(a.units, ui - 1);
            if (w.slot == u.slot && w.block == u.block - 1 && kv_part_unit_ok<PART>(a, w, start)) return;
        }
        n_tok = u.count;
        for (int i = 1; ok && i < span && ui + i < unit1 && (u.block + i) % span != 0; ++i) {
            const KvUnit w = kv_load_unit(a.units, ui + i);
            if (w.slot != u.slot || w.block != u.block + i) break;
            if (!kv_part_unit_ok<PART>(a, w, start)) break;   // reported by its own CTA
            ok = w.first == 0 && w.row == u.row + n_tok;
            n_tok += w.count;
        }
        if (!ok) {
            if (threadIdx.x == 0) atomicOr(a.err, kErrKvBounds);
            return;
        }
        last_seg = kv_seg_of(a, u.block);   // a span lies in one segment: span divides their starts
        seg0 = kv_part_seg0<PART>(a, start);
        seg += seg0;
        r0 = rt * P::R;
        if (seg > last_seg) return;
    }
    const int n_row = n_tok * a.G;
    if (r0 >= n_row) return;

    extern __shared__ __align__(1024) unsigned char sm[];
    uint64_t *bar64 = reinterpret_cast<uint64_t *>(sm + P::kBar);
    const uint32_t bar0 = smem_addr(bar64);
    auto bar = [&](int i) { return bar0 + 8 * i; };
    uint32_t *tslot = reinterpret_cast<uint32_t *>(sm + P::kSlot);
    uint32_t *bad_v = reinterpret_cast<uint32_t *>(sm + P::kBad);
    BlockInfo *info = reinterpret_cast<BlockInfo *>(sm + P::kInfo);
    float *row_q = reinterpret_cast<float *>(sm + P::kRow);
    float *raw_k = reinterpret_cast<float *>(sm + P::kRawK);
    const int t = threadIdx.x, warp = t >> 5, lane = t & 31;
    const int pos0 = u.block * kKvBlock + u.first;
    const int rows_here = min(P::R, n_row - r0);
    const int nt = rows_here > 128 ? 2 : 1;        // MMA tiles in use
    // blocks of this tile's rows, and the blocks of the pass: 8-bit [c0, c0 + n8), then raw from blo
    const int blo = PART == kKvShared ? u.block : (pos0 + r0 / a.G) / kKvBlock,
              bhi = PART == kKvShared ? u.block : (pos0 + (r0 + rows_here - 1) / a.G) / kKvBlock;
    const int c0 = PART == kKvShared ? seg * cut
                   : PART == kKvSuffix ? max(kv_seg_start(a, seg), a.starts[ui]) : kv_seg_start(a, seg);
    const int n8 = min(bhi, PART == kKvShared ? c0 + cut : kv_seg_start(a, seg + 1)) - c0;
    const int nb = n8 + (PART != kKvShared && seg == last_seg ? bhi - blo + 1 : 0);

    if (t == 0) {
        for (int i = 0; i < NS; ++i) {
            mbar_init(&bar64[P::bKFull + i], P::CW);
            mbar_init(&bar64[P::bVFull + i], P::CW);
            mbar_init(&bar64[P::bKFree + i], nt);
            mbar_init(&bar64[P::bVFree + i], nt);
        }
        for (int i = 0; i < 2 * P::NQ; ++i) {
            mbar_init(&bar64[P::bS + i], 1);
            mbar_init(&bar64[P::bP + i], 4);
        }
        for (int i = 0; i < P::NQ; ++i) mbar_init(&bar64[P::bPV + i], 1);
        mbar_init(&bar64[P::bDrain], nt);
        mbar_init(&bar64[P::bReady], P::NT / 32);
        mbar_init(&bar64[P::bQ], 4);
        mbar_init_fence();
        for (int i = 0; i < 4; ++i) bad_v[i] = 0;
    }
    if (warp == 0) {
        tmem_alloc(tslot, P::kTmemCols);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    constexpr uint32_t tmem = 0;   // all 512 columns are this CTA's
    const int limit = (int)min(a.wait_limit, 1LL << 30);
    bool alive = true;

    if (t < P::kKeys0) {
        // ---- the queries, by the issuing and the softmax warps while the first blocks are fetched: a warp takes 8 rows at a
        // time and 4 lanes a row, each every fourth piece of 8 columns. So two rows and two sectors go to a quarter warp's load,
        // and the 32 stores of a piece fill four K-major core matrices (8 rows x 16 bytes) side by side, free of conflicts ----
        constexpr int NP = D / 32, STEP = P::kKeys0 / 32 * 8;
        const int c = lane & 3;
        auto load_row = [&](int r, uint4 (&w)[NP]) {
            const int rr = r0 + r;
            if (r < rows_here) {
                const int tok = rr / a.G;
                const uint4 *src = reinterpret_cast<const uint4 *>(static_cast<const bf *>(a.q) +
                                                                   ((int64_t)(u.row + tok) * a.Hq + h * a.G + (rr - tok * a.G)) * D) + c;
#pragma unroll
                for (int i = 0; i < NP; ++i) w[i] = __ldg(src + 4 * i);
            } else {
#pragma unroll
                for (int i = 0; i < NP; ++i) w[i] = make_uint4(0, 0, 0, 0);
            }
        };
        auto put_row = [&](int r, const uint4 (&w)[NP]) {
            float f[8], top = 0.f;
#pragma unroll
            for (int i = 0; i < NP; ++i) {
                b8_to_f(w[i], f);
#pragma unroll
                for (int k = 0; k < 8; ++k) top = fmaxf(top, fabsf(f[k]));
            }
#pragma unroll
            for (int o = 2; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
            float back;
            const float up = pow2_to_2_15(top, back);
            unsigned char *dst = sm + P::kQ + (r >> 7) * P::kTile + ((r & 127) >> 3) * (D * 16) + c * 128 + (r & 7) * 16;
#pragma unroll
            for (int i = 0; i < NP; ++i) {
                b8_to_f(w[i], f);
#pragma unroll
                for (int k = 0; k < 8; ++k) f[k] *= up;
                *reinterpret_cast<uint4 *>(dst + 512 * i) = f8_to_h8(f);
            }
            if (c == 0) row_q[r] = back;
        };
        const int r1 = warp * 8 + (lane >> 2);
        if constexpr (PART == kKvShared && P::NQ == 2) {   // short passes: every row under way before the first is put down
            constexpr int IT = (P::R + STEP - 1) / STEP;
            uint4 w[IT][NP];
#pragma unroll
            for (int i = 0; i < IT; ++i)
                if (r1 + i * STEP < nt * 128) load_row(r1 + i * STEP, w[i]);
#pragma unroll
            for (int i = 0; i < IT; ++i)
                if (r1 + i * STEP < nt * 128) put_row(r1 + i * STEP, w[i]);
        } else {
#pragma unroll 1
            for (int r = r1; r < nt * 128; r += STEP) {
                uint4 w[NP];
                load_row(r, w);
                put_row(r, w);
            }
        }
        if constexpr (P::kQT) {   // each softmax thread its row, from the slots into TMEM
            kv_named_barrier(3, P::kKeys0);
            if (t >= P::kSoft0) {
                const int r = t - P::kSoft0;
                const unsigned char *src = sm + P::kQ + (r >> 3) * (D * 16) + (r & 7) * 16;
#pragma unroll 1
                for (int k = 0; k < D / 32; ++k) {
                    uint32_t w[16];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const uint4 x = *reinterpret_cast<const uint4 *>(src + (4 * k + i) * 128);
                        w[4 * i] = x.x; w[4 * i + 1] = x.y; w[4 * i + 2] = x.z; w[4 * i + 3] = x.w;
                    }
                    tmem_st16(tmem + ((uint32_t)(32 * (warp & 3)) << 16) + 128 + 16 * k, w);
                }
                tmem_wait_st();
                tc_fence_before();
                warp_arrive(bar(P::bQ));
            }
        } else {
            fence_proxy_async();
        }
        warp_arrive(bar(P::bReady));
        alive = lanes_wait(bar(P::bReady), 0, limit);
    }
    if (t < P::kSoft0) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 64;\n");
        // ---- the issuing warps, one per tile: whole warps in step, one elected lane issues (a lane of its own in a divergent
        // branch takes 84 cycles per MMA beside busy warps, an elected lane of a warp in step 53, measured) ----
        const int tile = __shfl_sync(0xffffffffu, warp, 0);   // the same in every lane, and the compiler sees it
        if (tile < nt) {
            constexpr uint32_t idS = umma_idesc_f16(128, 64, 0, 0), idO8 = umma_idesc_f16(128, D, 0, 1),
                               idOraw = umma_idesc_bf16(128, D, 0, 1);
            const bool elected = elect_one();
            if constexpr (P::kQT) alive = lanes_wait(bar(P::bQ), 0, limit) && alive;
            const uint64_t dq = umma_smem_desc(sm + P::kQ + tile * P::kTile, 128, D * 16),
                           dk0 = umma_smem_desc(sm, P::kCore, P::kGroup), dv0 = umma_smem_desc(sm, P::kGroup, P::kCore);
            const uint32_t s0_tm = tmem + 128 * tile, o_tm = tmem + P::kO + tile * D;
            auto issue_s = [&](int n) {
                const int slot = n % NS, b = n & 1;
                const uint64_t dk = dk0 + (P::key_slot(slot) >> 4);
                if (elected) {
#pragma unroll
                    for (int k = 0; k < D / 16; ++k) {
                        if constexpr (P::kQT) umma_bf16_ts(s0_tm + 64 * b, tmem + 128 + 8 * k, dk + 2 * P::kCore / 16 * k, idS, k > 0);
                        else umma_bf16(s0_tm + 64 * b, dq + 16 * k, dk + 2 * P::kCore / 16 * k, idS, k > 0);
                    }
                    bar_commit(bar(P::bS + 2 * tile + b));
                    bar_commit(bar(P::bKFree + slot));
                }
            };
            tc_fence_after();
            for (int n = 0; alive && n < min(nb, 2); ++n) {
                alive = __all_sync(0xffffffffu, bar_wait(bar(P::bKFull + n % NS), (n / NS) & 1, limit));
                tc_fence_after();
                if (alive) issue_s(n);
            }
#pragma unroll 1
            for (int n = 0; alive && n < nb; ++n) {
                const int slot = n % NS, b = n & 1;
                const bool more = n + 2 < nb;
                const int nk = more ? n + 2 : n;   // the keys of the product that follows (n: there already)
                alive = __all_sync(0xffffffffu, bar_wait3(bar(P::bVFull + slot), (n / NS) & 1, bar(P::bKFull + nk % NS), (nk / NS) & 1,
                                                      bar(P::bP + 2 * tile + b), (n >> 1) & 1, limit));
                if (!alive) break;
                tc_fence_after();
                const uint64_t dv = dv0 + (P::val_slot(slot) >> 4);
                const uint32_t p_tm = s0_tm + 64 * b, idO = n < n8 ? idO8 : idOraw;
                if (elected) {
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        umma_bf16_ts(o_tm, p_tm + 8 * k, dv + 2 * P::kGroup / 16 * k, idO, n > 0 || k > 0);
                    if (n >= n8) {   // the low parts of the raw block's weights
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            umma_bf16_ts(o_tm, p_tm + 32 + 8 * k, dv + 2 * P::kGroup / 16 * k, idO, 1);
                    }
                }
                if (more) issue_s(n + 2);
                if (elected) {
                    bar_commit(bar(P::bVFree + slot));
                    if (n == nb - 2) bar_commit(bar(P::bPV + tile));
                }
            }
            if (elected) {
                if (!alive) atomicOr(a.err, kErrTimeout);
                bar_commit(bar(P::bDrain));
                if (!bar_wait(bar(P::bDrain), 0, limit)) atomicOr(a.err, kErrTimeout);
            }
        }
    } else if (t >= P::kKeys0) {
        // ---- key and value warps: each role's convert a block at a time, its loads one block ahead (two ahead, with the
        // loop unrolled by two, measured slower: the roles share one instruction cache) ----
        asm volatile("setmaxnreg.dec.sync.aligned.u32 64;\n");
        const bool is_v = t >= P::kVals0;
        // load i of this warp: 8 keys x 64 columns, key group (cw + CW i) / kVec, column group (cw + CW i) % kVec
        uint4 w[P::kLoads];
        auto load_from = [&](const int8_t *src, int cw) {
#pragma unroll
            for (int i = 0; i < P::kLoads; ++i) {
                const int j = cw + P::CW * i;
                w[i] = __ldg(reinterpret_cast<const uint4 *>(src + j / P::kVec * (8 * D) + j % P::kVec * 64));
            }
        };
        // pages and scales of the pass's blocks, which the softmax warps read as well; with d = 256 and over shared blocks the
        // first block's loads before them (2.5 % of 290 x 16 rows over 41,802 keys; the two-tile form over whole contexts has no
        // registers left for that: 6 % slower)
        const int32_t *table = a.c.table + (int64_t)u.slot * a.c.max_blocks;
        constexpr bool kEarly = P::kQT || PART == kKvShared;
        if (kEarly && n8 > 0) {
            int page = table[c0];
            if ((unsigned)page >= (unsigned)a.c.n_pages) page = 0;
            load_from((is_v ? a.c.v : a.c.k) + ((int64_t)page * a.Hkv + h) * (kKvBlock * D) + (lane >> 2) * D + (lane & 3) * 16, warp % P::CW);
        }
        for (int i = t - P::kKeys0; i < nb; i += 64 * P::CW) {
            BlockInfo x = {0, a.scale_log2, 0.f};
            if (i < n8) {
                x.page = table[c0 + i];
                const bool in = (unsigned)x.page < (unsigned)a.c.n_pages;
                if (!in) {
                    x.page = 0;                        // in bounds; the result is reported as invalid
                    atomicOr(a.err, kErrKvBounds);
                }
                const int64_t ph = (int64_t)x.page * a.Hkv + h;
                const float ks = a.c.k_scale[ph], vs = a.c.v_scale[ph];
                x.c = in ? a.scale_log2 * ks : 0.f;
                x.lvs = in ? kv_log2_scale(vs) : INFINITY;
            }
            info[i] = x;
        }
        kv_named_barrier(2, 64 * P::CW);
        warp_arrive(bar(P::bReady));
        const int cw = warp % P::CW, kr = lane >> 2, ch = lane & 3;   // warp of the role; key of 8 and 16-byte chunk of 64
        const bf *tail = static_cast<const bf *>(a.c.tail);
        const int8_t *pool = (is_v ? a.c.v : a.c.k) + (int64_t)h * (kKvBlock * D) + kr * D + ch * 16;
        const int64_t stride = (int64_t)a.Hkv * (kKvBlock * D);
        const uint32_t full = bar(is_v ? P::bVFull : P::bKFull), free = bar(is_v ? P::bVFree : P::bKFree);
        auto load = [&](int n) { load_from(pool + info[min(n, nb - 1)].page * stride, cw); };   // a raw block: page 0, not used
        auto store = [&](unsigned char *dst) {
#pragma unroll
            for (int i = 0; i < P::kLoads; ++i) {
                const int j = cw + P::CW * i;
                const uint2 x0 = i8_to_f16x4(w[i].x), x1 = i8_to_f16x4(w[i].y), x2 = i8_to_f16x4(w[i].z), x3 = i8_to_f16x4(w[i].w);
                unsigned char *o = dst + j / P::kVec * P::kGroup + j % P::kVec * (8 * P::kCore);
                *reinterpret_cast<uint4 *>(o) = make_uint4(x0.x, x0.y, x1.x, x1.y);
                *reinterpret_cast<uint4 *>(o + P::kCore) = make_uint4(x2.x, x2.y, x3.x, x3.y);
            }
        };
        // a raw block: the tail's rows, then the new ones, zero past the last
        auto store_raw = [&](int block, unsigned char *dst) {
#pragma unroll 1
            for (int kg = cw; kg < 8; kg += P::CW) {
                const int off = kg * 8 + kr, pos = block * kKvBlock + off;
                const bf *src = nullptr;
                if (pos < pos0) src = tail + kv_tail_offset(u.slot, u.src, is_v, h, a.Hkv, D) + (int64_t)off * D;
                else if (pos < pos0 + n_tok)
                    src = static_cast<const bf *>(is_v ? a.v_new : a.k_new) + ((int64_t)(u.row + pos - pos0) * a.Hkv + h) * D;
                float top = 0.f, up = 1.f;
                if constexpr (PART == kKvSuffix) {
                    // raw blocks are most of such a pass: a row's pieces loaded together, where the loop below (whose few
                    // instructions leave the instruction cache to the complete blocks) waits for memory four times
                    uint4 y[P::kVec][2];
#pragma unroll
                    for (int dg = 0; dg < P::kVec; ++dg)
#pragma unroll
                        for (int k = 0; k < 2; ++k)
                            y[dg][k] = src ? reinterpret_cast<const uint4 *>(src + dg * 64 + ch * 16)[k] : make_uint4(0, 0, 0, 0);
                    if (!is_v) {
#pragma unroll
                        for (int dg = 0; dg < P::kVec; ++dg)
#pragma unroll
                            for (int k = 0; k < 2; ++k) {
                                float f[8];
                                b8_to_f(y[dg][k], f);
#pragma unroll
                                for (int x = 0; x < 8; ++x) top = fmaxf(top, fabsf(f[x]));
                            }
                        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
                        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
                        float back;
                        up = pow2_to_2_15(top, back);
                        if (ch == 0) raw_k[(block - blo) * 64 + off] = back;
                    }
#pragma unroll
                    for (int dg = 0; dg < P::kVec; ++dg)
#pragma unroll
                        for (int k = 0; k < 2; ++k) {
                            if (is_v) {
                                if (drop_not_finite(y[dg][k])) atomicOr(&bad_v[block - blo], 1u);   // added by the rows that see it
                            } else {
                                float f[8];
                                b8_to_f(y[dg][k], f);
#pragma unroll
                                for (int x = 0; x < 8; ++x) f[x] *= up;
                                y[dg][k] = f8_to_h8(f);
                            }
                            *reinterpret_cast<uint4 *>(dst + kg * P::kGroup + dg * (8 * P::kCore) + k * P::kCore) = y[dg][k];
                        }
                    continue;
                }
#pragma unroll 1
                for (int pass = is_v ? 1 : 0; pass < 2; ++pass) {   // keys: the largest element first, then the scaled key
#pragma unroll 1
                    for (int dg = 0; dg < P::kVec; ++dg) {
                        uint4 y[2] = {make_uint4(0, 0, 0, 0), make_uint4(0, 0, 0, 0)};
                        if (src) {
                            y[0] = reinterpret_cast<const uint4 *>(src + dg * 64 + ch * 16)[0];
                            y[1] = reinterpret_cast<const uint4 *>(src + dg * 64 + ch * 16)[1];
                        }
#pragma unroll
                        for (int k = 0; k < 2; ++k) {
                            if (is_v) {
                                // a value that is not finite would reach rows that do not see it (0 * inf): left out here,
                                // and added by the rows that do at the end
                                if (drop_not_finite(y[k])) atomicOr(&bad_v[block - blo], 1u);
                            } else {
                                float f[8];
                                b8_to_f(y[k], f);
#pragma unroll
                                for (int x = 0; x < 8; ++x) {
                                    top = fmaxf(top, fabsf(f[x]));
                                    f[x] *= up;
                                }
                                y[k] = f8_to_h8(f);
                            }
                            if (pass == 1) *reinterpret_cast<uint4 *>(dst + kg * P::kGroup + dg * (8 * P::kCore) + k * P::kCore) = y[k];
                        }
                    }
                    if (pass == 0) {
                        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
                        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
                        float back;
                        up = pow2_to_2_15(top, back);
                        if (ch == 0) raw_k[(block - blo) * 64 + off] = back;
                    }
                }
            }
        };
        if (!kEarly) load(0);
#pragma unroll 1
        for (int n = 0; n < nb; ++n) {
            const int slot = n % NS;
            if (n >= NS && !warp_wait(free + 8 * slot, (n / NS - 1) & 1, limit)) {
                alive = false;
                break;
            }
            if (P::kQT && n == 2 && !lanes_wait(bar(P::bQ), 0, limit)) {   // the queries leave the third slots
                alive = false;
                break;
            }
            unsigned char *dst = sm + (is_v ? P::val_slot(slot) : P::key_slot(slot)) + kr * 16 + ch * (2 * P::kCore);
            if (n < n8) {
                store(dst);
                load(n + 1);
            } else {
                store_raw(blo + n - n8, dst);
            }
            fence_proxy_async();
            if (n > 0 || is_v || a.skip_first_copy != 3) warp_arrive(full + 8 * slot);   // 3: the test hook
        }
        if (!alive && lane == 0) atomicOr(a.err, kErrTimeout);
        kv_named_barrier(1, P::NT - P::kSoft0);
    } else if (warp / 4 <= nt) {
        // ---- softmax warps ----
        asm volatile("setmaxnreg.inc.sync.aligned.u32 144;\n");
        const int tr = t - P::kSoft0, tile = tr >> 7, r = r0 + tr;   // tr = 128 tile + row
        const uint32_t lanes = (uint32_t)(32 * (warp & 3)) << 16;
        const int pos = pos0 + r / a.G, blk = pos / kKvBlock, off = pos % kKvBlock;
        const uint32_t o_tm = tmem + lanes + P::kO + tile * D;
        const float rq = row_q[tr];
        float m = -INFINITY, l = 0.f, lref = 0.f;
        auto block_step = [&](auto is_raw, int n) {
            constexpr bool raw = decltype(is_raw)::value;
            const int b = 2 * tile + (n & 1);
            const uint32_t s_tm = tmem + lanes + 64 * b;
            if (!warp_wait(bar(P::bS + b), (n >> 1) & 1, limit)) return false;
            // the key warps' scalings; no later block takes the slot (the pass ends with its at most NS raw blocks)
            if (raw && !lanes_wait(bar(P::bKFull + n % NS), (n / NS) & 1, limit)) return false;
            tc_fence_after();
            const BlockInfo x = info[n];
            // keys of the block that the row sees: all or none of an 8-bit block, up to its own offset of its raw block
            const int see = raw ? (blk == blo + n - n8 ? off + 1 : 0) : (PART == kKvShared || blk > c0 + n ? kKvBlock : 0);
            const float c = x.c * rq;
            float s[64];
            {
                uint32_t w[4][16];
#pragma unroll
                for (int j = 0; j < 4; ++j) tmem_ld16_nowait(s_tm + 16 * j, w[j]);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    tmem_wait_ld(w[j]);
#pragma unroll
                    for (int k = 0; k < 16; ++k) s[16 * j + k] = __uint_as_float(w[j][k]);
                }
            }
            if (raw) {
                const float *kf = raw_k + (n - n8) * 64;
#pragma unroll
                for (int j = 0; j < 64; ++j) s[j] = j < see ? s[j] * kf[j] : -INFINITY;
            }
            float mx[4] = {s[0], s[1], s[2], s[3]};
#pragma unroll
            for (int j = 4; j < 60; j += 8)
#pragma unroll
                for (int k = 0; k < 4; ++k) mx[k] = max3(mx[k], s[j + k], s[j + 4 + k]);
#pragma unroll
            for (int k = 0; k < 4; ++k) mx[k] = fmaxf(mx[k], s[60 + k]);
            // the block's values over the unit of O; a raw block's are their own, and the weights' power of two is exact
            float f = 1.f, dv = 0.f, raw_up = 1.f;   // f: what O is rescaled by
            if (raw) {
                if (fabsf(lref) > kRawSpan) {
                    f = pow2_of(lref);
                    lref = 0.f;
                }
                raw_up = pow2_of(-lref);
            } else {
                dv = kv_unit(x.lvs, lref, f);
            }
            const float top = fmaf(fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])), c, dv - kLift);
            if (see > 0 && top > m + kSlack) {    // also the row's first keys (m = -inf)
                const float g = ex2(m - top);  // 0 then
                m = top;
                l *= g;
                f *= g;
            }
            // O is rescaled once the product that is under way on it is done (a row's first keys meet O = 0)
            if (n > 0 && __any_sync(0xffffffffu, f != 1.f)) {
                // the next scores were issued after that product
                const bool last = n == nb - 1;
                if (!lanes_wait(bar(last ? P::bPV + tile : P::bS + 2 * tile + ((n + 1) & 1)), last ? 0 : ((n + 1) >> 1) & 1, limit))
                    return false;
                tc_fence_after();
#pragma unroll 1
                for (int k0 = 0; k0 < D; k0 += 32) {
                    uint32_t w[2][16];
#pragma unroll
                    for (int j = 0; j < 2; ++j) tmem_ld16_nowait(o_tm + k0 + 16 * j, w[j]);
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        tmem_wait_ld(w[j]);
#pragma unroll
                        for (int k = 0; k < 16; ++k) w[j][k] = __float_as_uint(__uint_as_float(w[j][k]) * f);
                        tmem_st16(o_tm + k0 + 16 * j, w[j]);
                    }
                }
                tmem_wait_st();
            }
            // the weights (8-bit blocks: times the value scale over the unit, which the sum takes out again); none of a block
            // that the row does not see
            const uint64_t cc = f2_pack(c, c);
            const float add = see == 0 ? -INFINITY : dv - (m == -INFINITY ? 0.f : m);
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
                    if (raw) split_bf16x2(p0 * raw_up, p1 * raw_up, w[k], lo[k]);
                    else w[k] = f2_to_h2(p0, p1);
                }
                tmem_st16(s_tm + 16 * j, w);
                if (raw) tmem_st16(s_tm + 32 + 16 * j, lo);
            }
            float s0, s1;
            f2_unpack(f2_add(sum[0], sum[1]), s0, s1);
            l = fmaf(s0 + s1, ex2(-dv), l);
            tmem_wait_st();
            tc_fence_before();
            warp_arrive(bar(P::bP + b));
            return true;
        };
#pragma unroll 1
        for (int n = 0; alive && n < n8; ++n) alive = block_step(std::false_type{}, n);
#pragma unroll 1
        for (int n = n8; alive && n < nb; ++n) alive = block_step(std::true_type{}, n);
        // every product is done, and the value warps have said what they left out: the rows
        kv_named_barrier(1, P::NT - P::kSoft0);
        if (alive) alive = lanes_wait(bar(P::bDrain), 0, limit);
        if (alive) {
            tc_fence_after();
            const bool live = tr < rows_here;
            const int head = h * a.G + r % a.G, tok = r / a.G;
            const bool one = PART == kKvWhole && last_seg == 0;
            const float inv = (one ? (l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l)) : 1.f) * pow2_of(lref);   // no key: zero; NaN stays
            int64_t pr = 0;
            if (live && !one) {
                pr = PART == kKvWhole ? kv_part_row(a, ui + blk - u.block, seg, blk == u.block ? tok : off, head)
                                      : kv_shared_part_row(a, PART == kKvShared ? seg : a.n_pre + seg - seg0, u.row + tok, head);
                a.part_ml[pr] = make_float2(m, l);
            }
            const bool fix = PART != kKvShared && live && seg == last_seg && bad_v[min(max(blk - blo, 0), 3)] != 0;
            // The warp's 32 rows pass through shared memory (the operands', which every product has read), 128 bytes of a row at a time
            // with the 16-byte chunks of row i at chunk ^ (i % 8), so that the stores to global memory are of whole rows.
            unsigned char *stage = sm + (warp - P::kSoft0 / 32) * (32 * 128);
            const int64_t dst_row = one ? (int64_t)(u.row + tok) * a.Hq + head : pr;
#pragma unroll 1
            for (int c = 0; c < D; c += 32) {
                uint32_t w[2][16];
#pragma unroll
                for (int j = 0; j < 2; ++j) tmem_ld16_nowait(o_tm + c + 16 * j, w[j]);
                float v[32];
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    tmem_wait_ld(w[j]);
#pragma unroll
                    for (int k = 0; k < 16; ++k) v[16 * j + k] = __uint_as_float(w[j][k]) * inv;
                }
                if (fix) {
                    for (int j = 0; j <= off; ++j) {
                        const int kp = blk * kKvBlock + j;
                        const bf *src = kp < pos0 ? static_cast<const bf *>(a.c.tail) + kv_tail_offset(u.slot, u.src, 1, h, a.Hkv, D) + (int64_t)j * D
                                                  : static_cast<const bf *>(a.v_new) + ((int64_t)(u.row + kp - pos0) * a.Hkv + h) * D;
#pragma unroll
                        for (int k = 0; k < 32; ++k) {
                            const float y = to_f(src[c + k]);
                            if (!(fabsf(y) <= 3.4e38f)) v[k] += y;
                        }
                    }
                }
                __syncwarp();
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    *reinterpret_cast<float4 *>(stage + lane * 128 + ((k ^ (lane & 7)) << 4)) =
                        make_float4(v[4 * k], v[4 * k + 1], v[4 * k + 2], v[4 * k + 3]);
                __syncwarp();
#pragma unroll 8
                for (int it = 0; it < 8; ++it) {   // 4 rows of 8 chunks a time
                    const int i = 4 * it + (lane >> 3), k = lane & 7;
                    const float4 x = *reinterpret_cast<const float4 *>(stage + i * 128 + ((k ^ (i & 7)) << 4));
                    const int64_t row = __shfl_sync(0xffffffffu, dst_row, i);
                    if (tr - lane + i >= rows_here) continue;
                    if (one) {
                        const __nv_bfloat162 y0 = __floats2bfloat162_rn(x.x, x.y), y1 = __floats2bfloat162_rn(x.z, x.w);
                        *reinterpret_cast<uint2 *>(static_cast<bf *>(a.out) + row * D + c + 4 * k) =
                            make_uint2(*reinterpret_cast<const uint32_t *>(&y0), *reinterpret_cast<const uint32_t *>(&y1));
                    } else {
                        *reinterpret_cast<float4 *>(a.part_o + row * D + c + 4 * k) = x;
                    }
                }
            }
        } else if (lane == 0) {
            atomicOr(a.err, kErrTimeout);
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 144;\n");
        kv_named_barrier(1, P::NT - P::kSoft0);   // the second tile's warps, without rows
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 0) tmem_dealloc(tmem, P::kTmemCols);
}

// n_units: units, or the most pieces of the shared blocks (kKvShared)
template <int D, int PART = kKvWhole>
cudaError_t launch_prompt(const KvAttn &a, int n_units, cudaStream_t st) {
    using P = PromptPlan<D>;
    cudaError_t e = cudaFuncSetAttribute(kv_attn_prompt_kernel<D, PART>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)P::kBytes);
    if (e != cudaSuccess) return e;
    if constexpr (PART == kKvShared) {
        e = gdn_launch_pdl(kv_attn_prompt_kernel<D, PART>, kv_shared_grid(a, n_units), P::NT, P::kBytes, st, a, 1, 1, n_units);
        return e != cudaSuccess ? e : cudaGetLastError();
    }
    // blocks of a span: enough rows to fill the tile where a block's tokens are too few (G = 1, 2), a power of two <= 4
    int span = 1;
    while (span < 4 && 2 * span * kKvBlock * a.G <= P::R) span *= 2;
    const int64_t rows_max = (int64_t)std::min(span * kKvBlock, a.max_new) * a.G;   // a span of several blocks is one tile
    const int row_tiles = (int)((rows_max + P::R - 1) / P::R);
    const dim3 grid((unsigned)((int64_t)n_units * row_tiles), (unsigned)a.Hkv, (unsigned)a.n_seg);
    e = gdn_launch_pdl(kv_attn_prompt_kernel<D, PART>, grid, P::NT, P::kBytes, st, a, row_tiles, span, n_units);
    return e != cudaSuccess ? e : cudaGetLastError();
}

template <int PART>
cudaError_t launch_prompt_part(const KvAttn &a, int d, int n, cudaStream_t st) {
    if (d == 64) return launch_prompt<64, PART>(a, n, st);
    if (d == 128) return launch_prompt<128, PART>(a, n, st);
    return launch_prompt<256, PART>(a, n, st);
}

}  // namespace gdn

// Attention of requests that share their first blocks, on the 5th-generation tensor core (bf16 inputs): the shared blocks for
// all rows of a group, and each request's own keys, by one set of persistent CTAs.
//
// The mathematics, the operands' formats and the steps of a block of 64 keys are those of kv_attn_prompt.cuh. What differs is
// what a CTA works on: a list of pieces, a piece being a row tile of one kv head over a run of blocks,
//   shared   R rows (token, query head) of a group, which stand side by side in the packed inputs whatever requests they are
//            of, over blocks [c0, c0 + L) of the group's shared ones: no row has a mask there;
//   own      R rows of a request's blocks (a span of kv_attn_prompt.cuh) over blocks past the shared ones, its own among them.
// Piece i goes to CTA i mod the CTAs, the shared ones (all of one cost) first. Every piece leaves (O, m, l) of its rows.
//
// The roles (two scheduling warps beside those of kv_attn_prompt.cuh) walk the list each at its own pace: keys and values of the
// next piece are converted while the softmax warps end the last one, its queries once the last scores are there. So a
// change of pieces costs the softmax warps' epilogue and one block's latency, where a CTA of its own took about 12 blocks'
// time. A piece's description, pages and scales stand in one of two places in shared memory, which all roles hand back.
#pragma once

#include "kv_attn_prompt.cuh"

namespace gdn {

struct __align__(16) KvPiece {
    int nb, n8;              // blocks of the pass, the first n8 of them from 8 bits; nb 0: the list's end
    int c0, blo;             // first block; block of the first raw one
    int h, slot, src;        // kv head; slot whose table is read, its tail buffer
    int row, r0, rows;       // packed row of the span's first token; first row (token x G) and number of rows of the tile
    int pos0, n_tok;         // position of that token, tokens of the span
    int seg, shared;         // segment of the partial results; whether every row sees every block
    int pad[2];
};
static_assert(sizeof(KvPiece) == 64, "piece record");

constexpr int kSharedMaxBlocks = kKvPieceBlocks;
constexpr int kSharedPieceCost = 4;     // a piece's own time, in blocks

template <int D>
struct SharedPlan : PromptPlan<D> {
    using B = PromptPlan<D>;
    static constexpr int kInfoLen = kSharedMaxBlocks + 4;
    static constexpr uint32_t kQ = 0, kK = B::kQT ? 0 : B::NQ * B::kTile, kV = kK + B::NS * B::kBlk, kInfo = kV + B::NS * B::kBlk;
    static constexpr uint32_t kPiece = kInfo + 2 * kInfoLen * 16, kRow = kPiece + 2 * sizeof(KvPiece);   // float [2][R]
    static constexpr uint32_t kRawK = kRow + 2 * B::R * 4, kBad = kRawK + 2 * 4 * 64 * 4;
    static constexpr uint32_t kTop = kBad + 2 * 16;          // kQT: float [4][128], a row's largest query element by quarter
    static constexpr uint32_t kBar = kTop + (B::kQT ? 4 * 128 * 4 : 0);
    static constexpr int NS = B::NS, NQ = B::NQ, CW = B::CW;
    // barriers: slots full and free, scores and weights by (tile, buffer), a tile's product before a piece's last, a tile's
    // products of a piece; per place of a piece: described, handed back, queries there, raw keys and values there; the
    // queries' largest elements; the end
    static constexpr int bKFull = 0, bKFree = NS, bVFull = 2 * NS, bVFree = 3 * NS, bS = 4 * NS, bP = bS + 2 * NQ, bPV = bP + 2 * NQ,
                         bDrain = bPV + NQ, bDesc = bDrain + NQ, bBack = bDesc + 2, bQ = bBack + 2, bRawK = bQ + 2,
                         bRawV = bRawK + 2, bTop = bRawV + 2, bEnd = bTop + 1, kNBar = bEnd + NQ;
    static constexpr uint32_t kSlot = kBar + (kNBar + 1) / 2 * 16;
    static constexpr uint32_t kBytes = kSlot + 16;
    static_assert(kBytes <= 227 * 1024, "shared memory");
};

// Blocks of a shared piece: those that make the fullest use of n_ctas CTAs; a lane tries a number of segments of the longest
// group. The same in every CTA and for the join, which reads it from *a.cut. *n_pieces: what it makes.
template <int R>
__device__ int kv_shared_cut(const KvAttn &a, int n_ctas, int &n_pieces) {
    const int lane = threadIdx.x & 31;
    int longest = 0, tiles = 0, blocks = 0;   // of the lane's last group
    long long work = 0;
    for (int g = lane; g < a.n_groups; g += 32) {
        const int4 r = a.groups[g];
        tiles = r.y > 0 ? (int)(((int64_t)r.y * a.G + R - 1) / R) : 0;
        blocks = max(r.w, 0);
        longest = max(longest, blocks);
        work += (long long)tiles * blocks;
    }
    longest = __reduce_max_sync(0xffffffffu, longest);
    n_pieces = 0;
    if (longest == 0) return 1;
    const int least = min((longest + a.n_pre - 1) / a.n_pre, kSharedMaxBlocks);
    if (a.n_groups > 32) {   // many groups: about four pieces a CTA
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) work += __shfl_xor_sync(0xffffffffu, work, o);
        const int cut = (int)min(max(work * a.Hkv / (4LL * n_ctas), (long long)least), (long long)kSharedMaxBlocks);
        long long n = 0;
        for (int g = lane; g < a.n_groups; g += 32) {
            const int4 r = a.groups[g];
            if (r.w > 0 && r.y > 0) n += ((int64_t)r.y * a.G + R - 1) / R * ((r.w + cut - 1) / cut);
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) n += __shfl_xor_sync(0xffffffffu, n, o);
        n_pieces = (int)min(n * a.Hkv, (long long)INT32_MAX);
        return cut;
    }
    // a segment more costs every row a partial result written and read again: in blocks of about 1 us
    const float part = (float)a.part_rows * (8.f * a.head_dim) / 4e6f;
    float best = INFINITY;
    int best_cut = kSharedMaxBlocks, best_n = 0;
#pragma unroll 1
    for (int round = 0; round < 2; ++round) {
        const unsigned s = round == 0 ? lane + 1 : 36 + 4 * lane;
        const unsigned c = (unsigned)min(max((int)((longest + s - 1) / s), least), kSharedMaxBlocks);
        long long n = 0;
        for (int g = 0; g < a.n_groups; ++g)
            n += (long long)__shfl_sync(0xffffffffu, tiles, g) * (((unsigned)__shfl_sync(0xffffffffu, blocks, g) + c - 1) / c);
        n *= a.Hkv;
        const float t = (float)((n + n_ctas - 1) / n_ctas) * (float)(c + kSharedPieceCost) + part * (float)((longest + c - 1) / c);
        if (t < best) {
            best = t;
            best_cut = (int)c;
            best_n = (int)min(n, (long long)INT32_MAX);
        }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {   // of equal ones the longer
        const float t = __shfl_xor_sync(0xffffffffu, best, o);
        const int c = __shfl_xor_sync(0xffffffffu, best_cut, o), n = __shfl_xor_sync(0xffffffffu, best_n, o);
        if (t < best || (t == best && c > best_cut)) {
            best = t;
            best_cut = c;
            best_n = n;
        }
    }
    n_pieces = best_n;
    return best_cut;
}

// 32 bytes of a partial result
__device__ __forceinline__ void st_global8(float *p, const float *v) {
    asm volatile("st.global.v8.f32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};\n" ::"l"(p), "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]),
                 "f"(v[5]), "f"(v[6]), "f"(v[7])
                 : "memory");
}

template <int D>
__global__ void __launch_bounds__(SharedPlan<D>::NT, 1) kv_attn_shared_kernel(const KvAttn a, int row_tiles, int span, int n_units) {
    using P = SharedPlan<D>;
    using bf = __nv_bfloat16;
    constexpr int NS = P::NS, NQ = P::NQ, R = P::R;
    extern __shared__ __align__(1024) unsigned char sm[];
    uint64_t *bar64 = reinterpret_cast<uint64_t *>(sm + P::kBar);
    const uint32_t bar0 = smem_addr(bar64);
    auto bar = [&](int i) { return bar0 + 8 * i; };
    uint32_t *tslot = reinterpret_cast<uint32_t *>(sm + P::kSlot);
    uint32_t *bad_all = reinterpret_cast<uint32_t *>(sm + P::kBad);
    BlockInfo *info_all = reinterpret_cast<BlockInfo *>(sm + P::kInfo);
    KvPiece *pieces = reinterpret_cast<KvPiece *>(sm + P::kPiece);
    float *row_all = reinterpret_cast<float *>(sm + P::kRow);
    float *raw_all = reinterpret_cast<float *>(sm + P::kRawK);
    const int t = threadIdx.x, warp = t >> 5, lane = t & 31;
    if (t == 0) {
        for (int i = 0; i < NS; ++i) {
            mbar_init(&bar64[P::bKFull + i], P::CW);
            mbar_init(&bar64[P::bVFull + i], P::CW);
            mbar_init(&bar64[P::bKFree + i], NQ);
            mbar_init(&bar64[P::bVFree + i], NQ);
        }
        for (int i = 0; i < 2 * NQ; ++i) {
            mbar_init(&bar64[P::bS + i], 1);
            mbar_init(&bar64[P::bP + i], 4);
        }
        for (int i = 0; i < NQ; ++i) {
            mbar_init(&bar64[P::bPV + i], 1);
            mbar_init(&bar64[P::bDrain + i], 1);
            mbar_init(&bar64[P::bEnd + i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&bar64[P::bDesc + i], 2);
            mbar_init(&bar64[P::bBack + i], 2 * P::CW + 5 * NQ);
            mbar_init(&bar64[P::bQ + i], 2 * P::CW);
            mbar_init(&bar64[P::bRawK + i], P::CW);
            mbar_init(&bar64[P::bRawV + i], P::CW);
        }
        mbar_init(&bar64[P::bTop], 2 * P::CW);
        mbar_init_fence();
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
    grid_dep_wait();
    grid_dep_launch();
    // a role's next piece: place i & 1, its uses counted by i >> 1
    auto next_piece = [&](int i) { return warp_wait(bar(P::bDesc + (i & 1)), (i >> 1) & 1, limit); };
    auto hand_back = [&](int i) { warp_arrive(bar(P::bBack + (i & 1))); };

    if (t < P::kSoft0) asm volatile("setmaxnreg.dec.sync.aligned.u32 64;\n");
    if (warp == 2 || warp == 3) {
        // ---- the scheduling warps: both find the same pieces, and share the blocks' pages and scales ----
        int i = 0, n_pieces;
        const int cut = kv_shared_cut<R>(a, gridDim.x, n_pieces);
        if (blockIdx.x == 0 && t == 64) *a.cut = cut;
        auto publish = [&](const KvPiece &x) {
            const int at = i & 1;
            if (i >= 2 && !lanes_wait(bar(P::bBack + at), ((i >> 1) - 1) & 1, limit)) return false;
            BlockInfo *info = info_all + at * P::kInfoLen;
            if (t == 64) pieces[at] = x;
            if (warp == 3 && lane < 4) bad_all[4 * at + lane] = 0;
            const int32_t *table = a.c.table + (int64_t)x.slot * a.c.max_blocks;
            for (int k = t - 64; k < x.nb; k += 64) {
                BlockInfo y = {0, a.scale_log2, 0.f};
                if (k < x.n8) {
                    y.page = table[x.c0 + k];
                    const bool in = (unsigned)y.page < (unsigned)a.c.n_pages;
                    if (!in) {
                        y.page = 0;                        // in bounds; the result is reported as invalid
                        atomicOr(a.err, kErrKvBounds);
                    }
                    const int64_t ph = (int64_t)y.page * a.Hkv + x.h;
                    const float ks = a.c.k_scale[ph], vs = a.c.v_scale[ph];
                    y.c = in ? a.scale_log2 * ks : 0.f;
                    y.lvs = in ? kv_log2_scale(vs) : INFINITY;
                }
                info[k] = y;
            }
            warp_arrive(bar(P::bDesc + at));
            ++i;
            return true;
        };
        int p = blockIdx.x;
#pragma unroll 1
        for (; alive && p < n_pieces; p += gridDim.x) {
            // the group that piece p is of: a warp looks at 32 groups at a time
            int x = p;
            int4 rec = make_int4(0, 0, 0, 0);
            for (int g0 = 0; g0 < a.n_groups; g0 += 32) {
                int4 r = make_int4(0, 0, 0, 0);
                if (g0 + lane < a.n_groups) r = a.groups[g0 + lane];
                const int here = r.w > 0 && r.y > 0 ? (int)(((int64_t)r.y * a.G + R - 1) / R) * a.Hkv * ((r.w + cut - 1) / cut) : 0;
                int upto = here;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const int y = __shfl_up_sync(0xffffffffu, upto, o);
                    if (lane >= o) upto += y;
                }
                const unsigned hit = __ballot_sync(0xffffffffu, upto > x);
                if (hit) {
                    const int w = __ffs(hit) - 1;
                    x -= __shfl_sync(0xffffffffu, upto - here, w);
                    rec.x = __shfl_sync(0xffffffffu, r.x, w);
                    rec.y = __shfl_sync(0xffffffffu, r.y, w);
                    rec.z = __shfl_sync(0xffffffffu, r.z, w);
                    rec.w = __shfl_sync(0xffffffffu, r.w, w);
                    break;
                }
                x -= __shfl_sync(0xffffffffu, upto, 31);
            }
            if (!kv_group_ok(a, rec)) {
                if (lane == 0) atomicOr(a.err, kErrKvBounds);
                continue;
            }
            const int tiles = (int)(((int64_t)rec.y * a.G + R - 1) / R), rest = x / tiles;   // row tiles of the same blocks together
            KvPiece y = {};
            y.h = rest % a.Hkv;
            y.seg = rest / a.Hkv;
            if (y.seg >= a.n_pre) continue;   // past max_len: of units that are left out
            y.c0 = y.seg * cut;
            y.nb = y.n8 = min(cut, rec.w - y.c0);
            y.blo = rec.w;
            y.slot = rec.z;
            y.row = rec.x;
            y.r0 = (x % tiles) * R;
            y.rows = min(R, rec.y * a.G - y.r0);
            y.n_tok = rec.y;
            y.shared = 1;
            if (!publish(y)) alive = false;
        }
        // own keys: candidates (segment, unit, row tile, kv head), 32 looked at together
        const int units = n_units > 0 ? min(n_units, a.counts[0]) : 0;
        const int64_t per_seg = (int64_t)units * row_tiles * a.Hkv, all = per_seg * a.n_seg;
#pragma unroll 1
        for (int64_t j0 = p - n_pieces; alive && j0 < all; j0 += 32LL * gridDim.x) {
            const int64_t j = j0 + (int64_t)lane * gridDim.x;
            KvPiece y = {};
            if (j < all) {
                const int seg = (int)(j / per_seg);
                int rest = (int)(j - seg * per_seg);
                y.h = rest % a.Hkv;
                rest /= a.Hkv;
                const int rt = rest % row_tiles, ui = rest / row_tiles;
                const KvUnit u = kv_load_unit(a.units, ui);
                const int start = a.starts[ui];
                bool ok = kv_suffix_unit_ok(a, u, start), first = true;
                // the span's first unit works for all of it (the first of a run of them, where one between is left out)
                if (ok && ui > 0 && u.block % span != 0) {
                    const KvUnit w = kv_load_unit(a.units, ui - 1);
                    first = !(w.slot == u.slot && w.block == u.block - 1 && kv_suffix_unit_ok(a, w, start));
                }
                int n_tok = u.count;
                for (int k = 1; ok && k < span && ui + k < units && (u.block + k) % span != 0; ++k) {
                    const KvUnit w = kv_load_unit(a.units, ui + k);
                    if (w.slot != u.slot || w.block != u.block + k) break;
                    if (!kv_suffix_unit_ok(a, w, start)) break;   // reported for itself
                    ok = w.first == 0 && w.row == u.row + n_tok;
                    n_tok += w.count;
                }
                if (!ok) atomicOr(a.err, kErrKvBounds);
                const int s = start / a.seg_blocks + seg, last = u.block / a.seg_blocks, n_row = n_tok * a.G;
                y.r0 = rt * R;
                if (ok && first && s <= last && y.r0 < n_row) {
                    y.rows = min(R, n_row - y.r0);
                    y.pos0 = u.block * kKvBlock + u.first;
                    y.blo = (y.pos0 + y.r0 / a.G) / kKvBlock;
                    const int bhi = (y.pos0 + (y.r0 + y.rows - 1) / a.G) / kKvBlock;
                    y.c0 = max(s * a.seg_blocks, start);
                    y.n8 = min(bhi, (s + 1) * a.seg_blocks) - y.c0;
                    y.nb = y.n8 + (s == last ? bhi - y.blo + 1 : 0);
                    y.slot = u.slot;
                    y.src = u.src;
                    y.row = u.row;
                    y.n_tok = n_tok;
                    y.seg = a.n_pre + seg;
                }
            }
            unsigned live = __ballot_sync(0xffffffffu, y.nb > 0);
            while (alive && live) {
                const int w = __ffs(live) - 1;
                live &= live - 1;
                KvPiece z;
                const int *from = reinterpret_cast<const int *>(&y);
                int *to = reinterpret_cast<int *>(&z);
#pragma unroll
                for (int k = 0; k < 14; ++k) to[k] = __shfl_sync(0xffffffffu, from[k], w);
                z.pad[0] = z.pad[1] = 0;
                if (!publish(z)) alive = false;
            }
        }
        if (alive) alive = publish(KvPiece{});
        if (!alive && lane == 0) atomicOr(a.err, kErrTimeout);
    } else if (warp < 2) {
        // ---- the issuing warps, one per tile ----
        const int tile = __shfl_sync(0xffffffffu, warp, 0);   // the same in every lane, and the compiler sees it
        if (tile < NQ) {
            constexpr uint32_t idS = umma_idesc_f16(128, 64, 0, 0), idO8 = umma_idesc_f16(128, D, 0, 1),
                               idOraw = umma_idesc_bf16(128, D, 0, 1);
            const bool elected = elect_one();
            const uint64_t dq = umma_smem_desc(sm + P::kQ + tile * P::kTile, 128, D * 16),
                           dk0 = umma_smem_desc(sm + P::kK, P::kCore, P::kGroup), dv0 = umma_smem_desc(sm + P::kV, P::kGroup, P::kCore);
            const uint32_t s0_tm = tmem + 128 * tile, o_tm = tmem + P::kO + tile * D;
            int gk = 0, gt = 0;   // blocks of the pieces before: all, and this tile's
#pragma unroll 1
            for (int i = 0; alive; ++i) {
                if (!next_piece(i)) {
                    alive = false;
                    break;
                }
                const int nb = pieces[i & 1].nb, n8 = pieces[i & 1].n8, rows = pieces[i & 1].rows;
                if (nb == 0) break;
                if (rows <= 128 * tile) {   // a piece of one tile: the slots go round all the same
#pragma unroll 1
                    for (int n = 0; alive && n < nb; ++n) {
                        const int slot = (gk + n) % NS, ph = (gk + n) / NS & 1;
                        alive = warp_wait(bar(P::bKFull + slot), ph, limit);
                        if (!alive) break;
                        warp_arrive(bar(P::bKFree + slot));
                        alive = warp_wait(bar(P::bVFull + slot), ph, limit);
                        if (!alive) break;
                        warp_arrive(bar(P::bVFree + slot));
                    }
                } else {
                    auto issue_s = [&](int n) {
                        const int slot = (gk + n) % NS, b = (gt + n) & 1;
                        const uint64_t dk = dk0 + (slot * P::kBlk >> 4);
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
                    alive = lanes_wait(bar(P::bQ + (i & 1)), (i >> 1) & 1, limit);
                    tc_fence_after();
                    for (int n = 0; alive && n < min(nb, 2); ++n) {
                        alive = __all_sync(0xffffffffu, bar_wait(bar(P::bKFull + (gk + n) % NS), (gk + n) / NS & 1, limit));
                        tc_fence_after();
                        if (alive) issue_s(n);
                    }
#pragma unroll 1
                    for (int n = 0; alive && n < nb; ++n) {
                        const int slot = (gk + n) % NS, b = (gt + n) & 1;
                        const bool more = n + 2 < nb;
                        const int nk = gk + (more ? n + 2 : n);   // the keys of the product that follows (n: there already)
                        if (more)
                            alive = __all_sync(0xffffffffu, bar_wait3(bar(P::bVFull + slot), (gk + n) / NS & 1, bar(P::bKFull + nk % NS),
                                                                      nk / NS & 1, bar(P::bP + 2 * tile + b), (gt + n) >> 1 & 1, limit));
                        else   // the keys' slot may have gone to the next piece
                            alive = __all_sync(0xffffffffu, bar_wait(bar(P::bVFull + slot), (gk + n) / NS & 1, limit) &&
                                                                bar_wait(bar(P::bP + 2 * tile + b), (gt + n) >> 1 & 1, limit));
                        if (!alive) break;
                        tc_fence_after();
                        const uint64_t dv = dv0 + (slot * P::kBlk >> 4);
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
                            if (n == max(nb - 2, 0)) bar_commit(bar(P::bPV + tile));
                        }
                    }
                    if (elected && alive) bar_commit(bar(P::bDrain + tile));
                    gt += nb;
                }
                gk += nb;
                if (alive) hand_back(i);
            }
            if (elected) {
                if (!alive) atomicOr(a.err, kErrTimeout);
                bar_commit(bar(P::bEnd + tile));   // nothing of this warp's is under way when TMEM goes
                if (!bar_wait(bar(P::bEnd + tile), 0, limit)) atomicOr(a.err, kErrTimeout);
            }
            __syncwarp();
        }
    } else if (t >= P::kKeys0) {
        // ---- key and value warps: a piece's queries, then its keys or values, the loads one block ahead ----
        asm volatile("setmaxnreg.dec.sync.aligned.u32 64;\n");
        const bool is_v = t >= P::kVals0;
        const int cw = warp % P::CW, kr = lane >> 2, ch = lane & 3;   // warp of the role; key of 8 and 16-byte chunk of 64
        const bf *tail = static_cast<const bf *>(a.c.tail);
        const int64_t stride = (int64_t)a.Hkv * (kKvBlock * D);
        const uint32_t full = bar(is_v ? P::bVFull : P::bKFull), free = bar(is_v ? P::bVFree : P::bKFree);
        unsigned char *slots = sm + (is_v ? P::kV : P::kK) + kr * 16 + ch * (2 * P::kCore);
        uint4 w[P::kLoads];   // load i: 8 keys x 64 columns, key group (cw + CW i) / kVec, column group (cw + CW i) % kVec
        int gk = 0;           // blocks of the pieces before
#pragma unroll 1
        for (int i = 0; alive; ++i) {
            if (!next_piece(i)) {
                alive = false;
                break;
            }
            const int at = i & 1;
            const KvPiece &x = pieces[at];
            const int nb = x.nb, n8 = x.n8, h = x.h;
            if (nb == 0) break;
            const BlockInfo *info = info_all + at * P::kInfoLen;
            const int8_t *pool = (is_v ? a.c.v : a.c.k) + (int64_t)h * (kKvBlock * D) + kr * D + ch * 16;
            auto load = [&](int n) {   // a raw block: page 0, not used
                const int8_t *src = pool + info[min(n, nb - 1)].page * stride;
#pragma unroll
                for (int k = 0; k < P::kLoads; ++k) {
                    const int j = cw + P::CW * k;
                    w[k] = __ldg(reinterpret_cast<const uint4 *>(src + j / P::kVec * (8 * D) + j % P::kVec * 64));
                }
            };
            auto store = [&](unsigned char *dst) {
#pragma unroll
                for (int k = 0; k < P::kLoads; ++k) {
                    const int j = cw + P::CW * k;
                    const uint2 x0 = i8_to_f16x4(w[k].x), x1 = i8_to_f16x4(w[k].y), x2 = i8_to_f16x4(w[k].z), x3 = i8_to_f16x4(w[k].w);
                    unsigned char *o = dst + j / P::kVec * P::kGroup + j % P::kVec * (8 * P::kCore);
                    *reinterpret_cast<uint4 *>(o) = make_uint4(x0.x, x0.y, x1.x, x1.y);
                    *reinterpret_cast<uint4 *>(o + P::kCore) = make_uint4(x2.x, x2.y, x3.x, x3.y);
                }
            };
            // a raw block: the tail's rows, then the new ones, zero past the last
            auto store_raw = [&](int block, unsigned char *dst) {
                float *raw_k = raw_all + at * 256;
#pragma unroll 1
                for (int kg = cw; kg < 8; kg += P::CW) {
                    const int off = kg * 8 + kr, pos = block * kKvBlock + off;
                    const bf *src = nullptr;
                    if (pos < x.pos0) src = tail + kv_tail_offset(x.slot, x.src, is_v, h, a.Hkv, D) + (int64_t)off * D;
                    else if (pos < x.pos0 + x.n_tok)
                        src = static_cast<const bf *>(is_v ? a.v_new : a.k_new) + ((int64_t)(x.row + pos - x.pos0) * a.Hkv + h) * D;
                    float top = 0.f, up = 1.f;
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
                                    // a value that is not finite would reach rows that do not see it (0 * inf): left out
                                    // here, and added by the rows that do at the end
                                    if (drop_not_finite(y[k])) atomicOr(&bad_all[4 * at + block - x.blo], 1u);
                                } else {
                                    float f[8];
                                    b8_to_f(y[k], f);
#pragma unroll
                                    for (int e = 0; e < 8; ++e) {
                                        top = fmaxf(top, fabsf(f[e]));
                                        f[e] *= up;
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
                            if (ch == 0) raw_k[(block - x.blo) * 64 + off] = back;
                        }
                    }
                }
            };
            load(0);
            // ---- the queries, once the scores of the piece before are there (their place is one) ----
            auto queries_free = [&] {
                return i == 0 || lanes_wait(bar(P::bKFree + (gk - 1) % NS), (gk - 1) / NS & 1, limit);
            };
            const bf *q = static_cast<const bf *>(a.q);
            float *row_q = row_all + at * R;
            const int rows = x.rows, r0 = x.r0, row = x.row;
            auto row_of = [&](int r) {   // of the tile
                const int rr = r0 + r, tok = rr / a.G;
                return q + ((int64_t)(row + tok) * a.Hq + h * a.G + (rr - tok * a.G)) * D;
            };
            if constexpr (P::kQT) {
                // a row by a lane, in TMEM; a quarter of its columns by a group of four warps, its largest element by way of
                // shared memory
                const int quarter = (warp - P::kKeys0 / 32) >> 2, r = 32 * (warp & 3) + lane;
                float *tops = reinterpret_cast<float *>(sm + P::kTop);
                uint4 y[D / 32];
#pragma unroll
                for (int k = 0; k < D / 32; ++k) y[k] = make_uint4(0, 0, 0, 0);
                if (r < rows) {
                    const uint4 *src = reinterpret_cast<const uint4 *>(row_of(r)) + D / 32 * quarter;
#pragma unroll
                    for (int k = 0; k < D / 32; ++k) y[k] = __ldg(src + k);
                }
                float f[8], top = 0.f, back;
#pragma unroll
                for (int k = 0; k < D / 32; ++k) {
                    b8_to_f(y[k], f);
#pragma unroll
                    for (int e = 0; e < 8; ++e) top = fmaxf(top, fabsf(f[e]));
                }
                if (!queries_free()) {   // (and every warp has read the last piece's largest elements)
                    alive = false;
                    break;
                }
                tc_fence_after();
                tops[128 * quarter + r] = top;
                warp_arrive(bar(P::bTop));
                if (!lanes_wait(bar(P::bTop), i & 1, limit)) {
                    alive = false;
                    break;
                }
#pragma unroll
                for (int k = 0; k < 4; ++k) top = fmaxf(top, tops[128 * k + r]);
                const float up = pow2_to_2_15(top, back);
                if (quarter == 0) row_q[r] = back;
#pragma unroll
                for (int j = 0; j < D / 128; ++j) {
                    uint32_t z[16];
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        b8_to_f(y[4 * j + k], f);
#pragma unroll
                        for (int e = 0; e < 8; ++e) f[e] *= up;
                        const uint4 v = f8_to_h8(f);
                        z[4 * k] = v.x; z[4 * k + 1] = v.y; z[4 * k + 2] = v.z; z[4 * k + 3] = v.w;
                    }
                    tmem_st16(tmem + ((uint32_t)(32 * (warp & 3)) << 16) + 128 + D / 8 * quarter + 16 * j, z);
                }
                tmem_wait_st();
                tc_fence_before();
            } else {
                // 8 rows a warp at a time, 4 lanes a row, each every fourth piece of 8 columns (as kv_attn_prompt.cuh)
                constexpr int NP = D / 32;
                const int c = lane & 3, qw = warp - P::kKeys0 / 32, tile_rows = rows > 128 ? 256 : 128;
                bool waited = false;
#pragma unroll 1
                for (int rb = qw * 8; rb < tile_rows; rb += 16 * P::CW * 2) {
                    uint4 y[2][NP];
#pragma unroll
                    for (int g = 0; g < 2; ++g) {
                        const int r = rb + 16 * P::CW * g + (lane >> 2);
#pragma unroll
                        for (int k = 0; k < NP; ++k) y[g][k] = make_uint4(0, 0, 0, 0);
                        if (r < rows) {
                            const uint4 *src = reinterpret_cast<const uint4 *>(row_of(r)) + c;
#pragma unroll
                            for (int k = 0; k < NP; ++k) y[g][k] = __ldg(src + 4 * k);
                        }
                    }
                    if (!waited && !queries_free()) {
                        alive = false;
                        break;
                    }
                    waited = true;
#pragma unroll
                    for (int g = 0; g < 2; ++g) {
                        const int r = rb + 16 * P::CW * g + (lane >> 2);
                        if (rb + 16 * P::CW * g >= tile_rows) break;
                        float f[8], top = 0.f;
#pragma unroll
                        for (int k = 0; k < NP; ++k) {
                            b8_to_f(y[g][k], f);
#pragma unroll
                            for (int e = 0; e < 8; ++e) top = fmaxf(top, fabsf(f[e]));
                        }
#pragma unroll
                        for (int o = 2; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
                        float back;
                        const float up = pow2_to_2_15(top, back);
                        unsigned char *dst = sm + P::kQ + (r >> 7) * P::kTile + ((r & 127) >> 3) * (D * 16) + c * 128 + (r & 7) * 16;
#pragma unroll
                        for (int k = 0; k < NP; ++k) {
                            b8_to_f(y[g][k], f);
#pragma unroll
                            for (int e = 0; e < 8; ++e) f[e] *= up;
                            *reinterpret_cast<uint4 *>(dst + 512 * k) = f8_to_h8(f);
                        }
                        if (c == 0) row_q[r] = back;
                    }
                }
                if (!alive) break;
                fence_proxy_async();
            }
            warp_arrive(bar(P::bQ + at));
#pragma unroll 1
            for (int n = 0; n < nb; ++n) {
                const int slot = (gk + n) % NS, use = (gk + n) / NS;
                if (use > 0 && !warp_wait(free + 8 * slot, (use - 1) & 1, limit)) {
                    alive = false;
                    break;
                }
                unsigned char *dst = slots + slot * P::kBlk;
                if (n < n8) {
                    store(dst);
                    load(n + 1);
                } else {
                    store_raw(x.blo + n - n8, dst);
                }
                fence_proxy_async();
                if (n > 0 || i > 0 || is_v || a.skip_first_copy != 3) warp_arrive(full + 8 * slot);   // 3: the test hook
            }
            if (!alive) break;
            gk += nb;
            warp_arrive(bar((is_v ? P::bRawV : P::bRawK) + at));
            hand_back(i);
        }
        if (!alive && lane == 0) atomicOr(a.err, kErrTimeout);
    } else {
        // ---- softmax warps ----
        asm volatile("setmaxnreg.inc.sync.aligned.u32 144;\n");
        const int tr = t - P::kSoft0, tile = tr >> 7;   // tr = 128 tile + row
        const uint32_t lanes = (uint32_t)(32 * (warp & 3)) << 16;
        const uint32_t o_tm = tmem + lanes + P::kO + tile * D;
        int gt = 0, done = 0;   // blocks and pieces of this tile before
#pragma unroll 1
        for (int i = 0; alive; ++i) {
            if (!next_piece(i)) {
                alive = false;
                break;
            }
            const int at = i & 1;
            const KvPiece &pc = pieces[at];
            const int nb = pc.nb, n8 = pc.n8, rows = pc.rows;
            if (nb == 0) break;
            if (rows <= 128 * tile) {
                hand_back(i);
                continue;
            }
            if (!lanes_wait(bar(P::bQ + at), (i >> 1) & 1, limit)) {
                alive = false;
                break;
            }
            const BlockInfo *info = info_all + at * P::kInfoLen;
            const float rq = row_all[at * R + tr];
            // of an own piece: blocks of 8 bits that the row sees (a shared one: all), its offset in its own block
            const int pos = pc.pos0 + (pc.r0 + tr) / a.G, own = pos / kKvBlock - pc.blo, off = pos % kKvBlock;
            const int n_see = pc.shared ? INT32_MAX : pos / kKvBlock - pc.c0;
            float m = -INFINITY, l = 0.f, lref = 0.f;
            auto block_step = [&](auto is_raw, int n) {
                constexpr bool raw = decltype(is_raw)::value;
                const int b = 2 * tile + ((gt + n) & 1);
                const uint32_t s_tm = tmem + lanes + 64 * b;
                if (!warp_wait(bar(P::bS + b), (gt + n) >> 1 & 1, limit)) return false;
                tc_fence_after();
                const BlockInfo x = info[n];
                // keys of the block that the row sees: all or none of an 8-bit block, up to its own offset of its raw block
                const int see = raw ? (own == n - n8 ? off + 1 : 0) : (n < n_see ? kKvBlock : 0);
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
                    const float *kf = raw_all + at * 256 + (n - n8) * 64;
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
                    if (!lanes_wait(bar(last ? P::bPV + tile : P::bS + 2 * tile + ((gt + n + 1) & 1)), last ? done & 1 : (gt + n + 1) >> 1 & 1, limit))
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
                // the weights (8-bit blocks: times the value scale over the unit, which the sum takes out again); none of a
                // block that the row does not see
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
            if (alive && nb > n8) alive = lanes_wait(bar(P::bRawK + at), (i >> 1) & 1, limit);   // the raw keys' scalings
#pragma unroll 1
            for (int n = n8; alive && n < nb; ++n) alive = block_step(std::true_type{}, n);
            // every product is done, and the value warps have said what they left out: the rows
            if (alive && nb > n8) alive = lanes_wait(bar(P::bRawV + at), (i >> 1) & 1, limit);
            if (alive) alive = lanes_wait(bar(P::bDrain + tile), done & 1, limit);
            if (!alive) break;
            tc_fence_after();
            const bool live = tr < rows;
            const int rr = pc.r0 + tr, tok = rr / a.G, head = pc.h * a.G + rr % a.G;
            const float unit = pow2_of(lref);
            const bool fix = live && nb > n8 && bad_all[4 * at + min(max(own, 0), 3)] != 0;
            const int64_t pr = live ? kv_shared_part_row(a, pc.seg, pc.row + tok, head) : 0;
            if (live) a.part_ml[pr] = make_float2(m, l);
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
                    for (int k = 0; k < 16; ++k) v[16 * j + k] = __uint_as_float(w[j][k]) * unit;
                }
                if (fix) {
                    for (int j = 0; j <= off; ++j) {
                        const int kp = pos - off + j;
                        const bf *src = kp < pc.pos0 ? static_cast<const bf *>(a.c.tail) + kv_tail_offset(pc.slot, pc.src, 1, pc.h, a.Hkv, D) + (int64_t)j * D
                                                     : static_cast<const bf *>(a.v_new) + ((int64_t)(pc.row + kp - pc.pos0) * a.Hkv + pc.h) * D;
#pragma unroll
                        for (int k = 0; k < 32; ++k) {
                            const float y = to_f(src[c + k]);
                            if (!(fabsf(y) <= 3.4e38f)) v[k] += y;
                        }
                    }
                }
                if (live) {
#pragma unroll
                    for (int k = 0; k < 4; ++k) st_global8(a.part_o + pr * D + c + 8 * k, v + 8 * k);
                }
            }
            tc_fence_before();   // the reads of O, before the next piece's weights are announced
            gt += nb;
            ++done;
            hand_back(i);
        }
        if (!alive && lane == 0) atomicOr(a.err, kErrTimeout);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 0) tmem_dealloc(tmem, P::kTmemCols);
}

// n_units: units whose own keys are in the list, or 0. n_pieces: the most pieces there can be.
template <int D>
cudaError_t launch_shared(const KvAttn &a, int n_units, int64_t n_pieces, cudaStream_t st) {
    using P = SharedPlan<D>;
    cudaError_t e = cudaFuncSetAttribute(kv_attn_shared_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)P::kBytes);
    if (e != cudaSuccess) return e;
    int sms = 1;
    if ((e = gdn_sm_count(&sms)) != cudaSuccess) return e;
    int span = 1;   // as kv_attn_prompt.cuh
    while (span < 4 && 2 * span * kKvBlock * a.G <= P::R) span *= 2;
    const int64_t rows_max = (int64_t)std::min(span * kKvBlock, a.max_new) * a.G;
    const int row_tiles = (int)((rows_max + P::R - 1) / P::R);
    const dim3 grid((unsigned)std::min<int64_t>(n_pieces, sms));
    e = gdn_launch_pdl(kv_attn_shared_kernel<D>, grid, P::NT, P::kBytes, st, a, row_tiles, span, n_units);
    return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace gdn

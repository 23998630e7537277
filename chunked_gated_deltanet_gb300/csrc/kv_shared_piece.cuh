// The pieces that the shared blocks of a plan's groups are worked off in: a row tile of R rows (token, query head) of a group,
// which stand side by side in the packed inputs whatever requests they are of, a kv head, and a run of `cut` blocks.
#pragma once

#include "kv.cuh"

namespace gdn {

constexpr int kSharedSms = 152;        // pieces at a time, one an SM
constexpr int kSharedPieceCost = 12;   // a piece's own time, in blocks
constexpr int kSharedGroups = 32, kSharedManyCut = 128;   // groups whose cut is searched for; the cut of more groups

// Blocks of a piece: those that make the fullest use of the SMs with no more pieces than the launch has CTAs. A lane tries a
// number of segments of the longest group. The same in every CTA and for the join, which reads it from *a.cut. (One group: the
// host's choice, made the same way, kv_api.cu.)
template <int R>
__device__ int kv_shared_cut(const KvAttn &a, int tiles, int blocks) {   // of the lane's group
    const int lane = threadIdx.x & 31;
    const int longest = __reduce_max_sync(0xffffffffu, blocks);
    const int least = min(max((longest + a.n_pre - 1) / a.n_pre, 1), kKvMaxSegBlocks);
    if (a.n_groups > kSharedGroups) return max(least, kSharedManyCut);   // they fill the SMs by themselves
    // a segment more costs every row a partial result written and read again: in blocks of about 0.9 us
    const float part = (float)a.part_rows * (8.f * a.head_dim) / 3.6e6f;
    float best = INFINITY;
    int best_cut = kKvMaxSegBlocks;
    const unsigned c = (unsigned)min(max((longest + lane) / (lane + 1), least), kKvMaxSegBlocks);
    unsigned n = 0;
    for (int g = 0; g < a.n_groups; ++g)
        n += (unsigned)__shfl_sync(0xffffffffu, tiles, g) * (((unsigned)__shfl_sync(0xffffffffu, blocks, g) + c - 1) / c);
    n *= a.Hkv;
    if (n <= gridDim.x) {
        best = (float)((n + kSharedSms - 1) / kSharedSms) * (float)(c + kSharedPieceCost) + part * (float)((longest + c - 1) / c);
        best_cut = (int)c;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {   // of equal ones the longer
        const float t = __shfl_xor_sync(0xffffffffu, best, o);
        const int x = __shfl_xor_sync(0xffffffffu, best_cut, o);
        if (t < best || (t == best && x > best_cut)) {
            best = t;
            best_cut = x;
        }
    }
    return best_cut;
}

// This CTA's piece: its group's record, first row of the tile, kv head and segment of `cut` blocks; false where there is none.
// One group: the launch's grid is (row tiles, kv heads, segments). Several: the CTA's number counts the pieces off, the row
// tiles of the same blocks in a row, so that CTAs that run together read the same pages (as the grid of one group has it).
template <int R>
__device__ bool kv_shared_piece(const KvAttn &a, int &r0, int &h, int &seg, int &cut, int4 &rec) {
    const int lane = threadIdx.x & 31;
    if (a.n_groups == 1) {
        rec = kv_load_group(a, 0);
        cut = a.pre_blocks;
        r0 = (int)blockIdx.x * R;
        h = blockIdx.y;
        seg = blockIdx.z;
        return rec.w > 0 && rec.y > 0 && r0 < (int64_t)rec.y * a.G && (int64_t)seg * cut < min(rec.w, (a.max_len - 1) / kKvBlock);
    }
    int p = blockIdx.x;
    for (int g0 = 0; g0 < a.n_groups; g0 += 32) {
        int4 r = make_int4(0, 0, 0, 0);
        if (g0 + lane < a.n_groups) r = kv_load_group(a, g0 + lane);
        const bool in = r.w > 0 && r.y > 0;
        const int most = (a.max_len - 1) / kKvBlock;   // blocks past max_len are of units that are left out
        const int tiles = in ? (int)(((int64_t)r.y * a.G + R - 1) / R) : 0, blocks = in ? min(r.w, most) : 0;
        if (g0 == 0) {
            int longest = blocks;   // more than 32 groups: the longest of all
            for (int g = 32 + lane; g < a.n_groups; g += 32) longest = max(longest, min(kv_load_group(a, g).w, most));
            cut = kv_shared_cut<R>(a, tiles, a.n_groups > 32 ? longest : blocks);
            if (blockIdx.x == 0 && threadIdx.x == 0) *a.cut = cut;
        }
        const int segs = (blocks + cut - 1) / cut;
        const int here = tiles * a.Hkv * segs;
        int upto = here;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, upto, o);
            if (lane >= o) upto += y;
        }
        const unsigned hit = __ballot_sync(0xffffffffu, upto > p);
        if (hit) {
            const int w = __ffs(hit) - 1;
            p -= __shfl_sync(0xffffffffu, upto - here, w);
            rec.x = __shfl_sync(0xffffffffu, r.x, w);
            rec.y = __shfl_sync(0xffffffffu, r.y, w);
            rec.z = __shfl_sync(0xffffffffu, r.z, w);
            rec.w = __shfl_sync(0xffffffffu, r.w, w);
            const int n = __shfl_sync(0xffffffffu, tiles, w), rest = p / n;
            // the same in every lane; said by a shuffle, as a quotient is not seen to be (loops over such a piece and the MMAs'
            // operands then went through vector registers: 8,000 x 16 rows over 37,760 keys 2,030 us instead of 1,740)
            r0 = __shfl_sync(0xffffffffu, (p - rest * n) * R, 0);
            h = __shfl_sync(0xffffffffu, rest % a.Hkv, 0);
            seg = __shfl_sync(0xffffffffu, rest / a.Hkv, 0);
            cut = __shfl_sync(0xffffffffu, cut, 0);
            return true;
        }
        p -= __shfl_sync(0xffffffffu, upto, 31);
    }
    return false;
}

// The launch's grid.
inline dim3 kv_shared_grid(const KvAttn &a, int n_pieces) {
    if (a.n_groups > 1) return dim3((unsigned)n_pieces);
    return dim3((unsigned)(n_pieces / (a.Hkv * a.n_pre)), (unsigned)a.Hkv, (unsigned)a.n_pre);
}

}  // namespace gdn

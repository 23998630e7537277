// Paged key/value cache held in 8 bits: structures shared by its kernels and the C ABI layer.
//
// The cache keeps keys and values in blocks of 64 tokens at absolute positions. A complete block lives in a page,
// int8 [Hkv][64][d] each for keys and values, with one fp32 scale per (page, head): scale = absmax / 127 over the
// block's 64 d elements, value = scale * q, q = x / scale rounded to nearest even. The open block at a session's end
// stays in the slot's tail as it came (in_dtype). So a block's 8-bit content is a function of its 64 tokens alone,
// however they were split into calls, and complete blocks never change: forks share their pages.
#pragma once

#include "common.cuh"

namespace gdn {

constexpr int kKvBlock = 64;
constexpr int kKvMaxRequests = 4096;

// One unit of a plan: the new tokens of one request inside one block (include/gdn.h lists the fields).
struct __align__(16) KvUnit {
    int32_t slot, block, page, first, count, row, src, dst;
};
static_assert(sizeof(KvUnit) == 32, "unit record");

// The cache's device buffers and sizes, as the kernels take them.
struct KvCache {
    int8_t *k, *v;                // [n_pages][Hkv][64][d]
    float *k_scale, *v_scale;     // [n_pages][Hkv]
    void *tail;                   // in_dtype [n_slots][2 buffers][k, v][Hkv][64][d]
    int32_t *state;               // [n_slots][2]: tokens held, tail buffer of the open block
    int32_t *table;               // [n_slots][max_blocks]: page of each complete block
    int32_t *free_pages, *n_free; // stack of free pages, its height
    int32_t *refs;                // [n_pages]: slots whose table names the page
    int32_t n_pages, n_slots, max_blocks;
};

constexpr unsigned kErrTimeout = 1u;  // device error word: a bounded wait ran out
constexpr unsigned kErrKvBounds = 2u; // a plan's unit lies outside the sizes given to the call

// A unit that every index computed from it stays inside the buffers for. n_rows: rows of the packed arrays.
__device__ __forceinline__ bool kv_unit_ok(const KvUnit &u, const KvCache &c, int64_t n_rows) {
    return u.slot >= 0 && u.slot < c.n_slots && u.first >= 0 && u.count >= 1 && u.first + u.count <= kKvBlock &&
           u.block >= 0 && u.row >= 0 && (int64_t)u.row + u.count <= n_rows && (unsigned)u.src < 2u &&
           u.block <= c.max_blocks && u.page < c.n_pages && (u.page >= 0 || (unsigned)u.dst < 2u);
}

__device__ __forceinline__ KvUnit kv_load_unit(const int32_t *units, int64_t i) {
    union { int4 v[2]; KvUnit u; } x;
    const int4 *p = reinterpret_cast<const int4 *>(units) + 2 * i;
    x.v[0] = p[0];
    x.v[1] = p[1];
    return x.u;
}

// First element of the tail rows of (slot, buffer, k or v, head): 64 rows of d.
__host__ __device__ __forceinline__ int64_t kv_tail_offset(int slot, int buf, int kv, int h, int Hkv, int d) {
    return ((((int64_t)slot * 2 + buf) * 2 + kv) * Hkv + h) * kKvBlock * d;
}

// Growing segments of the many-row bf16 form, in blocks: 32 below block 64, 64 below 128, 128 below 512, then 256. A segment
// costs its CTA about 12 blocks' time besides its own (queries in, outputs out) and the join a row of partial results, so
// long contexts want long ones, and short contexts short ones, to have CTAs for all SMs. Cut at absolute positions.
constexpr int kKvMaxSegBlocks = 256;
constexpr int kv_prompt_rows(int d) { return d == 256 ? 128 : 256; }   // rows of a CTA of that form
constexpr int kKvSimtRows = 64;                                        // and of its fp32 form
__host__ __device__ constexpr int kv_grown_seg(int block) {
    return block < 64 ? block / 32 : block < 128 ? 2 : block < 512 ? 2 + block / 128 : 4 + block / 256;
}
__host__ __device__ constexpr int kv_grown_start(int seg) { return seg < 3 ? 32 * seg : seg < 6 ? 128 * (seg - 2) : 256 * (seg - 4); }

// Attention launch. Rows of a unit for kv head h: r = t * G + g, token t of the unit and query head h * G + g.
struct KvAttn {
    const void *q, *k_new, *v_new;  // [n_rows][Hq][d], [n_rows][Hkv][d]
    void *out;                      // [n_rows][Hq][d]
    KvCache c;
    const int32_t *units, *counts;
    int64_t n_rows;
    int Hq, Hkv, G;
    float scale_log2;               // softmax scale * log2(e)
    float *part_o;                  // [segment][part_rows][d], unnormalised (kv_part_row)
    float2 *part_ml;                // [segment][part_rows]: running maximum (log2 domain), sum
    int64_t part_rows;              // units of the launch * tok_stride * Hq
    int unit0;                      // first unit of the launch (a call whose partials do not fit is several)
    int tok_stride;                 // most tokens of a unit: min(64, max_new)
    int seg_blocks, n_seg;          // segment s: blocks [s * seg_blocks, (s + 1) * seg_blocks), or by kv_grown_start with seg_blocks 0
    int max_new, max_len;           // the caller's bounds on a request's new tokens and on a slot's length after the plan
    long long wait_limit;           // polls before a bounded wait gives up
    int skip_first_copy;            // test hook: 3 = the prompt kernel never announces its first key tile
    unsigned int *err;
    // shared-prefix calls (KvPart): groups {first row, rows, slot, shared blocks}, and the shared blocks of each unit's group
    const int4 *groups;
    const int32_t *starts;
    int n_groups;
    int pre_blocks, n_pre;          // segments of the shared blocks, cut every pre_blocks (one group) or *cut; most of them
    int *cut;                       // several groups: the cut of the shared blocks, chosen on the GPU
    int head_dim, own_apart;
    int beside;                     // few rows: the launch before is the shared blocks' (KvBeside)
    int n_own;                      // few rows: CTAs [0, n_own) take units, the others row tiles of the groups
    int max_suffix;                 // the caller's bound on a request's tokens past its group's shared blocks
};

// What a launch of an attention kernel covers: a plan's units over all of their keys; the units over the keys past their
// group's shared blocks; the groups' rows over the shared blocks; the last two side by side (few rows). These leave partial
// results, by packed row.
enum KvPart { kKvWhole = 0, kKvSuffix = 1, kKvShared = 2, kKvFew = 3 };

// A launch over own keys runs beside the one over shared blocks before it, on the SMs that its last pieces leave: it reads
// nothing that one writes, and what came before that one is complete, as it lets the next launch start only after its own wait.
// So the wait stands at the end, in one CTA alone (the others make room for further ones): the join, which waits for this
// launch, thereby starts after both.
struct KvBeside {
    bool on;
    __device__ explicit KvBeside(bool beside) : on(beside) {
        if (!on) grid_dep_wait();
        grid_dep_launch();
    }
    __device__ ~KvBeside() {
        if (on && blockIdx.x == 0 && blockIdx.y == 0 && blockIdx.z == 0) grid_dep_wait();
    }
};

// Segment of a block, and a segment's first block.
__device__ __forceinline__ int kv_seg_of(const KvAttn &a, int block) { return a.seg_blocks ? block / a.seg_blocks : kv_grown_seg(block); }
__device__ __forceinline__ int kv_seg_start(const KvAttn &a, int seg) { return a.seg_blocks ? seg * a.seg_blocks : kv_grown_start(seg); }

// A unit inside the sizes that the call was given: what the attention and the join work on.
__device__ __forceinline__ bool kv_attn_unit_ok(const KvAttn &a, const KvUnit &u) {
    return kv_unit_ok(u, a.c, a.n_rows) && u.count <= a.max_new && (int64_t)u.block * kKvBlock + u.first + u.count <= a.max_len &&
           kv_seg_of(a, u.block) < a.n_seg;
}

// Shared-prefix calls. Segments of a unit's own keys, those of its blocks [start, block) and of its own block. Many rows: cut at
// absolute multiples of seg_blocks, the own block in the last one. Few rows: cut every seg_blocks from `start` on, so that each
// but the last complete one has a block for every warp (the kernel's loads a segment ahead count on that), and the own block a
// segment by itself.
__device__ __forceinline__ int kv_own_segs(const KvAttn &a, int block, int start) {
    if (!a.own_apart) return block / a.seg_blocks - start / a.seg_blocks + 1;
    return (block - start + a.seg_blocks - 1) / a.seg_blocks + 1;
}
// A unit's first block that is its own (its group's shared blocks lie before it); outside the sizes
// given with the call the unit is left out like any other.
__device__ __forceinline__ bool kv_suffix_unit_ok(const KvAttn &a, const KvUnit &u, int start) {
    return kv_unit_ok(u, a.c, a.n_rows) && u.count <= a.max_new && (int64_t)u.block * kKvBlock + u.first + u.count <= a.max_len &&
           start >= 0 && start <= u.block && (int64_t)(u.block - start) * kKvBlock + u.first + u.count <= a.max_suffix &&
           kv_own_segs(a, u.block, start) <= a.n_seg;
}
template <int PART>
__device__ __forceinline__ bool kv_part_unit_ok(const KvAttn &a, const KvUnit &u, int start) {
    if constexpr (PART != kKvWhole) return kv_suffix_unit_ok(a, u, start);
    else return kv_attn_unit_ok(a, u);
}
// Many rows: the segment that a unit's own keys start in, at `start`.
template <int PART>
__device__ __forceinline__ int kv_part_seg0(const KvAttn &a, int start) { return PART == kKvWhole ? 0 : start / a.seg_blocks; }
// Row of a shared-prefix call's partial results: (packed row, query head); the shared blocks' segments come first.
__device__ __forceinline__ int64_t kv_shared_part_row(const KvAttn &a, int seg, int64_t row, int head) {
    return seg * a.part_rows + row * a.Hq + head;
}

// A group's record, its rows no more than the call's (those past them are of units that are left out).
__device__ __forceinline__ int4 kv_load_group(const KvAttn &a, int g) {
    int4 r = a.groups[g];
    r.y = r.x < 0 ? 0 : (int)min((int64_t)r.y, max(a.n_rows - r.x, (int64_t)0));
    return r;
}
// Few rows: group of row tile x (of R rows), its record, and the tile's first row; -1 if there is none. The same in every lane.
template <int R>
__device__ __forceinline__ int kv_group_of_tile(const KvAttn &a, int x, int4 &rec) {
    const int lane = threadIdx.x & 31;
    for (int g0 = 0; g0 < a.n_groups; g0 += 32) {
        int4 r = make_int4(0, 0, 0, 0);
        if (g0 + lane < a.n_groups) r = kv_load_group(a, g0 + lane);
        const int tiles = r.w > 0 && r.y > 0 ? (int)(((int64_t)r.y * a.G + R - 1) / R) : 0;
        int upto = tiles;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, upto, o);
            if (lane >= o) upto += y;
        }
        const unsigned hit = __ballot_sync(0xffffffffu, upto > x);
        if (hit) {
            const int w = __ffs(hit) - 1;
            rec.x = __shfl_sync(0xffffffffu, r.x, w);
            rec.y = __shfl_sync(0xffffffffu, r.y, w);
            rec.z = __shfl_sync(0xffffffffu, r.z, w);
            rec.w = __shfl_sync(0xffffffffu, r.w, w);
            return (x - __shfl_sync(0xffffffffu, upto - tiles, w)) * R;
        }
        x -= __shfl_sync(0xffffffffu, upto, 31);
    }
    return -1;
}
__device__ __forceinline__ bool kv_group_ok(const KvAttn &a, const int4 &r) {
    return (unsigned)r.z < (unsigned)a.c.n_slots && r.w <= a.c.max_blocks;
}

// Row of the partial results: (unit, token of the unit, query head) of a segment.
__device__ __forceinline__ int64_t kv_part_row(const KvAttn &a, int unit, int seg, int tok, int head) {
    return seg * a.part_rows + ((int64_t)(unit - a.unit0) * a.tok_stride + tok) * a.Hq + head;
}

}  // namespace gdn

cudaError_t gdn_launch_kv_plan(const gdn::KvCache &c, const int32_t *slots, const int32_t *n_new, int n, int32_t *rows,
                               int32_t *units, int32_t *counts, int max_requests, int max_units, int32_t *state_out, int32_t *n_free_out,
                               cudaStream_t st);
cudaError_t gdn_launch_kv_append(const gdn::KvCache &c, const int32_t *units, const int32_t *counts, int unit_bound,
                                 const void *k, const void *v, int64_t n_rows, int Hkv, int d, int bf16, unsigned *err,
                                 cudaStream_t st);
cudaError_t gdn_launch_kv_fork(const gdn::KvCache &c, int src, int dst, int Hkv, int d, int elt, cudaStream_t st);
cudaError_t gdn_launch_kv_release(const gdn::KvCache &c, int slot, cudaStream_t st);
cudaError_t gdn_launch_kv_init(const gdn::KvCache &c, cudaStream_t st);
// Attention over unit_bound units from a.unit0. rows_max: the most rows (new tokens of one block x G) of a unit.
// fp32 inputs, few rows or many:
cudaError_t gdn_launch_kv_attn_simt(const gdn::KvAttn &a, int d, int unit_bound, int rows_max, int few, cudaStream_t st);
// bf16 inputs, rows_max <= 16:
cudaError_t gdn_launch_kv_attn_token(const gdn::KvAttn &a, int d, int unit_bound, int rows_max, cudaStream_t st);
// bf16 inputs, many rows:
cudaError_t gdn_launch_kv_attn_prompt(const gdn::KvAttn &a, int d, int unit_bound, cudaStream_t st);
// The parts of a shared-prefix call. Own keys: unit_bound units. Shared keys: at most n_pieces pieces. Few rows (bf16): own keys
// of up to rows_max rows a unit, and the shared keys of `tiles` row tiles at most (0: they are a launch of their own).
cudaError_t gdn_launch_kv_suffix(const gdn::KvAttn &a, int d, int bf16, int unit_bound, int rows_max, cudaStream_t st);
cudaError_t gdn_launch_kv_few(const gdn::KvAttn &a, int d, int unit_bound, int tiles, int rows_max, cudaStream_t st);
cudaError_t gdn_launch_kv_shared(const gdn::KvAttn &a, int d, int bf16, int n_pieces, cudaStream_t st);
cudaError_t gdn_launch_kv_shared_join(const gdn::KvAttn &a, int d, int bf16, int unit_bound, cudaStream_t st);
cudaError_t gdn_launch_kv_group(const gdn::KvCache &c, const int32_t *rows, const int32_t *units, const int32_t *counts,
                                int max_requests, int max_units, const int32_t *bounds, int n_groups, int max_groups,
                                int32_t *groups, int32_t *starts, unsigned *err, cudaStream_t st);
// Joins the segments' partial results of every row that has more than one.
cudaError_t gdn_launch_kv_join(const gdn::KvAttn &a, int d, int bf16, int unit_bound, int few, cudaStream_t st);

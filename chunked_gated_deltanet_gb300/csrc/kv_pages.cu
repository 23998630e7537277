// Slots of the paged cache forked or emptied in a batch, and the compaction of its page pool.
#include "kv_pages.cuh"

#include <algorithm>
#include <cooperative_groups.h>

namespace gdn {

namespace cg = cooperative_groups;

constexpr int kPageThreads = 1024, kPageCluster = 8;
constexpr int kFreedMark = INT32_MIN;   // a page's count between its last name's end and its way to the free stack

__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.aligned;\nbarrier.cluster.wait.aligned;\n" ::: "memory");
}

// Exclusive sum over the threads of a cluster in rank order; *total receives the sum of all. ws: 34 ints of shared memory,
// ws[32] this CTA's sum as the other CTAs read it.
__device__ int cluster_exclusive(int x, int *ws, int *total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int in = x;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, in, o);
        if (lane >= o) in += y;
    }
    __syncthreads();   // the last call's readers are done with ws
    if (lane == 31) ws[warp] = in;
    __syncthreads();
    if (warp == 0) {
        int w = ws[lane];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, w, o);
            if (lane >= o) w += y;
        }
        ws[lane] = w;
        if (lane == 31) ws[32] = w;
    }
    cluster_sync();
    const cg::cluster_group cl = cg::this_cluster();
    const int rank = (int)cl.block_rank(), n = (int)cl.num_blocks();
    const int v = lane < n ? *cl.map_shared_rank(&ws[32], lane) : 0;   // a lane a CTA
    const int sum = __reduce_add_sync(0xffffffffu, v), before = __reduce_add_sync(0xffffffffu, lane < rank ? v : 0);
    cluster_sync();   // every CTA has read the others' sums
    *total = sum;
    return before + (warp > 0 ? ws[warp - 1] : 0) + in - x;
}

// ---- forks and releases ----

struct __align__(16) ForkPair {
    int src, dst, now, before;   // slots; complete blocks that dst will name, and names
};

// Whether a batch's pairs are sound: slots in range, no slot twice among dst, no dst among src. Every CTA looks for itself.
__device__ bool fork_batch_ok(const int32_t *src, const int32_t *dst, int n, int n_slots, unsigned *bits) {
    const int t = threadIdx.x, words = (n_slots + 31) / 32;
    for (int i = t; i < words; i += kPageThreads) bits[i] = 0;
    __syncthreads();
    bool bad = false;
    for (int i = t; i < n; i += kPageThreads) {
        const int d = dst[i];
        if ((unsigned)d >= (unsigned)n_slots) bad = true;
        else if (atomicOr(&bits[d >> 5], 1u << (d & 31)) >> (d & 31) & 1u) bad = true;
    }
    __syncthreads();
    for (int i = t; i < n; i += kPageThreads) {
        const int s = src[i];
        if (s < -1 || s >= n_slots) bad = true;
        else if (s >= 0 && (bits[s >> 5] >> (s & 31) & 1u)) bad = true;
    }
    return __syncthreads_or(bad) == 0;
}

// Cluster 0 keeps the books: the sources' pages gain a name per fork; then each slot drops its old pages and takes its
// source's, and the pages that lost their last name go on the free stack in the order of their numbers, so that the
// stack does not depend on the order of the atomics. The other CTAs copy the open blocks' rows (nothing they read is
// written here: no source is a target).
// Bound: latency, five passes between cluster barriers (check, names, drops, count and push of freed pages), 6 us in a graph of
// such calls for 16 forks of 187 blocks; past some ten thousand entries (pairs times the longest one's blocks) the passes of
// names and drops over them on the cluster's eight SMs, 0.1 us a thousand: 256 forks of 187 blocks 12 us, of 653 24, 1,024 of 187
// 28. Not the atomics on a few sources' pages: forks of one, 12 or as many sources take 21, 25 and 24 us (256 of 653), 34, 27
// and 28 (1,024 of 187). 256 forks and releases of 8 to 653 blocks: 19 to 21 us.
__global__ void __launch_bounds__(kPageThreads) kv_fork_batch_kernel(const KvCache c, const int32_t *src, const int32_t *dst, int n,
                                                                     int Hkv, int row_vec, unsigned *err) {
    grid_dep_wait();
    grid_dep_launch();
    extern __shared__ __align__(16) unsigned char fork_smem[];
    __shared__ int ws[34], most;
    ForkPair *pairs = reinterpret_cast<ForkPair *>(fork_smem);
    unsigned *bits = reinterpret_cast<unsigned *>(pairs + n);
    const int t = threadIdx.x;
    const int2 *state = reinterpret_cast<const int2 *>(c.state);
    if (!fork_batch_ok(src, dst, n, c.n_slots, bits)) {
        if (blockIdx.x == 0 && t == 0) atomicOr(err, kErrKvBounds);
        return;   // the whole cluster
    }
    if (blockIdx.x >= kPageCluster) {
        const int64_t tasks = (int64_t)n * 2 * Hkv;
        for (int64_t k = blockIdx.x - kPageCluster; k < tasks; k += gridDim.x - kPageCluster) {
            const int i = (int)(k / (2 * Hkv)), part = (int)(k % (2 * Hkv)), s = src[i];
            if (s < 0) continue;
            const int2 st = state[s];
            const int vecs = max(st.x, 0) % kKvBlock * row_vec;
            const uint4 *from = static_cast<const uint4 *>(c.tail) + (((int64_t)s * 2 + (st.y & 1)) * 2 * Hkv + part) * kKvBlock * row_vec;
            uint4 *to = static_cast<uint4 *>(c.tail) + (((int64_t)dst[i] * 2 + (st.y & 1)) * 2 * Hkv + part) * kKvBlock * row_vec;
            for (int e = t; e < vecs; e += kPageThreads) to[e] = from[e];
        }
        return;
    }
    const int rank = blockIdx.x, first = rank * kPageThreads + t;
    constexpr int kAll = kPageCluster * kPageThreads;
    // the pairs, and the most blocks that one has to do with
    if (t == 0) most = 0;
    __syncthreads();
    for (int i = t; i < n; i += kPageThreads) {
        const int s = src[i], d = dst[i];
        auto blocks = [&](int slot) { return min(max(state[slot].x, 0) / kKvBlock, c.max_blocks); };
        const ForkPair p = {s, d, s >= 0 ? blocks(s) : 0, blocks(d)};
        pairs[i] = p;
        atomicMax(&most, max(p.now, p.before));
    }
    const int n_free = *c.n_free;
    __syncthreads();
    const unsigned nb = most;
    const int64_t entries = (int64_t)n * nb;
    // f(pair, block) over all of them, four a thread under way
    auto each = [&](auto f) {
        for (int64_t e0 = first; e0 < entries; e0 += 4 * kAll) {
            int64_t e = e0;
#pragma unroll
            for (int k = 0; k < 4; ++k, e += kAll) {
                if (e >= entries) break;
                const int i = entries <= UINT32_MAX ? (int)((unsigned)e / nb) : (int)(e / nb);
                f(pairs[i], (int)(e - (int64_t)i * nb));
            }
        }
    };
    each([&](const ForkPair &p, int b) {
        if (b >= p.now) return;
        const int page = c.table[(int64_t)p.src * c.max_blocks + b];
        if ((unsigned)page < (unsigned)c.n_pages) atomicAdd(&c.refs[page], 1);
    });
    cluster_sync();
    int freed = 0;
    each([&](const ForkPair &p, int b) {
        int32_t *mine = c.table + (int64_t)p.dst * c.max_blocks + b;
        const int to = b < p.now ? c.table[(int64_t)p.src * c.max_blocks + b] : -1, page = b < p.before ? *mine : -1;
        if ((unsigned)page < (unsigned)c.n_pages && atomicSub(&c.refs[page], 1) == 1) {
            c.refs[page] = kFreedMark;
            ++freed;
        }
        if (b < p.now) *mine = to;
    });
    int total;
    cluster_exclusive(freed, ws, &total);   // and the barrier after the last read of the old states
    for (int i = first; i < n; i += kAll) {
        const int s = src[i], d = dst[i];
        const int2 from = s >= 0 ? state[s] : make_int2(0, state[d].y);
        reinterpret_cast<int2 *>(c.state)[d] = make_int2(max(from.x, 0), from.y & 1);
    }
    if (total == 0) return;
    // freed pages in the order of their numbers: runs of consecutive pages per thread
    const int per = (int)((c.n_pages + (int64_t)kAll - 1) / kAll);
    const int64_t p0 = (int64_t)first * per, p1 = min(p0 + per, (int64_t)c.n_pages);
    int mine = 0;
    for (int64_t p = p0; p < p1; ++p) mine += c.refs[p] == kFreedMark;
    int at = n_free + cluster_exclusive(mine, ws, &total);
    if (mine) {
        for (int64_t p = p0; p < p1; ++p) {
            if (c.refs[p] != kFreedMark) continue;
            c.refs[p] = 0;
            if ((unsigned)at < (unsigned)c.n_pages) c.free_pages[at] = (int)p;
            ++at;
        }
    }
    if (first == 0) *c.n_free = min(n_free + total, c.n_pages);
}

// ---- compaction ----

// A cluster keeps the books. With U pages in use, page p >= U in use moves to a hole, a free page below U; both are counted
// off in the order of their numbers, so hole p is number p - (pages in use below p) and mover p number (pages in use
// between U and p). lists: holes, movers, and the new number of each page from U on.
// Bound: latency, four passes over the page counts between cluster barriers: 13 us for 20,000 pages, 5 us for 300.
__global__ void __launch_bounds__(kPageThreads) kv_compact_books_kernel(const KvCache c, const KvBooksOut o, int32_t *lists,
                                                                        int32_t *counts) {
    grid_dep_wait();
    grid_dep_launch();
    __shared__ int ws[34];
    constexpr int kAll = kPageCluster * kPageThreads;
    const int first = blockIdx.x * kPageThreads + threadIdx.x;
    const int per = (int)((c.n_pages + (int64_t)kAll - 1) / kAll);
    const int64_t p0 = (int64_t)first * per, p1 = min(p0 + per, (int64_t)c.n_pages);
    int32_t *holes = lists, *movers = lists + c.n_pages, *now = lists + 2 * (int64_t)c.n_pages;
    int mine = 0, used, moves;
    for (int64_t p = p0; p < p1; ++p) mine += c.refs[p] > 0;
    const int before = cluster_exclusive(mine, ws, &used);
    if (used > o.n_pages) {   // does not fit: nothing changes
        if (first == 0) {
            counts[0] = used;
            counts[1] = 1;
            counts[2] = 0;
        }
        return;
    }
    mine = 0;
    for (int64_t p = max(p0, (int64_t)used); p < p1; ++p) mine += c.refs[p] > 0;
    int mover = cluster_exclusive(mine, ws, &moves), below = before;
    for (int64_t p = p0; p < p1; ++p) {
        const bool in_use = c.refs[p] > 0;
        if (p < used) {
            if (!in_use) holes[p - below] = (int)p;
        } else if (in_use) {
            movers[mover++] = (int)p;
        } else {
            now[p] = (int)p;
        }
        below += in_use;
    }
    cluster_sync();
    for (int j = first; j < moves; j += kAll) now[movers[j]] = holes[j];
    // the counts: those of pages that stay, then the movers' in the holes, then none
    if (o.refs != c.refs)
        for (int64_t p = first; p < used; p += kAll) o.refs[p] = c.refs[p];
    cluster_sync();
    for (int j = first; j < moves; j += kAll) o.refs[holes[j]] = c.refs[movers[j]];
    cluster_sync();
    for (int64_t p = used + (int64_t)first; p < o.n_pages; p += kAll) o.refs[p] = 0;
    for (int i = first; i < o.n_pages - used; i += kAll) o.free_pages[i] = o.n_pages - 1 - i;
    if (first == 0) {
        *o.n_free = o.n_pages - used;
        counts[0] = used;
        counts[1] = 0;
        counts[2] = moves;
    }
}

constexpr int kMoveThreads = 256, kMoveVecs = 4;   // 16 KB of a page at a time
// The pages' bytes and scales, and the block tables. Bound: HBM, each moved byte read and written once, 16 KB a CTA at a time and
// eight CTAs an SM: 4,750 pages of 128 KB in 190 us, 6.5 TB/s.
__global__ void __launch_bounds__(kMoveThreads) kv_compact_move_kernel(const KvCache c, const KvBooksOut o, int Hkv, int64_t page_vecs,
                                                                       const int32_t *lists, const int32_t *counts) {
    grid_dep_wait();
    grid_dep_launch();
    if (counts[1] != 0) return;
    const int used = counts[0], moves = counts[2], t = threadIdx.x;
    const int32_t *holes = lists, *movers = lists + c.n_pages, *now = lists + 2 * (int64_t)c.n_pages;
    constexpr int kChunk = kMoveThreads * kMoveVecs;
    const int chunks = (int)((page_vecs + kChunk - 1) / kChunk);
    const int64_t tasks = 2LL * moves * chunks;
    for (int64_t k = blockIdx.x; k < tasks; k += gridDim.x) {
        const int64_t j = k / (2 * chunks);
        const int part = (int)(k - j * 2 * chunks), kv = part / chunks;
        const int64_t v0 = (int64_t)(part % chunks) * kChunk + t;
        int8_t *pool = kv ? c.v : c.k;
        const uint4 *from = reinterpret_cast<const uint4 *>(pool) + movers[j] * page_vecs;
        uint4 *to = reinterpret_cast<uint4 *>(pool) + holes[j] * page_vecs;
        uint4 w[kMoveVecs];
#pragma unroll
        for (int i = 0; i < kMoveVecs; ++i)
            if (v0 + i * kMoveThreads < page_vecs) w[i] = __ldcs(from + v0 + i * kMoveThreads);
#pragma unroll
        for (int i = 0; i < kMoveVecs; ++i)
            if (v0 + i * kMoveThreads < page_vecs) __stcs(to + v0 + i * kMoveThreads, w[i]);
    }
    const int64_t first = (int64_t)blockIdx.x * kMoveThreads + t, all = (int64_t)gridDim.x * kMoveThreads;
    for (int64_t e = first; e < 2LL * moves * Hkv; e += all) {
        const int64_t j = e / (2 * Hkv);
        const int x = (int)(e - j * 2 * Hkv), h = x % Hkv;
        float *s = x < Hkv ? c.k_scale : c.v_scale;
        s[(int64_t)holes[j] * Hkv + h] = s[(int64_t)movers[j] * Hkv + h];
    }
    for (int64_t e = first; e < (int64_t)c.n_slots * c.max_blocks; e += all) {
        const int slot = (int)(e / c.max_blocks), b = (int)(e - (int64_t)slot * c.max_blocks);
        if (b >= c.state[2 * slot] / kKvBlock) continue;
        int page = c.table[e];
        if (page >= used && page < c.n_pages) page = now[page];
        if (o.table != c.table || page != c.table[e]) o.table[e] = page;
    }
}

}  // namespace gdn

namespace {
template <class... K, class... A>
cudaError_t launch_clusters(void (*kernel)(K...), unsigned grid, size_t smem, cudaStream_t st, A &&...args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(gdn::kPageThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = gdn::kPageCluster;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, static_cast<A &&>(args)...);
    return e != cudaSuccess ? e : cudaGetLastError();
}
}  // namespace

cudaError_t gdn_launch_kv_fork_batch(const gdn::KvCache &c, const int32_t *src, const int32_t *dst, int n, int Hkv, int d, int elt,
                                     unsigned *err, cudaStream_t st) {
    using namespace gdn;
    const size_t smem = (size_t)n * sizeof(ForkPair) + ((size_t)c.n_slots + 31) / 32 * 4;
    if (smem > 32 * 1024) {
        const cudaError_t e = cudaFuncSetAttribute(kv_fork_batch_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                   (int)(kKvMaxRequests * sizeof(ForkPair) + kKvMaxBatchSlots / 8));
        if (e != cudaSuccess) return e;
    }
    const int64_t tasks = (int64_t)n * 2 * Hkv;   // copies, an eighth of a cluster each
    const unsigned copy = (unsigned)std::min<int64_t>((tasks + kPageCluster - 1) / kPageCluster, 16);
    return launch_clusters(kv_fork_batch_kernel, kPageCluster * (1 + copy), smem, st, c, src, dst, n, Hkv, d * elt / 16, err);
}

cudaError_t gdn_launch_kv_compact(const gdn::KvCache &c, const KvBooksOut &o, int Hkv, int d, int32_t *lists, int32_t *counts,
                                  cudaStream_t st) {
    using namespace gdn;
    cudaError_t e = launch_clusters(kv_compact_books_kernel, kPageCluster, 0, st, c, o, lists, counts);
    if (e != cudaSuccess) return e;
    int sms = 1;
    if ((e = gdn_sm_count(&sms)) != cudaSuccess) return e;
    const int64_t page_vecs = (int64_t)Hkv * kKvBlock * d / 16;
    e = gdn_launch_pdl(kv_compact_move_kernel, (unsigned)(8 * sms), kMoveThreads, 0, st, c, o, Hkv, page_vecs, lists, counts);
    return e != cudaSuccess ? e : cudaGetLastError();
}

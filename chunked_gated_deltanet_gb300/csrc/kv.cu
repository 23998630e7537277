// The paged 8-bit key/value cache's bookkeeping and writes: the plan of a batch (block tables and unit map from
// request lengths), the append (quantisation of complete blocks, raw copies into the tail), forks and releases.
#include "kv.cuh"

#include <algorithm>

namespace gdn {

constexpr int kPlanThreads = 1024;
constexpr int kPlanPer = kKvMaxRequests / kPlanThreads;   // requests per thread

struct Sum3 {
    long long rows;
    int units, pages;
};
__device__ __forceinline__ Sum3 add(const Sum3 &a, const Sum3 &b) {
    return {a.rows + b.rows, a.units + b.units, a.pages + b.pages};
}

// Exclusive sum over the CTA's threads in thread order; *total receives the sum of all. ws: one Sum3 per warp.
template <int NT>
__device__ Sum3 block_exclusive(Sum3 x, Sum3 *ws, Sum3 *total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    Sum3 in = x;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const Sum3 y = {__shfl_up_sync(0xffffffffu, in.rows, o), __shfl_up_sync(0xffffffffu, in.units, o),
                        __shfl_up_sync(0xffffffffu, in.pages, o)};
        if (lane >= o) in = add(in, y);
    }
    if (lane == 31) ws[warp] = in;
    __syncthreads();
    if (warp == 0) {
        Sum3 w = lane < NT / 32 ? ws[lane] : Sum3{0, 0, 0};
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const Sum3 y = {__shfl_up_sync(0xffffffffu, w.rows, o), __shfl_up_sync(0xffffffffu, w.units, o),
                            __shfl_up_sync(0xffffffffu, w.pages, o)};
            if (lane >= o) w = add(w, y);
        }
        ws[lane] = w;
    }
    __syncthreads();
    *total = ws[NT / 32 - 1];
    const Sum3 before = warp > 0 ? ws[warp - 1] : Sum3{0, 0, 0};
    return {before.rows + in.rows - x.rows, before.units + in.units - x.units, before.pages + in.pages - x.pages};
}

// Per request, in shared memory: what the expansion into units needs.
struct PlanReq {
    int ctx, count, slot, buf, unit0, page0, row0, pad;
};

// Plan of a batch in one CTA: per request i with ctx tokens held and n_new[i] to come, rows[i] = sum of earlier
// requests' new tokens, one unit per touched block, one page popped from the free stack per block that completes.
// Sums go in request order, so pages are handed out in unit order. A batch that does not fit (pages, table, unit
// map, a bad slot or count) leaves the cache as it was, with no unit and the reason in counts[1].
// Bound: latency (about 1 KB in and out per 16 requests): 3.1 us for one request, 8.6 us for 1,024 prompts. One CTA, or a cluster of kPlanCluster where the map has room for
// more units than a CTA has threads: every CTA sums over the requests by itself and expands its share of the units, and the
// cluster's barrier stands between the last read of the cache's state and its update in place.
constexpr int kPlanCluster = 8;
__global__ void __launch_bounds__(kPlanThreads) kv_plan_kernel(const KvCache c, const int32_t *slots, const int32_t *n_new,
                                                                int n, int32_t *rows, int32_t *units, int32_t *counts,
                                                                int max_units, int32_t *state_out, int32_t *n_free_out) {
    grid_dep_wait();
    grid_dep_launch();
    extern __shared__ __align__(16) unsigned char plan_smem[];
    PlanReq *req = reinterpret_cast<PlanReq *>(plan_smem);
    __shared__ Sum3 ws[32];
    __shared__ unsigned bad_all;
    const int t = threadIdx.x;
    const int per = (n + kPlanThreads - 1) / kPlanThreads;   // contiguous requests of this thread
    if (t == 0) bad_all = 0;
    const int n_free = *c.n_free;
    int slot[kPlanPer], cnt[kPlanPer], ctx[kPlanPer], buf[kPlanPer];
    Sum3 mine = {0, 0, 0};
    unsigned bad = 0;
#pragma unroll
    for (int j = 0; j < kPlanPer; ++j) {
        const int i = t * per + j;
        slot[j] = cnt[j] = ctx[j] = buf[j] = 0;
        if (j < per && i < n) {
            slot[j] = slots[i];
            cnt[j] = n_new[i];
            if ((unsigned)slot[j] >= (unsigned)c.n_slots || cnt[j] < 0) {
                bad |= 8u;
                slot[j] = cnt[j] = 0;
            } else {
                const int2 s = reinterpret_cast<const int2 *>(c.state)[slot[j]];
                ctx[j] = s.x;
                buf[j] = s.y & 1;
                const long long end = (long long)ctx[j] + cnt[j];
                if (ctx[j] < 0 || end / kKvBlock > c.max_blocks || end > INT32_MAX - kKvBlock) {
                    bad |= ctx[j] < 0 ? 8u : 2u;
                    ctx[j] = cnt[j] = 0;
                }
            }
            const int end = ctx[j] + cnt[j];
            mine.rows += cnt[j];
            if (cnt[j] > 0) mine.units += (end + kKvBlock - 1) / kKvBlock - ctx[j] / kKvBlock;
            mine.pages += end / kKvBlock - ctx[j] / kKvBlock;
        }
    }
    Sum3 total;
    Sum3 at = block_exclusive<kPlanThreads>(mine, ws, &total);
    if (bad) atomicOr(&bad_all, bad);
    if (t == 0) {
        if (total.pages > n_free || n_free > c.n_pages) atomicOr(&bad_all, 1u);
        if (total.units > max_units || total.rows > INT32_MAX) atomicOr(&bad_all, 4u);
    }
    __syncthreads();   // every read of the state and of the free stack's height is done, in the cluster's CTAs too
    if (gridDim.x > 1) {
        asm volatile("barrier.cluster.arrive.aligned;\nbarrier.cluster.wait.aligned;\n" ::: "memory");
    }
    const unsigned status = bad_all;
    const bool first = blockIdx.x == 0;   // writes what there is once
#pragma unroll
    for (int j = 0; j < kPlanPer; ++j) {
        const int i = t * per + j;
        if (j < per && i < n) {
            if (status == 0) {
                if (first) rows[i] = (int)at.rows;
                const int end = ctx[j] + cnt[j];
                const int fb = ctx[j] / kKvBlock, eb = end / kKvBlock;
                req[i] = {ctx[j], cnt[j], slot[j], buf[j], at.units, at.pages, (int)at.rows, 0};
                // the open block moves to the other tail buffer when it is a new block, so that the rows of the
                // block that closes in this call stay readable after its append
                if (first) reinterpret_cast<int2 *>(state_out)[slot[j]] = make_int2(end, eb != fb ? buf[j] ^ 1 : buf[j]);
                at.rows += cnt[j];
                if (cnt[j] > 0) at.units += (end + kKvBlock - 1) / kKvBlock - fb;
                at.pages += eb - fb;
            } else if (first) {
                rows[i] = 0;
            }
        }
    }
    if (t == 0 && first) {
        rows[n] = status == 0 ? (int)total.rows : 0;
        counts[0] = status == 0 ? total.units : 0;
        counts[1] = (int)status;
        *n_free_out = status == 0 ? n_free - total.pages : n_free;
    }
    if (status != 0) return;
    __syncthreads();
    // one thread per unit; its request is the last one whose first unit is not after it
    for (int u = blockIdx.x * kPlanThreads + t; u < total.units; u += gridDim.x * kPlanThreads) {
        int lo = 0, hi = n - 1;
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (req[mid].unit0 <= u) lo = mid;
            else hi = mid - 1;
        }
        const PlanReq r = req[lo];
        const int j = u - r.unit0, fb = r.ctx / kKvBlock, block = fb + j, end = r.ctx + r.count;
        const int start = max(r.ctx, block * kKvBlock), stop = min(end, block * kKvBlock + kKvBlock);
        const bool closes = stop == block * kKvBlock + kKvBlock;
        int page = -1;
        if (closes) {
            page = c.free_pages[n_free - 1 - (r.page0 + j)];
            if ((unsigned)page < (unsigned)c.n_pages) {
                c.table[(int64_t)r.slot * c.max_blocks + block] = page;
                c.refs[page] = 1;
            }
        }
        int4 *o = reinterpret_cast<int4 *>(units) + 2 * (int64_t)u;
        o[0] = make_int4(r.slot, block, page, start - block * kKvBlock);
        o[1] = make_int4(stop - start, r.row0 + start - r.ctx, r.buf, closes ? -1 : (end / kKvBlock != fb ? r.buf ^ 1 : r.buf));
    }
}

// ---- append ----

// x / scale rounded to nearest even as an IEEE division and rint give it, saturated, a NaN 0: every value of a block with
// values that are not finite, and the values of a vector whose quotient is near a tie.
__device__ __forceinline__ int kv_quant(float x, float scale) {
    const float q = rintf(x / scale);
    return q == q ? (int)fminf(fmaxf(q, -127.f), 127.f) : 0;   // 0 / 0 of an all-zero block, or a NaN: 0
}

template <typename T> struct Vec16;   // 16 bytes of T as floats
template <> struct Vec16<float> {
    static constexpr int N = 4;
    static constexpr uint32_t kInf = 0x7F800000u;
    static __device__ __forceinline__ void get(const uint4 &u, float (&f)[4]) {
        f[0] = __uint_as_float(u.x); f[1] = __uint_as_float(u.y); f[2] = __uint_as_float(u.z); f[3] = __uint_as_float(u.w);
    }
    // largest magnitude as bits (order-preserving for magnitudes; infinities and NaNs on top)
    static __device__ __forceinline__ uint32_t top(uint32_t m, const uint4 &u) {
        m = max(m, u.x & 0x7FFFFFFFu);
        m = max(m, u.y & 0x7FFFFFFFu);
        m = max(m, u.z & 0x7FFFFFFFu);
        return max(m, u.w & 0x7FFFFFFFu);
    }
    static __device__ __forceinline__ uint32_t bits(uint32_t m) { return m; }
};
template <> struct Vec16<__nv_bfloat16> {
    static constexpr int N = 8;
    static constexpr uint32_t kInf = 0x7F800000u;
    static __device__ __forceinline__ void get(const uint4 &u, float (&f)[8]) {
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f[2 * i] = __uint_as_float(w[i] << 16);
            f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
    }
    static __device__ __forceinline__ uint32_t top(uint32_t m, const uint4 &u) {   // two 16-bit magnitudes
        m = __vmaxu2(m, u.x & 0x7FFF7FFFu);
        m = __vmaxu2(m, u.y & 0x7FFF7FFFu);
        m = __vmaxu2(m, u.z & 0x7FFF7FFFu);
        return __vmaxu2(m, u.w & 0x7FFF7FFFu);
    }
    static __device__ __forceinline__ uint32_t bits(uint32_t m) { return max(m << 16, m & 0xFFFF0000u); }
};

// CTA (unit, kv head, k or v). A block that closes: its 64 rows (tail rows before `first`, then new ones) go through
// registers once: absmax, scale, int8 page. A block that stays open: its new rows are copied into the tail.
// Four 16-byte vectors per thread and 48 warps on an SM: enough bytes under way for the latency of a CTA's three steps
// (unit record, rows, page). A block of 64 x 128 bf16: 5.0 TB/s read and written.
template <typename InT, int D>
constexpr int kAppendThreads = kKvBlock * D / Vec16<InT>::N / 4;

template <typename InT, int D>
__global__ void __launch_bounds__(kAppendThreads<InT, D>, 1536 / kAppendThreads<InT, D>) kv_append_kernel(const KvCache c, const int32_t *units, const int32_t *counts,
                                                        const InT *kx, const InT *vx, int64_t n_rows, int Hkv,
                                                        unsigned *err) {
    grid_dep_wait();
    grid_dep_launch();
    const KvUnit u = kv_load_unit(units, blockIdx.x);   // inside the map whatever the count
    if ((int)blockIdx.x >= counts[0]) return;
    constexpr int NT = kAppendThreads<InT, D>, NW = NT / 32;
    constexpr int VN = Vec16<InT>::N, VPR = D / VN, NV = kKvBlock * VPR / NT;   // vectors per row, per thread
    __shared__ uint32_t red[NW];
    if (!kv_unit_ok(u, c, n_rows)) {
        if (threadIdx.x == 0 && blockIdx.y == 0 && blockIdx.z == 0) atomicOr(err, kErrKvBounds);
        return;
    }
    const int h = blockIdx.y, kv = blockIdx.z, t = threadIdx.x;
    const InT *x = kv ? vx : kx;
    const InT *old = static_cast<const InT *>(c.tail) + kv_tail_offset(u.slot, u.src, kv, h, Hkv, D);
    uint4 w[NV];
    const bool closes = u.page >= 0;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int e = t + NT * i, r = e / VPR, col = (e % VPR) * VN;
        const int o = r - u.first;
        w[i] = make_uint4(0, 0, 0, 0);
        if (o >= 0 && o < u.count) w[i] = *reinterpret_cast<const uint4 *>(x + ((int64_t)(u.row + o) * Hkv + h) * D + col);
        else if (o < 0 && closes) w[i] = *reinterpret_cast<const uint4 *>(old + r * D + col);
    }
    if (!closes) {
        InT *tail = static_cast<InT *>(c.tail) + kv_tail_offset(u.slot, u.dst, kv, h, Hkv, D);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int e = t + NT * i, r = e / VPR, col = (e % VPR) * VN;
            const int o = r - u.first;
            if (o >= 0 && o < u.count) *reinterpret_cast<uint4 *>(tail + r * D + col) = w[i];
        }
        return;
    }
    uint32_t mb = 0;
#pragma unroll
    for (int i = 0; i < NV; ++i) mb = Vec16<InT>::top(mb, w[i]);
    mb = __reduce_max_sync(0xffffffffu, Vec16<InT>::bits(mb));
    if ((t & 31) == 0) red[t >> 5] = mb;
    __syncthreads();
    mb = red[0];
#pragma unroll
    for (int i = 1; i < NW; ++i) mb = max(mb, red[i]);
    const bool finite = mb < Vec16<InT>::kInf;
    if (!finite) {   // the scale comes from the finite values
        mb = 0;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            float f[VN];
            Vec16<InT>::get(w[i], f);
#pragma unroll
            for (int j = 0; j < VN; ++j) {
                const uint32_t b = __float_as_uint(f[j]) & 0x7FFFFFFFu;
                if (b < Vec16<InT>::kInf) mb = max(mb, b);
            }
        }
        mb = __reduce_max_sync(0xffffffffu, mb);
        __syncthreads();
        if ((t & 31) == 0) red[t >> 5] = mb;
        __syncthreads();
        mb = red[0];
#pragma unroll
        for (int i = 1; i < NW; ++i) mb = max(mb, red[i]);
    }
    const float scale = __uint_as_float(mb) / 127.f, inv = 1.f / scale;
    const int64_t ph = (int64_t)u.page * Hkv + h;
    int8_t *page = (kv ? c.v : c.k) + ph * kKvBlock * D;
    if (t == 0) (kv ? c.v_scale : c.k_scale)[ph] = scale;
    // The quotient as the product with the reciprocal, off by at most 127 * 2^-23 < 1.6e-5, rounded by adding and taking away
    // 1.5 * 2^23, whose sum holds the integer in its low bits. Where that is within 5e-5 of a tie the vector is divided.
    const float magic = 12582912.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        float f[VN], d = 0.f;
        uint32_t q[VN], b[VN / 4];
        Vec16<InT>::get(w[i], f);
#pragma unroll
        for (int j = 0; j < VN; ++j) {
            const float y = f[j] * inv, z = y + magic;
            d = fmaxf(d, fabsf(y - (z - magic)));
            q[j] = __float_as_uint(z);
        }
        if (!finite || !(d < 0.49995f) || !(inv <= 3.4e38f)) {   // also a scale without a finite reciprocal
#pragma unroll
            for (int j = 0; j < VN; ++j) q[j] = (uint32_t)kv_quant(f[j], scale);
        }
#pragma unroll
        for (int j = 0; j < VN / 4; ++j)
            b[j] = __byte_perm(__byte_perm(q[4 * j], q[4 * j + 1], 0x0040), __byte_perm(q[4 * j + 2], q[4 * j + 3], 0x0040), 0x5410);
        const int e = t + NT * i, r = e / VPR, col = (e % VPR) * VN;
        if (VN == 8) *reinterpret_cast<uint2 *>(page + r * D + col) = make_uint2(b[0], b[VN / 4 - 1]);
        else *reinterpret_cast<uint32_t *>(page + r * D + col) = b[0];
    }
}

// ---- forks and releases ----

// Every slot empty, every page free (page 0 on top of the stack).
__global__ void __launch_bounds__(256) kv_init_kernel(const KvCache c) {
    grid_dep_wait();
    grid_dep_launch();
    const int i = blockIdx.x * 256 + threadIdx.x;
    if (i < c.n_pages) {
        c.free_pages[i] = c.n_pages - 1 - i;
        c.refs[i] = 0;
    }
    if (i < c.n_slots) reinterpret_cast<int2 *>(c.state)[i] = make_int2(0, 0);
    if (i == 0) *c.n_free = c.n_pages;
}

// Drops the slot's hold on its pages (CTA-wide): pages that no slot names any more go back on the free stack in
// block order. The slot then holds nothing.
__device__ void kv_drop(const KvCache &c, int slot, Sum3 *ws) {
    const int len = c.state[2 * slot], nb = min(max(len, 0) / kKvBlock, c.max_blocks);
    int height = *c.n_free;
    __syncthreads();
    for (int b0 = 0; b0 < nb; b0 += kPlanThreads) {
        const int b = b0 + threadIdx.x;
        int page = -1;
        bool freed = false;
        if (b < nb) {
            page = c.table[(int64_t)slot * c.max_blocks + b];
            if ((unsigned)page < (unsigned)c.n_pages) freed = --c.refs[page] == 0;
        }
        Sum3 total;
        const Sum3 at = block_exclusive<kPlanThreads>({0, 0, freed ? 1 : 0}, ws, &total);
        if (freed && height + at.pages < c.n_pages) c.free_pages[height + at.pages] = page;
        height += total.pages;
        __syncthreads();
    }
    if (threadIdx.x == 0) {
        *c.n_free = min(height, c.n_pages);
        c.state[2 * slot] = 0;
    }
    __syncthreads();
}

__global__ void __launch_bounds__(kPlanThreads) kv_release_kernel(const KvCache c, int slot) {
    __shared__ Sum3 ws[32];
    grid_dep_wait();
    grid_dep_launch();
    kv_drop(c, slot, ws);
}

// CTA 0: dst drops what it holds, then names src's complete blocks. The other CTAs copy src's open rows into the same
// tail buffer of dst (nothing they read is written here).
__global__ void __launch_bounds__(kPlanThreads) kv_fork_kernel(const KvCache c, int src, int dst, int Hkv, int row_vec) {
    __shared__ Sum3 ws[32];
    grid_dep_wait();
    grid_dep_launch();
    const int2 s = reinterpret_cast<const int2 *>(c.state)[src];
    const int len = max(s.x, 0), buf = s.y & 1;
    if (blockIdx.x == 0) {
        kv_drop(c, dst, ws);
        const int nb = min(len / kKvBlock, c.max_blocks);
        for (int b = threadIdx.x; b < nb; b += kPlanThreads) {
            const int page = c.table[(int64_t)src * c.max_blocks + b];
            c.table[(int64_t)dst * c.max_blocks + b] = page;
            if ((unsigned)page < (unsigned)c.n_pages) ++c.refs[page];
        }
        if (threadIdx.x == 0) reinterpret_cast<int2 *>(c.state)[dst] = make_int2(len, buf);
        return;
    }
    const int open = len % kKvBlock, per_head = open * row_vec;
    const int64_t n = 2LL * Hkv * per_head, stride = (int64_t)(gridDim.x - 1) * kPlanThreads;
    const uint4 *from = static_cast<const uint4 *>(c.tail) + ((int64_t)src * 2 + buf) * 2 * Hkv * kKvBlock * row_vec;
    uint4 *to = static_cast<uint4 *>(c.tail) + ((int64_t)dst * 2 + buf) * 2 * Hkv * kKvBlock * row_vec;
    for (int64_t i = (int64_t)(blockIdx.x - 1) * kPlanThreads + threadIdx.x; i < n; i += stride) {
        const int64_t e = i / per_head * kKvBlock * row_vec + i % per_head;
        to[e] = from[e];
    }
}

template <typename InT, int D>
cudaError_t launch_append(const KvCache &c, const int32_t *units, const int32_t *counts, int unit_bound, const void *k,
                          const void *v, int64_t n_rows, int Hkv, unsigned *err, cudaStream_t st) {
    const dim3 grid((unsigned)unit_bound, (unsigned)Hkv, 2);
    const cudaError_t e = gdn_launch_pdl(kv_append_kernel<InT, D>, grid, kAppendThreads<InT, D>, 0, st, c, units, counts,
                                         static_cast<const InT *>(k), static_cast<const InT *>(v), n_rows, Hkv, err);
    return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace gdn

cudaError_t gdn_launch_kv_plan(const gdn::KvCache &c, const int32_t *slots, const int32_t *n_new, int n, int32_t *rows,
                               int32_t *units, int32_t *counts, int max_units, int32_t *state_out, int32_t *n_free_out,
                               cudaStream_t st) {
    using namespace gdn;
    const size_t smem = (size_t)n * sizeof(PlanReq);
    cudaError_t e = cudaSuccess;
    if (smem > 32 * 1024) {
        e = cudaFuncSetAttribute(kv_plan_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 (int)(kKvMaxRequests * sizeof(PlanReq)));
        if (e != cudaSuccess) return e;
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(max_units > kPlanThreads ? kPlanCluster : 1);
    cfg.blockDim = dim3(kPlanThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = cfg.gridDim.x;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    e = cudaLaunchKernelEx(&cfg, kv_plan_kernel, c, slots, n_new, n, rows, units, counts, max_units, state_out, n_free_out);
    return e != cudaSuccess ? e : cudaGetLastError();
}

cudaError_t gdn_launch_kv_append(const gdn::KvCache &c, const int32_t *units, const int32_t *counts, int unit_bound,
                                 const void *k, const void *v, int64_t n_rows, int Hkv, int d, int bf16, unsigned *err,
                                 cudaStream_t st) {
    using namespace gdn;
    using bf = __nv_bfloat16;
    if (d == 64)
        return bf16 ? launch_append<bf, 64>(c, units, counts, unit_bound, k, v, n_rows, Hkv, err, st)
                    : launch_append<float, 64>(c, units, counts, unit_bound, k, v, n_rows, Hkv, err, st);
    if (d == 128)
        return bf16 ? launch_append<bf, 128>(c, units, counts, unit_bound, k, v, n_rows, Hkv, err, st)
                    : launch_append<float, 128>(c, units, counts, unit_bound, k, v, n_rows, Hkv, err, st);
    return bf16 ? launch_append<bf, 256>(c, units, counts, unit_bound, k, v, n_rows, Hkv, err, st)
                : launch_append<float, 256>(c, units, counts, unit_bound, k, v, n_rows, Hkv, err, st);
}

cudaError_t gdn_launch_kv_init(const gdn::KvCache &c, cudaStream_t st) {
    const int n = std::max(c.n_pages, c.n_slots);
    const cudaError_t e = gdn_launch_pdl(gdn::kv_init_kernel, (unsigned)((n + 255LL) / 256), 256, 0, st, c);
    return e != cudaSuccess ? e : cudaGetLastError();
}

cudaError_t gdn_launch_kv_fork(const gdn::KvCache &c, int src, int dst, int Hkv, int d, int elt, cudaStream_t st) {
    using namespace gdn;
    const int row_vec = d * elt / 16;
    const int copy = std::min<int64_t>(64, (2LL * Hkv * kKvBlock * row_vec + kPlanThreads - 1) / kPlanThreads);
    const cudaError_t e = gdn_launch_pdl(kv_fork_kernel, 1 + copy, kPlanThreads, 0, st, c, src, dst, Hkv, row_vec);
    return e != cudaSuccess ? e : cudaGetLastError();
}

cudaError_t gdn_launch_kv_release(const gdn::KvCache &c, int slot, cudaStream_t st) {
    const cudaError_t e = gdn_launch_pdl(gdn::kv_release_kernel, 1, gdn::kPlanThreads, 0, st, c, slot);
    return e != cudaSuccess ? e : cudaGetLastError();
}

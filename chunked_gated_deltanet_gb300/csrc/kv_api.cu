// C ABI of the paged 8-bit key/value cache and its attention (declared in include/gdn.h): argument validation on the
// host before any device work, workspace layout, choice of kernel and launches.
#include "gdn.h"
#include "host.h"
#include "kv.cuh"

#include <algorithm>
#include <array>
#include <cmath>

using namespace gdn_host;
using gdn::kKvBlock;

static_assert(GDN_KV_BLOCK == gdn::kKvBlock && GDN_KV_MAX_REQUESTS == gdn::kKvMaxRequests, "header constants");

namespace {

bool aligned(const void *p, uintptr_t n) { return p && (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

gdn_status check_attn(const gdn_attn_desc *d) {
    if (!d) return fail(GDN_ERR_INVALID_ARG, "attention description is NULL");
    if (d->n_kv_heads < 1 || d->n_q_heads < 1 || d->n_q_heads % d->n_kv_heads != 0 || d->n_q_heads > 65535)
        return fail(GDN_ERR_SHAPE, "heads: need 1 <= Hkv, Hq a multiple of Hkv, Hq <= 65535 (Hq=%d, Hkv=%d)", d->n_q_heads,
                    d->n_kv_heads);
    if (d->head_dim != 64 && d->head_dim != 128 && d->head_dim != 256)
        return fail(GDN_ERR_SHAPE, "head_dim must be 64, 128 or 256 (got %d)", d->head_dim);
    if (d->in_dtype != GDN_BF16 && d->in_dtype != GDN_FP32)
        return fail(GDN_ERR_SHAPE, "in_dtype must be GDN_BF16 or GDN_FP32 (got %d)", d->in_dtype);
    if (!(d->scale > 0.f) || !std::isfinite(d->scale)) return fail(GDN_ERR_INVALID_ARG, "scale must be finite and > 0");
    return GDN_OK;
}

// What a call needs of the cache: its bookkeeping, and its contents.
gdn_status check_cache(const gdn_kv_cache *c, bool books, bool contents) {
    if (!c) return fail(GDN_ERR_INVALID_ARG, "cache is NULL");
    if (c->n_pages < 1 || c->n_slots < 1 || c->max_blocks < 1)
        return fail(GDN_ERR_INVALID_ARG, "cache: n_pages, n_slots and max_blocks must be >= 1 (%d, %d, %d)", c->n_pages,
                    c->n_slots, c->max_blocks);
    if (!aligned(c->state, 8) || !aligned(c->table, 4))
        return fail(GDN_ERR_INVALID_ARG, "cache: state (8-byte aligned) and table must be non-NULL");
    if (books && (!aligned(c->free_pages, 4) || !aligned(c->n_free, 4) || !aligned(c->refs, 4)))
        return fail(GDN_ERR_INVALID_ARG, "cache: free_pages, n_free and refs must be non-NULL");
    if (contents && (!aligned(c->k, 16) || !aligned(c->v, 16) || !aligned(c->tail, 16) || !aligned(c->k_scale, 4) ||
                     !aligned(c->v_scale, 4)))
        return fail(GDN_ERR_INVALID_ARG, "cache: k, v, tail (16-byte aligned), k_scale and v_scale must be non-NULL");
    return GDN_OK;
}

gdn_status check_map(const gdn_kv_map *m) {
    if (!m) return fail(GDN_ERR_INVALID_ARG, "map is NULL");
    if (!aligned(m->rows, 4) || !aligned(m->units, 16) || !aligned(m->counts, 4))
        return fail(GDN_ERR_INVALID_ARG, "map: rows, units (16-byte aligned) and counts must be non-NULL");
    if (m->max_requests < 1 || m->max_requests > GDN_KV_MAX_REQUESTS || m->max_units < 1)
        return fail(GDN_ERR_INVALID_ARG, "map: max_requests must be in [1, %d] and max_units >= 1 (%d, %d)",
                    GDN_KV_MAX_REQUESTS, m->max_requests, m->max_units);
    return GDN_OK;
}

gdn::KvCache device_cache(const gdn_kv_cache *c) {
    return {c->k, c->v, c->k_scale, c->v_scale, c->tail, c->state, c->table, c->free_pages, c->n_free, c->refs,
            c->n_pages, c->n_slots, c->max_blocks};
}

// Units of a batch: a request of n tokens touches at most (n + 62) / 64 + 1 blocks, and at most n.
int64_t max_units(int64_t tokens, int32_t requests) { return std::min<int64_t>(tokens, tokens / kKvBlock + 2LL * requests); }

// Key segments of a row's attention, in blocks, cut at absolute positions. Few rows: 512 keys for fp32 and for up to three
// key/value heads, so that one token's long context fills the GPU, up to 4,096 for more heads, which fill it with longer
// ones. Many rows: by the CTAs of one request and segment. Up to 31, short segments fill the SMs; up to 159, growing ones
// (0, kv_grown_start's); more fill them alone. Against 64 blocks throughout (us, L2 flushed): 165 x 12 rows over 18,107
// keys 76 -> 66, 290 x 16 rows over 41,802 255 -> 229, 4,000 x 16 over 37,802 1,204 -> 1,115; requests that fill the GPU
// together lose: 16 of up to 200 x 16 rows over 12,000 204 -> 206, 6 of 165 x 12 over 18,107 144 -> 161. In fp32, where 64
// rows of one head take about 3 us a block: 256 keys up to 159 CTAs, then 512 (against 512 throughout: a prompt of 2,048 x 2
// rows 77 -> 47, 2 of 644 x 8 over 2,825 even; 2 of 2,099 x 32, which fill the SMs, lose 5 % with 256).
// A rule on the description and max_new: a row's segments do not depend on the batch.
int many_rows(const gdn_attn_desc *d) { return d->in_dtype == GDN_FP32 ? gdn::kKvSimtRows : gdn::kv_prompt_rows(d->head_dim); }
constexpr int kManySteps[] = {8, 32, 160}, kManySegs[] = {32, 48, 0, 128}, kManySegsFp32[] = {4, 4, 4, 8};
int seg_blocks(const gdn_attn_desc *d, bool few, int64_t max_new) {
    const bool fp32 = d->in_dtype == GDN_FP32;
    if (few) return fp32 || d->n_kv_heads < 4 ? 8 : d->n_kv_heads < 8 ? 16 : d->n_kv_heads < 16 ? 32 : 64;
    const int rows = many_rows(d), G = d->n_q_heads / d->n_kv_heads;   // rows of a CTA
    const int64_t ctas = (max_new * G + rows - 1) / rows * d->n_kv_heads;
    const int i = ctas < kManySteps[0] ? 0 : ctas < kManySteps[1] ? 1 : ctas < kManySteps[2] ? 2 : 3;
    return fp32 ? kManySegsFp32[i] : kManySegs[i];
}
constexpr int kFewRows = 16;   // rows (new tokens of a block x query heads per key/value head) of the few-row form

struct Form {
    bool few;
    int rows_max, tok_stride, seg_blocks;
    int64_t n_seg;
    size_t unit_bytes;   // partial results of one unit
};
Form form_of(const gdn_attn_desc *d, int64_t max_new, int64_t max_len) {
    Form f;
    const int G = d->n_q_heads / d->n_kv_heads;
    f.tok_stride = (int)std::min<int64_t>(max_new, kKvBlock);
    f.rows_max = f.tok_stride * G;
    f.few = max_new * G <= kFewRows;
    f.seg_blocks = seg_blocks(d, f.few, max_new);
    const int64_t blocks = std::max<int64_t>((max_len + kKvBlock - 1) / kKvBlock, 1);
    f.n_seg = f.seg_blocks ? (blocks + f.seg_blocks - 1) / f.seg_blocks : gdn::kv_grown_seg((int)blocks - 1) + 1;
    f.unit_bytes = f.n_seg == 1 ? 0 : (size_t)f.n_seg * f.tok_stride * d->n_q_heads * (d->head_dim * sizeof(float) + sizeof(float2));
    return f;
}
// The largest max_new of each of these forms, none above `most`: a form's partial results are the largest there.
std::array<int64_t, 5> form_tops(const gdn_attn_desc *d, int64_t most) {
    const int G = d->n_q_heads / d->n_kv_heads, rows = many_rows(d);
    std::array<int64_t, 5> tops = {kFewRows / G, most};
    for (int i = 0; i < 3; ++i) tops[2 + i] = (int64_t)((kManySteps[i] - 1) / d->n_kv_heads) * rows / G;
    for (int64_t &n : tops) n = std::min(std::max<int64_t>(n, 1), most);
    return tops;
}
constexpr size_t kWsTarget = size_t(2) << 30;   // a call's partial results beyond this go in several launches
constexpr size_t kWsSlack = 512;                // alignment of the two parts

}  // namespace

GDN_API gdn_status gdn_attn_desc_check(const gdn_attn_desc *d) { return check_attn(d); }

GDN_API int32_t gdn_kv_max_units(int64_t max_tokens, int32_t max_requests) {
    if (max_tokens < 0 || max_requests < 1 || max_tokens > INT32_MAX) return 0;
    return (int32_t)std::max<int64_t>(max_units(max_tokens, max_requests), 1);
}

GDN_API gdn_status gdn_kv_cache_init(const gdn_attn_desc *d, const gdn_kv_cache *c, gdn_stream_t stream) {
    gdn_status st = check_attn(d);
    if (st != GDN_OK || (st = check_cache(c, true, true)) != GDN_OK) return st;
    const cudaError_t e = launch_k(K_KV_STATE, (cudaStream_t)stream,
                                   [&] { return gdn_launch_kv_init(device_cache(c), (cudaStream_t)stream); });
    return e != cudaSuccess ? cuda_fail(e, "key/value cache initialisation") : GDN_OK;
}

GDN_API gdn_status gdn_kv_plan(const gdn_attn_desc *d, const gdn_kv_cache *c, const int32_t *slots, const int32_t *n_new,
                               int32_t n, const gdn_kv_map *m, int32_t *state_out, int32_t *n_free_out,
                               gdn_stream_t stream) {
    gdn_status st = check_attn(d);
    if (st != GDN_OK || (st = check_cache(c, true, false)) != GDN_OK || (st = check_map(m)) != GDN_OK) return st;
    if (n < 1 || n > m->max_requests)
        return fail(GDN_ERR_INVALID_ARG, "n_requests must be in [1, %d] (got %d)", m->max_requests, n);
    if (!aligned(slots, 4) || !aligned(n_new, 4)) return fail(GDN_ERR_INVALID_ARG, "slots and n_new must be non-NULL");
    if (!state_out) state_out = c->state;
    if (!n_free_out) n_free_out = c->n_free;
    if (!aligned(state_out, 8) || !aligned(n_free_out, 4))
        return fail(GDN_ERR_INVALID_ARG, "state_out must be 8-byte aligned, n_free_out 4-byte");
    cudaStream_t cst = (cudaStream_t)stream;
    const cudaError_t e = launch_k(K_KV_PLAN, cst, [&] {
        return gdn_launch_kv_plan(device_cache(c), slots, n_new, n, m->rows, m->units, m->counts, m->max_units, state_out,
                                  n_free_out, cst);
    });
    return e != cudaSuccess ? cuda_fail(e, "plan kernel") : GDN_OK;
}

GDN_API gdn_status gdn_kv_status(const gdn_kv_map *m, gdn_stream_t stream) {
    gdn_status st = check_map(m);
    if (st != GDN_OK) return st;
    int32_t counts[2] = {0, 0};
    cudaError_t e = cudaMemcpyAsync(counts, m->counts, sizeof(counts), cudaMemcpyDeviceToHost, (cudaStream_t)stream);
    if (e == cudaSuccess) e = cudaStreamSynchronize((cudaStream_t)stream);
    if (e != cudaSuccess) return cuda_fail(e, "plan status read");
    if (counts[1] == 0) return GDN_OK;
    return fail(GDN_ERR_CAPACITY, "the batch was not planned:%s%s%s%s", counts[1] & 1 ? " too few free pages;" : "",
                counts[1] & 2 ? " a request past max_blocks;" : "", counts[1] & 4 ? " more units or rows than the map holds;" : "",
                counts[1] & 8 ? " a slot, length or count out of range;" : "");
}

GDN_API gdn_status gdn_kv_append(const gdn_attn_desc *d, const gdn_kv_cache *c, const gdn_kv_map *m, const void *k,
                                 const void *v, int64_t n_rows, gdn_stream_t stream) {
    gdn_status st = check_attn(d);
    if (st != GDN_OK || (st = check_cache(c, false, true)) != GDN_OK || (st = check_map(m)) != GDN_OK) return st;
    if (n_rows < 0 || n_rows > INT32_MAX) return fail(GDN_ERR_INVALID_ARG, "n_rows out of range (%lld)", (long long)n_rows);
    if (n_rows == 0) return GDN_OK;
    if (!aligned(k, 16) || !aligned(v, 16)) return fail(GDN_ERR_INVALID_ARG, "k and v must be non-NULL and 16-byte aligned");
    unsigned *err = nullptr;
    cudaError_t e = gdn_device_error_word(&err);
    if (e != cudaSuccess) return cuda_fail(e, "device error word lookup");
    cudaStream_t cst = (cudaStream_t)stream;
    const int bound = (int)std::min<int64_t>(m->max_units, max_units(n_rows, m->max_requests));
    e = launch_k(K_KV_APPEND, cst, [&] {
        return gdn_launch_kv_append(device_cache(c), m->units, m->counts, bound, k, v, n_rows, d->n_kv_heads, d->head_dim,
                                    d->in_dtype == GDN_BF16, err, cst);
    });
    return e != cudaSuccess ? cuda_fail(e, "append kernel") : GDN_OK;
}

GDN_API size_t gdn_kv_attention_workspace_min(const gdn_attn_desc *d, int64_t max_len) {
    if (check_attn(d) != GDN_OK || max_len < 0 || max_len > INT32_MAX) return 0;
    size_t need = 0;
    for (const int64_t max_new : form_tops(d, INT32_MAX)) need = std::max(need, form_of(d, max_new, max_len).unit_bytes);
    return kWsSlack + need;
}

GDN_API size_t gdn_kv_attention_workspace(const gdn_attn_desc *d, int64_t max_tokens, int32_t max_requests, int64_t max_len) {
    if (check_attn(d) != GDN_OK || max_tokens < 0 || max_tokens > INT32_MAX || max_requests < 1 || max_len < 0 ||
        max_len > INT32_MAX)
        return 0;
    size_t need = 0;
    for (const int64_t max_new : form_tops(d, std::max<int64_t>(max_tokens, 1))) {
        const size_t units = (size_t)max_units(std::min<int64_t>(max_tokens, max_new * max_requests), max_requests);
        need = std::max(need, std::min(units * form_of(d, max_new, max_len).unit_bytes, kWsTarget));
    }
    return std::max(kWsSlack + need, gdn_kv_attention_workspace_min(d, max_len));
}

GDN_API gdn_status gdn_kv_attention(const gdn_attn_desc *d, const gdn_kv_cache *c, const gdn_kv_map *m, const void *q,
                                    const void *k, const void *v, void *out, int64_t n_rows, int32_t max_new,
                                    int64_t max_len, void *workspace, size_t workspace_bytes, gdn_stream_t stream) {
    gdn_status st = check_attn(d);
    if (st != GDN_OK || (st = check_cache(c, false, true)) != GDN_OK || (st = check_map(m)) != GDN_OK) return st;
    if (n_rows < 0 || n_rows > INT32_MAX) return fail(GDN_ERR_INVALID_ARG, "n_rows out of range (%lld)", (long long)n_rows);
    if (max_new < 1 || max_len < 1 || max_len > INT32_MAX)
        return fail(GDN_ERR_INVALID_ARG, "max_new and max_len must be >= 1 (%d, %lld)", max_new, (long long)max_len);
    if (n_rows == 0) return GDN_OK;
    if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(out, 16))
        return fail(GDN_ERR_INVALID_ARG, "q, k, v and out must be non-NULL and 16-byte aligned");
    max_new = (int32_t)std::min<int64_t>(max_new, n_rows);
    const Form f = form_of(d, max_new, max_len);
    if (f.n_seg > 65535) return fail(GDN_ERR_INVALID_ARG, "max_len %lld needs more than 65,535 segments", (long long)max_len);
    const int bound = (int)std::min<int64_t>(m->max_units, max_units(n_rows, m->max_requests));
    int64_t per_launch = bound;
    char *ws = nullptr;
    if (f.n_seg > 1) {
        if (!workspace || !aligned(workspace, 16) || workspace_bytes < kWsSlack + f.unit_bytes)
            return fail(GDN_ERR_WORKSPACE, "workspace needs at least %zu bytes (16-byte aligned), got %zu",
                        kWsSlack + f.unit_bytes, workspace ? workspace_bytes : (size_t)0);
        ws = reinterpret_cast<char *>((reinterpret_cast<uintptr_t>(workspace) + 255) & ~uintptr_t(255));
        per_launch = std::min<int64_t>(bound, (int64_t)((workspace_bytes - kWsSlack) / f.unit_bytes));
    }
    gdn::KvAttn a = {};
    a.q = q; a.k_new = k; a.v_new = v; a.out = out;
    a.c = device_cache(c);
    a.units = m->units; a.counts = m->counts;
    a.n_rows = n_rows;
    a.Hq = d->n_q_heads; a.Hkv = d->n_kv_heads; a.G = a.Hq / a.Hkv;
    a.scale_log2 = (float)((double)d->scale * 1.4426950408889634);
    a.seg_blocks = f.seg_blocks; a.n_seg = (int)f.n_seg;
    a.max_new = max_new; a.max_len = (int)max_len; a.tok_stride = f.tok_stride;
    a.wait_limit = g_wait_limit;
    a.skip_first_copy = g_skip_first_copy;
    cudaError_t e = gdn_device_error_word(&a.err);
    if (e != cudaSuccess) return cuda_fail(e, "device error word lookup");
    cudaStream_t cst = (cudaStream_t)stream;
    const bool bf16 = d->in_dtype == GDN_BF16;
    for (int64_t u0 = 0; u0 < bound; u0 += per_launch) {
        const int n = (int)std::min(per_launch, bound - u0);
        a.unit0 = (int)u0;
        a.part_rows = (int64_t)n * f.tok_stride * a.Hq;
        if (ws) {
            a.part_ml = reinterpret_cast<float2 *>(ws);
            a.part_o = reinterpret_cast<float *>(ws + (((size_t)f.n_seg * a.part_rows * sizeof(float2) + 255) & ~size_t(255)));
        }
        e = launch_k(K_KV_ATTN, cst, [&] {
            if (!bf16) return gdn_launch_kv_attn_simt(a, d->head_dim, n, f.rows_max, f.few, cst);
            return f.few ? gdn_launch_kv_attn_token(a, d->head_dim, n, f.rows_max, cst)
                         : gdn_launch_kv_attn_prompt(a, d->head_dim, n, cst);
        });
        if (e != cudaSuccess) return cuda_fail(e, "attention kernel");
        if (f.n_seg > 1) {
            e = launch_k(K_KV_JOIN, cst, [&] { return gdn_launch_kv_join(a, d->head_dim, bf16, n, f.few, cst); });
            if (e != cudaSuccess) return cuda_fail(e, "attention join kernel");
        }
    }
    return GDN_OK;
}

GDN_API gdn_status gdn_kv_fork(const gdn_attn_desc *d, const gdn_kv_cache *c, int32_t src, int32_t dst, gdn_stream_t stream) {
    gdn_status st = check_attn(d);
    if (st != GDN_OK || (st = check_cache(c, true, true)) != GDN_OK) return st;
    if (src < 0 || src >= c->n_slots || dst < 0 || dst >= c->n_slots || src == dst)
        return fail(GDN_ERR_INVALID_ARG, "src and dst must be two slots in [0, %d) (%d, %d)", c->n_slots, src, dst);
    cudaStream_t cst = (cudaStream_t)stream;
    const cudaError_t e = launch_k(K_KV_STATE, cst, [&] {
        return gdn_launch_kv_fork(device_cache(c), src, dst, d->n_kv_heads, d->head_dim, d->in_dtype == GDN_BF16 ? 2 : 4, cst);
    });
    return e != cudaSuccess ? cuda_fail(e, "fork kernel") : GDN_OK;
}

GDN_API gdn_status gdn_kv_release(const gdn_attn_desc *d, const gdn_kv_cache *c, int32_t slot, gdn_stream_t stream) {
    gdn_status st = check_attn(d);
    if (st != GDN_OK || (st = check_cache(c, true, false)) != GDN_OK) return st;
    if (slot < 0 || slot >= c->n_slots) return fail(GDN_ERR_INVALID_ARG, "slot must be in [0, %d) (got %d)", c->n_slots, slot);
    const cudaError_t e = launch_k(K_KV_STATE, (cudaStream_t)stream, [&] {
        return gdn_launch_kv_release(device_cache(c), slot, (cudaStream_t)stream);
    });
    return e != cudaSuccess ? cuda_fail(e, "release kernel") : GDN_OK;
}

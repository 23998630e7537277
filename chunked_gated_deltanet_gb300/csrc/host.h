// Host-side helpers shared by the C ABI's translation units: argument
// validation, the layer tag and the per-thread error message.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>
#include <vector>
#include "gdn.h"

#define GDN_API extern "C" __attribute__((visibility("default")))

namespace gdn_host {

// Records a printf-style message for gdn_last_error() on this host thread and returns st.
gdn_status fail(gdn_status st, const char *fmt, ...);
gdn_status cuda_fail(cudaError_t e, const char *what);
bool aligned16(const void *p);
int64_t channels(const gdn_layer_desc *d);          // conv channels: 2 Hk d_k + Hv d_v
size_t in_elt(const gdn_layer_desc *d);              // bytes per input element
gdn_status check_desc(const gdn_layer_desc *d);
uint64_t tag_of(const gdn_layer_desc *d);            // FNV-1a over the description (never 0)
gdn_status check_state(const gdn_layer_desc *d, const gdn_session *s, const char *what, bool need_present);

// Polls before a kernel's bounded wait gives up, and the test hook of gdn_debug_inject_wait_timeout.
extern long long g_wait_limit;
extern int g_skip_first_copy;

// ---- optional per-kernel event timing (gdn_timing_begin / gdn_timing_end) ----
enum Kind { K_PREP = 0, K_CONV = 1, K_STATE = 2, K_COPY = 3, K_DECODE = 4, K_GATES = 5, K_PREP_TAIL = 6, K_FUSED = 7,
            K_KV_PLAN = 8, K_KV_APPEND = 9, K_KV_STATE = 10, K_KV_ATTN = 11, K_KV_JOIN = 12, K_KV_GROUP = 13, K_ROPE = 14,
            K_KINDS = 15 };

struct Timing {
    bool on = false;
    int cap = 0, used = 0;
    std::vector<cudaEvent_t> ev;  // 2 per timed launch
    std::vector<int> kind;
    int64_t launches[K_KINDS] = {};
};
extern Timing g_timing;

// Runs the launch f, bracketed by an event pair on `st` while timing records.
template <class F>
cudaError_t launch_k(Kind k, cudaStream_t st, F &&f) {
    Timing &T = g_timing;
    if (!T.on) return f();
    T.launches[k]++;
    if (T.used >= T.cap) return f();
    cudaEvent_t a = T.ev[2 * T.used], b = T.ev[2 * T.used + 1];
    cudaError_t e = cudaEventRecord(a, st);
    if (e != cudaSuccess) return e;
    e = f();
    if (e != cudaSuccess) return e;
    e = cudaEventRecord(b, st);
    if (e == cudaSuccess) T.kind[T.used++] = k;
    return e;
}

}  // namespace gdn_host

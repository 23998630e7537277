// Slots forked or emptied in a batch, and the compaction of a page pool: launchers.
#pragma once

#include "kv.cuh"

constexpr int kKvMaxBatchSlots = 1 << 20;   // slots of a cache whose forks are batched: a bit each in shared memory

cudaError_t gdn_launch_kv_fork_batch(const gdn::KvCache &c, const int32_t *src, const int32_t *dst, int n, int Hkv, int d, int elt,
                                     unsigned *err, cudaStream_t st);

// The books after a compaction: the cache's own buffers or others.
struct KvBooksOut {
    int32_t *table, *refs, *free_pages, *n_free;
    int n_pages;
};
// lists: int32 [3][n_pages]; counts: {pages in use, status, pages moved}
cudaError_t gdn_launch_kv_compact(const gdn::KvCache &c, const KvBooksOut &o, int Hkv, int d, int32_t *lists, int32_t *counts,
                                  cudaStream_t st);

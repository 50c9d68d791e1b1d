// evict_internal.cuh -- arguments and launchers of the eviction (declared to
// callers in pfkv_evict.h).
#pragma once

#include "../../include/pfkv_evict.h"
#include "pfkv_internal.cuh"

namespace pfkv {

// One side's tables.
struct EvictTables {
    const int32_t *block_tables;
    long long bt_sb, bt_sh;
    const uint32_t *expected_tags;
    int max_pages;
};

struct EvictArgs {
    void *k_pages, *v_pages;
    float *k_scale, *v_scale;
    const uint32_t *page_tags;
    int num_pages, Hkv, B;
    EvictTables src, dst;
    const int32_t *seq_lens, *keep_lens;
    long long len_sb, len_sh;
    int keep_first, keep_last;
    const float *mass;
    long long mass_sb, mass_sh;
    int max_seq_len, max_keep;
    int32_t *new_lens;
    float *new_mass;
    long long nm_sb, nm_sh;
    int nm_len;
    int32_t *kept_out;      // the caller's, or null
    long long kept_sb, kept_sh;
    int2 *status;           // [B][Hkv] flag bits, and tokens kept (workspace)
    int32_t *kept;          // [B][Hkv][max_keep] old indices, in order (workspace)
    uint8_t *flags;
};

cudaError_t launch_evict(const EvictArgs &a, int D, bool fp8, int num_sms, cudaStream_t s);
cudaError_t preload_evict();

}  // namespace pfkv

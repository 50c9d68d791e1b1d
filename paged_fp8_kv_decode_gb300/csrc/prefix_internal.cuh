// prefix_internal.cuh -- arguments and launchers of the attention over shared
// prefixes (declared to callers in pfkv_prefix.h).
#pragma once

#include "../../include/pfkv_prefix.h"
#include "latent_internal.cuh"
#include "pfkv_internal.cuh"

namespace pfkv {

// One side's tables: those of the requests' own tokens, or of the prefixes.
struct PrefixTables {
    const int32_t *block_tables;
    long long bt_sb, bt_sh;
    const int32_t *seq_lens;
    long long len_sb, len_sh;
    const uint32_t *expected_tags;
    int max_pages, max_len;
    int count;              // requests, or prefixes
};

struct PrefixArgs {
    const void *k_pages, *v_pages;
    const float *k_scale, *v_scale;
    const uint32_t *page_tags;
    int num_pages, Hkv, G, B, kq;
    PrefixTables own, pre;  // count 0: none
    const int32_t *prefix_of;
    RowsArg q, out;
    float q_scale;          // sm_scale * log2(e): scores are kept in log2 units
    float *mass;
    long long mass_sb, mass_sh;
    uint8_t *flags;
    uint32_t *rflags;       // [B] flag bits (workspace)
};

cudaError_t launch_prefix(const PrefixArgs &a, int D, bool fp8, int num_sms, cudaStream_t s);
cudaError_t preload_prefix();

}  // namespace pfkv

// prefix_internal.cuh -- arguments and launchers of the attention over shared
// prefixes (declared to callers in pfkv_prefix.h).
#pragma once

#include "../../include/pfkv_prefix.h"
#include "latent_internal.cuh"
#include "pfkv_internal.cuh"

namespace pfkv {

constexpr int kPrefixTile = 128;   // tokens of a tile
constexpr int kPrefixBlock = 256;  // query rows of a segment, at most

// One side's tables: those of the requests' own tokens, or of the prefixes.
struct PrefixTables {
    const int32_t *block_tables;
    long long bt_sb, bt_sh;
    const int32_t *seq_lens;
    long long len_sb, len_sh;
    const uint32_t *expected_tags;
    int max_pages, max_len;
    int count;   // requests, or prefixes
    int htiles;  // check words a (row, head): ceil(max_pages / kValTile)
};

// What the plan kernel decides for the others (workspace).  A prefix's query rows are those of
// its requests in the order of the batch: row (position * kq + t) * G + g of kv head h.  A
// segment is a block of up to kPrefixBlock of them against the head's tokens.  The segments'
// tiles of kPrefixTile tokens are numbered through, and CTA c of W takes the tiles
// [ceil(c U / W), ceil((c + 1) U / W)) of all U; each leaves a partial result for every segment it
// touches.
struct PrefixHead {
    uint32_t timeout;  // PFKV_FLAG_DEVICE_TIMEOUT once a wait has given up
};
struct PrefixSeg {
    int p, h, row0, rows;
    int tile0, ntiles;  // its first tile's number, and how many
    int base;           // first row of its partial results: rows8 for each CTA that touches it
    int len;            // tokens
    int first, ctas;    // the first CTA that touches it, and how many do
    int pad[2];
};
static_assert(sizeof(PrefixSeg) == 48, "three 16-byte loads");
// Where a request's partial results are.
struct PrefixPlace {
    int row;   // first of its query rows among those of its prefix; -1: no prefix
    int seg;   // the prefix's first segment
    int nb;    // blocks of rows of a head
    int pad;
};
// A CTA's tiles x0 .. x1 - 1, and the segment of the first.
struct PrefixRange {
    int x0, x1, seg, pad;
};

__host__ __device__ inline int rows8(int rows) { return (rows + 7) & ~7; }

struct PrefixArgs {
    const void *k_pages, *v_pages;
    const float *k_scale, *v_scale;
    const uint32_t *page_tags;
    int num_pages, Hkv, G, B, kq;
    PrefixTables own, pre;  // count 0: none
    const int32_t *prefix_of;
    RowsArg q, out;
    float sm_scale;
    uint8_t *flags;
    uint8_t *rflags;                // the same for the mass pass, or null
    // workspace
    uint32_t *own_bits, *pre_bits;  // [count][Hkv][htiles] check bits
    float *pre_vmax;                // [prefixes][Hkv][htiles] largest |V scale| of the tile's pages
    PrefixHead *head;
    PrefixPlace *place;             // [B]
    int *pos, *members;             // [B] position among its prefix's requests (-1: none); requests by prefix
    int *mstart, *seg0;             // [prefixes + 1] first entry of members; first segment
    int2 *pair;                     // [prefixes][Hkv] first tile and length
    PrefixSeg *seg;
    PrefixRange *range;             // [ctas]
    float *po, *plse;               // partial results: [D / 4][rows8][4] and [rows8] a (segment, CTA)
    __nv_bfloat16 *packed_q;        // queries as the split kernel takes them, or null: they are so already
    int ctas;                       // of the attention kernel
    int tries;                      // of a wait in it
    int after_own;                  // the kernel before it is the own tokens' split kernel
};

// The split kernel's partial results of the requests' own tokens (null status: none), in groups of
// requests as its launches take them.
struct PrefixOwnRows {
    const uint32_t *status;
    const float *lse, *o;
    size_t group_bytes;  // from one group's arrays to the next's
    int *units;          // [groups][greq * kq * Hkv + 1] first unit of every segment (by the plan)
    int greq, workers, chunk_tokens;
    float *lse_fin;      // for the mass pass, or null
};

cudaError_t launch_prefix_plan(const PrefixArgs &a, const PrefixOwnRows &o, int D, bool fp8, cudaStream_t s);
cudaError_t launch_prefix_attn(const PrefixArgs &a, int D, bool fp8, cudaStream_t s);
cudaError_t launch_prefix_merge(const PrefixArgs &a, const PrefixOwnRows &o, int D, cudaStream_t s);
cudaError_t preload_prefix();
cudaError_t preload_prefix_attn();

}  // namespace pfkv

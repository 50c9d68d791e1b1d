// latent.cu -- the paged latent cache (declared in pfkv_latent.h): argument
// checks of its calls, and pfkv_latent_gather, which reads cached tokens out of
// their pages as contiguous rows.
#include <cmath>

#include "latent_internal.cuh"

namespace pfkv {

pfkv_status check_latent(const pfkv_latent_cache *c, const pfkv_pages *p) {
    if (!c) return PFKV_ERR_INVALID_ARG;
    if (c->page_size != kPage || c->latent_dim != PFKV_LATENT_DIM || c->rope_dim != PFKV_LATENT_ROPE)
        return PFKV_ERR_UNSUPPORTED;
    if (c->dtype != PFKV_KV_BF16 && c->dtype != PFKV_KV_FP8_E4M3) return PFKV_ERR_INVALID_ARG;
    if (c->num_pages <= 0 || !c->c_pages || !c->r_pages) return PFKV_ERR_INVALID_ARG;
    if (c->dtype == PFKV_KV_FP8_E4M3 && !c->c_scale) return PFKV_ERR_INVALID_ARG;
    if (!aligned(c->c_pages, 16) || !aligned(c->r_pages, 16)) return PFKV_ERR_ALIGNMENT;
    if (c->dtype == PFKV_KV_FP8_E4M3 && !aligned(c->c_scale, 4)) return PFKV_ERR_ALIGNMENT;
    if (c->page_tags && !aligned(c->page_tags, 4)) return PFKV_ERR_ALIGNMENT;
    pfkv_cache tags{};  // the table checks look at the tags alone
    tags.page_tags = c->page_tags;
    const pfkv_status st = check_pages(&tags, p);
    if (st != PFKV_OK) return st;
    if (p->batch > 0 && (p->bt_stride_h != 0 || p->len_stride_h != 0)) return PFKV_ERR_INVALID_ARG;
    return PFKV_OK;
}

LatentPool latent_pool(const pfkv_latent_cache *c, const pfkv_pages *p) {
    LatentPool a{};
    a.c_pages = c->c_pages;
    a.r_pages = static_cast<__nv_bfloat16 *>(c->r_pages);
    a.c_scale = c->c_scale;
    a.page_tags = c->page_tags;
    a.num_pages = c->num_pages;
    a.fp8 = c->dtype == PFKV_KV_FP8_E4M3;
    a.block_tables = p->block_tables;
    a.bt_sb = p->bt_stride_b;
    a.expected_tags = p->expected_tags;
    a.max_pages = p->max_pages;
    a.seq_lens = p->seq_lens;
    a.len_sb = p->len_stride_b;
    return a;
}

namespace {

// --------------------------------------------------------------------------
// Gather: a CTA takes one page of one request.  Every thread loads its 16-byte
// words of the page before it stores any: it is bound by memory (153 MB of FP8 pages
// and bf16 rows in 25 us, 6.1 TB/s, 89% of a copy).
// --------------------------------------------------------------------------
constexpr int kGatherThreads = 256;

struct GatherArgs {
    LatentPool pool;
    const int32_t *row_starts;
    long long total_rows, c_stride, r_stride;
    __nv_bfloat16 *c_out, *r_out;
    uint8_t *flags;
    int max_seq_len, tiles;
};

__device__ __forceinline__ uint32_t bf16_pair(float lo, float hi) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&h);
}

template <bool FP8>
__global__ void __launch_bounds__(kGatherThreads) latent_gather_kernel(GatherArgs a) {
    pdl_enter();
    const int b = blockIdx.x / a.tiles, k = blockIdx.x - b * a.tiles;
    const int n = a.pool.seq_lens[(long long)b * a.pool.len_sb];
    const int lo = a.row_starts[b], hi = a.row_starts[b + 1];
    const bool bad = n < 0 || (long long)n > (long long)a.pool.max_pages * kPage || n > a.max_seq_len || lo < 0 ||
                     (long long)lo + n > hi || hi > a.total_rows;
    if (bad) {
        if (k == 0 && threadIdx.x == 0 && a.flags) atomic_or_byte(a.flags, b, PFKV_FLAG_BAD_LENGTH);
        return;
    }
    const int cnt = min(kPage, n - k * kPage);
    if (cnt <= 0) return;
    const long long bi = (long long)b * a.pool.bt_sb + k;
    const int phys = a.pool.block_tables[bi];
    const uint32_t bits = latent_entry_bits(a.pool, phys, bi);
    if (bits && threadIdx.x == 0 && a.flags) atomic_or_byte(a.flags, b, bits);
    const long long row0 = (long long)lo + (long long)k * kPage;
    const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
    constexpr int WORDS = PFKV_LATENT_DIM / 8;                  // 16-byte words of an output row
    constexpr int PER = kPage * WORDS / kGatherThreads;
    uint4 w[PER];
    float scale = 1.f;
    if (FP8 && !bits) scale = a.pool.c_scale[phys];
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int e = threadIdx.x + i * kGatherThreads, r = e / WORDS;
        w[i] = zero;
        if (bits || r >= cnt) continue;
        if constexpr (FP8) {
            const uint2 v = reinterpret_cast<const uint2 *>(a.pool.c_pages)[(long long)phys * kPage * WORDS + e];
            w[i].x = v.x;
            w[i].y = v.y;
        } else {
            w[i] = reinterpret_cast<const uint4 *>(a.pool.c_pages)[(long long)phys * kPage * WORDS + e];
        }
    }
    constexpr int RWORDS = PFKV_LATENT_ROPE / 8;
    uint4 rw = zero;
    const int rr = threadIdx.x / RWORDS;
    if (rr < cnt && !bits)
        rw = reinterpret_cast<const uint4 *>(a.pool.r_pages)[(long long)phys * kPage * RWORDS + threadIdx.x];
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int e = threadIdx.x + i * kGatherThreads, r = e / WORDS;
        if (r >= cnt) continue;
        if constexpr (FP8) {
            const uint32_t in[2] = {w[i].x, w[i].y};
            uint32_t o[4];
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const float2 f = e4m3x2_to_float2((uint16_t)(in[u >> 1] >> (16 * (u & 1))));
                o[u] = bf16_pair(f.x * scale, f.y * scale);
            }
            w[i] = make_uint4(o[0], o[1], o[2], o[3]);
        }
        reinterpret_cast<uint4 *>(a.c_out + (row0 + r) * a.c_stride)[e % WORDS] = w[i];
    }
    if (rr < cnt) reinterpret_cast<uint4 *>(a.r_out + (row0 + rr) * a.r_stride)[threadIdx.x % RWORDS] = rw;
}

// Checks that the two attention calls share.
pfkv_status check_decode(const pfkv_latent_cache *cache, const pfkv_pages *pages, int32_t num_q_heads,
                         int32_t num_query_tokens, int32_t max_seq_len) {
    const pfkv_status st = check_latent(cache, pages);
    if (st != PFKV_OK) return st;
    if (num_q_heads <= 0 || num_query_tokens <= 0 || max_seq_len < 0) return PFKV_ERR_INVALID_ARG;
    const long long rows = (long long)num_q_heads * num_query_tokens;
    if (rows > (1 << 20) || rows * pages->batch > 0x7fffffffLL) return PFKV_ERR_UNSUPPORTED;
    return PFKV_OK;
}

}  // namespace

cudaError_t preload_latent() {
    const cudaError_t e = preload_kernel(latent_gather_kernel<true>);
    return e == cudaSuccess ? preload_kernel(latent_gather_kernel<false>) : e;
}

}  // namespace pfkv

using namespace pfkv;

extern "C" {

pfkv_status pfkv_latent_gather(const pfkv_latent_cache *cache, const pfkv_pages *pages, const int32_t *row_starts,
                               int64_t total_rows, int32_t max_seq_len, void *c_out, int64_t c_stride, void *r_out,
                               int64_t r_stride, uint8_t *flags, void *stream) {
    pfkv_status st = check_latent(cache, pages);
    if (st != PFKV_OK) return st;
    if (max_seq_len < 0 || total_rows < 0) return PFKV_ERR_INVALID_ARG;
    if (pages->batch == 0 || max_seq_len == 0) return PFKV_OK;
    if (!row_starts) return PFKV_ERR_INVALID_ARG;
    if (!aligned(row_starts, 4)) return PFKV_ERR_ALIGNMENT;
    if (total_rows > 0) {
        if (!c_out || !r_out) return PFKV_ERR_INVALID_ARG;
        if (c_stride < PFKV_LATENT_DIM || r_stride < PFKV_LATENT_ROPE) return PFKV_ERR_INVALID_ARG;
        if (!aligned(c_out, 16) || !aligned(r_out, 16) || ((c_stride | r_stride) & 7)) return PFKV_ERR_ALIGNMENT;
    }
    if (flags && !aligned(flags, 4)) return PFKV_ERR_ALIGNMENT;
    const long long tiles = ((long long)max_seq_len + kPage - 1) / kPage;
    if (tiles * pages->batch > 0x7fffffffLL) return PFKV_ERR_UNSUPPORTED;
    st = device_check(nullptr);
    if (st != PFKV_OK) return st;
    GatherArgs a{};
    a.pool = latent_pool(cache, pages);
    a.row_starts = row_starts;
    a.total_rows = total_rows;
    a.c_stride = c_stride;
    a.r_stride = r_stride;
    a.c_out = static_cast<__nv_bfloat16 *>(c_out);
    a.r_out = static_cast<__nv_bfloat16 *>(r_out);
    a.flags = flags;
    a.max_seq_len = max_seq_len;
    a.tiles = (int)tiles;
    const dim3 g((unsigned)(tiles * pages->batch));
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    const cudaError_t e = a.pool.fp8 ? launch_pdl(latent_gather_kernel<true>, g, dim3(kGatherThreads), 0, s, a)
                                     : launch_pdl(latent_gather_kernel<false>, g, dim3(kGatherThreads), 0, s, a);
    return e == cudaSuccess ? PFKV_OK : PFKV_ERR_CUDA;
}

pfkv_status pfkv_latent_decode_workspace_size(const pfkv_latent_cache *cache, const pfkv_pages *pages,
                                              int32_t num_q_heads, int32_t num_query_tokens, int32_t max_seq_len,
                                              size_t *bytes) {
    if (!bytes) return PFKV_ERR_INVALID_ARG;
    pfkv_status st = check_decode(cache, pages, num_q_heads, num_query_tokens, max_seq_len);
    if (st != PFKV_OK) return st;
    int sms = 0;
    st = device_check(&sms);
    if (st != PFKV_OK) return st;
    *bytes = latent_decode_workspace(pages->batch, num_q_heads, num_query_tokens, max_seq_len, sms);
    return PFKV_OK;
}

pfkv_status pfkv_latent_decode_attn(const pfkv_latent_cache *cache, const pfkv_pages *pages, const pfkv_rows *q_c,
                                    const pfkv_rows *q_r, int32_t num_q_heads, int32_t num_query_tokens,
                                    float sm_scale, int32_t max_seq_len, void *workspace, size_t workspace_bytes,
                                    const pfkv_rows *out, uint8_t *flags, void *stream) {
    return pfkv_selftest_latent_decode(kTries, cache, pages, q_c, q_r, num_q_heads, num_query_tokens, sm_scale,
                                       max_seq_len, workspace, workspace_bytes, out, flags, stream);
}

pfkv_status pfkv_selftest_latent_decode(int32_t tries, const pfkv_latent_cache *cache, const pfkv_pages *pages,
                                        const pfkv_rows *q_c, const pfkv_rows *q_r, int32_t num_q_heads,
                                        int32_t num_query_tokens, float sm_scale, int32_t max_seq_len, void *workspace,
                                        size_t workspace_bytes, const pfkv_rows *out, uint8_t *flags, void *stream) {
    if (tries < 0 || tries > kTries) return PFKV_ERR_INVALID_ARG;
    pfkv_status st = check_decode(cache, pages, num_q_heads, num_query_tokens, max_seq_len);
    if (st != PFKV_OK) return st;
    if (!std::isfinite(sm_scale)) return PFKV_ERR_INVALID_ARG;
    if (pages->batch == 0) return PFKV_OK;
    st = check_rows(q_c, true, true);
    if (st == PFKV_OK) st = check_rows(q_r, true, true);
    if (st == PFKV_OK) st = check_rows(out, true, true);
    if (st != PFKV_OK) return st;
    if (flags && !aligned(flags, 4)) return PFKV_ERR_ALIGNMENT;
    if (!workspace) return PFKV_ERR_WORKSPACE;
    if (!aligned(workspace, 256)) return PFKV_ERR_ALIGNMENT;
    int sms = 0;
    st = device_check(&sms);
    if (st != PFKV_OK) return st;
    if (workspace_bytes < latent_decode_workspace(pages->batch, num_q_heads, num_query_tokens, max_seq_len, sms))
        return PFKV_ERR_WORKSPACE;
    LatentDecodeArgs a{};
    a.pool = latent_pool(cache, pages);
    a.qc = rows_arg(q_c);
    a.qr = rows_arg(q_r);
    a.out = rows_arg(out);
    a.flags = flags;
    a.B = pages->batch;
    a.H = num_q_heads;
    a.kq = num_query_tokens;
    a.max_seq_len = max_seq_len;
    a.sm_scale = sm_scale;
    a.workspace = workspace;
    a.tries = tries;
    return launch_latent_decode(a, sms, static_cast<cudaStream_t>(stream)) == cudaSuccess ? PFKV_OK : PFKV_ERR_CUDA;
}

pfkv_status pfkv_latent_prefill_attn(int32_t batch, int32_t num_heads, const int32_t *q_starts,
                                     const int32_t *k_starts, int64_t total_q, int64_t total_k, int32_t max_q_len,
                                     const pfkv_rows *q_nope, const pfkv_rows *q_rope, const pfkv_rows *k_nope,
                                     const pfkv_rows *k_rope, const pfkv_rows *v, float sm_scale, int32_t causal,
                                     const pfkv_rows *out, uint8_t *flags, void *stream) {
    return pfkv_selftest_latent_prefill(kTries, batch, num_heads, q_starts, k_starts, total_q, total_k, max_q_len,
                                        q_nope, q_rope, k_nope, k_rope, v, sm_scale, causal, out, flags, stream);
}

pfkv_status pfkv_selftest_latent_prefill(int32_t tries, int32_t batch, int32_t num_heads, const int32_t *q_starts,
                                         const int32_t *k_starts, int64_t total_q, int64_t total_k, int32_t max_q_len,
                                         const pfkv_rows *q_nope, const pfkv_rows *q_rope, const pfkv_rows *k_nope,
                                         const pfkv_rows *k_rope, const pfkv_rows *v, float sm_scale, int32_t causal,
                                         const pfkv_rows *out, uint8_t *flags, void *stream) {
    if (tries < 0 || tries > kTries) return PFKV_ERR_INVALID_ARG;
    if (batch < 0 || num_heads <= 0 || total_q < 0 || total_k < 0 || max_q_len < 0) return PFKV_ERR_INVALID_ARG;
    if (!std::isfinite(sm_scale)) return PFKV_ERR_INVALID_ARG;
    if (batch == 0) return PFKV_OK;
    if (total_q > 0x7fffffffLL || total_k > 0x7fffffffLL || num_heads > 65535) return PFKV_ERR_UNSUPPORTED;
    if (!q_starts || !k_starts) return PFKV_ERR_INVALID_ARG;
    if (!aligned(q_starts, 4) || !aligned(k_starts, 4)) return PFKV_ERR_ALIGNMENT;
    if (flags && !aligned(flags, 4)) return PFKV_ERR_ALIGNMENT;
    // arrays without rows are not read; rows that share an address cannot be copied as a box
    auto check = [](const pfkv_rows *r, bool use_h, int64_t rows) {
        const pfkv_status st = check_rows(r, false, use_h, rows);
        return st == PFKV_OK && rows > 1 && r->stride_t == 0 ? PFKV_ERR_UNSUPPORTED : st;
    };
    pfkv_status st = check(q_nope, true, total_q);
    if (st == PFKV_OK) st = check(q_rope, true, total_q);
    if (st == PFKV_OK) st = check(out, true, total_q);
    if (st == PFKV_OK) st = check(k_nope, true, total_k);
    if (st == PFKV_OK) st = check(k_rope, false, total_k);
    if (st == PFKV_OK) st = check(v, true, total_k);
    if (st != PFKV_OK) return st;
    int sms = 0;
    st = device_check(&sms);
    if (st != PFKV_OK) return st;
    LatentPrefillArgs a{};
    a.qn = rows_arg(q_nope);
    a.qr = rows_arg(q_rope);
    a.kn = rows_arg(k_nope);
    a.kr = rows_arg(k_rope);
    a.v = rows_arg(v);
    a.out = rows_arg(out);
    a.q_starts = q_starts;
    a.k_starts = k_starts;
    a.total_q = total_q;
    a.total_k = total_k;
    a.flags = flags;
    a.B = batch;
    a.H = num_heads;
    a.max_q_len = max_q_len;
    a.causal = causal != 0;
    a.sm_scale = sm_scale;
    a.tries = tries;
    return launch_latent_prefill(a, sms, static_cast<cudaStream_t>(stream)) == cudaSuccess ? PFKV_OK : PFKV_ERR_CUDA;
}

}  // extern "C"

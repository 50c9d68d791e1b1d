// prefix.cu -- pfkv_prefix_decode_attn: attention of a batch whose requests share
// prefixes (declared in pfkv_prefix.h).
//
// The plainest form: one launch checks every request's lengths and table entries, a
// second attends, a CTA a (query token, kv head), over the prefix's and the request's
// own tokens with a running maximum and sum a warp.
#include <cmath>

#include "prefix_internal.cuh"

namespace pfkv {
namespace {

constexpr int kCheckThreads = 256, kAttnWarps = 4;

// Tokens of row i for head h; -1 where a bound does not hold.
__device__ __forceinline__ int table_len(const PrefixTables &t, int i, int h) {
    const int n = t.seq_lens[(long long)i * t.len_sb + (long long)h * t.len_sh];
    return n < 0 || n > t.max_len || (long long)n > (long long)t.max_pages * kPage ? -1 : n;
}

__device__ uint32_t table_bits(const PrefixArgs &a, const PrefixTables &t, int i) {
    uint32_t bits = 0u;
    for (int h = 0; h < a.Hkv; ++h) {
        const int n = table_len(t, i, h);
        if (n < 0) bits |= PFKV_FLAG_BAD_LENGTH;
        for (int p = threadIdx.x; p < (n + kPage - 1) / kPage; p += blockDim.x) {
            const long long e = (long long)i * t.bt_sb + (long long)h * t.bt_sh + p;
            const int id = t.block_tables[e];
            if (id < 0 || id >= a.num_pages) bits |= PFKV_FLAG_BAD_PAGE;
            else if (a.page_tags && a.page_tags[(long long)id * a.Hkv + h] != t.expected_tags[e]) bits |= PFKV_FLAG_TAG_MISMATCH;
        }
    }
    return bits;
}

__global__ void __launch_bounds__(kCheckThreads) prefix_check_kernel(PrefixArgs a) {
    pdl_enter();
    const int b = blockIdx.x, p = a.prefix_of[b];
    uint32_t bits = 0u;
    if (p < -1 || p >= a.pre.count) bits = PFKV_FLAG_BAD_PAGE;
    else if (p >= 0) bits = table_bits(a, a.pre, p);
    if (a.own.count > 0) bits |= table_bits(a, a.own, b);
    uint32_t all = 0u;
    for (const uint32_t f : {PFKV_FLAG_BAD_LENGTH, PFKV_FLAG_BAD_PAGE, PFKV_FLAG_TAG_MISMATCH})
        if (__syncthreads_or((bits & f) != 0u)) all |= f;
    if (threadIdx.x == 0) {
        a.rflags[b] = all;
        if (a.flags) a.flags[b] = (uint8_t)all;
    }
}

template <int D, bool FP8>
__device__ __forceinline__ void row_values(const void *pool, long long row, float scale, float (&x)[D / 32]) {
    const int lane = threadIdx.x & 31;
    if constexpr (FP8) {
        const uint8_t *p = static_cast<const uint8_t *>(pool) + row * D + lane * (D / 32);
#pragma unroll
        for (int i = 0; i < D / 32; i += 2) {
            const float2 v = e4m3x2_to_float2(*reinterpret_cast<const uint16_t *>(p + i));
            x[i] = v.x * scale;
            x[i + 1] = v.y * scale;
        }
    } else {
        const __nv_bfloat16 *p = static_cast<const __nv_bfloat16 *>(pool) + row * D + lane * (D / 32);
#pragma unroll
        for (int i = 0; i < D / 32; i += 2) {
            const float2 v = bf16x2_to_float2(*reinterpret_cast<const uint32_t *>(p + i));
            x[i] = v.x;
            x[i + 1] = v.y;
        }
    }
}

template <int D, bool FP8, int G>
__global__ void __launch_bounds__(kAttnWarps * 32) prefix_plain_kernel(PrefixArgs a) {
    pdl_enter();
    constexpr int V = D / 32;
    __shared__ float s_m[kAttnWarps][G], s_l[kAttnWarps][G], s_o[kAttnWarps][G][D];
    const int v = blockIdx.x, h = blockIdx.y, b = v / a.kq, t = v - b * a.kq;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const long long to = (long long)b * a.out.sb + (long long)t * a.out.st;
    if (a.rflags[b]) {
        for (int i = threadIdx.x; i < G * D; i += kAttnWarps * 32)
            a.out.p[to + (long long)(h * G + i / D) * a.out.sh + i % D] = __float2bfloat16(0.f);
        return;
    }
    float q[G][V], o[G][V], m[G], l[G];
#pragma unroll
    for (int g = 0; g < G; ++g) {
        const __nv_bfloat16 *src = a.q.p + (long long)b * a.q.sb + (long long)t * a.q.st + (long long)(h * G + g) * a.q.sh;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            q[g][i] = __bfloat162float(src[lane * V + i]) * a.q_scale;
            o[g][i] = 0.f;
        }
        m[g] = -INFINITY;
        l[g] = 0.f;
    }
    // the score of one token of a unit for head g, in every lane
    auto score = [&](const float (&k)[V], int g) {
        float s = 0.f;
#pragma unroll
        for (int i = 0; i < V; ++i) s = fmaf(q[g][i], k[i], s);
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
        return s;
    };
    const int p = a.prefix_of[b];
    const int seen = a.own.count > 0 ? max(0, table_len(a.own, b, h) - a.kq + 1 + t) : 0;
    for (int part = 0; part < 2; ++part) {
        const PrefixTables &tab = part ? a.own : a.pre;
        const int row = part ? b : p, n = part ? seen : p >= 0 ? table_len(a.pre, p, h) : 0;
        for (int page = warp; page < (n + kPage - 1) / kPage; page += kAttnWarps) {
            const int id = tab.block_tables[(long long)row * tab.bt_sb + (long long)h * tab.bt_sh + page];
            const long long unit = (long long)id * a.Hkv + h;
            const float ks = FP8 ? a.k_scale[unit] : 1.f, vs = FP8 ? a.v_scale[unit] : 1.f;
            for (int j = 0; j < min(kPage, n - page * kPage); ++j) {
                float k[V], x[V];
                row_values<D, FP8>(a.k_pages, unit * kPage + j, ks, k);
                row_values<D, FP8>(a.v_pages, unit * kPage + j, vs, x);
#pragma unroll
                for (int g = 0; g < G; ++g) {
                    const float s = score(k, g);
                    const float top = fmaxf(m[g], s), down = m[g] == top ? 1.f : exp2f(m[g] - top), w = exp2f(s - top);
                    m[g] = top;
                    l[g] = l[g] * down + w;
#pragma unroll
                    for (int i = 0; i < V; ++i) o[g][i] = fmaf(w, x[i], o[g][i] * down);
                }
            }
        }
    }
#pragma unroll
    for (int g = 0; g < G; ++g) {
        if (lane == 0) {
            s_m[warp][g] = m[g];
            s_l[warp][g] = l[g];
        }
#pragma unroll
        for (int i = 0; i < V; ++i) s_o[warp][g][lane * V + i] = o[g][i];
    }
    __syncthreads();
    for (int i = threadIdx.x; i < G * D; i += kAttnWarps * 32) {
        const int g = i / D;
        float top = -INFINITY, sum = 0.f, x = 0.f;
        for (int w = 0; w < kAttnWarps; ++w) top = fmaxf(top, s_m[w][g]);
        for (int w = 0; w < kAttnWarps; ++w) {
            const float f = s_l[w][g] == 0.f ? 0.f : exp2f(s_m[w][g] - top);
            sum += f * s_l[w][g];
            x += f * s_o[w][g][i % D];
        }
        a.out.p[to + (long long)(h * G + g) * a.out.sh + i % D] = __float2bfloat16(sum == 0.f ? 0.f : x / sum);
    }
    if (!a.mass) return;
    float lse[G];
#pragma unroll
    for (int g = 0; g < G; ++g) {
        float top = -INFINITY, sum = 0.f;
        for (int w = 0; w < kAttnWarps; ++w) top = fmaxf(top, s_m[w][g]);
        for (int w = 0; w < kAttnWarps; ++w) sum += s_l[w][g] == 0.f ? 0.f : exp2f(s_m[w][g] - top) * s_l[w][g];
        lse[g] = top + log2f(sum);
    }
    float *mass = a.mass + (long long)b * a.mass_sb + (long long)h * a.mass_sh;
    for (int page = warp; page < (seen + kPage - 1) / kPage; page += kAttnWarps) {
        const int id = a.own.block_tables[(long long)b * a.own.bt_sb + (long long)h * a.own.bt_sh + page];
        const long long unit = (long long)id * a.Hkv + h;
        for (int j = 0; j < min(kPage, seen - page * kPage); ++j) {
            float k[V], sum = 0.f;
            row_values<D, FP8>(a.k_pages, unit * kPage + j, FP8 ? a.k_scale[unit] : 1.f, k);
#pragma unroll
            for (int g = 0; g < G; ++g) sum += exp2f(score(k, g) - lse[g]);
            if (lane == 0) mass[page * kPage + j] += sum;
        }
    }
}

template <int D, bool FP8>
cudaError_t launch_plain(const PrefixArgs &a, cudaStream_t s) {
    const dim3 grid((unsigned)(a.B * a.kq), (unsigned)a.Hkv), block(kAttnWarps * 32);
    switch (a.G) {
        case 1: return launch_pdl(prefix_plain_kernel<D, FP8, 1>, grid, block, 0, s, a);
        case 2: return launch_pdl(prefix_plain_kernel<D, FP8, 2>, grid, block, 0, s, a);
        case 4: return launch_pdl(prefix_plain_kernel<D, FP8, 4>, grid, block, 0, s, a);
        case 8: return launch_pdl(prefix_plain_kernel<D, FP8, 8>, grid, block, 0, s, a);
    }
    return cudaErrorInvalidValue;
}

}  // namespace

cudaError_t launch_prefix(const PrefixArgs &a, int D, bool fp8, int num_sms, cudaStream_t s) {
    const cudaError_t e = launch_pdl(prefix_check_kernel, dim3((unsigned)a.B), dim3(kCheckThreads), 0, s, a);
    if (e != cudaSuccess) return e;
    if (D == 128) return fp8 ? launch_plain<128, true>(a, s) : launch_plain<128, false>(a, s);
    return fp8 ? launch_plain<64, true>(a, s) : launch_plain<64, false>(a, s);
}

cudaError_t preload_prefix() { return preload_kernel(prefix_check_kernel); }

namespace {

size_t up256(size_t x) { return (x + 255) & ~size_t(255); }

struct PrefixSizes {
    size_t off_rflags, total;
};

// Arguments that size the workspace.
pfkv_status prefix_sizes(const pfkv_cache *cache, const pfkv_pages *pages, const pfkv_pages *prefixes, int32_t batch,
                         int32_t num_q_heads, int32_t kq, int32_t max_seq_len, int32_t max_prefix_len, bool mass,
                         PrefixSizes *z) {
    pfkv_status st = check_cache(cache);
    if (st != PFKV_OK) return st;
    if (batch < 0) return PFKV_ERR_INVALID_ARG;
    if (pages) {
        st = check_pages(cache, pages);
        if (st != PFKV_OK) return st;
        if (pages->batch != batch || max_seq_len < 0) return PFKV_ERR_INVALID_ARG;
    }
    if (!prefixes || prefixes->batch < 0 || max_prefix_len < 0) return PFKV_ERR_INVALID_ARG;
    if (prefixes->batch > 0) {
        st = check_pages(cache, prefixes);
        if (st != PFKV_OK) return st;
    }
    if (prefixes->batch > PFKV_PREFIX_MAX) return PFKV_ERR_UNSUPPORTED;
    if (num_q_heads <= 0 || num_q_heads % cache->num_kv_heads != 0 || kq < 1) return PFKV_ERR_INVALID_ARG;
    const int G = num_q_heads / cache->num_kv_heads;
    if (G != 1 && G != 2 && G != 4 && G != 8) return PFKV_ERR_UNSUPPORTED;
    if ((long long)kq * cache->num_kv_heads > kPersMaxSegments) return PFKV_ERR_UNSUPPORTED;
    if (mass && !pages) return PFKV_ERR_INVALID_ARG;
    if (mass && kq != 1) return PFKV_ERR_UNSUPPORTED;
    if ((long long)batch * kq > 0x7fffffffLL / num_q_heads) return PFKV_ERR_UNSUPPORTED;
    z->off_rflags = 0;
    z->total = up256(sizeof(uint32_t) * (size_t)batch);
    return PFKV_OK;
}

PrefixTables prefix_tables(const pfkv_pages *p, int max_len) {
    return PrefixTables{p->block_tables, (long long)p->bt_stride_b, (long long)p->bt_stride_h, p->seq_lens,
                        (long long)p->len_stride_b, (long long)p->len_stride_h, p->expected_tags, p->max_pages, max_len,
                        p->batch};
}

}  // namespace
}  // namespace pfkv

using namespace pfkv;

extern "C" {

pfkv_status pfkv_prefix_decode_workspace_size(const pfkv_cache *cache, const pfkv_pages *pages,
                                              const pfkv_pages *prefixes, int32_t batch, int32_t num_q_heads,
                                              int32_t num_query_tokens, int32_t max_seq_len, int32_t max_prefix_len,
                                              int32_t with_mass, size_t *bytes) {
    if (!bytes) return PFKV_ERR_INVALID_ARG;
    PrefixSizes z{};
    const pfkv_status st = prefix_sizes(cache, pages, prefixes, batch, num_q_heads, num_query_tokens, max_seq_len,
                                        max_prefix_len, with_mass != 0, &z);
    if (st != PFKV_OK) return st;
    *bytes = z.total;
    return PFKV_OK;
}

pfkv_status pfkv_prefix_decode_attn(const pfkv_cache *cache, const pfkv_pages *pages, const pfkv_pages *prefixes,
                                    int32_t batch, const int32_t *prefix_of, const pfkv_rows *q, int32_t num_q_heads,
                                    int32_t num_query_tokens, float sm_scale, int32_t max_seq_len,
                                    int32_t max_prefix_len, void *workspace, size_t workspace_bytes,
                                    const pfkv_rows *out, float *attn_mass, int64_t mass_stride_b,
                                    int64_t mass_stride_h, uint8_t *flags, void *stream) {
    PrefixSizes z{};
    pfkv_status st = prefix_sizes(cache, pages, prefixes, batch, num_q_heads, num_query_tokens, max_seq_len,
                                  max_prefix_len, attn_mass != nullptr, &z);
    if (st != PFKV_OK) return st;
    if (!(sm_scale == sm_scale) || std::isinf(sm_scale)) return PFKV_ERR_INVALID_ARG;
    if (batch == 0) return PFKV_OK;
    if (!prefix_of) return PFKV_ERR_INVALID_ARG;
    st = check_rows(q, true, true);
    if (st == PFKV_OK) st = check_rows(out, true, true);
    if (st != PFKV_OK) return st;
    if (attn_mass && (mass_stride_b < 0 || mass_stride_h < 0)) return PFKV_ERR_INVALID_ARG;
    if (!aligned(prefix_of, 4) || !aligned(attn_mass, 4) || !aligned(flags, 4)) return PFKV_ERR_ALIGNMENT;
    if (!workspace || workspace_bytes < z.total) return PFKV_ERR_WORKSPACE;
    if (!aligned(workspace, 256)) return PFKV_ERR_ALIGNMENT;
    int sms = 0;
    st = device_check(&sms);
    if (st != PFKV_OK) return st;

    PrefixArgs a{};
    a.k_pages = cache->k_pages;
    a.v_pages = cache->v_pages;
    a.k_scale = cache->k_scale;
    a.v_scale = cache->v_scale;
    a.page_tags = cache->page_tags;
    a.num_pages = cache->num_pages;
    a.Hkv = cache->num_kv_heads;
    a.G = num_q_heads / cache->num_kv_heads;
    a.B = batch;
    a.kq = num_query_tokens;
    if (pages) a.own = prefix_tables(pages, max_seq_len);
    a.pre = prefix_tables(prefixes, max_prefix_len);
    a.prefix_of = prefix_of;
    a.q = rows_arg(q);
    a.out = rows_arg(out);
    a.q_scale = sm_scale * 1.4426950408889634f;  // log2(e): scores in log2 units
    a.mass = attn_mass;
    a.mass_sb = mass_stride_b;
    a.mass_sh = mass_stride_h;
    a.flags = flags;
    a.rflags = reinterpret_cast<uint32_t *>(static_cast<uint8_t *>(workspace) + z.off_rflags);
    return launch_prefix(a, cache->head_dim, cache->dtype == PFKV_KV_FP8_E4M3, sms, static_cast<cudaStream_t>(stream)) ==
                   cudaSuccess
               ? PFKV_OK
               : PFKV_ERR_CUDA;
}

}  // extern "C"

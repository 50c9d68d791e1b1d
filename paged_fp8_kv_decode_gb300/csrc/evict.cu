// evict.cu -- pfkv_kv_evict: keep the tokens of every (request, kv head) that
// received most attention and move them, in order, to new pages (declared in
// pfkv_evict.h).
//
// Two launches.  The first checks lengths and table entries and selects: the m-th
// largest of the totals between the protected ends is found digit by digit (a
// radix selection on the totals' bits), and one ordered pass then writes the kept
// tokens' indices: larger ones all, equal ones from the lowest index on.  The
// second moves them, a warp a destination unit.
#include "evict_internal.cuh"
#include "latent_internal.cuh"

namespace pfkv {
namespace {

constexpr int kSelThreads = 512, kSelWarps = kSelThreads / 32;
constexpr int kSelItems = 8;  // a warp's groups of 32 tokens a round of the ordered pass
constexpr int kMoveWarps = 8;

// Order of totals as that of unsigned numbers: NaN above all, -0 as 0.
__device__ __forceinline__ uint32_t order_key(float x) {
    const uint32_t u = __float_as_uint(x);
    if ((u & 0x7fffffffu) > 0x7f800000u) return 0xffffffffu;
    if ((u << 1) == 0u) return 0x80000000u;
    return (u & 0x80000000u) ? ~u : u | 0x80000000u;
}

__device__ __forceinline__ uint32_t entry_check(const EvictArgs &a, const EvictTables &t, int b, int h, int p) {
    const long long i = (long long)b * t.bt_sb + (long long)h * t.bt_sh + p;
    const int id = t.block_tables[i];
    if (id < 0 || id >= a.num_pages) return PFKV_FLAG_BAD_PAGE;
    if (a.page_tags && a.page_tags[(long long)id * a.Hkv + h] != t.expected_tags[i]) return PFKV_FLAG_TAG_MISMATCH;
    return 0u;
}

// Tokens of (b, h) and how many are kept; false where a bound does not hold.
__device__ __forceinline__ bool lengths(const EvictArgs &a, int b, int h, int &n, int &k) {
    const long long i = (long long)b * a.len_sb + (long long)h * a.len_sh;
    n = a.seq_lens[i];
    const int keep = a.keep_lens[i];
    k = min(keep, n);
    return n >= 0 && keep >= 0 && n <= a.max_seq_len && (long long)n <= (long long)a.src.max_pages * kPage &&
           k <= a.max_keep && (long long)k <= (long long)a.dst.max_pages * kPage;
}

__global__ void __launch_bounds__(kSelThreads) evict_select_kernel(EvictArgs a) {
    pdl_enter();
    __shared__ int hist[256];
    __shared__ int sum_gt[kSelWarps], sum_eq[kSelWarps];
    __shared__ uint32_t s_prefix;
    __shared__ int s_need;
    const int bh = blockIdx.x, b = bh / a.Hkv, h = bh - b * a.Hkv;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    int n, k;
    uint32_t bits = lengths(a, b, h, n, k) ? 0u : PFKV_FLAG_BAD_LENGTH;
    if (!bits) {
        for (int p = tid; p < (n + kPage - 1) / kPage; p += kSelThreads) bits |= entry_check(a, a.src, b, h, p);
        for (int p = tid; p < (k + kPage - 1) / kPage; p += kSelThreads) bits |= entry_check(a, a.dst, b, h, p);
    }
    uint32_t all = 0u;
    for (const uint32_t f : {PFKV_FLAG_BAD_LENGTH, PFKV_FLAG_BAD_PAGE, PFKV_FLAG_TAG_MISMATCH})
        if (__syncthreads_or((bits & f) != 0u)) all |= f;
    if (tid == 0) a.status[bh] = make_int2((int)all, k);
    if (all) return;

    const int f = min(a.keep_first, k), l = min(a.keep_last, k - f), m = k - f - l;
    int32_t *kept = a.kept + (long long)b * a.kept_sb + (long long)h * a.kept_sh;
    for (int j = tid; j < f; j += kSelThreads) kept[j] = j;
    for (int j = tid; j < l; j += kSelThreads) kept[k - l + j] = n - l + j;
    if (m == 0) return;
    const int L = n - l - f;  // candidates
    const float *mass = a.mass + (long long)b * a.mass_sb + (long long)h * a.mass_sh + f;

    // the m-th largest key: digits of eight bits, from the top
    uint32_t prefix = 0u;
    int need = m;
    for (int shift = 24; shift >= 0; shift -= 8) {
        if (tid < 256) hist[tid] = 0;
        __syncthreads();
        const uint32_t above = shift == 24 ? 0u : 0xffffffffu << (shift + 8);
        for (int j = tid; j < L; j += kSelThreads) {
            const uint32_t u = order_key(mass[j]);
            if ((u & above) == prefix) atomicAdd(&hist[(u >> shift) & 255], 1);
        }
        __syncthreads();
        if (tid == 0) {
            int left = need, d = 255;
            while (hist[d] < left) left -= hist[d--];
            s_prefix = prefix | ((uint32_t)d << shift);
            s_need = left;
        }
        __syncthreads();
        prefix = s_prefix;
        need = s_need;
    }

    // the ordered pass: of keys equal to the m-th, the first `need`
    int base_gt = 0, base_eq = 0;
    for (int j0 = 0; j0 < L; j0 += kSelThreads * kSelItems) {
        uint32_t gt[kSelItems], eq[kSelItems];
        int ngt = 0, neq = 0;
#pragma unroll
        for (int i = 0; i < kSelItems; ++i) {
            const int j = j0 + (warp * kSelItems + i) * 32 + lane;
            const uint32_t u = j < L ? order_key(mass[j]) : 0u;
            gt[i] = __ballot_sync(0xffffffffu, j < L && u > prefix);
            eq[i] = __ballot_sync(0xffffffffu, j < L && u == prefix);
            ngt += __popc(gt[i]);
            neq += __popc(eq[i]);
        }
        __syncthreads();
        if (lane == 0) {
            sum_gt[warp] = ngt;
            sum_eq[warp] = neq;
        }
        __syncthreads();
        int at_gt = base_gt, at_eq = base_eq;
        for (int w = 0; w < kSelWarps; ++w) {
            if (w < warp) {
                at_gt += sum_gt[w];
                at_eq += sum_eq[w];
            }
            base_gt += sum_gt[w];
            base_eq += sum_eq[w];
        }
        const uint32_t below = (1u << lane) - 1u;
#pragma unroll
        for (int i = 0; i < kSelItems; ++i) {
            const int j = j0 + (warp * kSelItems + i) * 32 + lane;
            const int before_eq = at_eq + __popc(eq[i] & below);
            const int to = at_gt + __popc(gt[i] & below) + min(before_eq, need);
            if (((gt[i] >> lane) & 1u) || (((eq[i] >> lane) & 1u) && before_eq < need)) kept[f + to] = f + j;
            at_gt += __popc(gt[i]);
            at_eq += __popc(eq[i]);
        }
    }
}

// One of K and V of a destination unit: slots < live take the rows of `row` (token rows of the
// pool, in units of 16) of lanes 0 .. 15.
template <int D, bool FP8>
__device__ __forceinline__ void move_unit(void *pool, float *scales, long long row, long long to, int live, int lane) {
    constexpr int ROWB = D * (FP8 ? 1 : 2), LPR = ROWB / 16, RPP = 32 / LPR, PASSES = kPage / RPP;
    uint8_t *bytes = static_cast<uint8_t *>(pool);
    const int r0 = lane / LPR, c = lane % LPR;
    uint4 w[PASSES];
#pragma unroll
    for (int i = 0; i < PASSES; ++i) {
        const int r = i * RPP + r0;
        const long long from = __shfl_sync(0xffffffffu, row, r);
        w[i] = r < live ? *reinterpret_cast<const uint4 *>(bytes + from * ROWB + c * 16) : make_uint4(0u, 0u, 0u, 0u);
    }
    if constexpr (FP8) {
        const long long unit = row / kPage, first = __shfl_sync(0xffffffffu, unit, 0);
        const bool one = __all_sync(0xffffffffu, lane >= live || unit == first);
        const float mine = lane < live ? scales[unit] : 0.f;
        if (one) {
            if (lane == 0) scales[to] = mine;
        } else {
            float z[PASSES];
            float top = 0.f;
#pragma unroll
            for (int i = 0; i < PASSES; ++i) {
                z[i] = __shfl_sync(0xffffffffu, mine, i * RPP + r0);
                const uint32_t u[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const float2 x = e4m3x2_to_float2((uint16_t)(u[e >> 1] >> (16 * (e & 1))));
                    top = fmaxf(top, fmaxf(fabsf(x.x * z[i]), fabsf(x.y * z[i])));
                }
            }
#pragma unroll
            for (int off = 16; off > 0; off >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
            const float scale = top == 0.f ? 1.f : __fdiv_rn(top, 448.f);
            if (lane == 0) scales[to] = scale;
#pragma unroll
            for (int i = 0; i < PASSES; ++i) {
                uint32_t u[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    uint32_t o = 0u;
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const float2 x = e4m3x2_to_float2((uint16_t)(u[q] >> (16 * e)));
                        o |= (uint32_t)float_to_e4m3(__fdiv_rn(x.x * z[i], scale)) << (16 * e);
                        o |= (uint32_t)float_to_e4m3(__fdiv_rn(x.y * z[i], scale)) << (16 * e + 8);
                    }
                    u[q] = o;
                }
                w[i] = make_uint4(u[0], u[1], u[2], u[3]);
            }
        }
    }
#pragma unroll
    for (int i = 0; i < PASSES; ++i) {
        const int r = i * RPP + r0;
        if (r < live) *reinterpret_cast<uint4 *>(bytes + (to * kPage + r) * ROWB + c * 16) = w[i];
    }
}

template <int D, bool FP8>
__global__ void __launch_bounds__(kMoveWarps * 32) evict_move_kernel(EvictArgs a, int units) {
    pdl_enter();
    const long long x = (long long)blockIdx.x * kMoveWarps + (threadIdx.x >> 5);
    const int lane = threadIdx.x & 31;
    const long long bh = x / units;
    if (bh >= (long long)a.B * a.Hkv) return;
    const int u = (int)(x - bh * units), b = (int)(bh / a.Hkv), h = (int)(bh - (long long)b * a.Hkv);
    uint32_t bits = 0u;
    for (int i = lane; i < a.Hkv; i += 32) bits |= (uint32_t)a.status[(long long)b * a.Hkv + i].x;
    bits = __reduce_or_sync(0xffffffffu, bits);
    const int k = a.status[bh].y;
    if (u == 0 && lane == 0) {
        if (h == 0 || a.len_sh != 0) a.new_lens[(long long)b * a.len_sb + (long long)h * a.len_sh] = bits ? 0 : k;
        if (h == 0 && a.flags) a.flags[b] = (uint8_t)bits;
    }
    if (bits) return;
    const int j = u * kPage + (lane & 15), live = min(kPage, k - u * kPage);
    int from = 0;
    long long row = 0;
    if (lane < live) {
        from = a.kept[(long long)b * a.kept_sb + (long long)h * a.kept_sh + j];
        const int id = a.src.block_tables[(long long)b * a.src.bt_sb + (long long)h * a.src.bt_sh + from / kPage];
        row = ((long long)id * a.Hkv + h) * kPage + from % kPage;
    }
    if (a.new_mass && lane < kPage && j < a.nm_len)
        a.new_mass[(long long)b * a.nm_sb + (long long)h * a.nm_sh + j] =
            lane < live ? a.mass[(long long)b * a.mass_sb + (long long)h * a.mass_sh + from] : 0.f;
    if (live <= 0) return;
    const int id = a.dst.block_tables[(long long)b * a.dst.bt_sb + (long long)h * a.dst.bt_sh + u];
    const long long to = (long long)id * a.Hkv + h;
    move_unit<D, FP8>(a.k_pages, a.k_scale, row, to, live, lane);
    move_unit<D, FP8>(a.v_pages, a.v_scale, row, to, live, lane);
}

}  // namespace

cudaError_t launch_evict(const EvictArgs &a, int D, bool fp8, int num_sms, cudaStream_t s) {
    cudaError_t e = launch_pdl(evict_select_kernel, dim3((unsigned)(a.B * a.Hkv)), dim3(kSelThreads), 0, s, a);
    if (e != cudaSuccess) return e;
    const int units = max(1, (max(a.max_keep, a.new_mass ? a.nm_len : 0) + kPage - 1) / kPage);
    const long long ctas = ((long long)a.B * a.Hkv * units + kMoveWarps - 1) / kMoveWarps;
    const dim3 grid((unsigned)ctas), block(kMoveWarps * 32);
    auto *const kernel = D == 128 ? (fp8 ? evict_move_kernel<128, true> : evict_move_kernel<128, false>)
                                  : (fp8 ? evict_move_kernel<64, true> : evict_move_kernel<64, false>);
    return launch_pdl(kernel, grid, block, 0, s, a, units);
}

cudaError_t preload_evict() {
    cudaError_t e = preload_kernel(evict_select_kernel);
    for (auto *const kernel : {evict_move_kernel<128, true>, evict_move_kernel<128, false>, evict_move_kernel<64, true>,
                               evict_move_kernel<64, false>})
        if (e == cudaSuccess) e = preload_kernel(kernel);
    return e;
}

namespace {

size_t up256(size_t x) { return (x + 255) & ~size_t(255); }

// Arguments that size the workspace.
pfkv_status evict_sizes(const pfkv_cache *cache, const pfkv_pages *src, int32_t max_seq_len, int32_t max_keep_len,
                        size_t *status_bytes, size_t *total) {
    pfkv_status st = check_cache(cache);
    if (st != PFKV_OK) return st;
    st = check_pages(cache, src);
    if (st != PFKV_OK) return st;
    if (max_seq_len < 0 || max_keep_len < 0) return PFKV_ERR_INVALID_ARG;
    const long long bh = (long long)src->batch * cache->num_kv_heads;
    if (bh > 0x7fffffffLL) return PFKV_ERR_UNSUPPORTED;
    *status_bytes = up256(sizeof(int2) * (size_t)bh);
    *total = *status_bytes + up256(sizeof(int32_t) * (size_t)bh * (size_t)max_keep_len);
    return PFKV_OK;
}

}  // namespace
}  // namespace pfkv

using namespace pfkv;

extern "C" {

pfkv_status pfkv_kv_evict_workspace_size(const pfkv_cache *cache, const pfkv_pages *src, int32_t max_seq_len,
                                         int32_t max_keep_len, size_t *bytes) {
    if (!bytes) return PFKV_ERR_INVALID_ARG;
    size_t status_bytes = 0, total = 0;
    const pfkv_status st = evict_sizes(cache, src, max_seq_len, max_keep_len, &status_bytes, &total);
    if (st == PFKV_OK) *bytes = total;
    return st;
}

pfkv_status pfkv_kv_evict(const pfkv_cache *cache, const pfkv_pages *src, const pfkv_pages *dst,
                          const int32_t *keep_lens, int32_t keep_first, int32_t keep_last, const float *attn_mass,
                          int64_t mass_stride_b, int64_t mass_stride_h, int32_t max_seq_len, int32_t max_keep_len,
                          void *workspace, size_t workspace_bytes, int32_t *new_lens, float *new_mass,
                          int64_t new_mass_stride_b, int64_t new_mass_stride_h, int32_t new_mass_len, int32_t *kept,
                          int64_t kept_stride_b, int64_t kept_stride_h, uint8_t *flags, void *stream) {
    size_t status_bytes = 0, total = 0;
    pfkv_status st = evict_sizes(cache, src, max_seq_len, max_keep_len, &status_bytes, &total);
    if (st != PFKV_OK) return st;
    if (!dst || dst->batch != src->batch) return PFKV_ERR_INVALID_ARG;
    if (src->batch == 0) return PFKV_OK;
    pfkv_pages to = *dst;  // its lengths are not read
    to.seq_lens = src->seq_lens;
    to.len_stride_b = to.len_stride_h = 0;
    st = check_pages(cache, &to);
    if (st != PFKV_OK) return st;
    if (keep_first < 0 || keep_last < 0) return PFKV_ERR_INVALID_ARG;
    if (!keep_lens || !attn_mass || !new_lens) return PFKV_ERR_INVALID_ARG;
    if (mass_stride_b < 0 || mass_stride_h < 0) return PFKV_ERR_INVALID_ARG;
    if (new_mass && (new_mass_stride_b < 0 || new_mass_stride_h < 0 || new_mass_len < max_keep_len))
        return PFKV_ERR_INVALID_ARG;
    if (kept && (kept_stride_b < 0 || kept_stride_h < 0)) return PFKV_ERR_INVALID_ARG;
    // rows that results are written to, of max_keep_len or new_mass_len elements, must not overlap
    const auto apart = [&](int64_t sb, int64_t sh, int64_t len) {
        const int64_t B = src->batch, H = cache->num_kv_heads;
        if (len == 0) return true;
        if (B == 1) return H == 1 || sh >= len;
        if (H == 1) return sb >= len;
        return (sh >= len && (sb - len) / (H - 1) >= sh) || (sb >= len && (sh - len) / (B - 1) >= sb);
    };
    if (new_mass && !apart(new_mass_stride_b, new_mass_stride_h, new_mass_len)) return PFKV_ERR_INVALID_ARG;
    if (kept && !apart(kept_stride_b, kept_stride_h, max_keep_len)) return PFKV_ERR_INVALID_ARG;
    if (src->batch > 1 && src->len_stride_b == 0) return PFKV_ERR_INVALID_ARG;  // new_lens: one a request
    if (!aligned(keep_lens, 4) || !aligned(attn_mass, 4) || !aligned(new_lens, 4) || !aligned(new_mass, 4) ||
        !aligned(kept, 4) || (flags && !aligned(flags, 4)))
        return PFKV_ERR_ALIGNMENT;
    if (!workspace || workspace_bytes < total) return PFKV_ERR_WORKSPACE;
    if (!aligned(workspace, 256)) return PFKV_ERR_ALIGNMENT;
    const long long units = (max(max_keep_len, new_mass ? new_mass_len : 0) + 15LL) / kPage;
    if ((long long)src->batch * cache->num_kv_heads * units > 0x7fffffffLL) return PFKV_ERR_UNSUPPORTED;
    int sms = 0;
    st = device_check(&sms);
    if (st != PFKV_OK) return st;

    EvictArgs a{};
    a.k_pages = cache->k_pages;
    a.v_pages = cache->v_pages;
    a.k_scale = cache->k_scale;
    a.v_scale = cache->v_scale;
    a.page_tags = cache->page_tags;
    a.num_pages = cache->num_pages;
    a.Hkv = cache->num_kv_heads;
    a.B = src->batch;
    const auto tables = [](const pfkv_pages *p) {
        return EvictTables{p->block_tables, (long long)p->bt_stride_b, (long long)p->bt_stride_h, p->expected_tags,
                           p->max_pages};
    };
    a.src = tables(src);
    a.dst = tables(dst);
    a.seq_lens = src->seq_lens;
    a.keep_lens = keep_lens;
    a.len_sb = src->len_stride_b;
    a.len_sh = src->len_stride_h;
    a.keep_first = keep_first;
    a.keep_last = keep_last;
    a.mass = attn_mass;
    a.mass_sb = mass_stride_b;
    a.mass_sh = mass_stride_h;
    a.max_seq_len = max_seq_len;
    a.max_keep = max_keep_len;
    a.new_lens = new_lens;
    a.new_mass = new_mass;
    a.nm_sb = new_mass_stride_b;
    a.nm_sh = new_mass_stride_h;
    a.nm_len = new_mass_len;
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    a.status = reinterpret_cast<int2 *>(ws);
    a.kept = kept ? kept : reinterpret_cast<int32_t *>(ws + status_bytes);
    a.kept_sb = kept ? kept_stride_b : (long long)cache->num_kv_heads * max_keep_len;
    a.kept_sh = kept ? kept_stride_h : (long long)max_keep_len;
    a.flags = flags;
    return launch_evict(a, cache->head_dim, cache->dtype == PFKV_KV_FP8_E4M3, sms, static_cast<cudaStream_t>(stream)) ==
                   cudaSuccess
               ? PFKV_OK
               : PFKV_ERR_CUDA;
}

}  // extern "C"

// evict.cu -- pfkv_kv_evict: keep the tokens of every (request, kv head) that
// received most attention and move them, in order, to new pages (declared in
// pfkv_evict.h).
//
// Two launches.  The first checks lengths and table entries and selects; the second
// moves the kept tokens, a warp a destination unit.
#include "evict_internal.cuh"
#include "latent_internal.cuh"

namespace pfkv {
namespace {

constexpr int kSelThreads = 1024, kSelWarps = kSelThreads / 32;
constexpr int kSelBins = 2048;            // 11 bits a digit
constexpr int kSelCluster = 8;            // CTAs a (request, kv head), at most
constexpr int kSelSlice = 8192;           // totals that a CTA takes while there are CTAs to share with
constexpr int kSelKeys = 48 * 1024;       // keys that a CTA keeps in shared memory, at most
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

// --------------------------------------------------------------------------
// The selection.  A cluster of one to eight CTAs a (request, kv head), each with a slice of the
// totals between the protected ends, which it reads once and keeps as ordered keys in shared
// memory (what does not fit is read again).  The m-th largest key is found digit by digit, from
// the top (11, 11 and 10 bits): every CTA counts its keys' digits, the counts are added up over the
// cluster, and the digit is the one in which the m-th falls.  Then every warp counts, over its part
// of the slice, the keys above the m-th and those equal to it; with the sums of the parts before
// it, it knows where its kept tokens go: larger ones all, equal ones from the lowest index on.
// --------------------------------------------------------------------------
__device__ __forceinline__ uint32_t cta_of_cluster() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void sync_cluster(int ctas) {
    if (ctas == 1) __syncthreads();
    else asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// The word at this address in CTA `rank` of the cluster.
__device__ __forceinline__ int word_of_cta(const int *p, uint32_t rank) {
    int v;
    asm volatile("{\n\t.reg .b32 a;\n\tmapa.shared::cluster.u32 a, %1, %2;\n\tld.shared::cluster.u32 %0, [a];\n\t}"
                 : "=r"(v)
                 : "r"(smem_addr(p)), "r"(rank)
                 : "memory");
    return v;
}

struct SelShared {
    int hist[3][kSelBins];     // a digit's counts: one array a pass, so that one is read while the next is made
    int warp_sum[kSelWarps], warp_eq[kSelWarps];
    int gt, eq;                // keys above and equal to the m-th in this CTA
    uint32_t bits;             // flag bits
    int digit, need;
};

__global__ void __launch_bounds__(kSelThreads) evict_select_kernel(EvictArgs a, int ctas, int room) {
    extern __shared__ uint32_t keys[];
    __shared__ SelShared sm;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int rank = ctas == 1 ? 0 : (int)cta_of_cluster();
    const int bh = blockIdx.x / ctas, b = bh / a.Hkv, h = bh - b * a.Hkv;
    for (int i = tid; i < 3 * kSelBins; i += kSelThreads) sm.hist[0][i] = 0;
    if (tid == 0) sm.bits = 0u;
    pdl_enter();
    int n, k;
    const bool sound = lengths(a, b, h, n, k);
    uint32_t bits = sound ? 0u : PFKV_FLAG_BAD_LENGTH;
    if (sound) {
        const int step = ctas * kSelThreads, first = rank * kSelThreads + tid;
        for (int p = first; p < (n + kPage - 1) / kPage; p += step) bits |= entry_check(a, a.src, b, h, p);
        for (int p = first; p < (k + kPage - 1) / kPage; p += step) bits |= entry_check(a, a.dst, b, h, p);
    } else {
        n = k = 0;
    }
    const int f = min(a.keep_first, k), l = min(a.keep_last, k - f), m = k - f - l;
    const int L = n - l - f;  // candidates
    // this CTA's slice of them, in whole warps' worth
    const int per = ((L + ctas - 1) / ctas + 31) & ~31, s0 = min(L, rank * per), len = min(L, s0 + per) - s0;
    const float *mass = a.mass + (long long)b * a.mass_sb + (long long)h * a.mass_sh + f + s0;
    const int have = min(len, room);
    auto key_at = [&](int j) { return j < have ? keys[j] : order_key(mass[j]); };
    __syncthreads();  // the counts are zero
    if (m > 0 && m < L) {
        // keys, and the first digit's counts
#pragma unroll 4
        for (int j = tid; j < len; j += kSelThreads) {
            const uint32_t u = order_key(mass[j]);
            if (j < have) keys[j] = u;
            atomicAdd(&sm.hist[0][u >> 21], 1);
        }
    }
    bits = __reduce_or_sync(0xffffffffu, bits);
    if (lane == 0 && bits) atomicOr(&sm.bits, bits);
    sync_cluster(ctas);
    bits = sm.bits;
    for (int r = 0; r < ctas && ctas > 1; ++r) bits |= (uint32_t)word_of_cta(reinterpret_cast<const int *>(&sm.bits), r);
    if (rank == 0 && tid == 0) a.status[bh] = make_int2((int)bits, k);
    int32_t *kept = a.kept + (long long)b * a.kept_sb + (long long)h * a.kept_sh;
    if (bits || m == 0 || m == L) {
        // nothing to choose; the cluster's CTAs leave together (their shared memory is read by others)
        if (!bits)
            for (int j = rank * kSelThreads + tid; j < k; j += ctas * kSelThreads) kept[j] = j < f + (m == L ? m : 0) ? j : n - k + j;
        if (ctas > 1) sync_cluster(ctas);
        return;
    }
    for (int j = rank * kSelThreads + tid; j < f; j += ctas * kSelThreads) kept[j] = j;
    for (int j = rank * kSelThreads + tid; j < l; j += ctas * kSelThreads) kept[k - l + j] = n - l + j;

    uint32_t found = 0u;
    int need = m;
    constexpr int kShift[3] = {21, 10, 0};
#pragma unroll
    for (int pass = 0; pass < 3; ++pass) {
        const int shift = kShift[pass];
        if (pass > 0) {
            const uint32_t above = pass == 1 ? 0xffe00000u : 0xfffffc00u;
            const uint32_t mask = pass == 1 ? 2047u : 1023u;
            for (int j = tid; j < len; j += kSelThreads) {
                const uint32_t u = key_at(j);
                if ((u & above) == found) atomicAdd(&sm.hist[pass][(u >> shift) & mask], 1);
            }
            sync_cluster(ctas);
        }
        // the digit: counts from the top, two bins a thread (thread 0 has the highest)
        const int top = kSelBins - 1 - 2 * tid;
        int c0 = 0, c1 = 0;
        if (ctas == 1) {
            c0 = sm.hist[pass][top];
            c1 = sm.hist[pass][top - 1];
        } else {
            for (int r = 0; r < ctas; ++r) {
                c0 += word_of_cta(&sm.hist[pass][top], r);
                c1 += word_of_cta(&sm.hist[pass][top - 1], r);
            }
        }
        int x = c0 + c1;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, x, off);
            if (lane >= off) x += y;
        }
        if (lane == 31) sm.warp_sum[warp] = x;
        __syncthreads();
        const int w = sm.warp_sum[lane];
        const int before = __reduce_add_sync(0xffffffffu, lane < warp ? w : 0) + x - c0 - c1;
        if (before < need && before + c0 + c1 >= need) {  // one thread
            const bool second = before + c0 < need;
            sm.digit = second ? top - 1 : top;
            sm.need = need - before - (second ? c0 : 0);
        }
        __syncthreads();
        found |= (uint32_t)sm.digit << shift;
        need = sm.need;
    }

    // where the kept ones go: a warp's part of the slice, 32 keys at a time
    const int part = ((len + kSelWarps - 1) / kSelWarps + 31) & ~31;
    const int p0 = min(len, warp * part), p1 = min(len, p0 + part);
    int gt = 0, eq = 0;
    for (int j = p0 + lane; j < p1; j += 32) {
        const uint32_t u = key_at(j);
        gt += u > found;
        eq += u == found;
    }
    gt = __reduce_add_sync(0xffffffffu, gt);
    eq = __reduce_add_sync(0xffffffffu, eq);
    if (lane == 0) {
        sm.warp_sum[warp] = gt;
        sm.warp_eq[warp] = eq;
    }
    __syncthreads();
    const int wg = sm.warp_sum[lane], we = sm.warp_eq[lane];
    int at_gt = __reduce_add_sync(0xffffffffu, lane < warp ? wg : 0);
    int at_eq = __reduce_add_sync(0xffffffffu, lane < warp ? we : 0);
    if (ctas > 1) {
        if (warp == 0) {
            const int all_gt = __reduce_add_sync(0xffffffffu, wg), all_eq = __reduce_add_sync(0xffffffffu, we);
            if (lane == 0) {
                sm.gt = all_gt;
                sm.eq = all_eq;
            }
        }
        sync_cluster(ctas);
        for (int r = 0; r < rank; ++r) {
            at_gt += word_of_cta(&sm.gt, r);
            at_eq += word_of_cta(&sm.eq, r);
        }
        // no CTA leaves while another reads its shared memory
        asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    }
    const uint32_t below = (1u << lane) - 1u;
    for (int j0 = p0; j0 < p1; j0 += 32) {
        const int j = j0 + lane;
        const uint32_t u = j < p1 ? key_at(j) : 0u;
        const uint32_t is_gt = __ballot_sync(0xffffffffu, j < p1 && u > found);
        const uint32_t is_eq = __ballot_sync(0xffffffffu, j < p1 && u == found);
        const int before_eq = at_eq + __popc(is_eq & below);
        const bool keep = ((is_gt >> lane) & 1u) || (((is_eq >> lane) & 1u) && before_eq < need);
        if (keep) kept[f + at_gt + __popc(is_gt & below) + min(before_eq, need)] = f + s0 + j;
        at_gt += __popc(is_gt);
        at_eq += __popc(is_eq);
    }
    if (ctas > 1) asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// --------------------------------------------------------------------------
// The move.
// --------------------------------------------------------------------------
// Bytes of a row a lane takes, and which.
template <int D, bool FP8>
struct MoveCfg {
    static constexpr int ROWB = D * (FP8 ? 1 : 2), LPR = ROWB / 16, RPP = 32 / LPR, PASSES = kPage / RPP;
};

template <int D, bool FP8>
__device__ __forceinline__ void load_rows(uint4 (&w)[MoveCfg<D, FP8>::PASSES], const void *pool, long long row, int live, int lane) {
    using C = MoveCfg<D, FP8>;
    const uint8_t *bytes = static_cast<const uint8_t *>(pool);
#pragma unroll
    for (int i = 0; i < C::PASSES; ++i) {
        const int r = i * C::RPP + lane / C::LPR;
        const long long from = __shfl_sync(0xffffffffu, row, r);
        w[i] = r < live ? *reinterpret_cast<const uint4 *>(bytes + from * C::ROWB + lane % C::LPR * 16) : make_uint4(0u, 0u, 0u, 0u);
    }
}

template <int D, bool FP8>
__device__ __forceinline__ void store_rows(const uint4 (&w)[MoveCfg<D, FP8>::PASSES], void *pool, long long to, int live, int lane) {
    using C = MoveCfg<D, FP8>;
    uint8_t *bytes = static_cast<uint8_t *>(pool) + to * kPage * C::ROWB;
#pragma unroll
    for (int i = 0; i < C::PASSES; ++i) {
        const int r = i * C::RPP + lane / C::LPR;
        if (r < live) *reinterpret_cast<uint4 *>(bytes + r * C::ROWB + lane % C::LPR * 16) = w[i];
    }
}

// A pair of e4m3 codes as f16 (exact).
__device__ __forceinline__ __half2 codes_to_half2(uint32_t two) {
    __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)two, __NV_E4M3);
    return *reinterpret_cast<__half2 *>(&h);
}

// New codes of a destination unit's rows, in registers as load_rows left them; `mine`: the scale of
// row `lane` (lanes below `live`).  Returns the unit's new scale.
//
// The code of fl(fl(c s) / z) for old code c, old scale s and new scale z.  Taken as the code of
// c fl(s / z): both are within 2^-23 (relative) of c s / z, so they differ at most if a border
// between codes lies within 2^-21 of the product.  A code's significand is one of eight, and
// borders are multiples of 1/16 of a power of two (of 1/8 and coarser below the normal range), so
// eight products a row say whether any code of it comes near one; then all of the unit's codes are
// taken by the definition.  A ratio within 2^-21 of one keeps every code.
template <int D>
__device__ __forceinline__ float new_codes(uint4 (&w)[MoveCfg<D, true>::PASSES], float mine, int live, int lane) {
    using C = MoveCfg<D, true>;
    // absolute maxima of rows as codes (exact in f16), then of values
    float top = 0.f;
    float z[C::PASSES];
#pragma unroll
    for (int i = 0; i < C::PASSES; ++i) {
        const int r = i * C::RPP + lane / C::LPR;
        z[i] = __shfl_sync(0xffffffffu, mine, r);
        const uint32_t u[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
        __half2 t = __float2half2_rn(0.f);
#pragma unroll
        for (int q = 0; q < 4; ++q)
            t = __hmax2(t, __hmax2(__habs2(codes_to_half2(u[q] & 0xffffu)), __habs2(codes_to_half2(u[q] >> 16))));
        const float2 t2 = __half22float2(t);
        top = fmaxf(top, fabsf(fmaxf(t2.x, t2.y) * z[i]));
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
    const float scale = top == 0.f ? 1.f : __fdiv_rn(top, 448.f);
    // a row's ratio by the lane that has its scale; its products with half of the significands, and
    // lane + 16 has the other half
    const float from = __shfl_sync(0xffffffffu, mine, lane & 15);
    const float ratio = __fdiv_rn(from, scale);
    bool near = !(from > 1e-24f && from < 1e30f && scale > 1e-24f && scale < 1e30f && ratio > 1e-20f && ratio < 1e20f);
    if (!(fabsf(ratio - 1.f) <= 0x1p-21f)) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const float y = ratio * (float)(8 + 4 * (lane >> 4) + e);
            near |= ((__float_as_uint(y) + 16u) & 0x7ffffu) <= 32u;
        }
    }
    const bool exact = __any_sync(0xffffffffu, (lane & 15) < live && near);
#pragma unroll
    for (int i = 0; i < C::PASSES; ++i) {
        const float f = __shfl_sync(0xffffffffu, ratio, i * C::RPP + lane / C::LPR);
        uint32_t u[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const float2 x0 = __half22float2(codes_to_half2(u[q] & 0xffffu)), x1 = __half22float2(codes_to_half2(u[q] >> 16));
            float2 y0, y1;
            if (!exact) {
                y0 = mul2(x0, make_float2(f, f));
                y1 = mul2(x1, make_float2(f, f));
            } else {
                y0 = make_float2(__fdiv_rn(x0.x * z[i], scale), __fdiv_rn(x0.y * z[i], scale));
                y1 = make_float2(__fdiv_rn(x1.x * z[i], scale), __fdiv_rn(x1.y * z[i], scale));
            }
            u[q] = (uint32_t)__nv_cvt_float2_to_fp8x2(y0, __NV_SATFINITE, __NV_E4M3) |
                   (uint32_t)__nv_cvt_float2_to_fp8x2(y1, __NV_SATFINITE, __NV_E4M3) << 16;
        }
        w[i] = make_uint4(u[0], u[1], u[2], u[3]);
    }
    return scale;
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
    using C = MoveCfg<D, FP8>;
    uint4 wk[C::PASSES], wv[C::PASSES];
    load_rows<D, FP8>(wk, a.k_pages, row, live, lane);
    load_rows<D, FP8>(wv, a.v_pages, row, live, lane);
    if constexpr (FP8) {
        const long long unit = row / kPage, first = __shfl_sync(0xffffffffu, unit, 0);
        float ks = 0.f, vs = 0.f;
        if (lane < live) {
            ks = a.k_scale[unit];
            vs = a.v_scale[unit];
        }
        // of one unit: bytes and scales as they are
        if (!__all_sync(0xffffffffu, lane >= live || unit == first)) {
            ks = new_codes<D>(wk, ks, live, lane);
            vs = new_codes<D>(wv, vs, live, lane);
        }
        if (lane == 0) {
            a.k_scale[to] = ks;
            a.v_scale[to] = vs;
        }
    }
    store_rows<D, FP8>(wk, a.k_pages, to, live, lane);
    store_rows<D, FP8>(wv, a.v_pages, to, live, lane);
}

}  // namespace

cudaError_t launch_evict(const EvictArgs &a, int D, bool fp8, int num_sms, cudaStream_t s) {
    // As many CTAs a (request, head) as keep a slice of at most kSelSlice totals, while all run at once
    // or a slice would not fit in shared memory otherwise.
    const long long bh = (long long)a.B * a.Hkv;
    int ctas = 1;
    while (ctas < kSelCluster && a.max_seq_len > ctas * kSelSlice &&
           (bh * ctas * 2 <= 2LL * num_sms || a.max_seq_len > ctas * kSelKeys))
        ctas *= 2;
    const int room = min(kSelKeys, (a.max_seq_len + ctas - 1) / ctas + 32);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(bh * ctas));
    cfg.blockDim = dim3(kSelThreads);
    cfg.dynamicSmemBytes = sizeof(uint32_t) * (size_t)room;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)ctas;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = ctas > 1 ? 2 : 1;
    cudaError_t e = cudaLaunchKernelEx(&cfg, evict_select_kernel, a, ctas, room);
    if (e != cudaSuccess) return e;
    const int units = max(1, (max(a.max_keep, a.new_mass ? a.nm_len : 0) + kPage - 1) / kPage);
    const long long grid_x = (bh * units + kMoveWarps - 1) / kMoveWarps;
    const dim3 grid((unsigned)grid_x), block(kMoveWarps * 32);
    auto *const kernel = D == 128 ? (fp8 ? evict_move_kernel<128, true> : evict_move_kernel<128, false>)
                                  : (fp8 ? evict_move_kernel<64, true> : evict_move_kernel<64, false>);
    return launch_pdl(kernel, grid, block, 0, s, a, units);
}

cudaError_t preload_evict() {
    cudaError_t e = cudaFuncSetAttribute(evict_select_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         (int)(sizeof(uint32_t) * kSelKeys));
    if (e == cudaSuccess) e = preload_kernel(evict_select_kernel);
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
    if ((long long)src->batch * cache->num_kv_heads * max(units, (long long)kSelCluster) > 0x7fffffffLL) return PFKV_ERR_UNSUPPORTED;
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

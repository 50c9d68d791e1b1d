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

constexpr int kSelThreads = 512, kSelWarps = kSelThreads / 32;
constexpr int kSelBins = 256;             // eight bits a digit
constexpr int kSelCluster = 12;           // CTAs a (request, kv head), at most
constexpr int kGroup = 128;               // keys that a warp takes at a time
constexpr int kSelSlice = 8192;           // totals that a CTA takes while there are CTAs to share with
constexpr int kSelKeys = 48 * 1024;       // keys that a CTA keeps in shared memory, at most
constexpr int kMoveWarps = 8;
constexpr int kMaxTokens = 1 << 30;       // of a (request, head): indices and their round-ups are ints

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
// The selection.  A cluster of one to twelve CTAs a (request, kv head), each with a slice of the
// totals between the protected ends, which it reads once and keeps as ordered keys in shared
// memory (what does not fit is read again).  The m-th largest key is found digit by digit, from
// the top, eight bits each: every CTA counts its keys' digits, the counts are added up over the
// cluster, and the digit is the one in which the m-th falls.  Then every warp counts, over its part
// of the slice, the keys above the m-th and those equal to it; with the sums of the parts before it,
// it knows where its kept tokens go: larger ones all, equal ones from the lowest index on.
//
// Bound by the latency of its passes: 15 us for 32 x 8 heads of 512 to 8,192 totals (one CTA each), 34 us
// for 2 x 8 of 200,000 to 262,144 (twelve CTAs each).  Clusters of 16 take 112 us a call there, of 12 103,
// as the chip runs 15 of the former at once and the 16th came after.  The rule does not look at the
// number of heads: 8 of them, up to 262,144 totals, take 67 us with 16 and 72 with 12; 24 and 32 the same.
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

// Sum of the words at this address in CTAs 0 .. n - 1 of the cluster, four on their way at once.
__device__ __forceinline__ int sum_of_ctas(const int *p, int n) {
    int sum = 0;
    for (int r = 0; r < n; r += 4) {
        int y[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) y[i] = word_of_cta(p, min(r + i, n - 1));
#pragma unroll
        for (int i = 0; i < 4; ++i) sum += r + i < n ? y[i] : 0;
    }
    return sum;
}

struct SelShared {
    int hist[4][kSelBins];     // a digit's counts
    int warp_sum[kSelWarps], warp_eq[kSelWarps];
    int gt, eq;                // keys above and equal to the m-th in this CTA
    uint32_t bits, all_bits;   // flag bits, and those of the cluster
    int digit, need;
};

__global__ void __launch_bounds__(kSelThreads, 2) evict_select_kernel(EvictArgs a, int ctas, int room) {
    extern __shared__ __align__(16) uint32_t keys[];
    __shared__ SelShared sm;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int rank = ctas == 1 ? 0 : (int)cta_of_cluster();
    const int bh = blockIdx.x / ctas, b = bh / a.Hkv, h = bh - b * a.Hkv;
    for (int i = tid; i < 4 * kSelBins; i += kSelThreads) sm.hist[0][i] = 0;
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
    const int per = ((L + ctas - 1) / ctas + kGroup - 1) / kGroup * kGroup, s0 = min(L, rank * per), len = min(L, s0 + per) - s0;
    const float *mass = a.mass + (long long)b * a.mass_sb + (long long)h * a.mass_sh + f + s0;
    const int groups = (len + kGroup - 1) / kGroup, have = min(groups, room / kGroup);
    // four keys that follow each other, of lane's place in a group; zero, which is below all keys, past the last
    auto four_keys = [&](int g) {
        if (g < have) return reinterpret_cast<const uint4 *>(keys)[g * 32 + lane];
        uint4 u = make_uint4(0u, 0u, 0u, 0u);
        const int j = g * kGroup + lane * 4;
        if (j < len) u.x = order_key(mass[j]);
        if (j + 1 < len) u.y = order_key(mass[j + 1]);
        if (j + 2 < len) u.z = order_key(mass[j + 2]);
        if (j + 3 < len) u.w = order_key(mass[j + 3]);
        return u;
    };
    __syncthreads();  // the counts are zero
    if (m > 0 && m < L) {
        // keys, and the first digit's counts; the loads of kAhead groups are on their way together
        constexpr int kAhead = 4;
        for (int g0 = warp; g0 < groups; g0 += kAhead * kSelWarps) {
            float x[kAhead][4];
#pragma unroll
            for (int i = 0; i < kAhead; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int j = (g0 + i * kSelWarps) * kGroup + e * 32 + lane;
                    x[i][e] = j < len ? mass[j] : 0.f;
                }
#pragma unroll
            for (int i = 0; i < kAhead; ++i) {
                const int g = g0 + i * kSelWarps;
                if (g >= groups) break;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int j = g * kGroup + e * 32 + lane;
                    const uint32_t u = j < len ? order_key(x[i][e]) : 0u;
                    if (g < have) keys[j] = u;
                    atomicAdd(&sm.hist[0][u >> 24], 1);
                }
            }
        }
    }
    bits = __reduce_or_sync(0xffffffffu, bits);
    if (lane == 0 && bits) atomicOr(&sm.bits, bits);
    sync_cluster(ctas);
    bits = sm.bits;
    if (ctas > 1) {
        if (warp == 0) {  // a CTA a lane
            const uint32_t all = __reduce_or_sync(
                0xffffffffu, (uint32_t)word_of_cta(reinterpret_cast<const int *>(&sm.bits), min(lane, ctas - 1)));
            if (lane == 0) sm.all_bits = all;
        }
        __syncthreads();
        bits = sm.all_bits;
    }
    if (rank == 0 && tid == 0) a.status[bh] = make_int2((int)bits, k);
    int32_t *kept = a.kept + (long long)bh * a.max_keep;
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
#pragma unroll 1
    for (int pass = 0; pass < 4; ++pass) {
        const int shift = 24 - 8 * pass;
        if (pass > 0) {
            const uint32_t above = 0xffffffffu << (shift + 8);
            auto count = [&](uint32_t u) {
                if ((u & above) == found) atomicAdd(&sm.hist[pass][(u >> shift) & 255u], 1);
            };
#pragma unroll 2
            for (int g = warp; g < groups; g += kSelWarps) {
                const uint4 u = four_keys(g);
                count(u.x);
                count(u.y);
                count(u.z);
                count(u.w);
            }
            sync_cluster(ctas);
        }
        const int *const sum = sm.hist[pass];
        // the digit: counts from the top, a bin a thread (thread 0 has the highest)
        int c = 0, x = 0;
        const int bin = kSelBins - 1 - tid;
        if (tid < kSelBins) {
            if (ctas == 1) c = sum[bin];
            else c = sum_of_ctas(&sum[bin], ctas);
            x = c;
#pragma unroll
            for (int off = 1; off < 32; off <<= 1) {
                const int y = __shfl_up_sync(0xffffffffu, x, off);
                if (lane >= off) x += y;
            }
            if (lane == 31) sm.warp_sum[warp] = x;
        }
        __syncthreads();
        if (tid < kSelBins) {
            const int w = lane < kSelBins / 32 ? sm.warp_sum[lane] : 0;
            const int before = __reduce_add_sync(0xffffffffu, lane < warp ? w : 0) + x - c;
            if (before < need && before + c >= need) {  // one thread
                sm.digit = bin;
                sm.need = need - before;
            }
        }
        __syncthreads();
        found |= (uint32_t)sm.digit << shift;
        need = sm.need;
    }

    // where the kept ones go: a warp's part of the slice, a group at a time
    const int part = (groups + kSelWarps - 1) / kSelWarps, g0 = min(groups, warp * part), g1 = min(groups, g0 + part);
    int gt = 0, eq = 0;
#pragma unroll 2
    for (int g = g0; g < g1; ++g) {
        const uint4 u = four_keys(g);
        gt += (u.x > found) + (u.y > found) + (u.z > found) + (u.w > found);
        eq += (u.x == found) + (u.y == found) + (u.z == found) + (u.w == found);
    }
    gt = __reduce_add_sync(0xffffffffu, gt);
    eq = __reduce_add_sync(0xffffffffu, eq);
    if (lane == 0) {
        sm.warp_sum[warp] = gt;
        sm.warp_eq[warp] = eq;
    }
    __syncthreads();
    const int wg = lane < kSelWarps ? sm.warp_sum[lane] : 0, we = lane < kSelWarps ? sm.warp_eq[lane] : 0;
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
        // those of the CTAs before: a CTA a lane
        at_gt += __reduce_add_sync(0xffffffffu, lane < rank ? word_of_cta(&sm.gt, min(lane, ctas - 1)) : 0);
        at_eq += __reduce_add_sync(0xffffffffu, lane < rank ? word_of_cta(&sm.eq, min(lane, ctas - 1)) : 0);
        // no CTA leaves while another reads its shared memory
        asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    }
    const uint32_t below = (1u << lane) - 1u;
#pragma unroll 1
    for (int g = g0; g < g1; ++g) {
        const uint4 u4 = four_keys(g);
        const uint32_t u[4] = {u4.x, u4.y, u4.z, u4.w};
        uint32_t is_gt[4], is_eq[4];
        int gt_before = at_gt, eq_before = at_eq;  // of this lane's four
        int any = 0;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            is_gt[e] = __ballot_sync(0xffffffffu, u[e] > found);
            is_eq[e] = __ballot_sync(0xffffffffu, u[e] == found);
            any |= is_eq[e];
            gt_before += __popc(is_gt[e] & below);
            at_gt += __popc(is_gt[e]);
        }
        if (any) {  // (equal ones are few)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                eq_before += __popc(is_eq[e] & below);
                at_eq += __popc(is_eq[e]);
            }
        }
        int32_t *const to = kept + f;
        const int j = f + s0 + g * kGroup + lane * 4;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const bool larger = u[e] > found, equal = u[e] == found;
            if (larger || (equal && eq_before < need)) to[gt_before + min(eq_before, need)] = j + e;
            gt_before += larger;
            eq_before += equal;
        }
    }
    if (ctas > 1) asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// --------------------------------------------------------------------------
// The move: a warp a destination unit, its 16 rows gathered in 16-byte loads.  Bytes: both rows read and
// written.  BF16: near memory's rate (24 us for 16 x 4 heads of 33 to 20,000 tokens of 64, half kept).  FP8:
// 46 us for 32 x 8 heads of 512 to 8,192 tokens, a quarter kept, and nothing is at its limit (ALU 56% busy
// with conversions of codes, issue slots 60%, DRAM 35%): latency, at two fifths of the warps, which is what
// 64 registers (some spilled) and two units a warp, one after the other, leave of it.  (The whole call: 96
// us while units with a code near a border took divisions, 57 now.)
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

// The rows of a destination unit by the definition: code of fl(fl(c s) / z).  (A call, not inlined:
// few units need it, and its registers would be every unit's.)
template <int D>
__device__ __noinline__ float by_definition(void *pool, long long row, float mine, long long to, int live, int lane) {
    using C = MoveCfg<D, true>;
    uint4 w[C::PASSES];
    load_rows<D, true>(w, pool, row, live, lane);
    float z[C::PASSES];
    float top = 0.f;  // (a NaN is no maximum)
#pragma unroll
    for (int i = 0; i < C::PASSES; ++i) z[i] = __shfl_sync(0xffffffffu, mine, i * C::RPP + lane / C::LPR);
#pragma unroll
    for (int i = 0; i < C::PASSES; ++i) {
        const uint32_t u[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
#pragma unroll
        for (int q = 0; q < 8; ++q) {
            const float2 x = e4m3x2_to_float2((uint16_t)(u[q >> 1] >> (16 * (q & 1))));
            top = fmaxf(top, fmaxf(fabsf(x.x * z[i]), fabsf(x.y * z[i])));
        }
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
    const float sound = top == 0.f ? 1.f : __fdiv_rn(top, 448.f);
#pragma unroll
    for (int i = 0; i < C::PASSES; ++i) {
        uint32_t u[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const float2 x0 = e4m3x2_to_float2((uint16_t)u[q]), x1 = e4m3x2_to_float2((uint16_t)(u[q] >> 16));
            const float2 y0 = make_float2(__fdiv_rn(x0.x * z[i], sound), __fdiv_rn(x0.y * z[i], sound));
            const float2 y1 = make_float2(__fdiv_rn(x1.x * z[i], sound), __fdiv_rn(x1.y * z[i], sound));
            u[q] = (uint32_t)__nv_cvt_float2_to_fp8x2(y0, __NV_SATFINITE, __NV_E4M3) |
                   (uint32_t)__nv_cvt_float2_to_fp8x2(y1, __NV_SATFINITE, __NV_E4M3) << 16;
        }
        w[i] = make_uint4(u[0], u[1], u[2], u[3]);
    }
    store_rows<D, true>(w, pool, to, live, lane);
    return sound;
}

// Writes a destination unit's rows, in registers as load_rows left them, with new codes; `mine`: the
// scale of row `lane` (lanes below `live`).  Returns the unit's new scale.
//
// The code of fl(fl(c s) / z) for old code c, old scale s and new scale z, in one of three ways:
//
// (1) As the code of c fl(s / z).  Both are within 2^-23 (relative) of c s / z, so the codes are the
// same unless a border between codes lies within 2^-21 of the product.  With c = m 2^q, m = 8 .. 15 (a
// subnormal c as a multiple of its own), and t = m s / z, borders are at odd multiples of 1/16 of t's
// power of two; or, where the new code is subnormal, at odd multiples o < 16 of 2^-10, so that t is
// a multiple of 1/8 of its power of two and below 8, or o (m even), 2 o (m = 8, 12) or 4 o (m = 8), where
// c is subnormal.  Eight t a row say whether any code of it may come near a border.  A ratio
// within 2^-21 of one keeps every code.  (Borders are met often: z is a code's value over 448, so
// in the row of the largest, ratios are 14 / m.)
// (2) Otherwise (for the rows that are loaded together with such a row, not for the whole unit)
// with a correctly rounded quotient, by Markstein's theorem (IBM J. Res. Dev. 34, 1990): two
// corrections of x times the correctly rounded reciprocal of z.  Magnitudes: a sum would lose a
// zero's sign.
// (3) By divisions, for scales so small or large that (1) or (2) might not hold, and codes of NaN.
template <int D>
__device__ __forceinline__ float new_codes(uint4 (&w)[MoveCfg<D, true>::PASSES], void *pool, long long row, float mine,
                                           long long to, int live, int lane) {
    using C = MoveCfg<D, true>;
    // absolute maxima of rows as codes, whose order is that of their values; then of values
    float top = 0.f;
    uint32_t most = 0u;
    float z[C::PASSES];
#pragma unroll
    for (int i = 0; i < C::PASSES; ++i) {
        z[i] = __shfl_sync(0xffffffffu, mine, i * C::RPP + lane / C::LPR);
        // the upper and the lower bytes of 16-bit halves
        uint32_t hi = __vimax3_u16x2(w[i].x & 0x7fff7fffu, w[i].y & 0x7fff7fffu, w[i].z & 0x7fff7fffu);
        uint32_t lo = __vimax3_u16x2(w[i].x & 0x007f007fu, w[i].y & 0x007f007fu, w[i].z & 0x007f007fu);
        hi = __vimax3_u16x2(hi, w[i].w & 0x7fff7fffu, 0u) >> 8;
        lo = __vimax3_u16x2(lo, w[i].w & 0x007f007fu, 0u);
        const uint32_t code = max(max(hi & 0xffu, hi >> 16), max(lo & 0xffffu, lo >> 16));
        most = max(most, code);
        top = fmaxf(top, fabsf(e4m3x2_to_float2((uint16_t)code).x * z[i]));
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
    const float scale = top == 0.f ? 1.f : __fdiv_rn(top, 448.f);
    // a row's ratio by the lane that has its scale; its products with half of the significands, and
    // lane + 16 has the other half
    const float from = __shfl_sync(0xffffffffu, mine, lane & 15);
    const float ratio = __fdiv_rn(from, scale);
    const bool odd = !(from > 1e-24f && from < 1e30f && scale > 1e-24f && scale < 1e30f && ratio > 1e-20f && ratio < 1e20f);
    bool near = false;
    if (!(fabsf(ratio - 1.f) <= 0x1p-21f)) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int sig = 8 + 4 * (lane >> 4) + e;
            const float t = ratio * (float)sig;
            const uint32_t u = __float_as_uint(t) + 16u;  // near: within 16 steps
            if ((u & 0x7ffffu) > 32u) continue;           // of no multiple of 1/16
            const int n = (int)(t + 0.5f);                // t itself where it matters below: 8 <= t < 61
            const int twos = n & -n;
            near |= (u & 0x80000u) != 0u || t < 7.9f || (t < 60.1f && twos <= (sig == 8 ? 4 : sig == 12 ? 2 : (sig & 1) ? 0 : 1));
        }
    }
    if (__any_sync(0xffffffffu, ((lane & 15) < live && odd) || most == 0x7fu))
        return by_definition<D>(pool, row, mine, to, live, lane);
    const uint32_t lanes = __ballot_sync(0xffffffffu, (lane & 15) < live && near), rows = lanes | (lanes >> 16);
    const float inv = __frcp_rn(scale);
    const float2 inv2 = make_float2(inv, inv), down = make_float2(-scale, -scale);
#pragma unroll
    for (int i = 0; i < C::PASSES; ++i) {
        uint32_t u[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
        if ((rows >> (i * C::RPP)) & ((1u << C::RPP) - 1u)) {  // the same for all lanes
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const uint32_t size = u[q] & 0x7f7f7f7fu;
                uint32_t code = u[q] & 0x80808080u;
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    const float2 x = mul2(__half22float2(codes_to_half2(size >> (16 * half))), make_float2(z[i], z[i]));
                    float2 y = mul2(x, inv2);
                    y = fma2(fma2(y, down, x), inv2, y);
                    y = fma2(fma2(y, down, x), inv2, y);
                    code |= (uint32_t)__nv_cvt_float2_to_fp8x2(y, __NV_SATFINITE, __NV_E4M3) << (16 * half);
                }
                u[q] = code;
            }
        } else {
            const float f = __shfl_sync(0xffffffffu, ratio, i * C::RPP + lane / C::LPR);
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const float2 y0 = mul2(__half22float2(codes_to_half2(u[q])), make_float2(f, f));
                const float2 y1 = mul2(__half22float2(codes_to_half2(u[q] >> 16)), make_float2(f, f));
                u[q] = (uint32_t)__nv_cvt_float2_to_fp8x2(y0, __NV_SATFINITE, __NV_E4M3) |
                       (uint32_t)__nv_cvt_float2_to_fp8x2(y1, __NV_SATFINITE, __NV_E4M3) << 16;
            }
        }
        w[i] = make_uint4(u[0], u[1], u[2], u[3]);
    }
    store_rows<D, true>(w, pool, to, live, lane);
    return scale;
}


// A warp takes `each` units (at most kMoveUnits) of one (request, head), kMoveWarps apart.  What
// leads to their rows (status, indices and new pages, then old pages) is loaded for all of them at
// once, half a warp a unit: one after the other, these loads took most of a unit's time.
constexpr int kMoveUnits = 2;

template <int D, bool FP8>
__global__ void __launch_bounds__(kMoveWarps * 32, FP8 || D == 64 ? 4 : 3) evict_move_kernel(EvictArgs a, int chunks, int each) {
    pdl_enter();
    using C = MoveCfg<D, FP8>;
    const int bh = blockIdx.x / chunks, chunk = blockIdx.x - bh * chunks;
    const int b = bh / a.Hkv, h = bh - b * a.Hkv;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, slot = lane & 15;
    const int u0 = chunk * each * kMoveWarps + warp;
    uint32_t bits = 0u;
    for (int i = lane; i < a.Hkv; i += 32) bits |= (uint32_t)a.status[(long long)b * a.Hkv + i].x;
    const int k = a.status[bh].y;
    const int32_t *kept = a.kept + (long long)bh * a.max_keep;
    const int at = lane >> 4, j = (u0 + at * kMoveWarps) * kPage + slot;  // this lane's unit and slot
    const int from = at < each && j < a.max_keep ? kept[j] : 0;
    // a new page a unit, in lane `unit`
    const int up = u0 + min(lane, each - 1) * kMoveWarps;
    const int new_id = up < a.dst.max_pages ? a.dst.block_tables[(long long)b * a.dst.bt_sb + (long long)h * a.dst.bt_sh + up] : 0;
    bits = __reduce_or_sync(0xffffffffu, bits);
    if (u0 == 0 && lane == 0) {
        if (h == 0 || a.len_sh != 0) a.new_lens[(long long)b * a.len_sb + (long long)h * a.len_sh] = bits ? 0 : k;
        if (h == 0 && a.flags) a.flags[b] = (uint8_t)bits;
    }
    if (bits) return;
    const int32_t *table = a.src.block_tables + (long long)b * a.src.bt_sb + (long long)h * a.src.bt_sh;
    const bool there = at < each && j < k;
    const int id = there ? table[from / kPage] : -1;
    if (a.kept_out && there) a.kept_out[(long long)b * a.kept_sb + (long long)h * a.kept_sh + j] = from;
    if (a.new_mass && at < each && j < a.nm_len)
        a.new_mass[(long long)b * a.nm_sb + (long long)h * a.nm_sh + j] =
            there ? a.mass[(long long)b * a.mass_sb + (long long)h * a.mass_sh + from] : 0.f;
#pragma unroll 1
    for (int i = 0; i < each; ++i) {
        const int u = u0 + i * kMoveWarps, live = min(kPage, k - u * kPage);
        if (live <= 0) return;
        const int page = __shfl_sync(0xffffffffu, id, i * 16 + slot), token = __shfl_sync(0xffffffffu, from, i * 16 + slot);
        const long long unit = (long long)page * a.Hkv + h, row = unit * kPage + token % kPage;
        const long long to = (long long)__shfl_sync(0xffffffffu, new_id, i) * a.Hkv + h;
        uint4 wk[C::PASSES], wv[C::PASSES];
        load_rows<D, FP8>(wk, a.k_pages, row, live, lane);
        load_rows<D, FP8>(wv, a.v_pages, row, live, lane);
        if constexpr (FP8) {
            const long long first = __shfl_sync(0xffffffffu, unit, 0);
            float ks = 0.f, vs = 0.f;
            if (lane < live) {
                ks = a.k_scale[unit];
                vs = a.v_scale[unit];
            }
            // of one unit: bytes and scales as they are
            if (!__all_sync(0xffffffffu, lane >= live || unit == first)) {
                // K, then V: one copy of the code, which is long
                void *pool = a.k_pages;
#pragma unroll 1
                for (int which = 0; which < 2; ++which) {
                    const float z = new_codes<D>(wk, pool, row, which ? vs : ks, to, live, lane);
                    if (which) {
                        vs = z;
                    } else {
                        ks = z;
                        pool = a.v_pages;
#pragma unroll
                        for (int q = 0; q < C::PASSES; ++q) wk[q] = wv[q];
                    }
                }
            } else {
                store_rows<D, FP8>(wk, a.k_pages, to, live, lane);
                store_rows<D, FP8>(wv, a.v_pages, to, live, lane);
            }
            if (lane == 0) {
                a.k_scale[to] = ks;
                a.v_scale[to] = vs;
            }
        } else {
            store_rows<D, FP8>(wk, a.k_pages, to, live, lane);
            store_rows<D, FP8>(wv, a.v_pages, to, live, lane);
        }
    }
}

}  // namespace

cudaError_t launch_evict(const EvictArgs &a, int D, bool fp8, int num_sms, cudaStream_t s) {
    // As many CTAs a (request, head) as keep a slice of at most kSelSlice totals, while all run at once
    // or a slice would not fit in shared memory otherwise.  All by the bounds, which the host knows, not
    // by the lengths: shared memory, clusters and grids for more than there is cost time.  32 x 8 heads of
    // 512 to 8,192 tokens, a quarter kept, take 58 us with exact bounds, 79 with four times them, 185 with
    // sixteen times; 2 x 8 heads 29, 30 and 31.
    const long long bh = (long long)a.B * a.Hkv;
    int ctas = 1;
    while (ctas < kSelCluster && a.max_seq_len > ctas * kSelSlice &&
           (bh * ctas * 2 <= 2LL * num_sms || a.max_seq_len > ctas * kSelKeys))
        ctas = min(2 * ctas, kSelCluster);
    const int room = min(kSelKeys, ((a.max_seq_len + ctas - 1) / ctas + kGroup - 1) / kGroup * kGroup);
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
    // one unit a warp while all warps run at once
    const int each = (int)min((long long)kMoveUnits, max(1LL, bh * units / ((long long)num_sms * 32)));
    const int chunks = (units + each * kMoveWarps - 1) / (each * kMoveWarps);
    const dim3 grid((unsigned)(bh * chunks)), block(kMoveWarps * 32);
    auto *const kernel = D == 128 ? (fp8 ? evict_move_kernel<128, true> : evict_move_kernel<128, false>)
                                  : (fp8 ? evict_move_kernel<64, true> : evict_move_kernel<64, false>);
    return launch_pdl(kernel, grid, block, 0, s, a, chunks, each);
}

cudaError_t preload_evict() {
    cudaError_t e = cudaFuncSetAttribute(evict_select_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         (int)(sizeof(uint32_t) * kSelKeys));
    if (e == cudaSuccess) e = cudaFuncSetAttribute(evict_select_kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
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
    if (max_seq_len > kMaxTokens || max_keep_len > kMaxTokens) return PFKV_ERR_UNSUPPORTED;
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
    if (new_mass && new_mass_len > kMaxTokens) return PFKV_ERR_UNSUPPORTED;
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
    a.kept = reinterpret_cast<int32_t *>(ws + status_bytes);
    a.kept_out = kept;
    a.kept_sb = kept_stride_b;
    a.kept_sh = kept_stride_h;
    a.flags = flags;
    return launch_evict(a, cache->head_dim, cache->dtype == PFKV_KV_FP8_E4M3, sms, static_cast<cudaStream_t>(stream)) ==
                   cudaSuccess
               ? PFKV_OK
               : PFKV_ERR_CUDA;
}

}  // extern "C"

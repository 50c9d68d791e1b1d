// prefix.cu -- pfkv_prefix_decode_attn: attention of a batch whose requests share
// prefixes (declared in pfkv_prefix.h).
//
// Four launches.  The plan checks every table, sorts the requests by their prefix and cuts the
// work of the prefixes into equal shares (below).  The split kernel of pfkv_paged_decode_attn
// (decode_pers.cuh) attends over the requests' own tokens, and the kernel of prefix_attn.cu over the
// prefixes; both leave normalised partial results with their log2-sum-exp, which the merge joins.
#include <cmath>

#include "prefix_internal.cuh"

namespace pfkv {
namespace {

// --------------------------------------------------------------------------
// The plan: the first CTA counts the requests of every prefix and cuts the work into
// segments and partial results; the others check one tile of a table row each, like
// validate_kernel, with the tags as far as they are tracked, or pack the queries.  It waits for
// its predecessor before it lets the next kernel start, so the call's inputs are final then.  Bound by
// latency: 5 us for 32 requests of 8 heads, 8 us for 256 (whose tables would be 2,048 CTAs: see
// short_rows).
// --------------------------------------------------------------------------
// Exclusive sums over the block of two numbers a thread; the totals in total.  Ends synchronised.
struct Two {
    int x, y;
};
__device__ __forceinline__ Two block_sums_before(Two v, Two *part, Two *total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    constexpr int W = kValThreads / 32;
    Two s = v;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const int x = __shfl_up_sync(0xffffffffu, s.x, off), y = __shfl_up_sync(0xffffffffu, s.y, off);
        if (lane >= off) {
            s.x += x;
            s.y += y;
        }
    }
    __syncthreads();
    if (lane == 31) part[warp] = s;
    __syncthreads();
    const Two p = lane < W ? part[lane] : Two{0, 0};
    const Two before{__reduce_add_sync(0xffffffffu, lane < warp ? p.x : 0), __reduce_add_sync(0xffffffffu, lane < warp ? p.y : 0)};
    *total = Two{__reduce_add_sync(0xffffffffu, p.x), __reduce_add_sync(0xffffffffu, p.y)};
    return Two{before.x + s.x - v.x, before.y + s.y - v.y};
}

// Tokens of row i for head h; -1 where a bound does not hold.
__device__ __forceinline__ int table_len(const PrefixTables &t, int i, int h) {
    const int n = t.seq_lens[(long long)i * t.len_sb + (long long)h * t.len_sh];
    return n < 0 || n > t.max_len || (long long)n > (long long)t.max_pages * kPage ? -1 : n;
}

constexpr int kPlanChunk = 2048;
constexpr int kPrefixFew = 512, kSegFew = 1024, kPairFew = 512;  // what shared memory has room for

// count: requests of a prefix.
__device__ void plan_segments(const PrefixArgs &a, int *count) {
    __shared__ int of[kPlanChunk], first_member[kPrefixFew], first_seg[kPrefixFew], seg_tile[kSegFew];
    __shared__ int2 pair_tile[kPairFew];
    __shared__ Two part[kValThreads / 32];
    Two total;
    const int tid = threadIdx.x, lane = tid & 31, NP = a.pre.count;
    if (tid == 0) a.head->timeout = 0u;
    for (int b = tid; b < a.B; b += kValThreads) {  // the merge adds the bits
        if (a.flags) a.flags[b] = 0;
        if (a.rflags) a.rflags[b] = 0;
    }
    for (int p = tid; p < NP; p += kValThreads) count[p] = 0;
    // lengths are on their way while requests are counted (one a thread: the usual case)
    const int pairs = NP * a.Hkv, per = (pairs + kValThreads - 1) / kValThreads;
    const int x0 = min(pairs, tid * per), x1 = min(pairs, x0 + per);
    const auto len_of = [&](int x) { return max(0, table_len(a.pre, x / a.Hkv, x % a.Hkv)); };
    const int len0 = x0 < x1 ? len_of(x0) : 0;
    // positions, in the order of the batch: one warp takes 32 requests at a time
    for (int b0 = 0; b0 < a.B; b0 += kPlanChunk) {
        const int n = min(kPlanChunk, a.B - b0);
        __syncthreads();
        for (int i = tid; i < n; i += kValThreads) of[i] = a.prefix_of[b0 + i];
        __syncthreads();
        if (tid < 32) {
            for (int i = lane; i - lane < n; i += 32) {
                const int p = i < n ? of[i] : -1;
                const bool valid = p >= 0 && p < NP;
                const uint32_t same = __match_any_sync(0xffffffffu, valid ? p : -1 - lane);
                const int rank = __popc(same & ((1u << lane) - 1u));
                const int before = valid ? count[p] : 0;
                __syncwarp();
                if (valid && rank == 0) count[p] = before + __popc(same);
                __syncwarp();
                if (i < n) {
                    of[i] = valid ? before + rank : -1;
                    a.pos[b0 + i] = of[i];
                }
            }
        }
    }
    __syncthreads();
    // first members and first segments
    const auto blocks = [&](int p) { return (int)(((long long)count[p] * a.kq * a.G + kPrefixBlock - 1) / kPrefixBlock); };
    int segs = 0;
    const bool few = NP <= kPrefixFew && a.B <= kPlanChunk;  // all in shared memory
    {
        const int each = (NP + kValThreads - 1) / kValThreads, p0 = min(NP, tid * each), p1 = min(NP, p0 + each);
        Two v{0, 0};
        for (int p = p0; p < p1; ++p) {
            v.x += count[p];
            v.y += blocks(p) * a.Hkv;
        }
        v = block_sums_before(v, part, &total);
        segs = total.y;
        if (tid == 0) {
            a.mstart[NP] = total.x;
            a.seg0[NP] = total.y;
        }
        for (int p = p0; p < p1; ++p) {
            a.mstart[p] = v.x;
            a.seg0[p] = v.y;
            if (few) {
                first_member[p] = v.x;
                first_seg[p] = v.y;
            }
            v.x += count[p];
            v.y += blocks(p) * a.Hkv;
        }
    }
    __syncthreads();
    for (int b = tid; b < a.B; b += kValThreads) {
        const int at = few ? of[b] : a.pos[b];
        PrefixPlace w{-1, 0, 0, 0};
        if (at >= 0) {
            const int p = a.prefix_of[b];
            a.members[(few ? first_member[p] : a.mstart[p]) + at] = b;
            w = PrefixPlace{at * a.kq * a.G, few ? first_seg[p] : a.seg0[p], blocks(p), 0};
        }
        a.place[b] = w;
    }
    // tiles: first ones of every (prefix, head)
    Two v{0, 0};
    for (int x = x0; x < x1; ++x)
        v.x += blocks(x / a.Hkv) * (((x == x0 ? len0 : len_of(x)) + kPrefixTile - 1) / kPrefixTile);
    v.x = block_sums_before(v, part, &total).x;
    const int U = total.x, W = min(a.ctas, U);
    for (int x = x0; x < x1; ++x) {
        const int len = x == x0 ? len0 : len_of(x);
        const int2 y = make_int2(v.x, len);
        if (x < kPairFew) pair_tile[x] = y;
        else a.pair[x] = y;
        v.x += blocks(x / a.Hkv) * ((len + kPrefixTile - 1) / kPrefixTile);
    }
    __syncthreads();
    // CTAs without work; the others' ranges follow
    for (int c = W + tid; c < a.ctas; c += kValThreads) a.range[c] = PrefixRange{0, 0, 0, 0};
    // segments, and the rows of their partial results
    const int each = (segs + kValThreads - 1) / kValThreads, k0 = min(segs, tid * each), k1 = min(segs, k0 + each);
    const auto segment = [&](int k) {
        int lo = 0, hi = NP;  // the last prefix whose first segment is at most k
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if ((few ? first_seg[mid] : a.seg0[mid]) <= k) lo = mid;
            else hi = mid;
        }
        const int nb = blocks(lo), at = k - (few ? first_seg[lo] : a.seg0[lo]), h = at / nb, rb = at - h * nb;
        const int x = lo * a.Hkv + h;
        const int2 y = x < kPairFew ? pair_tile[x] : a.pair[x];
        PrefixSeg s{};
        s.p = lo;
        s.h = h;
        s.row0 = rb * kPrefixBlock;
        s.rows = (int)min((long long)kPrefixBlock, (long long)count[lo] * a.kq * a.G - s.row0);
        s.len = y.y;
        s.ntiles = (y.y + kPrefixTile - 1) / kPrefixTile;
        s.tile0 = y.x + rb * s.ntiles;
        s.first = s.ntiles > 0 ? pers_worker_of(s.tile0, U, W) : 0;
        s.ctas = s.ntiles > 0 ? pers_worker_of(s.tile0 + s.ntiles - 1, U, W) - s.first + 1 : 0;
        return s;
    };
    int rows = 0;
    PrefixSeg s{};
    for (int k = k0; k < k1; ++k) {
        s = segment(k);
        rows += rows8(s.rows) * s.ctas;
    }
    rows = block_sums_before(Two{rows, 0}, part, &total).x;
    for (int k = k0; k < k1; ++k) {
        if (each > 1) s = segment(k);
        s.base = rows;
        rows += rows8(s.rows) * s.ctas;
        a.seg[k] = s;
        if (k < kSegFew) seg_tile[k] = s.tile0;
    }
    __syncthreads();
    // the segment of every CTA's first tile
    for (int c = tid; c < W; c += kValThreads) {
        const int t0 = (int)(((long long)c * U + W - 1) / W);
        int lo = 0, hi = segs;
        while (hi - lo > 1) {  // (of equal first tiles the last segment, the one that has tiles)
            const int mid = (lo + hi) >> 1;
            if ((segs <= kSegFew ? seg_tile[mid] : a.seg[mid].tile0) <= t0) lo = mid;
            else hi = mid;
        }
        a.range[c] = PrefixRange{t0, (int)(((long long)(c + 1) * U + W - 1) / W), lo, 0};
    }
}

// First units of the own tokens' segments, group by group, as the split kernel counts them.
__device__ void plan_own_units(const PrefixArgs &a, const PrefixOwnRows &o, int *count) {
    __shared__ Two part[kValThreads / 32];
    for (int r0 = 0, g = 0; r0 < a.B; r0 += o.greq, ++g) {
        const int K = min(o.greq, a.B - r0) * a.kq * a.Hkv, per = (K + kValThreads - 1) / kValThreads;
        int *units = o.units + (long long)g * (o.greq * a.kq * a.Hkv + 1);
        __syncthreads();
#pragma unroll 2
        for (int k = threadIdx.x; k < K; k += kValThreads) {
            const int v = k / a.Hkv, r = v / a.kq, n = table_len(a.own, r0 + r, k - v * a.Hkv);
            count[k] = segment_units(n < 0 ? -1 : max(0, n - a.kq + 1 + (v - r * a.kq)), 0, o.chunk_tokens);
        }
        __syncthreads();
        const int k0 = min(K, (int)threadIdx.x * per), k1 = min(K, k0 + per);
        Two mine{0, 0}, total;
#pragma unroll 1
        for (int k = k0; k < k1; ++k) mine.x += count[k];
        int at = block_sums_before(mine, part, &total).x;
#pragma unroll 1
        for (int k = k0; k < k1; ++k) {
            units[k] = at;
            at += count[k];
        }
        if (threadIdx.x == 0) units[K] = total.x;
    }
}

// Check bits of one tile of kValTile entries of table row i, head h; VMAX: and its pages' largest |V scale|.
// Rows: a warp a row of at most kValTile / 8 entries, eight rows a CTA (a batch of 256 requests of 8 heads
// would be 2,048 CTAs).
__host__ __device__ inline bool short_rows(const PrefixTables &t) { return t.max_pages <= kValTile / (kValThreads / 32); }

template <bool VMAX, bool Rows>
__device__ void check_tile(const PrefixArgs &a, const PrefixTables &t, int ih, int tile, uint32_t *bits_out, float *vmax_out) {
    constexpr int STEP = Rows ? 32 : kValThreads;
    if constexpr (Rows) {
        ih = ih * (kValThreads / 32) + (threadIdx.x >> 5);
        if (ih >= t.count * a.Hkv) return;
    }
    const int i = ih / a.Hkv, h = ih - i * a.Hkv;
    const int n = table_len(t, i, h), np = (n + kPage - 1) / kPage;
    const int p0 = tile * kValTile + threadIdx.x % STEP;
    const long long row = (long long)i * t.bt_sb + (long long)h * t.bt_sh;
    int id[kValPer];
    uint32_t want[kValPer], tag[kValPer];
#pragma unroll
    for (int j = 0; j < kValPer; ++j) {
        const int p = p0 + j * STEP;
        id[j] = p < t.max_pages ? t.block_tables[row + p] : 0;
        want[j] = p < t.max_pages && a.page_tags ? t.expected_tags[row + p] : 0u;
    }
    uint32_t bits = n < 0 ? PFKV_FLAG_BAD_LENGTH : 0u;
    float scale[kValPer];
#pragma unroll
    for (int j = 0; j < kValPer; ++j) {
        const bool live = p0 + j * STEP < np, in_pool = id[j] >= 0 && id[j] < a.num_pages;
        if (live && !in_pool) bits |= PFKV_FLAG_BAD_PAGE;
        const long long unit = live && in_pool ? (long long)id[j] * a.Hkv + h : -1;
        tag[j] = unit >= 0 && a.page_tags ? a.page_tags[unit] : want[j];
        scale[j] = VMAX && unit >= 0 ? fabsf(a.v_scale[unit]) : 0.f;
        if (unit < 0) want[j] = tag[j];
    }
    float top = 0.f;
#pragma unroll
    for (int j = 0; j < kValPer; ++j) {
        if (tag[j] != want[j]) bits |= PFKV_FLAG_TAG_MISMATCH;
        top = fmaxf(top, scale[j]);
    }
    bits = __reduce_or_sync(0xffffffffu, bits);
    const uint32_t high = __reduce_max_sync(0xffffffffu, __float_as_uint(top));  // not negative: ordered as numbers
    if constexpr (Rows) {
        if ((threadIdx.x & 31) == 0) {
            bits_out[ih] = bits;  // one word a row
            if (VMAX) vmax_out[ih] = __uint_as_float(high);
        }
        return;
    }
    __shared__ uint32_t all, most;
    if (threadIdx.x == 0) all = most = 0u;
    __syncthreads();
    if ((threadIdx.x & 31) == 0) {
        if (bits) atomicOr(&all, bits);
        if (VMAX) atomicMax(&most, high);
    }
    __syncthreads();
    if (threadIdx.x == 0) {
        bits_out[(long long)ih * t.htiles + tile] = all;
        if (VMAX) vmax_out[(long long)ih * t.htiles + tile] = __uint_as_float(most);
    }
}

constexpr int kPackPer = 4;  // 16-byte chunks a thread packs

template <bool FP8>
__global__ void __launch_bounds__(kValThreads) prefix_plan_kernel(PrefixArgs a, PrefixOwnRows o, int D, int pre_tiles, int own_tiles) {
    pdl_enter();
    static_assert(PFKV_PREFIX_MAX <= kPersMaxSegments, "room for either");
    __shared__ int count[kPersMaxSegments];
    int x = blockIdx.x;
    if (x == 0) {
        plan_segments(a, count);
        return;
    }
    if (x == 1) {
        if (o.status) plan_own_units(a, o, count);
        return;
    }
    x -= 2;
    if (x < pre_tiles) {
        if (short_rows(a.pre)) check_tile<FP8, true>(a, a.pre, x, 0, a.pre_bits, a.pre_vmax);
        else check_tile<FP8, false>(a, a.pre, x / a.pre.htiles, x % a.pre.htiles, a.pre_bits, a.pre_vmax);
        return;
    }
    x -= pre_tiles;
    if (x < own_tiles) {
        if (short_rows(a.own)) check_tile<false, true>(a, a.own, x, 0, a.own_bits, nullptr);
        else check_tile<false, false>(a, a.own, x / a.own.htiles, x % a.own.htiles, a.own_bits, nullptr);
        return;
    }
    // queries as rows that follow each other
    x -= own_tiles;
    const int per = D / 8, Hq = a.Hkv * a.G;
    const long long chunks = (long long)a.B * a.kq * Hq * per;
#pragma unroll
    for (int j = 0; j < kPackPer; ++j) {
        const long long at = ((long long)x * kPackPer + j) * kValThreads + threadIdx.x;
        if (at >= chunks) return;
        const long long row = at / per;
        const int c = (int)(at - row * per), hq = (int)(row % Hq);
        const long long v = row / Hq;
        const int b = (int)(v / a.kq), t = (int)(v - (long long)b * a.kq);
        reinterpret_cast<uint4 *>(a.packed_q)[at] = *reinterpret_cast<const uint4 *>(
            a.q.p + (long long)b * a.q.sb + (long long)t * a.q.st + (long long)hq * a.q.sh + c * 8);
    }
}

// --------------------------------------------------------------------------
// The merge: a CTA a (request, query token, kv head).  Its partial results are those that the
// CTAs of the attention over the prefix left for its rows, and those that the workers of the own
// tokens' split kernel left for its segment; out = sum 2^(lse - M) o / sum 2^(lse - M).
//
// What it needs of the plan (and no partial result) is read before its wait: the plan had ended
// when the kernel before this one let it start (`early`; not where the plan itself is that kernel; the
// rules are at launch_pdl).
//
// Bound by the latency of its rows, hence several a thread on their way at once: 9 us for 32 requests
// of 32 heads, 17 us for 256 of 64 (about 44 MB of partial rows, 2.6 TB/s).
// --------------------------------------------------------------------------
constexpr int kMergeThreads = 256;

template <int D, int G>
__global__ void __launch_bounds__(kMergeThreads, G == 8 ? 5 : 4) prefix_merge_kernel(PrefixArgs a, PrefixOwnRows own, int early) {
    constexpr int C4 = D / 4, TPR = G * C4, WAYS = kMergeThreads / TPR;
    static_assert(WAYS >= 1 && TPR * WAYS == kMergeThreads, "every thread has a place");
    __shared__ uint32_t s_flags;
    __shared__ float s_m[WAYS][G], s_s[WAYS][G];
    __shared__ float4 s_o[WAYS][TPR];
    if (!early) pdl_enter();
    const int v = blockIdx.x / a.Hkv, h = blockIdx.x - v * a.Hkv, b = v / a.kq, t = v - b * a.kq;
    const int tid = threadIdx.x, lane = tid & 31;
    if (tid == 0) s_flags = 0u;
    // the request's flags, but for waits that gave up
    const int p = a.prefix_of[b];
    const PrefixPlace place = a.place[b];
    const bool member = place.row >= 0;
    uint32_t f = p < -1 || p >= a.pre.count ? PFKV_FLAG_BAD_PAGE : 0u;
    if (member)
        for (int i = tid; i < a.Hkv * a.pre.htiles; i += kMergeThreads) f |= a.pre_bits[(long long)p * a.Hkv * a.pre.htiles + i];
    // own tokens: rows k + worker of the request's group of launches
    long long own_row = 0;
    int own_n = 0;
    size_t shift = 0;
    if (own.status) {
        for (int i = tid; i < a.Hkv * a.own.htiles; i += kMergeThreads) f |= a.own_bits[(long long)b * a.Hkv * a.own.htiles + i];
        const int grp = b / own.greq, r0 = grp * own.greq, Bg = min(own.greq, a.B - r0);
        shift = (size_t)grp * own.group_bytes;
        const int *units = own.units + (long long)grp * (own.greq * a.kq * a.Hkv + 1);
        const int U = units[Bg * a.kq * a.Hkv], W = min(own.workers, U);
        const int k = ((b - r0) * a.kq + t) * a.Hkv + h, u0 = units[k], u1 = units[k + 1];
        if (u1 > u0) {
            const int w0 = pers_worker_of(u0, U, W);
            own_row = k + w0;
            own_n = pers_worker_of(u1 - 1, U, W) - w0 + 1;
        }
    }
    // the prefix's: one a CTA that touched the rows' segment
    int pre_n = 0, pre_rows = 0, base = 0, block_row = 0;
    if (member) {
        const int R = place.row + t * G;
        const PrefixSeg sg = a.seg[place.seg + h * place.nb + R / kPrefixBlock];
        pre_n = sg.ctas;
        pre_rows = rows8(sg.rows);
        base = sg.base;
        block_row = R % kPrefixBlock;
    }
    __syncthreads();  // s_flags
    if (early) pdl_enter();

    // rows, several on their way together.  Threads of a way: query heads first, so that a warp reads
    // pieces of G rows (64 bytes with four heads) of a prefix's result.
    const int way = tid / TPR, e = tid - way * TPR, g = e % G, c = e / G;
    const uint32_t *own_status = reinterpret_cast<const uint32_t *>(reinterpret_cast<const uint8_t *>(own.status) + shift);
    const float *own_lse = reinterpret_cast<const float *>(reinterpret_cast<const uint8_t *>(own.lse) + shift);
    const float *own_o = reinterpret_cast<const float *>(reinterpret_cast<const uint8_t *>(own.o) + shift);
    float M = -INFINITY, S = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    const int n = pre_n + own_n;
    constexpr int RB = G == 8 ? 4 : 6;
    uint32_t gave_up = member && tid == 0 ? a.head->timeout : 0u;
    for (int j0 = way; j0 < n; j0 += RB * WAYS) {
        float l[RB];
        float4 x[RB];
        uint32_t st[RB];
#pragma unroll
        for (int r = 0; r < RB; ++r) {
            const int j = j0 + r * WAYS;
            l[r] = -INFINITY;
            x[r] = make_float4(0.f, 0.f, 0.f, 0.f);
            st[r] = 0u;
            if (j < pre_n) {
                const long long first = base + (long long)j * pre_rows;
                l[r] = a.plse[first + block_row + g];
                x[r] = reinterpret_cast<const float4 *>(a.po + first * D)[(long long)c * pre_rows + block_row + g];
            } else if (j < n) {
                const long long row = own_row + j - pre_n;
                l[r] = own_lse[row * G + g];
                x[r] = reinterpret_cast<const float4 *>(own_o + (row * G + g) * D)[c];
                if (e == 0) st[r] = own_status[row];
            }
        }
#pragma unroll
        for (int r = 0; r < RB; ++r) {
            gave_up |= st[r];
            if (l[r] == -INFINITY) continue;  // no token
            if (l[r] > M) {
                const float down = exp2f(M - l[r]);
                S *= down;
                acc = make_float4(acc.x * down, acc.y * down, acc.z * down, acc.w * down);
                M = l[r];
            }
            const float w = exp2f(l[r] - M);
            S += w;
            acc = make_float4(fmaf(w, x[r].x, acc.x), fmaf(w, x[r].y, acc.y), fmaf(w, x[r].z, acc.z), fmaf(w, x[r].w, acc.w));
        }
    }
    f |= gave_up;
    f = __reduce_or_sync(0xffffffffu, f);
    if (lane == 0 && f) atomicOr(&s_flags, f);
    if (WAYS > 1) {
        if (c == 0) {
            s_m[way][g] = M;
            s_s[way][g] = S;
        }
        s_o[way][e] = acc;
    }
    __syncthreads();
    // The bits of checks are those of every CTA of the request; a wait that gave up in the own tokens'
    // workers is known to the CTA of their head alone.
    const uint32_t flags = s_flags;
    if (flags && tid == 0) {
        if (a.flags) atomic_or_byte(a.flags, b, flags);
        if (a.rflags) atomic_or_byte(a.rflags, b, flags);
    }
    if (way != 0) return;
    __nv_bfloat16 *out = a.out.p + (long long)b * a.out.sb + (long long)t * a.out.st + (long long)(h * G + g) * a.out.sh + c * 4;
    if (flags) {
        *reinterpret_cast<uint2 *>(out) = make_uint2(0u, 0u);
        return;
    }
#pragma unroll
    for (int w2 = 1; w2 < WAYS; ++w2) {
        const float M2 = s_m[w2][g], S2 = s_s[w2][g];
        const float4 y = s_o[w2][e];
        if (S2 == 0.f) continue;
        const float top = fmaxf(M, M2), f1 = M == top ? 1.f : exp2f(M - top), f2 = M2 == top ? 1.f : exp2f(M2 - top);
        S = S * f1 + S2 * f2;
        acc = make_float4(acc.x * f1 + y.x * f2, acc.y * f1 + y.y * f2, acc.z * f1 + y.z * f2, acc.w * f1 + y.w * f2);
        M = top;
    }
    if (c == 0 && own.lse_fin) own.lse_fin[((long long)v * a.Hkv + h) * G + g] = S == 0.f ? -INFINITY : M + log2f(S);
    const float inv = S == 0.f ? 0.f : 1.f / S;
    const __nv_bfloat162 lo = __floats2bfloat162_rn(acc.x * inv, acc.y * inv), hi = __floats2bfloat162_rn(acc.z * inv, acc.w * inv);
    *reinterpret_cast<uint2 *>(out) = make_uint2(*reinterpret_cast<const uint32_t *>(&lo), *reinterpret_cast<const uint32_t *>(&hi));
}

template <int D>
cudaError_t launch_merge_d(const PrefixArgs &a, const PrefixOwnRows &o, cudaStream_t s) {
    const dim3 grid((unsigned)((long long)a.B * a.kq * a.Hkv)), block(kMergeThreads);
    const int early = o.status != nullptr || a.pre.count > 0;
    switch (a.G) {
        case 1: return launch_pdl(prefix_merge_kernel<D, 1>, grid, block, 0, s, a, o, early);
        case 2: return launch_pdl(prefix_merge_kernel<D, 2>, grid, block, 0, s, a, o, early);
        case 4: return launch_pdl(prefix_merge_kernel<D, 4>, grid, block, 0, s, a, o, early);
        case 8: return launch_pdl(prefix_merge_kernel<D, 8>, grid, block, 0, s, a, o, early);
    }
    return cudaErrorInvalidValue;
}

template <int D>
cudaError_t preload_merge_d() {
    cudaError_t e = preload_kernel(prefix_merge_kernel<D, 1>);
    if (e == cudaSuccess) e = preload_kernel(prefix_merge_kernel<D, 2>);
    if (e == cudaSuccess) e = preload_kernel(prefix_merge_kernel<D, 4>);
    if (e == cudaSuccess) e = preload_kernel(prefix_merge_kernel<D, 8>);
    return e;
}

}  // namespace

cudaError_t launch_prefix_plan(const PrefixArgs &a, const PrefixOwnRows &o, int D, bool fp8, cudaStream_t s) {
    const auto checks = [&](const PrefixTables &t) {
        const long long rows = (long long)t.count * a.Hkv;
        return short_rows(t) ? (rows + kValThreads / 32 - 1) / (kValThreads / 32) : rows * t.htiles;
    };
    const long long pre = checks(a.pre), own = checks(a.own);
    const long long chunks = a.packed_q ? (long long)a.B * a.kq * a.Hkv * a.G * (D / 8) : 0;
    const long long pack = (chunks + kPackPer * kValThreads - 1) / (kPackPer * kValThreads);
    const dim3 grid((unsigned)(2 + pre + own + pack)), block(kValThreads);
    return launch_pdl(fp8 ? prefix_plan_kernel<true> : prefix_plan_kernel<false>, grid, block, 0, s, a, o, D, (int)pre, (int)own);
}

cudaError_t launch_prefix_merge(const PrefixArgs &a, const PrefixOwnRows &o, int D, cudaStream_t s) {
    return D == 128 ? launch_merge_d<128>(a, o, s) : launch_merge_d<64>(a, o, s);
}

cudaError_t preload_prefix() {
    cudaError_t e = preload_kernel(prefix_plan_kernel<false>);
    if (e == cudaSuccess) e = preload_kernel(prefix_plan_kernel<true>);
    if (e == cudaSuccess) e = preload_merge_d<128>();
    if (e == cudaSuccess) e = preload_merge_d<64>();
    if (e == cudaSuccess) e = preload_prefix_attn();
    return e;
}

namespace {

size_t up256(size_t x) { return (x + 255) & ~size_t(255); }

constexpr int kMaxTokens = 1 << 30;  // of a request or prefix: indices and their round-ups are ints

// Checks of what sizes a call (no CUDA call).
pfkv_status check_prefix(const pfkv_cache *cache, const pfkv_pages *pages, const pfkv_pages *prefixes, int32_t batch,
                         int32_t num_q_heads, int32_t kq, int32_t max_seq_len, int32_t max_prefix_len, bool mass) {
    pfkv_status st = check_cache(cache);
    if (st != PFKV_OK) return st;
    if (batch < 0) return PFKV_ERR_INVALID_ARG;
    if (pages) {
        st = check_pages(cache, pages);
        if (st != PFKV_OK) return st;
        if (pages->batch != batch || max_seq_len < 0) return PFKV_ERR_INVALID_ARG;
        if (max_seq_len > kMaxTokens) return PFKV_ERR_UNSUPPORTED;
    }
    if (!prefixes || prefixes->batch < 0 || max_prefix_len < 0) return PFKV_ERR_INVALID_ARG;
    if (prefixes->batch > 0) {
        st = check_pages(cache, prefixes);
        if (st != PFKV_OK) return st;
    }
    if (prefixes->batch > PFKV_PREFIX_MAX || max_prefix_len > kMaxTokens) return PFKV_ERR_UNSUPPORTED;
    if (num_q_heads <= 0 || num_q_heads % cache->num_kv_heads != 0 || kq < 1) return PFKV_ERR_INVALID_ARG;
    const int G = num_q_heads / cache->num_kv_heads;
    if (G != 1 && G != 2 && G != 4 && G != 8) return PFKV_ERR_UNSUPPORTED;
    if ((long long)kq * cache->num_kv_heads > kPersMaxSegments) return PFKV_ERR_UNSUPPORTED;
    if (mass && !pages) return PFKV_ERR_INVALID_ARG;
    if (mass && kq != 1) return PFKV_ERR_UNSUPPORTED;
    if ((long long)batch * kq > 0x7fffffffLL / num_q_heads) return PFKV_ERR_UNSUPPORTED;
    return PFKV_OK;
}

// Units a worker above which the split kernel takes 12 workers (by the bound of the lengths).  Behind a
// prefix requests' own tokens are few and of many lengths.  Calls behind 16,384 tokens, 8 heads, lengths
// up to n, with 8 and with 12 workers (us): 32 requests, n = 300: 42, 43; 600: 45, 44; 1,200 (just below
// the border): 50, 48; 1,300 (just above): 51, 49; 2,048: 54, 52; 64 requests, n = 600: 60, 58; 650: 62, 58;
// 128, n = 256: 87, 82; 350: 99, 86.  So 12 gain most where there are many requests and lose where few are long
// (8 requests, n = 4,800: 49, 51; 5,200: 49, 53), which a border in units cannot tell apart.
constexpr int kOwnUnitsPerWorker = 16;

int check_words(const pfkv_pages *p) { return max(1, (p->max_pages + kValTile - 1) / kValTile); }

// Where everything lies in the workspace.
struct Layout {
    size_t head, pre_bits, pre_vmax, own_bits, place, pos, members, mstart, seg0, pair, seg, range, units, plse, po, packed, own, mass, total;
    size_t group_bytes;
    DecodePlan plan;  // of the own tokens
};

pfkv_status lay_out(const pfkv_cache *c, const pfkv_pages *pages, const pfkv_pages *prefixes, int32_t batch,
                    int32_t num_q_heads, int32_t kq, int32_t max_seq_len, int32_t max_prefix_len, bool mass, int sms,
                    Layout *l) {
    const long long H = c->num_kv_heads, NP = prefixes->batch, rows = (long long)batch * kq * (num_q_heads / H);
    const int pre_words = NP > 0 ? check_words(prefixes) : 0, own_words = pages ? check_words(pages) : 0;
    // segments, tiles and rows of partial results, at most
    const long long S = NP > 0 ? H * (min(NP, (long long)batch) + rows / kPrefixBlock) : 0;
    const long long tiles = ((long long)max_prefix_len + kPrefixTile - 1) / kPrefixTile;
    if (S > 0x7fffffffLL || (tiles > 0 && S > 0x7fffffffLL / tiles)) return PFKV_ERR_UNSUPPORTED;
    const long long partial = NP > 0 ? H * rows + 8 * S + (long long)sms * kPrefixBlock : 0;
    const long long words = NP * H * pre_words + batch * H * own_words;
    const long long pack = rows * H * c->head_dim / (8 * kPackPer * kValThreads) + 1;
    if (partial > 0x7fffffffLL || words + pack + 2 > 0x7fffffffLL) return PFKV_ERR_UNSUPPORTED;
    size_t off = 0;
    auto take = [&](size_t bytes) {
        const size_t at = off;
        off = up256(off + bytes);
        return at;
    };
    l->head = take(sizeof(PrefixHead));
    l->pre_bits = take(4 * (size_t)(NP * H * pre_words));
    l->pre_vmax = take(c->dtype == PFKV_KV_FP8_E4M3 ? 4 * (size_t)(NP * H * pre_words) : 0);
    l->own_bits = take(4 * (size_t)(batch * H * own_words));
    l->place = take(sizeof(PrefixPlace) * (size_t)batch);
    l->pos = take(4 * (size_t)batch);
    l->members = take(4 * (size_t)batch);
    l->mstart = take(4 * (size_t)(NP + 1));
    l->seg0 = take(4 * (size_t)(NP + 1));
    l->pair = take(sizeof(int2) * (size_t)(NP * H));
    l->seg = take(sizeof(PrefixSeg) * (size_t)S);
    l->range = take(sizeof(PrefixRange) * (size_t)sms);
    l->plse = take(4 * (size_t)partial);
    l->po = take(4 * (size_t)partial * c->head_dim);
    l->packed = take(pages ? 2 * (size_t)(rows * H) * c->head_dim : 0);
    l->own = l->mass = off;
    l->group_bytes = 0;
    if (pages) {
        const pfkv_status st = make_plan(c, pages, num_q_heads, 0, max_seq_len, sms, &l->plan, mass, kq, false, kOwnUnitsPerWorker);
        if (st != PFKV_OK) return st;
        if (l->plan.kind != 1 || l->plan.nchunks != 1) return PFKV_ERR_UNSUPPORTED;
        // a group of launches keeps its results until the merge; the mass pass's arrays are the call's
        l->group_bytes = l->plan.off_mscore - l->plan.off_prefix;
        l->own = take(l->group_bytes * (size_t)l->plan.ngroups);
        l->mass = take(l->plan.total - l->plan.off_mscore);
        l->units = take(4 * (size_t)l->plan.ngroups * ((size_t)l->plan.greq * kq * H + 1));
    }
    l->total = off;
    return PFKV_OK;
}

// Whether the queries lie as the split kernel reads them.
bool rows_follow(const pfkv_rows *q, int B, int kq, int Hq, int D) {
    return (Hq == 1 || q->stride_h == D) && (kq == 1 || q->stride_t == (int64_t)Hq * D) &&
           (B == 1 || q->stride_b == (int64_t)kq * Hq * D);
}

PrefixTables prefix_tables(const pfkv_pages *p, int max_len) {
    return PrefixTables{p->block_tables, (long long)p->bt_stride_b, (long long)p->bt_stride_h, p->seq_lens,
                        (long long)p->len_stride_b, (long long)p->len_stride_h, p->expected_tags, p->max_pages, max_len,
                        p->batch, check_words(p)};
}

pfkv_status prefix_attn(int tries, const pfkv_cache *cache, const pfkv_pages *pages, const pfkv_pages *prefixes,
                        int32_t batch, const int32_t *prefix_of, const pfkv_rows *q, int32_t num_q_heads, int32_t kq,
                        float sm_scale, int32_t max_seq_len, int32_t max_prefix_len, void *workspace,
                        size_t workspace_bytes, const pfkv_rows *out, float *attn_mass, int64_t mass_stride_b,
                        int64_t mass_stride_h, uint8_t *flags, void *stream) {
    const bool mass = attn_mass != nullptr;
    pfkv_status st = check_prefix(cache, pages, prefixes, batch, num_q_heads, kq, max_seq_len, max_prefix_len, mass);
    if (st != PFKV_OK) return st;
    if (!(sm_scale == sm_scale) || std::isinf(sm_scale)) return PFKV_ERR_INVALID_ARG;
    if (batch == 0) return PFKV_OK;
    if (!prefix_of) return PFKV_ERR_INVALID_ARG;
    st = check_rows(q, true, true);
    if (st == PFKV_OK) st = check_rows(out, true, true);
    if (st != PFKV_OK) return st;
    if (mass && (mass_stride_b < 0 || mass_stride_h < 0)) return PFKV_ERR_INVALID_ARG;
    if (!aligned(prefix_of, 4) || !aligned(attn_mass, 4) || !aligned(flags, 4)) return PFKV_ERR_ALIGNMENT;
    if (!workspace || workspace_bytes < sizeof(PrefixHead)) return PFKV_ERR_WORKSPACE;
    if (!aligned(workspace, 256)) return PFKV_ERR_ALIGNMENT;
    int sms = 0;
    st = device_check(&sms);
    if (st != PFKV_OK) return st;
    Layout l{};
    st = lay_out(cache, pages, prefixes, batch, num_q_heads, kq, max_seq_len, max_prefix_len, mass, sms, &l);
    if (st != PFKV_OK) return st;
    if (workspace_bytes < l.total) return PFKV_ERR_WORKSPACE;

    const int D = cache->head_dim;
    const bool fp8 = cache->dtype == PFKV_KV_FP8_E4M3;
    uint8_t *ws = static_cast<uint8_t *>(workspace);
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
    a.kq = kq;
    if (pages) a.own = prefix_tables(pages, max_seq_len);
    if (prefixes->batch > 0) a.pre = prefix_tables(prefixes, max_prefix_len);
    a.prefix_of = prefix_of;
    a.q = rows_arg(q);
    a.out = rows_arg(out);
    a.sm_scale = sm_scale;
    a.flags = flags;
    a.own_bits = reinterpret_cast<uint32_t *>(ws + l.own_bits);
    a.pre_bits = reinterpret_cast<uint32_t *>(ws + l.pre_bits);
    a.pre_vmax = reinterpret_cast<float *>(ws + l.pre_vmax);
    a.head = reinterpret_cast<PrefixHead *>(ws + l.head);
    a.place = reinterpret_cast<PrefixPlace *>(ws + l.place);
    a.pos = reinterpret_cast<int *>(ws + l.pos);
    a.members = reinterpret_cast<int *>(ws + l.members);
    a.mstart = reinterpret_cast<int *>(ws + l.mstart);
    a.seg0 = reinterpret_cast<int *>(ws + l.seg0);
    a.pair = reinterpret_cast<int2 *>(ws + l.pair);
    a.seg = reinterpret_cast<PrefixSeg *>(ws + l.seg);
    a.range = reinterpret_cast<PrefixRange *>(ws + l.range);
    a.plse = reinterpret_cast<float *>(ws + l.plse);
    a.po = reinterpret_cast<float *>(ws + l.po);
    const bool packs = pages && !rows_follow(q, batch, kq, num_q_heads, D);
    a.packed_q = packs ? reinterpret_cast<__nv_bfloat16 *>(ws + l.packed) : nullptr;
    a.ctas = sms;
    a.tries = tries;
    a.after_own = pages != nullptr;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    DecodeArgs d{};
    PrefixOwnRows own{};
    if (pages) {
        const DecodePlan &plan = l.plan;
        uint8_t *part = ws + l.own - plan.off_prefix;  // of the plan's offsets
        d.k_pages = cache->k_pages;
        d.v_pages = cache->v_pages;
        d.k_scale = cache->k_scale;
        d.v_scale = cache->v_scale;
        d.num_pages = cache->num_pages;
        d.block_tables = pages->block_tables;
        d.bt_sb = pages->bt_stride_b;
        d.bt_sh = pages->bt_stride_h;
        d.seq_lens = pages->seq_lens;
        d.len_sb = pages->len_stride_b;
        d.len_sh = pages->len_stride_h;
        d.max_pages = pages->max_pages;
        d.max_seq_len = max_seq_len;
        d.q = packs ? a.packed_q : a.q.p;
        d.q_scale = sm_scale * 1.4426950408889634f;  // log2(e): scores in log2 units
        d.hflags = a.own_bits;
        d.htiles = plan.htiles;
        d.kq = kq;
        d.status = reinterpret_cast<uint32_t *>(part + plan.off_status);
        d.lse = reinterpret_cast<float *>(part + plan.off_lse);
        d.o = reinterpret_cast<float *>(part + plan.off_o);
        d.ws_prefix = reinterpret_cast<int *>(part + plan.off_prefix);
        // the plan kernel checks tables and lengths as the validation kernel does; the split kernel may
        // read queries before it has ended unless they are packed there
        d.early = packs ? 0 : 1;
        if (mass) {
            uint8_t *m = ws + l.mass - plan.off_mscore;
            d.mscore = reinterpret_cast<float *>(m + plan.off_mscore);
            d.mlen = max_seq_len;
            d.lse_fin = reinterpret_cast<float *>(m + plan.off_lsefin);
            d.rflags = m + plan.off_rflags;
            d.mass = attn_mass;
            d.mass_sb = mass_stride_b;
            d.mass_sh = mass_stride_h;
        }
        own = PrefixOwnRows{d.status, d.lse, d.o, l.group_bytes, reinterpret_cast<int *>(ws + l.units), plan.greq,
                            plan.workers, plan.chunk_tokens, d.lse_fin};
        a.rflags = d.rflags;
    }
    if (launch_prefix_plan(a, own, D, fp8, s) != cudaSuccess) return PFKV_ERR_CUDA;
    if (pages) {
        const DecodePlan &plan = l.plan;
        for (int g = 0; g < plan.ngroups; ++g) {
            DecodePlan pg = plan;
            pg.Breq = min(plan.greq, plan.Breq - g * plan.greq);
            pg.B = pg.Breq * kq;
            DecodeArgs dg = group_args(d, plan, g * plan.greq);
            const size_t shift = (size_t)g * l.group_bytes;
            const auto moved = [&](auto *p) { return reinterpret_cast<decltype(p)>(reinterpret_cast<uint8_t *>(p) + shift); };
            dg.status = moved(d.status);
            dg.lse = moved(d.lse);
            dg.o = moved(d.o);
            dg.ws_prefix = moved(d.ws_prefix);
            if (launch_split(dg, pg, s) != cudaSuccess) return PFKV_ERR_CUDA;
        }
    }
    if (prefixes->batch > 0 && launch_prefix_attn(a, D, fp8, s) != cudaSuccess) return PFKV_ERR_CUDA;
    if (launch_prefix_merge(a, own, D, s) != cudaSuccess) return PFKV_ERR_CUDA;
    if (mass && launch_mass(d, l.plan, s) != cudaSuccess) return PFKV_ERR_CUDA;
    return PFKV_OK;
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
    pfkv_status st = check_prefix(cache, pages, prefixes, batch, num_q_heads, num_query_tokens, max_seq_len,
                                  max_prefix_len, with_mass != 0);
    if (st != PFKV_OK) return st;
    int sms = 0;
    st = device_check(&sms);
    if (st != PFKV_OK) return st;
    Layout l{};
    st = lay_out(cache, pages, prefixes, batch, num_q_heads, num_query_tokens, max_seq_len, max_prefix_len,
                 with_mass != 0, sms, &l);
    if (st != PFKV_OK) return st;
    *bytes = l.total;
    return PFKV_OK;
}

pfkv_status pfkv_prefix_decode_attn(const pfkv_cache *cache, const pfkv_pages *pages, const pfkv_pages *prefixes,
                                    int32_t batch, const int32_t *prefix_of, const pfkv_rows *q, int32_t num_q_heads,
                                    int32_t num_query_tokens, float sm_scale, int32_t max_seq_len,
                                    int32_t max_prefix_len, void *workspace, size_t workspace_bytes,
                                    const pfkv_rows *out, float *attn_mass, int64_t mass_stride_b,
                                    int64_t mass_stride_h, uint8_t *flags, void *stream) {
    return prefix_attn(kTries, cache, pages, prefixes, batch, prefix_of, q, num_q_heads, num_query_tokens, sm_scale,
                       max_seq_len, max_prefix_len, workspace, workspace_bytes, out, attn_mass, mass_stride_b,
                       mass_stride_h, flags, stream);
}

pfkv_status pfkv_selftest_prefix_decode(int32_t tries, const pfkv_cache *cache, const pfkv_pages *pages,
                                        const pfkv_pages *prefixes, int32_t batch, const int32_t *prefix_of,
                                        const pfkv_rows *q, int32_t num_q_heads, int32_t num_query_tokens,
                                        float sm_scale, int32_t max_seq_len, int32_t max_prefix_len, void *workspace,
                                        size_t workspace_bytes, const pfkv_rows *out, float *attn_mass,
                                        int64_t mass_stride_b, int64_t mass_stride_h, uint8_t *flags, void *stream) {
    if (tries < 0 || tries > kTries) return PFKV_ERR_INVALID_ARG;
    return prefix_attn(tries, cache, pages, prefixes, batch, prefix_of, q, num_q_heads, num_query_tokens, sm_scale,
                       max_seq_len, max_prefix_len, workspace, workspace_bytes, out, attn_mass, mass_stride_b,
                       mass_stride_h, flags, stream);
}

}  // extern "C"

// latent_decode.cu -- pfkv_latent_decode_attn: attention in the absorbed form
// over a paged latent cache (declared in pfkv_latent.h).
//
// Mathematics.  R = query tokens x heads rows of a request share every token's
// latent c_j (512 values) and rotated key r_j (64):
//     S = scale (Q_c C^T + Q_r R^T),   O = softmax(S) C,
// 2 R (576 + 512) operations a token for 1,152 bytes (BF16) or 640 (FP8): at 128
// rows 242 or 435 operations a byte, where this GPU turns from memory-bound to
// tensor-bound (288 at the measured rates).  So both products run on the
// fifth-generation tensor cores, and every latent is to be read from HBM once.
//
// Why a pair of CTAs.  A row's result is 512 fp32 values: 128 rows of it fill a
// streaming multiprocessor's whole tensor memory, and the scores have no room.
// With 64 rows a CTA the products run at half rate (measured with operands in
// place: 128 x 128 x 16 on one CTA 64 cycles, 64 x 128 x 16 the same 64).  Two
// CTAs of a cluster issued as one (cta_group::2) do 128 rows at full rate (128 x
// 128 x 16 in 32 cycles), each holding 64 rows: 256 columns for O, two buffers of
// 64 or 128 for S.
//
// A tile is 128 tokens (8 pages).  For S each CTA brings 64 of them (K: nine
// chunks of 64 values, 8 KB each); for O each brings all 128 tokens of 256 of the
// values (V: four chunks, 16 KB each), as V's columns are split between the
// CTAs.  Each latent is thus read from HBM once, and from L2 twice.  Shared
// memory (Q 72 KB, K 72 KB, V 64 KB, P 16 KB) leaves no room for second buffers;
// instead every chunk's slot is refilled as soon as its last product has
// completed, and an L2 prefetch runs two tiles ahead.
//
// Softmax: one pass.  Two threads hold a row (64 tokens each), in log2 units, with
// a running reference that moves only when the maximum has grown by 2^8 (then O
// is rescaled in tensor memory).  FP8: a weight enters the second product times
// its page's scale z_j; the reference is of s_j + log2 z_j, so that the f16
// weights stay in range and the largest keep their 11 bits however far apart the
// scales are; the weights' sum takes the rounded weight over z_j.
//
// Work: the tiles of all (request, 128-row block) pairs are one list, cut into
// equal ranges for the clusters.  A pair that lies in one range is written out
// directly; parts of a pair go to the workspace (normalised rows and their
// log2-sum-exp) and a second kernel merges them.
//
// Roles of a CTA's sixteen warps: 0-3 softmax and output; 4 issues the products
// (even CTA) or passes on to it that the odd CTA's operands are in place; 5 and 6
// load K and V (BF16: TMA, one box of 16 tokens x 64 values a page and chunk); FP8:
// 8-11 and 12-15 convert K and V to f16 between L2 and shared memory; 8-11 load Q.
#include <type_traits>

#include "latent_internal.cuh"
#include "umma.cuh"

namespace pfkv {
namespace {

constexpr int kDC = PFKV_LATENT_DIM;
constexpr int kTile = 128;                    // tokens a tile
constexpr int kTilePages = kTile / kPage;
constexpr int kRowsCta = 64, kRowBlock = 128;
constexpr int kKChunks = 9;                   // 8 of latents, 1 of rotated keys
constexpr uint32_t kChunkB = kRowsCta * 128;  // Q, K and P chunks: 64 rows of 128 bytes
constexpr uint32_t kVChunkB = kTile * 128;
constexpr int kThreads = 512;
constexpr uint32_t kOffQ = 0, kOffK = kKChunks * kChunkB, kOffV = 2 * kKChunks * kChunkB,
                   kOffP = kOffV + 4 * kVChunkB, kOffMisc = kOffP + 2 * kChunkB;
constexpr float kLazyGrowth = 8.f;
constexpr float kLog2e = 1.4426950408889634f;
// FP8: weights are kept 2^7 above the reference.  The largest then lies between
// 2^7 and 2^15 (f16 holds 2^16), and f16's smallest step is 2^-31 of it or less.
template <bool FP8>
constexpr float kWeightBias = FP8 ? 7.f : 0.f;
constexpr uint32_t kColS = 256;               // tensor memory: O in columns 0-255, S above
constexpr float kNegInf = -INFINITY;

struct Misc {
    uint64_t kfull[kKChunks], kempty[kKChunks], pk[kKChunks];
    uint64_t vfull[2], vempty[2], pv[2];
    uint64_t sfull[2], sq[2], pready, pvdone, qfull, pq, qfree, drain;
    long long warp_sum[kThreads / 32];
    long long x0, x1, off;
    int b0;
    uint32_t tmem, gave_up;
    float xm[kRowBlock];
    float qscale[2][kRowsCta];
};
constexpr size_t kSmemBytes = kOffMisc + sizeof(Misc) + 1024;
static_assert(kSmemBytes <= 232448, "shared memory of one CTA");

// Workspace: normalised partial rows and their log2-sum-exp, two blocks a
// cluster (the part of a pair that began before its range, and the part of one
// that ends after it), and a word a CTA that says whether its waits gave up.
struct Parts {
    float *o;        // [clusters][2][rows][512]
    float *lse;      // [clusters][2][rows]
    uint32_t *gave_up;  // [clusters][2]
    int rows;        // min(R, 128)
};

struct DecodePlan2 {
    int R, blocks, W;
};

// Tokens of request b, 0 for a length that is refused.
__device__ __forceinline__ int live_len(const LatentDecodeArgs &a, int b) {
    const int n = a.pool.seq_lens[(long long)b * a.pool.len_sb];
    return n < 0 || (long long)n > (long long)a.pool.max_pages * kPage || n > a.max_seq_len ? 0 : n;
}
__device__ __forceinline__ int tiles_of(int n) { return (n + kTile - 1) / kTile; }

// First unit of cluster w's range, U units over W clusters.
__device__ __forceinline__ long long range_start(long long w, long long U, int W) { return (w * U + W - 1) / W; }

// One (request, row block) part of a cluster's range: tiles t0 .. t1 - 1.
struct Segment {
    int b, block, t0, t1, tiles, n;
};

// Walks a range of the list of tiles.
struct Walk {
    long long x, x1, off;
    int b;
    __device__ __forceinline__ bool next(const LatentDecodeArgs &a, int blocks, Segment &s) {
        if (x >= x1) return false;
        int n, tiles;
        while (true) {
            n = live_len(a, b);
            tiles = tiles_of(n);
            if (off < (long long)tiles * blocks) break;
            ++b;
            off = 0;
        }
        s.b = b;
        s.n = n;
        s.tiles = tiles;
        s.block = (int)(off / tiles);
        s.t0 = (int)(off - (long long)s.block * tiles);
        s.t1 = (int)min((long long)tiles, s.t0 + (x1 - x));
        x += s.t1 - s.t0;
        off += s.t1 - s.t0;
        return true;
    }
};

// The same, a tile at a time.
struct TileWalk {
    Walk w;
    Segment s;
    int t;
    bool first, last, live;
    __device__ __forceinline__ void start(const LatentDecodeArgs &a, int blocks, const Walk &walk) {
        w = walk;
        live = w.next(a, blocks, s);
        t = live ? s.t0 : 0;
        first = true;
        last = live && t + 1 == s.t1;
    }
    __device__ __forceinline__ void step(const LatentDecodeArgs &a, int blocks) {
        if (++t < s.t1) {
            first = false;
        } else {
            live = w.next(a, blocks, s);
            t = live ? s.t0 : 0;
            first = true;
        }
        last = live && t + 1 == s.t1;
    }
};

// The physical page of logical page p of request b, or -1 for one that is not to
// be read (past the length, a bad id, a stale tag: the merge kernel flags those
// and zeroes the request).
__device__ __forceinline__ int page_of(const LatentDecodeArgs &a, int b, int p, int n) {
    if (p >= (n + kPage - 1) / kPage) return -1;
    const long long bi = (long long)b * a.pool.bt_sb + p;
    const int id = a.pool.block_tables[bi];
    return latent_entry_bits(a.pool, id, bi) ? -1 : id;
}

__device__ __forceinline__ uint4 cvt_e4m3x8(uint32_t lo, uint32_t hi) {
    uint4 r;
    asm("{\n\t.reg .b16 a, b, c, d;\n\tmov.b32 {a, b}, %4;\n\tmov.b32 {c, d}, %5;\n\t"
        "cvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t"
        "cvt.rn.f16x2.e4m3x2 %2, c;\n\tcvt.rn.f16x2.e4m3x2 %3, d;\n\t}"
        : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
        : "r"(lo), "r"(hi));
    return r;
}

// Piece c (16 bytes) of row r of a swizzled chunk.
__device__ __forceinline__ uint4 *piece(uint8_t *chunk, int r, int c) {
    return reinterpret_cast<uint4 *>(chunk + r * 128 + ((c ^ (r & 7)) << 4));
}

// Query rows of one segment into shared memory, by 128 threads: two a row.  FP8:
// the latent part as f16 over a power of two that puts its largest element in
// [1, 2); the rotated part stays bf16.  Rows past the last are zero.
template <bool FP8>
__device__ __forceinline__ void load_queries(const LatentDecodeArgs &a, const Segment &s, int R, uint32_t rank,
                                             uint8_t *q, float *qscale, int i) {
    const int r = i >> 1, sub = i & 1;
    const int row = s.block * kRowBlock + (int)rank * kRowsCta + r;
    const bool live = row < R;
    const int t = live ? row / a.H : 0, h = live ? row - t * a.H : 0;
    const uint4 *c = reinterpret_cast<const uint4 *>(a.qc.p + (long long)s.b * a.qc.sb + (long long)t * a.qc.st +
                                                     (long long)h * a.qc.sh);
    const uint4 *e = reinterpret_cast<const uint4 *>(a.qr.p + (long long)s.b * a.qr.sb + (long long)t * a.qr.st +
                                                     (long long)h * a.qr.sh);
    const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
    float inv = 1.f;
    if constexpr (FP8) {
        uint32_t top = 0;  // largest magnitude as bf16 bits (integers order as magnitudes do)
#pragma unroll
        for (int g = 0; g < 2; ++g) {
            uint4 w[16];
#pragma unroll
            for (int j = 0; j < 16; ++j) w[j] = live ? c[(g * 16 + j) * 2 + sub] : zero;
#pragma unroll
            for (int j = 0; j < 16; ++j) {
                const uint32_t u[4] = {w[j].x, w[j].y, w[j].z, w[j].w};
#pragma unroll
                for (int k = 0; k < 4; ++k) top = max(top, max(u[k] & 0x7FFFu, (u[k] >> 16) & 0x7FFFu));
            }
        }
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
        // biased exponent, kept where both 2^e and 2^-e are normal fp32 numbers
        const int eb = min(253, max(1, (int)(top >> 7)));
        inv = __uint_as_float((uint32_t)(254 - eb) << 23);
        if (sub == 0) qscale[r] = __uint_as_float((uint32_t)eb << 23);
    }
#pragma unroll
    for (int g = 0; g < 4; ++g) {
        uint4 w[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) w[j] = live ? c[(g * 8 + j) * 2 + sub] : zero;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int p = (g * 8 + j) * 2 + sub;
            if constexpr (FP8) {
                const uint32_t u[4] = {w[j].x, w[j].y, w[j].z, w[j].w};
                uint32_t o[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const float2 f = bf16x2_to_float2(u[k]);
                    const __half2 v = __floats2half2_rn(f.x * inv, f.y * inv);
                    o[k] = *reinterpret_cast<const uint32_t *>(&v);
                }
                w[j] = make_uint4(o[0], o[1], o[2], o[3]);
            }
            *piece(q + (p >> 3) * kChunkB, r, p & 7) = w[j];
        }
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) *piece(q + 8 * kChunkB, r, j * 2 + sub) = live ? e[j * 2 + sub] : zero;
}

// Rows valid .. 127 of the two V chunks at `v`, by one warp: slots past the last
// token may hold anything, NaN among it, and meet weights of zero.
__device__ __forceinline__ void zero_rows(uint8_t *v, int valid, int lane) {
    for (int i = valid * 8 + lane; i < kTile * 8; i += 32) {
        reinterpret_cast<uint4 *>(v)[i] = make_uint4(0u, 0u, 0u, 0u);
        reinterpret_cast<uint4 *>(v + kVChunkB)[i] = make_uint4(0u, 0u, 0u, 0u);
    }
}

template <bool FP8>
__global__ void __launch_bounds__(kThreads, 1)
    latent_split_kernel(const __grid_constant__ CUtensorMap mapc, const __grid_constant__ CUtensorMap mapr,
                        LatentDecodeArgs a, int R, int blocks, int clusters, Parts parts) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t *sm = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    Misc &m = *reinterpret_cast<Misc *>(sm + kOffMisc);
    uint8_t *const q = sm + kOffQ, *const k = sm + kOffK, *const v = sm + kOffV, *const p = sm + kOffP;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t rank = cluster_rank();
    const int w = blockIdx.x >> 1;
    if (tid == 0) {
        for (int c = 0; c < kKChunks; ++c) {
            mbar_init(&m.kfull[c], FP8 && c < 8 ? 4 : 1);
            mbar_init(&m.kempty[c], 1);
            mbar_init(&m.pk[c], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&m.vfull[i], FP8 ? 4 : 1);
            mbar_init(&m.vempty[i], 1);
            mbar_init(&m.pv[i], 1);
            mbar_init(&m.sfull[i], 1);
            mbar_init(&m.sq[i], 4);
        }
        mbar_init(&m.pready, 8);
        mbar_init(&m.pvdone, 1);
        mbar_init(&m.qfull, 4);
        mbar_init(&m.pq, 1);
        mbar_init(&m.qfree, 1);
        mbar_init(&m.drain, 1);
        m.gave_up = 0u;
        m.x0 = m.x1 = 0;
        m.off = 0;
        m.b0 = 0;
        fence_mbar_init();
    }
    if (warp == 4) tmem_alloc512<2>(&m.tmem);
    pdl_enter();

    // this cluster's range of the list of tiles
    {
        const int per = (a.B + kThreads - 1) / kThreads;
        const int lo = min(a.B, tid * per), hi = min(a.B, lo + per);
        long long mine = 0;
        for (int b = lo; b < hi; ++b) mine += (long long)tiles_of(live_len(a, b)) * blocks;
        long long incl = mine;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const long long y = __shfl_up_sync(0xffffffffu, incl, d);
            if (lane >= d) incl += y;
        }
        if (lane == 31) m.warp_sum[warp] = incl;
        tmem_fence_before();
        __syncthreads();
        tmem_fence_after();
        long long before = 0, U = 0;
        for (int i = 0; i < kThreads / 32; ++i) {
            if (i < warp) before += m.warp_sum[i];
            U += m.warp_sum[i];
        }
        const int W = (int)min((long long)clusters, U);
        const long long x0 = w < W ? range_start(w, U, W) : 0, x1 = w < W ? range_start(w + 1, U, W) : 0;
        before += incl - mine;
        if (x0 < x1 && before <= x0 && x0 < before + mine) {
            long long at = before;
            int b = lo;
            for (;; ++b) {
                const long long u = (long long)tiles_of(live_len(a, b)) * blocks;
                if (x0 < at + u) break;
                at += u;
            }
            m.b0 = b;
            m.off = x0 - at;
            m.x0 = x0;
            m.x1 = x1;
        }
    }
    __syncthreads();
    cluster_sync();  // both CTAs' barriers are initialised
    const Walk walk{m.x0, m.x1, m.off, m.b0};
    const uint32_t tmem = m.tmem;
    volatile uint32_t *const gave_up = &m.gave_up;

    if (warp < 4) {
        // ------------------------- softmax and output -------------------------
        const int half = warp >> 1, r = tid & 63;    // lanes 64-127 hold tokens 64-127 of rows 0-63
        const uint32_t lanes = tmem + ((uint32_t)(warp * 32) << 16);
        const float a2 = a.sm_scale * kLog2e;
        TileWalk tw, nx;
        tw.start(a, blocks, walk);
        nx = tw;
        float z[4] = {1.f, 1.f, 1.f, 1.f};
        int zid[4] = {-1, -1, -1, -1};
        auto load_ids = [&](const TileWalk &t) {  // pages of this half of the tile (FP8: their scales)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                zid[i] = t.live ? page_of(a, t.s.b, t.t * kTilePages + half * 4 + i, t.s.n) : -1;
        };
        if constexpr (FP8) {
            load_ids(tw);
#pragma unroll
            for (int i = 0; i < 4; ++i) z[i] = zid[i] >= 0 ? a.pool.c_scale[zid[i]] : 1.f;
            if (nx.live) nx.step(a, blocks);
            load_ids(nx);
        }
        float ref = kNegInf, sum = 0.f, qs = 0.f;
        int lim = 0, row = 0, seg = 0;
        bool live = false, any_live = false;
        for (int t = 0; tw.live; ++t) {
            if (tw.first) {
                row = tw.s.block * kRowBlock + (int)rank * kRowsCta + r;
                live = row < R;
                any_live = __any_sync(0xffffffffu, live);
                lim = tw.s.n - a.kq + 1 + (live ? row / a.H : a.kq - 1);
                ref = kNegInf;
                sum = 0.f;
            }
            float zn[4];
            if constexpr (FP8) {
#pragma unroll
                for (int i = 0; i < 4; ++i) zn[i] = zid[i] >= 0 ? a.pool.c_scale[zid[i]] : 1.f;
            }
            bar_wait(&m.sfull[t & 1], (t >> 1) & 1, gave_up);
            tmem_fence_after();
            if (FP8 && tw.first) {
                bar_wait(&m.sq[seg & 1], (seg >> 1) & 1, gave_up);
                qs = a2 * m.qscale[seg & 1][r];
            }
            seg += tw.last;
            bool waited = false;
            if (any_live) {
                float x[2][32];
                const uint32_t cs = lanes + kColS + (t & 1) * 128;
                tmem_ld32(cs, x[0]);
                tmem_ld32(cs + 32, x[1]);
                tmem_wait_ld();
                float lz[4], iz[4];
                if constexpr (FP8) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float zc = fmaxf(z[i], 7.888609052210118e-31f);  // 2^-100
                        lz[i] = __log2f(zc);
                        iz[i] = __frcp_rn(zc);
                    }
#pragma unroll
                    for (int g = 0; g < 2; ++g) {
                        float y[32];
                        tmem_ld32(cs + 64 + g * 32, y);
                        tmem_wait_ld();
#pragma unroll
                        for (int j = 0; j < 32; ++j) {
                            const int i = g * 2 + (j >> 4);
                            x[g][j] = fmaf(x[g][j], qs * z[i], fmaf(y[j], a2, lz[i]));
                        }
                    }
                } else {
#pragma unroll
                    for (int g = 0; g < 2; ++g)
#pragma unroll
                        for (int j = 0; j < 32; ++j) x[g][j] *= a2;
                }
                const int seen = lim - (tw.t * kTile + half * 64);  // of this thread's 64 tokens
                if (seen < 64) {
#pragma unroll
                    for (int g = 0; g < 2; ++g)
#pragma unroll
                        for (int j = 0; j < 32; ++j)
                            if (g * 32 + j >= seen) x[g][j] = kNegInf;
                }
                float top = kNegInf;
#pragma unroll
                for (int g = 0; g < 2; ++g)
#pragma unroll
                    for (int j = 0; j < 32; ++j) top = fmaxf(top, x[g][j]);
                m.xm[tid] = top;
                // rows' two halves: warps w and w + 2
                asm volatile("bar.sync %0, 64;" ::"r"(1 + (warp & 1)) : "memory");
                top = fmaxf(top, m.xm[tid ^ 64]);
                asm volatile("bar.sync %0, 64;" ::"r"(1 + (warp & 1)) : "memory");
                float shrink = 1.f;
                if (top > ref + kLazyGrowth || (ref == kNegInf && top > kNegInf)) {
                    shrink = fast_exp2(ref - top);  // 0 when nothing was seen yet
                    sum *= shrink;
                    ref = top;
                }
                if (t > 0) {
                    bar_wait(&m.pvdone, (t - 1) & 1, gave_up);  // P is free, O is at rest
                    tmem_fence_after();
                    waited = true;
                }
                if (!tw.first && __any_sync(0xffffffffu, shrink != 1.f)) {
#pragma unroll 1
                    for (int g = 0; g < 8; ++g) {
                        float o[32];
                        tmem_ld32(lanes + g * 32, o);
                        tmem_wait_ld();
                        uint32_t u[32];
#pragma unroll
                        for (int j = 0; j < 32; ++j) u[j] = __float_as_uint(o[j] * shrink);
                        tmem_st32(lanes + g * 32, u);
                    }
                    tmem_wait_st();
                }
                const float base = ref == kNegInf ? 0.f : ref - kWeightBias<FP8>;
                uint8_t *pc = p + half * kChunkB;
#pragma unroll
                for (int c = 0; c < 8; ++c) {
                    uint32_t o[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int j = c * 8 + e * 2;
                        const float w0 = fast_exp2(x[j >> 5][j & 31] - base);
                        const float w1 = fast_exp2(x[(j + 1) >> 5][(j + 1) & 31] - base);
                        if constexpr (FP8) {
                            const __half2 hw = __floats2half2_rn(w0, w1);
                            const float2 f = __half22float2(hw);
                            sum = fmaf(f.x + f.y, iz[c >> 1], sum);
                            o[e] = *reinterpret_cast<const uint32_t *>(&hw);
                        } else {
                            const __nv_bfloat162 hw = __floats2bfloat162_rn(w0, w1);
                            const float2 f = __bfloat1622float2(hw);
                            sum += f.x + f.y;
                            o[e] = *reinterpret_cast<const uint32_t *>(&hw);
                        }
                    }
                    *piece(pc, r, c) = make_uint4(o[0], o[1], o[2], o[3]);
                }
                fence_proxy_async_smem();
            }
            if (!waited && t > 0) bar_wait(&m.pvdone, (t - 1) & 1, gave_up);
            tmem_fence_before();
            __syncwarp();
            if (lane == 0) bar_arrive_at(&m.pready, 0);
            if (tw.last) {
                bar_wait(&m.pvdone, t & 1, gave_up);
                tmem_fence_after();
                if (any_live) {
                    m.xm[tid] = sum;
                    asm volatile("bar.sync %0, 64;" ::"r"(1 + (warp & 1)) : "memory");
                    const float total = sum + m.xm[tid ^ 64];
                    asm volatile("bar.sync %0, 64;" ::"r"(1 + (warp & 1)) : "memory");
                    const float inv = total > 0.f ? __fdiv_rn(1.f, total) : total == 0.f ? 0.f : total;  // NaN stays
                    const bool whole = tw.s.t1 - tw.s.t0 == tw.s.tiles;
                    const int brow = (int)rank * kRowsCta + r;
                    const int slot = w * 2 + (tw.s.t0 == 0 ? 1 : 0);
                    float *po = parts.o + ((long long)slot * parts.rows + brow) * kDC;
                    if (!whole && live && half == 0)
                        parts.lse[(long long)slot * parts.rows + brow] = total == 0.f ? kNegInf : ref - kWeightBias<FP8> + __log2f(total);
                    __nv_bfloat16 *out = a.out.p;
                    if (live) {
                        const int tok = row / a.H;
                        out += (long long)tw.s.b * a.out.sb + (long long)tok * a.out.st +
                               (long long)(row - tok * a.H) * a.out.sh;
                    }
#pragma unroll 1
                    for (int g = 0; g < 8; ++g) {
                        float o[32];
                        tmem_ld32(lanes + g * 32, o);
                        tmem_wait_ld();
                        // columns 0-127: values 0-255, 128-255: values 256-511; each half a row's threads' share
                        const int d = (g >> 2) * 256 + half * 128 + (g & 3) * 32;
                        if (!live) continue;
#pragma unroll
                        for (int j = 0; j < 32; ++j) o[j] = total == 0.f ? 0.f : o[j] * inv;
                        if (whole) {
#pragma unroll
                            for (int j = 0; j < 32; j += 8) {
                                uint32_t u[4];
#pragma unroll
                                for (int e = 0; e < 4; ++e) {
                                    const __nv_bfloat162 h = __floats2bfloat162_rn(o[j + 2 * e], o[j + 2 * e + 1]);
                                    u[e] = *reinterpret_cast<const uint32_t *>(&h);
                                }
                                *reinterpret_cast<uint4 *>(out + d + j) = make_uint4(u[0], u[1], u[2], u[3]);
                            }
                        } else {
#pragma unroll
                            for (int j = 0; j < 32; j += 4)
                                *reinterpret_cast<float4 *>(po + d + j) = make_float4(o[j], o[j + 1], o[j + 2], o[j + 3]);
                        }
                    }
                }
                tmem_fence_before();
            }
            tw.step(a, blocks);
            if constexpr (FP8) {
#pragma unroll
                for (int i = 0; i < 4; ++i) z[i] = zn[i];
                if (nx.live) nx.step(a, blocks);
                load_ids(nx);
            }
        }
    } else if (warp == 4) {
        // ---------------- products (even CTA), relay (odd CTA) ----------------
        const uint32_t qa = smem_addr(q), ka = smem_addr(k), va = smem_addr(v), pa = smem_addr(p);
        constexpr uint32_t idS = umma_idesc(kRowBlock, kTile, !FP8, false, false);
        constexpr uint32_t idR = umma_idesc(kRowBlock, kTile, true, false, false);
        constexpr uint32_t idO = umma_idesc(kRowBlock, 256, !FP8, false, true);
        auto scores = [&](int t, bool first, bool last, int seg) {
            if (first) {
                bar_wait(&m.qfull, seg & 1, gave_up);
                if (rank == 0) bar_wait(&m.pq, seg & 1, gave_up);
                else if (lane == 0) bar_arrive_at(&m.pq, 0);
            }
            const uint32_t cs = tmem + kColS + (t & 1) * 128;
#pragma unroll 1
            for (int c = 0; c < kKChunks; ++c) {
                bar_wait(&m.kfull[c], t & 1, gave_up);
                if (rank != 0) {
                    __syncwarp();
                    if (lane == 0) bar_arrive_at(&m.pk[c], 0);
                    continue;
                }
                bar_wait(&m.pk[c], t & 1, gave_up);
                tmem_fence_after();
                __syncwarp();
                if (!*gave_up && elect_one()) {
                    const bool rope = FP8 && c == 8;
                    const uint64_t da = umma_desc(qa + c * kChunkB, 16, 1024), db = umma_desc(ka + c * kChunkB, 16, 1024);
#pragma unroll
                    for (int s = 0; s < 4; ++s)
                        umma_ss<2>(rope ? cs + 64 : cs, da + 2 * s, db + 2 * s, rope ? idR : idS,
                                   s > 0 || (c > 0 && !rope));
                    umma_commit_pair(&m.kempty[c]);
                    if (c == kKChunks - 1) {
                        umma_commit_pair(&m.sfull[t & 1]);
                        if (last) umma_commit_pair(&m.qfree);
                    }
                }
                __syncwarp();
            }
        };
        auto values = [&](int t, bool first, int valid) {
            if (rank == 0) bar_wait(&m.pready, t & 1, gave_up);
#pragma unroll 1
            for (int nb = 0; nb < 2; ++nb) {
                bar_wait(&m.vfull[nb], t & 1, gave_up);
                if (!FP8 && valid < kTile) {
                    zero_rows(v + nb * 2 * kVChunkB, valid, lane);
                    fence_proxy_async_smem();
                }
                if (rank != 0) {
                    __syncwarp();
                    if (lane == 0) bar_arrive_at(&m.pv[nb], 0);
                    continue;
                }
                bar_wait(&m.pv[nb], t & 1, gave_up);
                tmem_fence_after();
                __syncwarp();
                if (!*gave_up && elect_one()) {
                    const uint64_t da = umma_desc(pa, 16, 1024);
                    const uint64_t db = umma_desc(va + nb * 2 * kVChunkB, kVChunkB, 1024);
#pragma unroll
                    for (int s = 0; s < 8; ++s)
                        umma_ss<2>(tmem + nb * 128, da + (s >> 2) * (kChunkB >> 4) + 2 * (s & 3), db + s * 128, idO,
                                   s > 0 || !first);
                    umma_commit_pair(&m.vempty[nb]);
                    if (nb == 1) umma_commit_pair(&m.pvdone);
                }
                __syncwarp();
            }
        };
        TileWalk tw;
        tw.start(a, blocks, walk);
        int t = 0, seg = 0, pvalid = 0;
        bool pending = false, pfirst = false;
        for (; tw.live; ++t) {
            if (tw.first && pending) {
                values(t - 1, pfirst, pvalid);
                pending = false;
            }
            scores(t, tw.first, tw.last, seg);
            if (pending) values(t - 1, pfirst, pvalid);
            pending = true;
            pfirst = tw.first;
            pvalid = tw.s.n - tw.t * kTile;
            seg += tw.last;
            tw.step(a, blocks);
        }
        if (pending) values(t - 1, pfirst, pvalid);
        if (rank == 0) {  // nothing in flight when the CTAs leave
            __syncwarp();
            if (elect_one()) umma_commit_pair(&m.drain);
            __syncwarp();
            bar_drain(&m.drain, 0);
        }
    } else if (warp == 5) {
        // ---------------- K: TMA (FP8: the rotated keys alone) ----------------
        const uint64_t pol = l2_policy_evict_normal();
        TileWalk tw, ah;
        tw.start(a, blocks, walk);
        ah = tw;
        // own pages of a tile into L2: this CTA's half, its peer takes the other
        auto ahead = [&]() {
            if (ah.live) ah.step(a, blocks);
            if (ah.live && lane < 4) {
                const int id = page_of(a, ah.s.b, ah.t * kTilePages + (int)rank * 4 + lane, ah.s.n);
                if (id >= 0) {
                    const uint32_t cb = kPage * kDC * (FP8 ? 1 : 2);
                    l2_prefetch(static_cast<const uint8_t *>(a.pool.c_pages) + (long long)id * cb, cb);
                    l2_prefetch(a.pool.r_pages + (long long)id * kPage * PFKV_LATENT_ROPE, kPage * PFKV_LATENT_ROPE * 2);
                }
            }
        };
        ahead();
        int t = 0;
        for (; tw.live; ++t) {
            ahead();
            const int id = lane < 4 ? page_of(a, tw.s.b, tw.t * kTilePages + (int)rank * 4 + lane, tw.s.n) : -1;
            const uint32_t bytes = 2048u * __popc(__ballot_sync(0xffffffffu, id >= 0));
#pragma unroll 1
            for (int c = FP8 ? 8 : 0; c < kKChunks; ++c) {
                bar_wait(&m.kempty[c], (t & 1) ^ 1, gave_up);
                if (*gave_up) break;
                if (lane == 0) mbar_arrive_expect_tx(&m.kfull[c], bytes);
                __syncwarp();
                if (id >= 0) {
                    uint8_t *dst = k + c * kChunkB + lane * 2048;
                    if (c < 8) tma_box3(dst, &mapc, c * 64, 0, id, &m.kfull[c], pol);
                    else tma_box3(dst, &mapr, 0, 0, id, &m.kfull[c], pol);
                }
            }
            __syncwarp();
            if (*gave_up) break;
            tw.step(a, blocks);
        }
        __syncwarp();
        if (*gave_up)  // copies in flight: of this tile and the last
            for (int c = FP8 ? 8 : 0; c < kKChunks; ++c) {
                bar_drain(&m.kfull[c], 0);
                bar_drain(&m.kfull[c], 1);
            }
    } else if (warp == 6 && !FP8) {
        // ------------------------------ V: TMA ------------------------------
        const uint64_t pol = l2_policy_evict_normal();
        TileWalk tw;
        tw.start(a, blocks, walk);
        for (int t = 0; tw.live; ++t) {
            const int id = lane < 16 ? page_of(a, tw.s.b, tw.t * kTilePages + (lane & 7), tw.s.n) : -1;
            const uint32_t bytes = 2048u * __popc(__ballot_sync(0xffffffffu, id >= 0));
#pragma unroll 1
            for (int nb = 0; nb < 2; ++nb) {
                bar_wait(&m.vempty[nb], (t & 1) ^ 1, gave_up);
                if (*gave_up) break;
                if (lane == 0) mbar_arrive_expect_tx(&m.vfull[nb], bytes);
                __syncwarp();
                if (id >= 0)
                    tma_box3(v + (nb * 2 + (lane >> 3)) * kVChunkB + (lane & 7) * 2048, &mapc,
                             (nb * 4 + (int)rank * 2 + (lane >> 3)) * 64, 0, id, &m.vfull[nb], pol);
            }
            __syncwarp();
            if (*gave_up) break;
            tw.step(a, blocks);
        }
        __syncwarp();
        if (*gave_up)
            for (int nb = 0; nb < 2; ++nb) {
                bar_drain(&m.vfull[nb], 0);
                bar_drain(&m.vfull[nb], 1);
            }
    } else if (warp >= 8 && warp < 12) {
        // ------------------- Q; FP8: K converted on the way -------------------
        const int i = tid - 256;
        const int kr = i >> 2, part = i & 3;  // row (+ 32) and 16-byte piece of a chunk's 64 bytes
        TileWalk tw, nx;
        tw.start(a, blocks, walk);
        nx = tw;
        uint4 raw[8][2];
        int ids[2];
        bool in[2];
        const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
        auto load_ids = [&](const TileWalk &t) {
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const int key = (int)rank * 64 + u * 32 + kr;
                ids[u] = t.live ? page_of(a, t.s.b, t.t * kTilePages + key / kPage, t.s.n) : -1;
                in[u] = ids[u] >= 0 && t.t * kTile + key < t.s.n;
            }
        };
        auto load = [&](int c) {
#pragma unroll
            for (int u = 0; u < 2; ++u)
                raw[c][u] = in[u] ? reinterpret_cast<const uint4 *>(a.pool.c_pages)[((long long)ids[u] * kPage + (kr & 15)) * (kDC / 16) + c * 4 + part]
                                  : zero;
        };
        if constexpr (FP8) {
            load_ids(tw);
            for (int c = 0; c < 8; ++c) load(c);
            if (nx.live) nx.step(a, blocks);
            load_ids(nx);
        }
        int seg = 0;
        for (int t = 0; tw.live; ++t) {
            if (tw.first) {
                bar_wait(&m.qfree, (seg & 1) ^ 1, gave_up);
                load_queries<FP8>(a, tw.s, R, rank, q, m.qscale[seg & 1], i);
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) {
                    bar_arrive(&m.qfull);
                    bar_arrive(&m.sq[seg & 1]);
                }
                ++seg;
            }
            if constexpr (FP8) {
#pragma unroll
                for (int c = 0; c < 8; ++c) {
                    bar_wait(&m.kempty[c], (t & 1) ^ 1, gave_up);
#pragma unroll
                    for (int u = 0; u < 2; ++u) {
                        const int r = u * 32 + kr;
                        *piece(k + c * kChunkB, r, 2 * part) = cvt_e4m3x8(raw[c][u].x, raw[c][u].y);
                        *piece(k + c * kChunkB, r, 2 * part + 1) = cvt_e4m3x8(raw[c][u].z, raw[c][u].w);
                    }
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) bar_arrive(&m.kfull[c]);
                    load(c);  // the next tile's
                }
                if (nx.live) nx.step(a, blocks);
                load_ids(nx);
            }
            tw.step(a, blocks);
        }
    } else if (warp >= 12 && FP8) {
        // ---------------------- V converted on the way ----------------------
        const int i = tid - 384;
        const int kr = i >> 2, part = i & 3;
        TileWalk tw, nx;
        tw.start(a, blocks, walk);
        nx = tw;
        uint4 raw[4][4];
        int ids[4];
        bool in[4];
        const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
        auto load_ids = [&](const TileWalk &t) {
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const int key = u * 32 + kr;
                ids[u] = t.live ? page_of(a, t.s.b, t.t * kTilePages + key / kPage, t.s.n) : -1;
                in[u] = ids[u] >= 0 && t.t * kTile + key < t.s.n;
            }
        };
        auto load = [&](int s) {  // chunk s holds values (s / 2) * 256 + rank * 128 + (s & 1) * 64 ...
            const int g = (s >> 1) * 4 + (int)rank * 2 + (s & 1);
#pragma unroll
            for (int u = 0; u < 4; ++u)
                raw[s][u] = in[u] ? reinterpret_cast<const uint4 *>(a.pool.c_pages)[((long long)ids[u] * kPage + (kr & 15)) * (kDC / 16) + g * 4 + part]
                                  : zero;
        };
        load_ids(tw);
        for (int s = 0; s < 4; ++s) load(s);
        if (nx.live) nx.step(a, blocks);
        load_ids(nx);
        for (int t = 0; tw.live; ++t) {
#pragma unroll
            for (int s = 0; s < 4; ++s) {
                if ((s & 1) == 0) bar_wait(&m.vempty[s >> 1], (t & 1) ^ 1, gave_up);
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    const int r = u * 32 + kr;
                    *piece(v + s * kVChunkB, r, 2 * part) = cvt_e4m3x8(raw[s][u].x, raw[s][u].y);
                    *piece(v + s * kVChunkB, r, 2 * part + 1) = cvt_e4m3x8(raw[s][u].z, raw[s][u].w);
                }
                load(s);
                if (s & 1) {
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) bar_arrive(&m.vfull[s >> 1]);
                }
            }
            if (nx.live) nx.step(a, blocks);
            load_ids(nx);
            tw.step(a, blocks);
        }
    }
    __syncthreads();
    if (tid == 0) parts.gave_up[w * 2 + rank] = m.gave_up;
    tmem_fence_before();
    cluster_sync();  // the even CTA's products read the odd one's shared memory
    tmem_fence_after();
    if (warp == 4) tmem_free512<2>(tmem);
}

// --------------------------------------------------------------------------
// Merge: a warp a row.  Before its wait for the split kernel it checks what the
// flags depend on: the length, and the id and tag of every live page.
// --------------------------------------------------------------------------
constexpr int kMergeWarps = 8;

__global__ void __launch_bounds__(kMergeWarps * 32)
    latent_merge_kernel(LatentDecodeArgs a, int R, int blocks, int clusters, Parts parts, int groups) {
    __shared__ long long sums[2][kMergeWarps];
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int b = blockIdx.x / groups, g = blockIdx.x - b * groups;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int raw = a.pool.seq_lens[(long long)b * a.pool.len_sb];
    const int n = live_len(a, b);
    uint32_t bits = raw != n ? PFKV_FLAG_BAD_LENGTH : 0u;
    for (int i = tid; i < (n + kPage - 1) / kPage; i += blockDim.x) {
        const long long bi = (long long)b * a.pool.bt_sb + i;
        bits |= latent_entry_bits(a.pool, a.pool.block_tables[bi], bi);
    }
    long long before = 0, all = 0;
    for (int i = tid; i < a.B; i += blockDim.x) {
        const long long u = (long long)tiles_of(live_len(a, i)) * blocks;
        all += u;
        if (i < b) before += u;
    }
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) {
        before += __shfl_xor_sync(0xffffffffu, before, d);
        all += __shfl_xor_sync(0xffffffffu, all, d);
        bits |= __shfl_xor_sync(0xffffffffu, bits, d);
    }
    if (lane == 0) {
        sums[0][warp] = before;
        sums[1][warp] = all;
    }
    uint32_t flag = 0;
#pragma unroll
    for (uint32_t f = 1; f < 8; f <<= 1)
        if (__syncthreads_or(bits & f)) flag |= f;
    before = all = 0;
    for (int i = 0; i < kMergeWarps; ++i) {
        before += sums[0][i];
        all += sums[1][i];
    }
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int tiles = tiles_of(n);
    const int W = (int)min((long long)clusters, all);
    auto cluster_of = [&](long long x) { return (int)(x * W / all); };
    if (tiles > 0) {
        const int w0 = cluster_of(before), w1 = cluster_of(before + (long long)tiles * blocks - 1);
        int up = 0;
        for (int i = w0 * 2 + tid; i < (w1 + 1) * 2; i += blockDim.x) up |= parts.gave_up[i] != 0u;
        if (__syncthreads_or(up)) flag |= PFKV_FLAG_DEVICE_TIMEOUT;
    }
    if (g == 0 && tid == 0 && a.flags) a.flags[b] = (uint8_t)flag;
    const int row = g * kMergeWarps + warp;
    if (row >= R) return;
    const int t = row / a.H, h = row - t * a.H;
    __nv_bfloat16 *out = a.out.p + (long long)b * a.out.sb + (long long)t * a.out.st + (long long)h * a.out.sh;
    // lane l: values 4 l + 128 i .. + 3
    float o[4][4] = {};
    if (!flag && tiles > 0) {
        const int block = row / kRowBlock, brow = row - block * kRowBlock;
        const long long first = before + (long long)block * tiles;
        const int w0 = cluster_of(first), w1 = cluster_of(first + tiles - 1);
        if (w0 == w1) return;  // one part: written by the split kernel
        float ref = kNegInf, sum = 0.f;
        for (int w = w0; w <= w1; ++w) {
            const long long at = (long long)(w * 2 + (w == w0 ? 1 : 0)) * parts.rows + brow;
            const float l = parts.lse[at];
            if (l == kNegInf) continue;
            const float4 *src = reinterpret_cast<const float4 *>(parts.o + at * kDC) + lane;
            const float top = fmaxf(ref, l);
            const float old = ref == kNegInf ? 0.f : exp2f(ref - top), now = exp2f(l - top);
            ref = top;
            sum = sum * old + now;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float4 y = src[i * 32];
                o[i][0] = o[i][0] * old + y.x * now;
                o[i][1] = o[i][1] * old + y.y * now;
                o[i][2] = o[i][2] * old + y.z * now;
                o[i][3] = o[i][3] * old + y.w * now;
            }
        }
        const float inv = sum == 0.f ? 0.f : 1.f / sum;
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[i][e] *= inv;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 x = __floats2bfloat162_rn(o[i][0], o[i][1]), y = __floats2bfloat162_rn(o[i][2], o[i][3]);
        *reinterpret_cast<uint2 *>(out + 4 * lane + 128 * i) =
            make_uint2(*reinterpret_cast<const uint32_t *>(&x), *reinterpret_cast<const uint32_t *>(&y));
    }
}

struct Layout {
    size_t lse, gave_up, total;
    int rows;
};

Layout workspace_layout(int R, int clusters) {
    Layout l;
    l.rows = R < kRowBlock ? R : kRowBlock;
    auto up = [](size_t x) { return (x + 255) & ~size_t(255); };
    const size_t rows = (size_t)clusters * 2 * l.rows;
    l.lse = up(rows * kDC * sizeof(float));
    l.gave_up = l.lse + up(rows * sizeof(float));
    l.total = l.gave_up + up((size_t)clusters * 2 * sizeof(uint32_t));
    return l;
}

template <bool FP8>
cudaError_t launch_split(const CUtensorMap &mapc, const CUtensorMap &mapr, const LatentDecodeArgs &a, int R, int blocks,
                         int clusters, const Parts &parts, cudaStream_t s) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)clusters * 2);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = kSmemBytes;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, latent_split_kernel<FP8>, mapc, mapr, a, R, blocks, clusters, parts);
}

}  // namespace

size_t latent_decode_workspace(int, int H, int kq, int, int num_sms) {
    return workspace_layout(H * kq, max(1, num_sms / 2)).total;
}

cudaError_t launch_latent_decode(const LatentDecodeArgs &a, int num_sms, cudaStream_t s) {
    const int R = a.H * a.kq, blocks = (R + kRowBlock - 1) / kRowBlock, clusters = max(1, num_sms / 2);
    const Layout l = workspace_layout(R, clusters);
    uint8_t *ws = static_cast<uint8_t *>(a.workspace);
    const Parts parts{reinterpret_cast<float *>(ws), reinterpret_cast<float *>(ws + l.lse),
                      reinterpret_cast<uint32_t *>(ws + l.gave_up), l.rows};
    alignas(64) CUtensorMap mapc, mapr;
    const uint64_t np = (uint64_t)a.pool.num_pages;
    cudaError_t e = bf16_map3(&mapr, a.pool.r_pages, PFKV_LATENT_ROPE, kPage, np, PFKV_LATENT_ROPE,
                              kPage * PFKV_LATENT_ROPE, kPage, 1);
    if (e != cudaSuccess) return e;
    mapc = mapr;  // FP8 pools: not read
    if (!a.pool.fp8) {
        e = bf16_map3(&mapc, a.pool.c_pages, kDC, kPage, np, kDC, kPage * kDC, kPage, 1);
        if (e != cudaSuccess) return e;
    }
    e = a.pool.fp8 ? launch_split<true>(mapc, mapr, a, R, blocks, clusters, parts, s)
                   : launch_split<false>(mapc, mapr, a, R, blocks, clusters, parts, s);
    if (e != cudaSuccess) return e;
    const int groups = (R + kMergeWarps - 1) / kMergeWarps;
    if ((long long)groups * a.B > 0x7fffffffLL) return cudaErrorInvalidValue;
    return launch_pdl(latent_merge_kernel, dim3((unsigned)(groups * a.B)), dim3(kMergeWarps * 32), 0, s, a, R, blocks,
                      clusters, parts, groups);
}

cudaError_t preload_latent_decode() {
    cudaError_t e = cudaFuncSetAttribute(latent_split_kernel<true>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmemBytes);
    if (e == cudaSuccess)
        e = cudaFuncSetAttribute(latent_split_kernel<false>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmemBytes);
    if (e == cudaSuccess) e = preload_kernel(latent_merge_kernel);
    return e;
}

}  // namespace pfkv

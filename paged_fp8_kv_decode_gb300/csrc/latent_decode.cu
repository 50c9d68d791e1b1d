// latent_decode.cu -- pfkv_latent_decode_attn: attention in the absorbed form
// over a paged latent cache (declared in pfkv_latent.h).
//
// Mathematics.  R = query tokens x heads rows of a request share every token's
// latent c_j (512 values) and rotated key r_j (64):
//     S = scale (Q_c C^T + Q_r R^T),   O = softmax(S) C,
// 2 R (576 + 512) operations a token for 1,152 bytes (BF16) or 640 (FP8): at 128
// rows 242 or 435 operations a byte, where this GPU turns from memory-bound to
// tensor-bound (288 at the measured rates).  So both products run on the
// fifth-generation tensor cores, and every latent is to be read from HBM once for up to
// 128 rows (each further block of 128 reads it again).
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
// CTAs.  A block's rows thus read each latent from HBM once, and from L2 twice.  Shared
// memory (Q 72 KB, K 72 KB, V 64 KB, P 16 KB) leaves no room for second buffers;
// instead every stage's slot is refilled as soon as its last product has completed,
// and an L2 prefetch runs ahead of that.
//
// Softmax: one pass.  Four threads hold a row (32 tokens each), in log2 units, with
// a running reference that moves only when the maximum has grown by 2^8 (then O
// is rescaled in tensor memory).  FP8: a weight enters the second product times
// its page's scale z_j; the reference is of s_j + log2 z_j, so that the f16
// weights stay in range and the largest keep their 11 bits however far apart the
// scales are; the weights' sum takes the weight in fp32 over z_j.
//
// Work: the tiles of all (request, 128-row block) pairs are one list, cut into
// ranges of equal cost for the clusters (below).  A pair that lies in one range is
// written out directly; parts of a pair go to the workspace (normalised rows and
// their log2-sum-exp) and a second kernel merges them.
//
// Measured: a tile takes 1.85 us with BF16 pages (6.1 TB/s over 76 clusters, 90% of a
// copy) and 2.45 us with FP8 ones, where 400 KB pass through shared memory a tile
// (converted K and V stored, operands read, weights): 1.6 us at 128 bytes a cycle, and
// the softmax's chain (scores read, maxima exchanged, weights stored when the last
// products have ended) is 1.9 us long.  A call has 20-24 us besides: start 8, a part's end 4-6, merge 5.
//
// Tokens that a row does not see have weights of zero.  So that values which are not finite do
// not reach it, a tile's tokens past the last that any row of the block sees are zero in the
// second product, and those that only some rows see (several query tokens) are looked at.
//
// Roles of a CTA's twenty warps: 0-7 softmax and output (four threads a row); 8, in
// the even CTA, issues the pair's products; 9 and 10 load rotated keys, K and V by TMA
// (K and V of BF16 pools: through registers, K of BF16 cost 2.7 us a tile, by TMA
// 2.15); 11 looks up pages, checks and scales four tiles ahead of their use and
// prefetches them into L2; FP8: 12-15 and 16-19 carry K and V through registers and
// convert them to f16, the next tile's loaded while this one is stored.
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
constexpr int kKStages = 5;                   // two chunks each, the rotated keys alone
constexpr int kRing = 4;                      // tiles looked up ahead (and at least 3: see the issuing role).
                                              // BF16, a tile: 6 ahead 2.14 us, 4 1.82, 3 1.82 (FP8 2.30, 2.33, 2.41)
constexpr uint32_t kChunkB = kRowsCta * 128;  // Q, K and P chunks: 64 rows of 128 bytes
constexpr uint32_t kVChunkB = kTile * 128;
// V of one block of 256 values: two chunks of 64.  FP8: chunk by chunk, 128 tokens
// each.  BF16: page by page, both chunks of 16 tokens each, as one TMA box brings them.
template <bool FP8>
constexpr uint32_t kVLbo = FP8 ? kVChunkB : 2048u;  // to the next chunk
template <bool FP8>
constexpr uint32_t kVStep = FP8 ? 2048u : 4096u;    // to the next page
constexpr int kThreads = 640;
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

// What the roles need to know of a tile.
struct Tile {
    int id[kTilePages];      // physical pages, -1 for one that is not to be read
    float z[kTilePages], lz[kTilePages], iz[kTilePages];  // FP8: scales, their logarithms and reciprocals
    int b, block, left;      // request, row block, the request's tokens from this tile's first on
    // Of those, the ones that some row of the block sees: a value past them is taken for zero (it
    // would meet weights of zero, harmless where it is finite).  And the ones before the first
    // that a row does not see and that is not finite (else as many as are held): past them, what is
    // not finite is zero; rows that see it have it in their scores.
    int held, sound;
    uint32_t flags;
};
constexpr uint32_t kFirst = 1, kLast = 2, kWhole = 4, kBegins = 8;  // of the part of a (request, row block)

struct Misc {
    // operands of both CTAs in place (in the even CTA), slots free again (in both)
    uint64_t kfull[kKStages], vfull[2], pready, kempty[kKStages], vempty[2];
    uint64_t mfull[kRing], mempty[kRing];
    uint64_t sfull[2], pvdone, qfull, drain;
    Tile tile[kRing];
    union {
        long long warp_sum[2][kThreads / 32];
        float xm[2][4][kRowsCta];  // what a row's four threads exchange: maxima by the tile's parity
    };
    long long x0, x1, off;
    int b0;
    uint32_t tmem, gave_up;
};
constexpr size_t kSmemBytes = kOffMisc + sizeof(Misc);
static_assert(kSmemBytes <= 232448, "shared memory of one CTA");

// Workspace: normalised partial rows and their log2-sum-exp, two blocks a
// cluster (the part of a pair that began before its range, and the part of one
// that ends after it), and a word a CTA that says whether its waits gave up.
struct Parts {
    float *o;        // [clusters][2][rows][512]
    float *lse;      // [clusters][2][rows]
    uint32_t *gave_up;  // [clusters][2]
    uint32_t *status;   // [request x row block + cluster]: flags of the pages that the cluster looked up
    int rows;        // min(R, 128)
};

// Tokens of request b, 0 for a length that is refused.
__device__ __forceinline__ int live_len(const LatentDecodeArgs &a, int b) {
    const int n = a.pool.seq_lens[(long long)b * a.pool.len_sb];
    return n < 0 || (long long)n > (long long)a.pool.max_pages * kPage || n > a.max_seq_len ? 0 : n;
}
__device__ __forceinline__ int tiles_of(int n) { return (n + kTile - 1) / kTile; }

// The list of (request, row block) parts is dealt to the clusters by cost: a tile is
// one unit, and the start of a part (new queries, the part before written out while
// the products wait: 5 to 6 us) as many as kPartUnits tiles.  32 requests of 512 to
// 8,192 tokens: equal tiles 76.2 us, 2 units 70.6, 3 71.5, 4 71.7, 6 74.1.
constexpr int kPartUnits = 2;
__device__ __forceinline__ long long units_of(int tiles) { return tiles > 0 ? tiles + kPartUnits : 0; }

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

__device__ __forceinline__ uint4 cvt_e4m3x8(uint32_t lo, uint32_t hi) {
    uint4 r;
    asm("{\n\t.reg .b16 a, b, c, d;\n\tmov.b32 {a, b}, %4;\n\tmov.b32 {c, d}, %5;\n\t"
        "cvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t"
        "cvt.rn.f16x2.e4m3x2 %2, c;\n\tcvt.rn.f16x2.e4m3x2 %3, d;\n\t}"
        : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
        : "r"(lo), "r"(hi));
    return r;
}

__device__ __forceinline__ void store_shared(uint32_t at, const uint4 &w) {
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(w.x), "r"(w.y), "r"(w.z), "r"(w.w) : "memory");
}

// Piece c (16 bytes) of row r of a swizzled chunk.
__device__ __forceinline__ uint4 *piece(uint8_t *chunk, int r, int c) {
    return reinterpret_cast<uint4 *>(chunk + r * 128 + ((c ^ (r & 7)) << 4));
}

// Eight query rows, r0 .. r0 + 7 of the CTA's 64, into shared memory by one warp, all
// copies in flight at once; rows past the last are zero.
__device__ __forceinline__ void copy_queries(const LatentDecodeArgs &a, int b, int block, int R, uint32_t rank,
                                             uint8_t *q, int r0, int lane) {
#pragma unroll
    for (int g = 0; g < 2; ++g) {
        const int r = r0 + g * 4 + (lane >> 3), pc = lane & 7;
        const int row = block * kRowBlock + (int)rank * kRowsCta + r;
        const bool live = row < R;
        const int t = live ? row / a.H : 0, h = live ? row - t * a.H : 0;
        const __nv_bfloat16 *c = a.qc.p + (long long)b * a.qc.sb + (long long)t * a.qc.st + (long long)h * a.qc.sh;
        const __nv_bfloat16 *e = a.qr.p + (long long)b * a.qr.sb + (long long)t * a.qr.st + (long long)h * a.qr.sh;
        const uint32_t bytes = live ? 16u : 0u;  // the rest of a copy's 16 bytes is filled with zeros
#pragma unroll
        for (int j = 0; j < kKChunks; ++j) {
            const __nv_bfloat16 *src = (j < 8 ? c + j * 64 : e) + pc * 8;
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_addr(piece(q + j * kChunkB, r, pc))),
                         "l"(src), "r"(bytes)
                         : "memory");
        }
    }
}

// FP8: the latent part of a row's quarter, in place, to f16 over the power of two
// that puts the row's largest element in [1, 2) (the rotated part stays bf16).
// First its largest magnitude, as bf16 bits (integers order as magnitudes do).
__device__ __forceinline__ uint32_t largest_query(uint8_t *q, int r, int part) {
    uint32_t top = 0;
#pragma unroll
    for (int j = 0; j < 16; ++j) {
        const uint4 w = *piece(q + (part * 2 + (j >> 3)) * kChunkB, r, j & 7);
        top = max(max(top, max(w.x & 0x7FFFu, (w.x >> 16) & 0x7FFFu)), max(w.y & 0x7FFFu, (w.y >> 16) & 0x7FFFu));
        top = max(max(top, max(w.z & 0x7FFFu, (w.z >> 16) & 0x7FFFu)), max(w.w & 0x7FFFu, (w.w >> 16) & 0x7FFFu));
    }
    return top;
}
__device__ __forceinline__ uint32_t scaled_half2(uint32_t w, float f) {
    const float2 x = bf16x2_to_float2(w);
    const __half2 v = __floats2half2_rn(x.x * f, x.y * f);
    return *reinterpret_cast<const uint32_t *>(&v);
}
__device__ __forceinline__ void convert_query(uint8_t *q, int r, int part, float inv) {
#pragma unroll
    for (int j = 0; j < 16; j += 4) {
        uint4 w[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) w[u] = *piece(q + (part * 2 + (j >> 3)) * kChunkB, r, (j + u) & 7);
#pragma unroll
        for (int u = 0; u < 4; ++u)
            *piece(q + (part * 2 + (j >> 3)) * kChunkB, r, (j + u) & 7) =
                make_uint4(scaled_half2(w[u].x, inv), scaled_half2(w[u].y, inv), scaled_half2(w[u].z, inv),
                           scaled_half2(w[u].w, inv));
    }
}

// What a block's rows see in part (num_query_tokens > 1) is looked at before it is used, as a
// weight of zero does not hide a value that is not finite.  (Inlined: the roles that do it have 64
// and 88 registers, and a call may take any of the kernel's 96.)

// Whether tokens k0 .. k1 - 1 of a tile, whose page ids the lanes from `lane0` on hold, have such a latent.
template <bool FP8>
__device__ __forceinline__ bool odd_latents(const void *pages, int id, int lane0, int k0, int k1, int lane) {
    uint32_t odd = 0;
#pragma unroll 4
    for (int k = k0; k < k1; ++k) {
        const int page = __shfl_sync(0xffffffffu, id, lane0 + k / kPage);
        const uint4 *c = reinterpret_cast<const uint4 *>(static_cast<const uint8_t *>(pages) +
                                                         ((long long)max(page, 0) * kPage + k % kPage) * (kDC * (FP8 ? 1 : 2)));
        const uint4 w = c[lane];
        if constexpr (FP8) {
            odd |= e4m3_nan(w.x) | e4m3_nan(w.y) | e4m3_nan(w.z) | e4m3_nan(w.w);
        } else {
            const uint4 u = c[lane + 32];
            odd |= not_finite(w.x) | not_finite(w.y) | not_finite(w.z) | not_finite(w.w);
            odd |= not_finite(u.x) | not_finite(u.y) | not_finite(u.z) | not_finite(u.w);
        }
    }
    return __any_sync(0xffffffffu, odd != 0u);
}

// BF16: rows 16 full .. rows - 1 of a tile's V, without what is not finite from row `sound` on (a
// lane's pieces are those that it stored as zeros before).
__device__ __forceinline__ void copy_sound_latents(const void *pages, const Tile &ti, uint8_t *v, int full, int sound, int rows,
                                                int x, int lane) {
#pragma unroll 1
    for (int e = lane; e < (rows - full * kPage) * 16; e += 32) {
        const int r = full * kPage + (e >> 4), c = e & 15, id = ti.id[r / kPage];
        if (id < 0) continue;
        uint4 w = static_cast<const uint4 *>(pages)[((long long)id * kPage + (r & 15)) * (kDC / 8) + x / 8 + c];
        if (r >= sound) {
            w.x &= ~((not_finite(w.x) >> 15) * 0xFFFFu);
            w.y &= ~((not_finite(w.y) >> 15) * 0xFFFFu);
            w.z &= ~((not_finite(w.z) >> 15) * 0xFFFFu);
            w.w &= ~((not_finite(w.w) >> 15) * 0xFFFFu);
        }
        *piece(v + (r >> 4) * 4096 + (c >> 3) * 2048, r & 15, c & 7) = w;
    }
}

// FP8: the same to a lane's converted values, rows 8 u + r_in of a chunk from row `sound` on (NaN
// codes have become the f16 of all ones).
__device__ __forceinline__ void zero_odd_values(uint8_t *chunk, int pc, int r_in, int sound) {
#pragma unroll 1
    for (int u = 0; u < 32; ++u) {
        const int r = (u >> 1) * 8 + r_in;
        if (r < sound) continue;
        uint32_t *w = reinterpret_cast<uint32_t *>(piece(chunk, r, 2 * pc + (u & 1)));
        for (int i = 0; i < 4; ++i) w[i] &= ~((((w[i] & 0x7C007C00u) + 0x04000400u) >> 15 & 0x00010001u) * 0xFFFFu);
    }
}

// A barrier of 128 threads that tells whether any of them says so.
__device__ __forceinline__ bool bar_any(int id, bool says) {
    uint32_t r;
    asm volatile("{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %2, 0;\n\tbar.red.or.pred q, %1, 128, p;\n\t"
                 "selp.u32 %0, 1, 0, q;\n\t}"
                 : "=r"(r)
                 : "r"(id), "r"((uint32_t)says)
                 : "memory");
    return r != 0;
}

// Selftest: waits of as many tries as the call says.
template <bool FP8, bool Selftest>
__global__ void __launch_bounds__(kThreads, 1)
    latent_split_kernel(const __grid_constant__ CUtensorMap mapc, const __grid_constant__ CUtensorMap mapr,
                        const __grid_constant__ CUtensorMap mapk,
                        LatentDecodeArgs a, int R, int blocks, int clusters, Parts parts) {
    extern __shared__ __align__(1024) uint8_t sm[];  // no static shared memory: the window's aligned base
    Misc &m = *reinterpret_cast<Misc *>(sm + kOffMisc);
    uint8_t *const q = sm + kOffQ, *const k = sm + kOffK, *const v = sm + kOffV, *const p = sm + kOffP;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t rank = cluster_rank();
    const int w = blockIdx.x >> 1;
    if (tid == 0) {
        for (int c = 0; c < kKStages; ++c) {
            mbar_init(&m.kfull[c], 2);  // both CTAs, whether or not they bring keys
            mbar_init(&m.kempty[c], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&m.vfull[i], FP8 ? 4 : 2);
            mbar_init(&m.vempty[i], 1);
            mbar_init(&m.sfull[i], 1);
        }
        for (int i = 0; i < kRing; ++i) {
            mbar_init(&m.mfull[i], 1);
            mbar_init(&m.mempty[i], 1);
        }
        mbar_init(&m.pready, 16);
        mbar_init(&m.pvdone, 1);
        mbar_init(&m.qfull, 16);
        mbar_init(&m.drain, 1);
        m.gave_up = (smem_addr(sm) & 1023u) != 0u;  // nothing runs on a base that the swizzle cannot take
        m.x0 = m.x1 = 0;
        m.off = 0;
        m.b0 = 0;
        fence_mbar_init();
    }
    if (warp == 8) tmem_alloc512<2>(&m.tmem);
    tmem_fence_before();
    __syncthreads();
    cluster_sync();  // both CTAs' barriers are initialised
    tmem_fence_after();
    pdl_enter();

    {
        // the block tables into L2, while the list of tiles is counted
        const int lines = (a.pool.max_pages * 4 + 127) / 128 + 1;
        for (long long i = (long long)blockIdx.x * kThreads + tid; i < (long long)a.B * lines; i += (long long)gridDim.x * kThreads) {
            const int b = (int)(i / lines);
            const long long e = min((i - (long long)b * lines) * 32, (long long)a.pool.max_pages - 1);
            asm volatile("prefetch.global.L2 [%0];" ::"l"(a.pool.block_tables + (long long)b * a.pool.bt_sb + e));
        }
    }
    // this cluster's range of the list of tiles
    {
        const int per = (a.B + kThreads - 1) / kThreads;
        const int lo = min(a.B, tid * per), hi = min(a.B, lo + per);
        long long mine[2] = {0, 0};  // units, and tiles
        for (int b = lo; b < hi; ++b) {
            const int tiles = tiles_of(live_len(a, b));
            mine[0] += units_of(tiles) * blocks;
            mine[1] += (long long)tiles * blocks;
        }
        long long before[2] = {mine[0], mine[1]}, all[2] = {0, 0};
#pragma unroll
        for (int d = 1; d < 32; d <<= 1)
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const long long y = __shfl_up_sync(0xffffffffu, before[k], d);
                if (lane >= d) before[k] += y;
            }
        if (lane == 31) {
            m.warp_sum[0][warp] = before[0];
            m.warp_sum[1][warp] = before[1];
        }
        __syncthreads();
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            before[k] -= mine[k];
            for (int i = 0; i < kThreads / 32; ++i) {
                if (i < warp) before[k] += m.warp_sum[k][i];
                all[k] += m.warp_sum[k][i];
            }
        }
        const int W = (int)min((long long)clusters, all[1]);
        if (w < W && !m.gave_up) {
#pragma unroll 1
            for (int end = 0; end < 2; ++end) {  // the tiles at which the range begins and ends
                const long long x = range_start(w + end, all[0], W);
                if (x == all[0] && tid == 0) m.x1 = all[1];
                if (x < before[0] || x >= before[0] + mine[0]) continue;
                long long at = before[0], tile = before[1];
                for (int b = lo;; ++b) {
                    const int tiles = tiles_of(live_len(a, b));
                    const long long u = units_of(tiles);
                    if (x >= at + u * blocks) {
                        at += u * blocks;
                        tile += (long long)tiles * blocks;
                        continue;
                    }
                    const long long block = (x - at) / u;
                    const long long off = block * tiles + max(0LL, x - at - block * u - kPartUnits);
                    if (end) {
                        m.x1 = tile + off;
                    } else {
                        m.x0 = tile + off;
                        m.b0 = b;
                        m.off = off;
                    }
                    break;
                }
            }
        }
    }
    __syncthreads();
    const int N = (int)(m.x1 - m.x0);  // tiles of this cluster: every role counts them
    const uint32_t tmem = m.tmem;
    volatile uint32_t *const gave_up = &m.gave_up;
    const int tries = Selftest ? a.tries : kTries;
    // Waits until tile t is looked up; false when a wait of this CTA has given up
    // (the entry may then be anything, and is not used).
    auto looked_up = [&](int t) { return bar_wait(&m.mfull[t % kRing], (t / kRing) & 1, gave_up, tries); };

    // Registers of the five warpgroups, of 5 x 96 at launch: 2 x 120 + 64 + 2 x 88.  No role
    // may spill: with 230 KB of shared memory there is next to no L1 to catch it.

    // After waits have given up: copies in flight (into either CTA) are left time to land.
    auto drain_copies = [&]() {
        const unsigned long long t0 = globaltimer_ns();
        while (globaltimer_ns() - t0 < kWaitLimitNs) {}
    };

    if (warp < 8) {
        // ------------------------- softmax and output -------------------------
        // lanes 64-127 of tensor memory hold tokens 64-127 of rows 0-63; warps 4-7
        // take the upper 32 of each 64 tokens, and columns 128-255 of O
        reg_share_more<120>();
        const int quad = warp & 3, half = quad >> 1, cw = warp >> 2, r = (quad & 1) * 32 + lane;
        const int part = half * 2 + cw;  // of a row's four threads
        const int bar = 1 + (quad & 1);
        const uint32_t lanes = tmem + ((uint32_t)(quad * 32) << 16);
        const float a2 = a.sm_scale * kLog2e;
        float ref = kNegInf, sum = 0.f, qs = 0.f;
        int hidden = 0, row = 0;  // hidden: candidates after this row's own
        bool live = false, any_live = false;
        // Q of the part that begins with tile t; its slots are free once the scores of
        // the tile before are there.  The copies run while the last part is written out.
        auto fetch_queries = [&](int b, int block) {
            copy_queries(a, b, block, R, rank, q, (quad & 1) * 32 + part * 8, lane);
        };
        auto finish_queries = [&](float (&xm)[4][kRowsCta]) {
            asm volatile("cp.async.wait_all;" ::: "memory");
            if constexpr (FP8) {
                asm volatile("bar.sync %0, 128;" ::"r"(bar) : "memory");  // the row block's copies are in
                const uint32_t mine = largest_query(q, r, part);
                xm[part][r] = __uint_as_float(mine);
                asm volatile("bar.sync %0, 128;" ::"r"(bar) : "memory");
                const uint32_t top = max(max(__float_as_uint(xm[0][r]), __float_as_uint(xm[1][r])),
                                         max(__float_as_uint(xm[2][r]), __float_as_uint(xm[3][r])));
                // biased exponent, kept where both 2^e and 2^-e are normal fp32 numbers
                const int eb = min(253, max(1, (int)(top >> 7)));
                convert_query(q, r, part, __uint_as_float((uint32_t)(254 - eb) << 23));
                qs = a2 * __uint_as_float((uint32_t)eb << 23);
                asm volatile("bar.sync %0, 128;" ::"r"(bar) : "memory");  // xm is free
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) bar_arrive_at(&m.qfull, 0);
        };
        if (N > 0) {
            fetch_queries(m.b0, (int)(m.off / tiles_of(live_len(a, m.b0))));
            finish_queries(m.xm[1]);
        }
        for (int t = 0; t < N; ++t) {
            const bool ok = looked_up(t);
            const Tile &ti = m.tile[t % kRing];
            uint32_t flags = ok ? ti.flags : 0u;
            const int b = ti.b;
            if (flags & kFirst) {
                row = ti.block * kRowBlock + (int)rank * kRowsCta + r;
                live = row < R;
                hidden = a.kq - 1 - (live ? row / a.H : a.kq - 1);
                ref = kNegInf;
                sum = 0.f;
            }
            live = live && ok;
            any_live = __any_sync(0xffffffffu, live);
            const int seen = ti.left - hidden - part * 32;  // of this thread's 32 tokens
            float z[2], lz[2], iz[2];
            if constexpr (FP8) {
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    z[i] = ti.z[part * 2 + i];
                    lz[i] = ti.lz[part * 2 + i];
                    iz[i] = ti.iz[part * 2 + i];
                }
            }
            bar_wait(&m.sfull[t & 1], (t >> 1) & 1, gave_up, tries);
            tmem_fence_after();
            float x[32];
            float top = kNegInf;
            if (any_live) {
                const uint32_t cs = lanes + kColS + (t & 1) * 128 + cw * 32;
                tmem_ld32(cs, x);
                if constexpr (FP8) {
#pragma unroll
                    for (int g = 0; g < 2; ++g) {
                        float y[16];
                        tmem_ld16(cs + 64 + g * 16, y);
                        tmem_wait_ld();
#pragma unroll
                        for (int j = 0; j < 16; j += 2) {
                            const float2 turned = fma2(make_float2(y[j], y[j + 1]), make_float2(a2, a2), make_float2(lz[g], lz[g]));
                            const float2 v = fma2(make_float2(x[g * 16 + j], x[g * 16 + j + 1]), make_float2(qs * z[g], qs * z[g]), turned);
                            x[g * 16 + j] = v.x;
                            x[g * 16 + j + 1] = v.y;
                        }
                    }
                } else {
                    tmem_wait_ld();
#pragma unroll
                    for (int j = 0; j < 32; ++j) x[j] *= a2;
                }
                if (seen < 32) {
#pragma unroll
                    for (int j = 0; j < 32; ++j)
                        if (j >= seen) x[j] = kNegInf;
                }
                float tops[4] = {x[0], x[1], x[2], x[3]};  // four chains, not one
#pragma unroll
                for (int j = 4; j < 32; ++j) tops[j & 3] = fmaxf(tops[j & 3], x[j]);
                top = fmaxf(fmaxf(tops[0], tops[1]), fmaxf(tops[2], tops[3]));
            }
            float (&xm)[4][kRowsCta] = m.xm[t & 1];
            xm[part][r] = top;
            // all of the row block's threads know the tile, or none goes by it: they meet at
            // the barriers below by its flags
            if (bar_any(bar, !ok)) flags = 0u;
            top = fmaxf(fmaxf(xm[0][r], xm[1][r]), fmaxf(xm[2][r], xm[3][r]));
            float shrink = 1.f;
            if (top > ref + kLazyGrowth || (ref == kNegInf && top > kNegInf)) {
                shrink = fast_exp2(ref - top);  // 0 when nothing was seen yet
                sum *= shrink;
                ref = top;
            }
            // the weights, in registers until P's slot is free
            uint32_t pw[16];
            if (any_live) {
                const float base = ref == kNegInf ? 0.f : ref - kWeightBias<FP8>;
                float2 sums[2][2] = {};  // of 16 tokens (a page) each
#pragma unroll
                for (int j = 0; j < 32; j += 2) {
                    const float2 y = add2(make_float2(x[j], x[j + 1]), make_float2(-base, -base));
                    const float2 f = make_float2(fast_exp2(y.x), fast_exp2(y.y));
                    sums[j >> 4][(j >> 1) & 1] = add2(sums[j >> 4][(j >> 1) & 1], f);
                    if constexpr (FP8) {
                        const __half2 hw = __floats2half2_rn(f.x, f.y);
                        pw[j >> 1] = *reinterpret_cast<const uint32_t *>(&hw);
                    } else {
                        const __nv_bfloat162 hw = __floats2bfloat162_rn(f.x, f.y);
                        pw[j >> 1] = *reinterpret_cast<const uint32_t *>(&hw);
                    }
                }
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const float2 f = add2(sums[i][0], sums[i][1]);
                    if constexpr (FP8) sum = fmaf(f.x + f.y, iz[i], sum);
                    else sum += f.x + f.y;
                }
            }
            if (t > 0) {
                bar_wait(&m.pvdone, (t - 1) & 1, gave_up, tries);  // P is free, O is at rest
                tmem_fence_after();
            }
            if (any_live) {
#pragma unroll
                for (int c = 0; c < 4; ++c)
                    *piece(p + half * kChunkB, r, cw * 4 + c) = make_uint4(pw[4 * c], pw[4 * c + 1], pw[4 * c + 2], pw[4 * c + 3]);
                if (!(flags & kFirst) && __any_sync(0xffffffffu, shrink != 1.f)) {
#pragma unroll 1
                    for (int g = 0; g < 8; ++g) {
                        float o[16];
                        tmem_ld16(lanes + cw * 128 + g * 16, o);
                        tmem_wait_ld();
#pragma unroll
                        for (int j = 0; j < 16; ++j) o[j] *= shrink;
                        tmem_st16(lanes + cw * 128 + g * 16, o);
                    }
                    tmem_wait_st();
                }
                fence_proxy_async_smem();
            }
            tmem_fence_before();
            __syncwarp();
            if (lane == 0) bar_arrive_at(&m.pready, 0);
            if (flags & kLast) {
                if (t + 1 < N && looked_up(t + 1)) fetch_queries(m.tile[(t + 1) % kRing].b, m.tile[(t + 1) % kRing].block);
                const bool whole = (flags & kWhole) != 0;
                const int slot = w * 2 + ((flags & kBegins) ? 1 : 0);
                const bool done = bar_wait(&m.pvdone, t & 1, gave_up, tries);
                tmem_fence_after();
                float (&sums)[4][kRowsCta] = m.xm[(t & 1) ^ 1];  // read before this tile's first barrier
                sums[part][r] = sum;
                asm volatile("bar.sync %0, 128;" ::"r"(bar) : "memory");
                const float total = (sums[0][r] + sums[1][r]) + (sums[2][r] + sums[3][r]);
                if (t + 1 < N) {  // the next part's scores are taken while this one is written
                    asm volatile("bar.sync %0, 128;" ::"r"(bar) : "memory");  // the sums have been read
                    finish_queries(sums);
                }
                if (any_live) {
                    const float inv = total > 0.f ? __fdiv_rn(1.f, total) : total;  // zero and NaN stay
                    const bool store = live && done;
                    if (!whole && store && part == 0)
                        parts.lse[(long long)slot * parts.rows + rank * kRowsCta + r] =
                            total == 0.f ? kNegInf : ref - kWeightBias<FP8> + __log2f(total);
                    // Columns 128 cw ..: values 256 cw .., each half a row's threads' share.
                    // Sixteen columns at a time pass through 2 KB of P's slots a warp, so that a store
                    // covers 64 bytes of eight rows (a thread's own row would make it 32 rows); the
                    // slots are those of the row block's own weights, which its next barrier guards.
                    const int d = cw * 256 + half * 128;
                    float4 *const stage = reinterpret_cast<float4 *>(p + half * kChunkB + (quad & 1) * 4096 + cw * 2048);
                    const int r4 = lane >> 2, c4 = lane & 3;
                    const uint32_t rows = __ballot_sync(0xffffffffu, store);
                    // this lane's eight-row steps: rows r4, r4 + 8, ..
                    long long at[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int rr = (quad & 1) * 32 + i * 8 + r4, br = (int)rank * kRowsCta + rr;
                        const int gr = row - r + rr;  // row of the request
                        if (whole) {
                            const int tok = gr / a.H;
                            at[i] = (long long)b * a.out.sb + (long long)tok * a.out.st + (long long)(gr - tok * a.H) * a.out.sh;
                        } else {
                            at[i] = ((long long)slot * parts.rows + br) * kDC;
                        }
                    }
                    float o[16];
                    tmem_ld16(lanes + cw * 128, o);
#pragma unroll 1
                    for (int g = 0; g < 8; ++g) {
                        tmem_wait_ld();
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            float4 x = make_float4(o[4 * j] * inv, o[4 * j + 1] * inv, o[4 * j + 2] * inv, o[4 * j + 3] * inv);
                            if (total == 0.f) x = make_float4(0.f, 0.f, 0.f, 0.f);
                            stage[lane * 4 + (j ^ ((lane >> 1) & 3))] = x;
                        }
                        if (g < 7) tmem_ld16(lanes + cw * 128 + (g + 1) * 16, o);
                        __syncwarp();
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const int rr = i * 8 + r4;
                            const float4 x = stage[rr * 4 + (c4 ^ ((rr >> 1) & 3))];
                            if (!((rows >> rr) & 1u)) continue;
                            if (whole) {
                                const __nv_bfloat162 lo = __floats2bfloat162_rn(x.x, x.y), hi = __floats2bfloat162_rn(x.z, x.w);
                                *reinterpret_cast<uint2 *>(a.out.p + at[i] + d + g * 16 + c4 * 4) =
                                    make_uint2(*reinterpret_cast<const uint32_t *>(&lo), *reinterpret_cast<const uint32_t *>(&hi));
                            } else {
                                *reinterpret_cast<float4 *>(parts.o + at[i] + d + g * 16 + c4 * 4) = x;
                            }
                        }
                        __syncwarp();
                    }
                }
                tmem_fence_before();
            }
        }
    } else if (warp == 8) {
        // ----------------------- products (even CTA) -----------------------
        reg_share_less<64>();
        // One thread runs the whole role: the compiler then knows that descriptors are
        // those of a single thread.
        if (rank == 0 && elect_one()) {
            const uint32_t qa = smem_addr(q), ka = smem_addr(k), va = smem_addr(v), pa = smem_addr(p);
            constexpr uint32_t idS = umma_idesc(kRowBlock, kTile, !FP8, false, false);
            constexpr uint32_t idR = umma_idesc(kRowBlock, kTile, true, false, false);
            constexpr uint32_t idO = umma_idesc(kRowBlock, 256, !FP8, false, true);
            auto values = [&](int t, bool first) {
                const bool ok = bar_wait(&m.pready, t & 1, gave_up, tries);
                const uint32_t da = umma_desc(pa, 16);
#pragma unroll 1
                for (int nb = 0; nb < 2; ++nb) {
                    if (!bar_wait(&m.vfull[nb], t & 1, gave_up, tries) || !ok) continue;
                    tmem_fence_after();
                    const uint32_t db = umma_desc(va + nb * 2 * kVChunkB, kVLbo<FP8>);
#pragma unroll
                    for (int s = 0; s < 8; ++s)  // a page a step
                        umma_ss<2>(tmem + nb * 128, da + (s >> 2) * (kChunkB >> 4) + 2 * (s & 3),
                                   db + s * (kVStep<FP8> >> 4), idO, s > 0 || !first);
                    umma_commit_pair(&m.vempty[nb]);
                }
                if (ok) {
                    umma_commit_pair(&m.pvdone);
                    umma_commit_pair(&m.mempty[t % kRing]);
                }
            };
            int seg = 0;
            bool pfirst = false;
            uint32_t flags = N > 0 && looked_up(0) ? m.tile[0].flags : 0u, next = 0;
            for (int t = 0; t < N; ++t, flags = next) {
                const bool first = (flags & kFirst) != 0;
                // the products of the tile before this one's scores when Q changes between them
                if (t > 0 && first) values(t - 1, pfirst);
                if (first) bar_wait(&m.qfull, seg & 1, gave_up, tries);
                const uint32_t cs = tmem + kColS + (t & 1) * 128;
                // The rotated keys come first: their one slot is refilled by TMA, which then has
                // the rest of the tile's time.  (Loops over stages stay loops: unrolled, their
                // descriptors cost the registers that the other roles need.)
                bool ok = bar_wait(&m.kfull[4], t & 1, gave_up, tries);
                uint32_t da = umma_desc(qa, 16), db = umma_desc(ka, 16);
                if (ok) {
                    tmem_fence_after();
                    constexpr uint32_t last = 8 * kChunkB >> 4;
#pragma unroll
                    for (int s = 0; s < 4; ++s)
                        umma_ss<2>(FP8 ? cs + 64 : cs, da + last + 2 * s, db + last + 2 * s, idR, s > 0);
                    umma_commit_pair(&m.kempty[4]);
                }
#pragma unroll 1
                for (int c = 0; c < 4; ++c, da += 2 * kChunkB >> 4, db += 2 * kChunkB >> 4) {
                    ok = bar_wait(&m.kfull[c], t & 1, gave_up, tries) && ok;
                    if (!ok) continue;
                    tmem_fence_after();
#pragma unroll
                    for (int s = 0; s < 8; ++s) {
                        const uint32_t step = (s >> 2) * (kChunkB >> 4) + 2 * (s & 3);
                        umma_ss<2>(cs, da + step, db + step, idS, !FP8 || s > 0 || c > 0);
                    }
                    umma_commit_pair(&m.kempty[c]);
                }
                if (ok) umma_commit_pair(&m.sfull[t & 1]);
                next = t + 1 < N && looked_up(t + 1) ? m.tile[(t + 1) % kRing].flags : 0u;
                if (t > 0 && !first) values(t - 1, pfirst);
                pfirst = first;
                if (flags & kLast) ++seg;
            }
            if (N > 0) values(N - 1, pfirst);
            umma_commit_pair(&m.drain);
        }
        __syncwarp();
    } else if (warp == 9) {
        // ------------- rotated keys, and K of BF16 pools: TMA -------------
        reg_share_less<64>();
        if (elect_one()) {
            const uint64_t pol = l2_policy_evict_normal();
            for (int t = 0; t < N && looked_up(t); ++t) {
                const Tile &ti = m.tile[t % kRing];
                int id[4];
                uint32_t pages = 0;
#pragma unroll
                for (int i = 0; i < kTilePages; ++i) pages += ti.id[i] >= 0;
#pragma unroll
                for (int i = 0; i < 4; ++i) id[i] = ti.id[rank * 4 + i];
                if (!bar_wait(&m.kempty[4], (t & 1) ^ 1, gave_up, tries)) break;
                // The odd CTA arrives too, with its ids in registers: where its four pages are
                // past the last token its bytes hold nothing up, and the ring's entry and the
                // barriers' phases would go on without it.
                if (rank == 0) mbar_arrive_expect_tx(&m.kfull[4], pages * 2048u);  // both CTAs' bytes
                else bar_arrive_at(&m.kfull[4], 0);
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (id[i] >= 0) tma_box3_pair(k + 8 * kChunkB + i * 2048, &mapr, 0, 0, id[i], &m.kfull[4], pol);
                if constexpr (!FP8) {
#pragma unroll 1
                    for (int c = 0; c < 4; ++c) {
                        if (!bar_wait(&m.kempty[c], (t & 1) ^ 1, gave_up, tries)) break;
                        if (rank == 0) mbar_arrive_expect_tx(&m.kfull[c], pages * 4096u);
                        else bar_arrive_at(&m.kfull[c], 0);
                        uint8_t *dst = k + 2 * c * kChunkB;
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            if (id[i] < 0) continue;
                            tma_box3_pair(dst + i * 2048, &mapk, c * 128, 0, id[i], &m.kfull[c], pol);
                            tma_box3_pair(dst + kChunkB + i * 2048, &mapk, c * 128 + 64, 0, id[i], &m.kfull[c], pol);
                        }
                    }
                }
            }
            if (*gave_up) drain_copies();
        }
        __syncwarp();
    } else if (warp == 10) {
        // ------------------------------ V: TMA ------------------------------
        reg_share_less<64>();
        const uint64_t pol = l2_policy_evict_normal();
        for (int t = 0; !FP8 && t < N; ++t) {
            if (!__all_sync(0xffffffffu, looked_up(t))) break;
            const Tile &ti = m.tile[t % kRing];
            const int held = ti.held, sound = ti.sound;
            const int full = min(kTilePages, max(0, sound) / kPage);  // pages whose slots are all taken as they are
#pragma unroll 1
            for (int nb = 0; nb < 2; ++nb) {
                if (!__all_sync(0xffffffffu, bar_wait(&m.vempty[nb], (t & 1) ^ 1, gave_up, tries))) break;
                uint8_t *dst = v + nb * 2 * kVChunkB;
                const int x = (nb * 4 + (int)rank * 2) * 64;
                if (elect_one()) {
                    // The ids are read before the arrival: where no page is to be read nothing
                    // else holds up the products, and with them the entry's refill.
                    int id[kTilePages];
                    uint32_t pages = 0;
#pragma unroll
                    for (int i = 0; i < kTilePages; ++i) {
                        id[i] = i < full ? ti.id[i] : -1;
                        pages += id[i] >= 0;
                    }
                    // the even CTA counts both CTAs' bytes
                    if (rank == 0 && full == kTilePages) mbar_arrive_expect_tx(&m.vfull[nb], pages * 8192u);
                    else if (rank == 0) bar_expect_tx(&m.vfull[nb], pages * 8192u);
                    else if (full == kTilePages) bar_arrive_at(&m.vfull[nb], 0);
#pragma unroll
                    for (int i = 0; i < kTilePages; ++i) {
                        if (id[i] < 0) continue;
                        tma_box4_pair(dst + i * 4096, &mapc, 0, 0, x / 64, id[i], &m.vfull[nb], pol);
                    }
                }
                __syncwarp();
                if (full < kTilePages) {
                    // the pages behind those, and zeros for every slot past the last token that is
                    // held: those may hold anything, NaN among it, and meet weights of zero
                    const int id = sound == held && held % kPage ? ti.id[full] : -1;
                    const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
                    for (int e = lane; e < (kTile - full * kPage) * 16; e += 32) {
                        const int r = full * kPage + (e >> 4), c = e & 15;  // row, 16-byte piece of its 256
                        uint4 w = zero;
                        if (r < held && id >= 0)
                            w = reinterpret_cast<const uint4 *>(a.pool.c_pages)[((long long)id * kPage + (r & 15)) * (kDC / 8) + x / 8 + c];
                        *piece(dst + (r >> 4) * 4096 + (c >> 3) * 2048, r & 15, c & 7) = w;
                    }
                    if (sound < held) copy_sound_latents(a.pool.c_pages, ti, dst, full, sound, min(kTile, held), x, lane);
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) bar_arrive_at(&m.vfull[nb], 0);
                }
            }
        }
        if (!FP8 && *gave_up) drain_copies();
        __syncwarp();
    } else if (warp == 11) {
        // ------------- pages, checks, scales; two tiles at a time -------------
        reg_share_less<64>();
        Walk walk{m.x0, m.x1, m.off, m.b0};
        Segment s;
        const int i = (lane >> 3) & 1, pg = lane & 7;  // tile of the two, page of the tile
        int t = 0;
        while (walk.next(a, blocks, s)) {
            uint32_t bits = 0;
            int seen_all = s.n, seen_any = s.n;  // tokens that all rows of the block see, and that one does
            if (a.kq > 1) {
                seen_all += 1 - a.kq + s.block * kRowBlock / a.H;
                seen_any += min(0, 1 - a.kq + (s.block * kRowBlock + kRowBlock - 1) / a.H);
            }
            for (int at = s.t0; at < s.t1; at += 2) {
                const int tile = at + i, lp = tile * kTilePages + pg;
                int id = -1;
                uint32_t bad = 0;
                float z = 1.f;
                if (lane < 16 && tile < s.t1 && lp < (s.n + kPage - 1) / kPage) {
                    const long long bi = (long long)s.b * a.pool.bt_sb + lp;
                    id = a.pool.block_tables[bi];
                    bad = latent_entry_bits(a.pool, id, bi);
                    if (bad) id = -1;  // not read; the merge kernel flags and zeroes the request
                }
                bits |= bad;
                if (id >= 0 && FP8) {
                    z = a.pool.c_scale[id];
                    if (z < 7.888609052210118e-31f) z = 7.888609052210118e-31f;  // 2^-100
                }
                for (int j = 0; j < min(2, s.t1 - at); ++j, ++t) {
                    const int first = (at + j) * kTile, held = seen_any - first;
                    int sound = held;
                    if (seen_all < seen_any && seen_any > first && seen_all < first + kTile &&
                        odd_latents<FP8>(a.pool.c_pages, id, j * 8, max(0, seen_all - first), min(kTile, held), lane))
                        sound = seen_all - first;
                    Tile &ti = m.tile[t % kRing];
                    if (!__all_sync(0xffffffffu, bar_wait(&m.mempty[t % kRing], ((t / kRing) & 1) ^ 1, gave_up, tries))) continue;
                    if (lane < 16 && i == j) {
                        ti.id[pg] = id;
                        ti.z[pg] = z;
                        if constexpr (FP8) {
                            ti.lz[pg] = __log2f(z);
                            ti.iz[pg] = __frcp_rn(z);
                        }
                        if (pg == 0) {
                            ti.b = s.b;
                            ti.block = s.block;
                            ti.left = s.n - tile * kTile;
                            ti.held = held;
                            ti.sound = sound;
                            ti.flags = (tile == s.t0 ? kFirst : 0u) | (tile + 1 == s.t1 ? kLast : 0u) |
                                       (s.t1 - s.t0 == s.tiles ? kWhole : 0u) | (s.t0 == 0 ? kBegins : 0u);
                        }
                        // this CTA's half into L2; its peer takes the other
                        if (id >= 0 && (uint32_t)(pg >> 2) == rank) {
                            const uint32_t cb = kPage * kDC * (FP8 ? 1 : 2);
                            l2_prefetch(static_cast<const uint8_t *>(a.pool.c_pages) + (long long)id * cb, cb);
                            l2_prefetch(a.pool.r_pages + (long long)id * kPage * PFKV_LATENT_ROPE,
                                        kPage * PFKV_LATENT_ROPE * 2);
                        }
                    }
                    __syncwarp();
                    if (lane == 0) bar_arrive(&m.mfull[t % kRing]);
                }
            }
            bits = __reduce_or_sync(0xffffffffu, bits);
            if (lane == 0 && rank == 0) parts.status[(long long)s.b * blocks + s.block + w] = bits;
        }
    } else if (!FP8) {
        reg_share_less<24>();  // BF16: nothing to convert
    } else if (warp < 16) {
        // ------------------ FP8: K converted on the way, a warp a stage ------------------
        // stage j holds chunks 2j and 2j + 1 of 64 tokens, 8 lanes a row of 128 bytes; a
        // thread's words of the next tile are loaded as soon as this tile's are stored
        reg_share_less<88>();
        const int j = warp - 12, r_in = lane >> 3, pc = lane & 7;
        // A page that is not to be read is read as page 0, which exists: its rows are past
        // the last token and stored as zeros, or its request is flagged and zeroed.
        const uint8_t *const src = static_cast<const uint8_t *>(a.pool.c_pages) + r_in * kDC + j * 128 + pc * 16;
        // where the thread's first piece of rows 4 i + r_in goes
        uint32_t at[2];
#pragma unroll
        for (int i = 0; i < 2; ++i)
            at[i] = smem_addr(k + 2 * j * kChunkB) + (pc >> 2) * kChunkB + r_in * 128 +
                    (((2 * (pc & 3)) ^ (4 * i + r_in)) << 4);
        uint4 raw[16];
        int left = 0;
        auto load = [&](int t) {
            const bool ok = t < N && looked_up(t);
            const Tile &ti = m.tile[t % kRing];
            left = ok ? ti.left - (int)rank * 64 : 0;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint8_t *page = src + (long long)(kPage * kDC) * (ok ? max(0, ti.id[rank * 4 + i]) : 0);
#pragma unroll
                for (int u = 0; u < 4; ++u) raw[4 * i + u] = *reinterpret_cast<const uint4 *>(page + u * 4 * kDC);
            }
        };
        load(0);
        for (int t = 0; t < N; ++t) {
            if (left < 64) {
#pragma unroll
                for (int u = 0; u < 16; ++u)
                    if (u * 4 + r_in >= left) raw[u] = make_uint4(0u, 0u, 0u, 0u);
            }
            bar_wait(&m.kempty[j], (t & 1) ^ 1, gave_up, tries);
#pragma unroll
            for (int u = 0; u < 16; ++u) {
                const uint32_t to = at[u & 1] + u * 512;
                store_shared(to, cvt_e4m3x8(raw[u].x, raw[u].y));
                store_shared(to ^ 16u, cvt_e4m3x8(raw[u].z, raw[u].w));
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) bar_arrive_at(&m.kfull[j], 0);
            load(t + 1);
        }
    } else {
        // ------------------ FP8: V converted on the way, a warp a chunk ------------------
        const int s = warp - 16;
        const int g = (s >> 1) * 4 + (int)rank * 2 + (s & 1);  // chunk of the latent's eight
        const int r_in = lane >> 2, pc = lane & 3;
        uint8_t *const dst = v + s * kVChunkB;
        const uint8_t *const src = static_cast<const uint8_t *>(a.pool.c_pages) + r_in * kDC + g * 64 + pc * 16;
        const uint32_t at = smem_addr(dst) + r_in * 128 + (((2 * pc) ^ r_in) << 4);
        reg_share_less<88>();
        uint4 raw[16];
        int held = 0, sound = 0;
        auto load = [&](int t) {
            const bool ok = t < N && looked_up(t);
            const Tile &ti = m.tile[t % kRing];
            held = ok ? ti.held : 0;
            sound = ok ? ti.sound : 0;
#pragma unroll
            for (int i = 0; i < kTilePages; ++i) {
                const uint8_t *page = src + (long long)(kPage * kDC) * (ok ? max(0, ti.id[i]) : 0);
                raw[2 * i] = *reinterpret_cast<const uint4 *>(page);
                raw[2 * i + 1] = *reinterpret_cast<const uint4 *>(page + 8 * kDC);
            }
        };
        load(0);
        for (int t = 0; t < N; ++t) {
            if (held < kTile) {
#pragma unroll
                for (int u = 0; u < 16; ++u)
                    if (u * 8 + r_in >= held) raw[u] = make_uint4(0u, 0u, 0u, 0u);
            }
            bar_wait(&m.vempty[s >> 1], (t & 1) ^ 1, gave_up, tries);
#pragma unroll
            for (int u = 0; u < 16; ++u) {  // row u * 8 + r_in
                store_shared(at + u * 1024, cvt_e4m3x8(raw[u].x, raw[u].y));
                store_shared((at ^ 16u) + u * 1024, cvt_e4m3x8(raw[u].z, raw[u].w));
            }
            if (sound < held) zero_odd_values(dst, pc, r_in, sound);
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) bar_arrive_at(&m.vfull[s >> 1], 0);
            load(t + 1);
        }
    }
    __syncthreads();
    if (tid == 0) parts.gave_up[w * 2 + rank] = m.gave_up;
    // Nothing in flight when the CTAs leave: the products' last arrivals come to the barriers
    // of both, and each waits for its own (that the even CTA's have come says nothing of the
    // odd one's).
    if (warp == 8 && elect_one()) bar_drain(&m.drain, 0);
    __syncwarp();
    tmem_fence_before();
    cluster_sync();  // the even CTA's products read the odd one's shared memory
    tmem_fence_after();
    if (warp == 8) tmem_free512<2>(tmem);
}

// --------------------------------------------------------------------------
// Merge: a warp half a row, or a quarter of its parts.  What depends on the call's
// inputs alone (the list of tiles) comes before its wait for the split kernel.
// --------------------------------------------------------------------------
constexpr int kMergeWarps = 8;

// Ways: warps that share a half row's parts.
template <int Ways>
__global__ void __launch_bounds__(kMergeWarps * 32)
    latent_merge_kernel(LatentDecodeArgs a, int R, int blocks, int clusters, Parts parts, int groups) {
    constexpr int kRows = kMergeWarps / 2 / Ways;
    __shared__ long long sums[3][kMergeWarps];
    __shared__ float4 shared_o[Ways > 1 ? kMergeWarps : 1][2][32];
    __shared__ float shared_ref[kMergeWarps], shared_sum[kMergeWarps];
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int b = blockIdx.x / groups, g = blockIdx.x - b * groups;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int raw = a.pool.seq_lens[(long long)b * a.pool.len_sb];
    const int n = live_len(a, b);
    long long before = 0, all = 0, tiles_all = 0;
    for (int i = tid; i < a.B; i += blockDim.x) {
        const int tiles = tiles_of(live_len(a, i));
        const long long u = units_of(tiles) * blocks;
        tiles_all += (long long)tiles * blocks;
        all += u;
        if (i < b) before += u;
    }
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) {
        before += __shfl_xor_sync(0xffffffffu, before, d);
        all += __shfl_xor_sync(0xffffffffu, all, d);
        tiles_all += __shfl_xor_sync(0xffffffffu, tiles_all, d);
    }
    if (lane == 0) {
        sums[0][warp] = before;
        sums[1][warp] = all;
        sums[2][warp] = tiles_all;
    }
    __syncthreads();
    before = all = tiles_all = 0;
    for (int i = 0; i < kMergeWarps; ++i) {
        before += sums[0][i];
        all += sums[1][i];
        tiles_all += sums[2][i];
    }
    const int tiles = tiles_of(n);
    const int W = (int)min((long long)clusters, tiles_all);
    // the cluster of tile j of row block k
    auto cluster_of = [&](int k, int j) {
        return (int)((before + k * units_of(tiles) + kPartUnits + j) * W / all);
    };
    asm volatile("griddepcontrol.wait;" ::: "memory");
    uint32_t flag = raw != n ? PFKV_FLAG_BAD_LENGTH : 0u;
    if (tiles > 0) {
        const int w0 = cluster_of(0, 0), w1 = cluster_of(blocks - 1, tiles - 1);
        uint32_t bits = 0;
        for (int i = w0 * 2 + tid; i < (w1 + 1) * 2; i += blockDim.x)
            if (parts.gave_up[i]) bits |= PFKV_FLAG_DEVICE_TIMEOUT;
        for (int k = 0; k < blocks; ++k) {  // every cluster that holds a part of row block k
            const int last = cluster_of(k, tiles - 1);
            for (int i = cluster_of(k, 0) + tid; i <= last; i += blockDim.x)
                bits |= parts.status[(long long)b * blocks + k + i];
        }
#pragma unroll
        for (uint32_t f = 1; f < 16; f <<= 1)
            if (__syncthreads_or(bits & f)) flag |= f;
    }
    if (g == 0 && tid == 0 && a.flags) a.flags[b] = (uint8_t)flag;
    const int half = warp & 1, way = (warp >> 1) % Ways, row = g * kRows + (warp >> 1) / Ways;
    if (Ways == 1 && row >= R) return;  // otherwise a row a CTA, and all are there
    const int t = row / a.H, h = row - t * a.H;
    __nv_bfloat16 *out = a.out.p + (long long)b * a.out.sb + (long long)t * a.out.st + (long long)h * a.out.sh + half * 256;
    // lane l: values 4 l + 128 i .. + 3 of the half
    float o[2][4] = {};
    if (!flag && tiles > 0) {
        const int block = row / kRowBlock, brow = row - block * kRowBlock;
        const int w0 = cluster_of(block, 0), w1 = cluster_of(block, tiles - 1);
        if (w0 == w1) return;  // one part: written by the split kernel
        // this warp's parts: those of clusters w0 + way, w0 + way + Ways, ..
        const int mine_all = (w1 - w0 - way + Ways) / Ways;
        auto place = [&](int i) {
            const int w = w0 + way + i * Ways;
            return (long long)(w * 2 + (w == w0 ? 1 : 0)) * parts.rows + brow;
        };
        float ref = kNegInf, sum = 0.f;
        for (int at = 0; at < mine_all; at += 32) {  // 32 parts at once: a lane has one's weight
            const float l = at + lane < mine_all ? parts.lse[place(at + lane)] : kNegInf;
            if (__all_sync(0xffffffffu, l == kNegInf)) continue;  // (a NaN goes on, and into the sum)
            float top = l;
#pragma unroll
            for (int d = 16; d > 0; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
            top = fmaxf(ref, top);
            const float old = exp2f(ref - top), mine = exp2f(l - top);
            ref = top;
            float s = mine;
#pragma unroll
            for (int d = 16; d > 0; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
            sum = sum * old + s;
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e) o[i][e] *= old;
            const int count = min(32, mine_all - at);
            for (int j = 0; j < count; j += 8) {  // eight parts' loads in flight
                float4 y[8][2];
#pragma unroll
                for (int u = 0; u < 8; ++u) {
                    const float *from = parts.o + place(min(at + j + u, mine_all - 1)) * kDC + half * 256;
                    const float4 *src = reinterpret_cast<const float4 *>(from) + lane;
                    y[u][0] = src[0];
                    y[u][1] = src[32];
                }
#pragma unroll
                for (int u = 0; u < 8; ++u) {
                    const float f = __shfl_sync(0xffffffffu, mine, min(31, j + u));
                    if (j + u >= count || f == 0.f) continue;  // parts that saw nothing hold zeros
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        o[i][0] += y[u][i].x * f;
                        o[i][1] += y[u][i].y * f;
                        o[i][2] += y[u][i].z * f;
                        o[i][3] += y[u][i].w * f;
                    }
                }
            }
        }
        if constexpr (Ways > 1) {
            if (lane == 0) {
                shared_ref[warp] = ref;
                shared_sum[warp] = sum;
            }
#pragma unroll
            for (int i = 0; i < 2; ++i) shared_o[warp][i][lane] = make_float4(o[i][0], o[i][1], o[i][2], o[i][3]);
            __syncthreads();  // the flags and the parts are the CTA's: all its warps are here
            if (way > 0) return;
            float top = ref;
#pragma unroll
            for (int k = 1; k < Ways; ++k) top = fmaxf(top, shared_ref[warp + 2 * k]);
            const float own = top == kNegInf ? 0.f : exp2f(ref - top);
            sum *= own;
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e) o[i][e] *= own;
#pragma unroll
            for (int k = 1; k < Ways; ++k) {
                const float f = top == kNegInf ? 0.f : exp2f(shared_ref[warp + 2 * k] - top);
                sum += shared_sum[warp + 2 * k] * f;
                if (f == 0.f) continue;
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const float4 y = shared_o[warp + 2 * k][i][lane];
                    o[i][0] += y.x * f;
                    o[i][1] += y.y * f;
                    o[i][2] += y.z * f;
                    o[i][3] += y.w * f;
                }
            }
        }
        const float inv = sum == 0.f ? 0.f : 1.f / sum;
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[i][e] *= inv;
    } else if (Ways > 1 && way > 0) {
        return;
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const __nv_bfloat162 x = __floats2bfloat162_rn(o[i][0], o[i][1]), y = __floats2bfloat162_rn(o[i][2], o[i][3]);
        *reinterpret_cast<uint2 *>(out + 4 * lane + 128 * i) =
            make_uint2(*reinterpret_cast<const uint32_t *>(&x), *reinterpret_cast<const uint32_t *>(&y));
    }
}

struct Layout {
    size_t lse, gave_up, status, total;
    int rows;
};

Layout workspace_layout(int B, int R, int clusters) {
    Layout l;
    l.rows = R < kRowBlock ? R : kRowBlock;
    auto up = [](size_t x) { return (x + 255) & ~size_t(255); };
    const size_t rows = (size_t)clusters * 2 * l.rows;
    l.lse = up(rows * kDC * sizeof(float));
    l.gave_up = l.lse + up(rows * sizeof(float));
    l.status = l.gave_up + up((size_t)clusters * 2 * sizeof(uint32_t));
    const size_t pairs = (size_t)B * ((R + kRowBlock - 1) / kRowBlock);
    l.total = l.status + up((pairs + clusters) * sizeof(uint32_t));
    return l;
}

template <bool FP8>
cudaError_t launch_split(const CUtensorMap &mapc, const CUtensorMap &mapr, const CUtensorMap &mapk,
                         const LatentDecodeArgs &a, int R, int blocks, int clusters, const Parts &parts,
                         cudaStream_t s) {
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
    auto *const kernel = a.tries == kTries ? latent_split_kernel<FP8, false> : latent_split_kernel<FP8, true>;
    return cudaLaunchKernelEx(&cfg, kernel, mapc, mapr, mapk, a, R, blocks, clusters, parts);
}

}  // namespace

size_t latent_decode_workspace(int B, int H, int kq, int, int num_sms) {
    return workspace_layout(B, H * kq, max(1, num_sms / 2)).total;
}

cudaError_t launch_latent_decode(const LatentDecodeArgs &a, int num_sms, cudaStream_t s) {
    const int R = a.H * a.kq, blocks = (R + kRowBlock - 1) / kRowBlock, clusters = max(1, num_sms / 2);
    const Layout l = workspace_layout(a.B, R, clusters);
    uint8_t *ws = static_cast<uint8_t *>(a.workspace);
    const Parts parts{reinterpret_cast<float *>(ws), reinterpret_cast<float *>(ws + l.lse),
                      reinterpret_cast<uint32_t *>(ws + l.gave_up), reinterpret_cast<uint32_t *>(ws + l.status),
                      l.rows};
    alignas(64) CUtensorMap mapc, mapr, mapk;
    const uint64_t np = (uint64_t)a.pool.num_pages;
    cudaError_t e = bf16_map3(&mapr, a.pool.r_pages, PFKV_LATENT_ROPE, kPage, np, PFKV_LATENT_ROPE,
                              kPage * PFKV_LATENT_ROPE, kPage, 1);
    if (e != cudaSuccess) return e;
    mapc = mapk = mapr;  // FP8 pools: not read
    if (!a.pool.fp8) {
        e = bf16_map3(&mapk, a.pool.c_pages, kDC, kPage, np, kDC, kPage * kDC, kPage, 1);
        if (e != cudaSuccess) return e;
        e = bf16_map4(&mapc, a.pool.c_pages, kPage, kDC / 64, np, kDC, 64, kPage * kDC, kPage, 2);
        if (e != cudaSuccess) return e;
    }
    e = a.pool.fp8 ? launch_split<true>(mapc, mapr, mapk, a, R, blocks, clusters, parts, s)
                   : launch_split<false>(mapc, mapr, mapk, a, R, blocks, clusters, parts, s);
    if (e != cudaSuccess) return e;
    if ((long long)R * a.B > 0x7fffffffLL) return cudaErrorInvalidValue;
    // Few rows have many parts: then a CTA a row, its parts dealt to four warps a half (one
    // request of 78,000 tokens, 128 rows: 50.9 us a call with four rows a CTA, 39.6 so).
    const bool few = (long long)(R + 3) / 4 * a.B < num_sms;
    const int groups = few ? R : (R + 3) / 4;
    auto *const merge = few ? latent_merge_kernel<4> : latent_merge_kernel<1>;
    return launch_pdl(merge, dim3((unsigned)(groups * a.B)), dim3(kMergeWarps * 32), 0, s, a, R, blocks, clusters, parts,
                      groups);
}

cudaError_t preload_latent_decode() {
    cudaError_t e = cudaSuccess;
    for (auto *const kernel : {latent_split_kernel<true, false>, latent_split_kernel<false, false>,
                               latent_split_kernel<true, true>, latent_split_kernel<false, true>})
        if (e == cudaSuccess) e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmemBytes);
    if (e == cudaSuccess) e = preload_kernel(latent_merge_kernel<1>);
    if (e == cudaSuccess) e = preload_kernel(latent_merge_kernel<4>);
    return e;
}

}  // namespace pfkv

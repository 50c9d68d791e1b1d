// rope.cu -- rotary position embedding fused with the cache append (declared in
// pfkv_rope.h and pfkv_latent.h): queries and keys are turned by their
// positions, keys and values (or latents) are quantised or copied into their
// page slots, in one launch.
//
// Mathematics.  The pair (x_i, x_j) turns by a = position * inv_freq[i].  With
// u = inv_freq / 2 pi as a 64-bit fraction of a turn, position * u modulo 2^64
// is the angle's fraction of a turn exactly (integers wrap as angles do), so a
// position of 2^20 is as accurate as a position of 2: no fp64 arithmetic a
// token, one fp64 product a frequency.
#include <cmath>

#include "latent_internal.cuh"

namespace pfkv {
namespace {

constexpr int kRopeWarps = 8;
constexpr int kRopeThreads = kRopeWarps * 32;
constexpr int kRowsAhead = 2;               // groups of query rows of a warp in flight
constexpr int kMaxPairs = 64;               // rot_dim / 2 at most
constexpr int kTrigRows = 2 * kPage - 1;    // tokens whose angles a CTA may need

struct TokenArgs {
    const int32_t *positions, *new_lens;
    long long len_sb, len_sh;
    const int32_t *rope_pos, *row_starts;
    long long total_rows;
    int T;
};

struct TurnArgs {
    const float *inv_freq;
    int rot, inter;
    float scale;
};

struct RopeAppendArgs {
    AppendArgs ap;  // pool, tables, flags (k_new, v_new, positions are not read)
    TokenArgs tok;
    TurnArgs turn;
    RowsArg k, v, q, q_out;
    int Hq, tiles;
};

struct LatentAppendArgs {
    LatentPool pool;
    uint8_t *flags;
    TokenArgs tok;
    TurnArgs turn;
    RowsArg c, r, q, q_out;
    int Hq, tiles;
};

// The rows of request b's new tokens.
struct Span {
    int n;             // tokens, at most T
    long long row0;    // first row (packed), 0 otherwise
    bool bad;
};

__device__ __forceinline__ Span request_span(const TokenArgs &t, int b) {
    Span s{t.T, 0, false};
    if (t.row_starts) {
        const int lo = t.row_starts[b], hi = t.row_starts[b + 1];
        s.bad = lo < 0 || hi < lo || hi > t.total_rows || (long long)hi - lo > t.T;
        s.n = s.bad ? 0 : hi - lo;
        s.row0 = lo;
    }
    return s;
}

__device__ __forceinline__ int head_tokens(const TokenArgs &t, const Span &s, long long li) {
    return t.new_lens ? min(t.new_lens[li], s.n) : s.n;
}

__device__ __forceinline__ __nv_bfloat16 *row_of(const RowsArg &r, const TokenArgs &tok, const Span &s, int b,
                                                 int t, int h) {
    const long long lead = tok.row_starts ? (s.row0 + t) * r.st : (long long)b * r.sb + (long long)t * r.st;
    return r.p + lead + (long long)h * r.sh;
}

// Cosines and sines (times scale) of the tokens tlo .. tlo + kTrigRows - 1, a
// float4 holding two frequencies: pair i of token t in half i & 1 of
// cs[t - tlo][(i & 7) / 2][i / 8], so that lane p of a row reads its eight
// pairs 8p .. 8p + 7 as four words without bank conflicts.
struct Trig {
    float4 cs[kTrigRows][4][8];
    unsigned long long step[kMaxPairs];
};

// Fills the tokens t0 .. t1 - 1 (t0 >= tlo); `pos0` is token 0's position.
__device__ __forceinline__ void fill_trig(Trig &tr, const TurnArgs &a, long long pos0, int tlo, int t0, int t1) {
    const int pairs = a.rot / 2;
    for (int i = threadIdx.x; i < pairs; i += kRopeThreads) {
        // turns a position, without the whole ones, as a 64-bit fraction
        double u = (double)a.inv_freq[i] * 0.15915494309189533577;
        u -= floor(u);
        tr.step[i] = (unsigned long long)(u * 18446744073709551616.0);
    }
    __syncthreads();
    for (int e = threadIdx.x; e < (t1 - t0) * pairs; e += kRopeThreads) {
        const int r = e / pairs, i = e - r * pairs;
        const unsigned long long frac = (unsigned long long)(pos0 + t0 + r) * tr.step[i];
        // half turns in [-1, 1): the top 32 bits, rounded
        const float x = (float)(int)((frac + 0x80000000ull) >> 32) * 4.656612873077393e-10f;
        float s, c;
        sincospif(x, &s, &c);
        float *dst = reinterpret_cast<float *>(&tr.cs[t0 + r - tlo][(i & 7) >> 1][i >> 3]) + 2 * (i & 1);
        dst[0] = c * a.scale;
        dst[1] = s * a.scale;
    }
    __syncthreads();
}

// A lane's share of a row of D elements: sixteen, as two 16-byte chunks that
// hold eight whole pairs.  Rotated with halves apart, the chunks are p and p +
// rot / 16; otherwise (interleaved, or past rot) 2p and 2p + 1.
struct Share {
    int c0, c1;
    bool turned;
};

__device__ __forceinline__ Share lane_share(const TurnArgs &a, int p) {
    Share s;
    s.turned = p < a.rot / 16;
    const bool halves = s.turned && !a.inter;
    s.c0 = halves ? p : 2 * p;
    s.c1 = halves ? p + a.rot / 16 : 2 * p + 1;
    return s;
}

__device__ __forceinline__ void unpack8(const uint4 &w, float *x) {
    const uint32_t v[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 f = bf16x2_to_float2(v[i]);
        x[2 * i] = f.x;
        x[2 * i + 1] = f.y;
    }
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&h);
}

__device__ __forceinline__ uint4 pack8(const float *x) {
    return make_uint4(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4], x[5]), pack_bf16(x[6], x[7]));
}

// Turns a lane's sixteen elements (its two chunks in order).  One branch for all of
// them: inside the loops the compiler would issue both forms.
template <bool Inter>
__device__ __forceinline__ void turn16(float *x, const float4 (&cs)[4][8], int p) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const float4 w = cs[k][p];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const int i = 2 * k + u, at = Inter ? 2 * i : i, to = Inter ? 2 * i + 1 : 8 + i;
            const float c = u ? w.z : w.x, s = u ? w.w : w.y, a = x[at], b = x[to];
            x[at] = a * c - b * s;
            x[to] = b * c + a * s;
        }
    }
}

__device__ __forceinline__ void turn16(float *x, const float4 (&cs)[4][8], int p, int inter) {
    if (inter) turn16<true>(x, cs, p);
    else turn16<false>(x, cs, p);
}

// A unit's scale, its reciprocal, and whether quotients may be taken by it: in a unit that
// this call opens they are at most 448, and far enough above fp32's smallest numbers
// their remainders are exact.
struct Quant {
    float scale, inv;
    bool quick;
};

__device__ __forceinline__ Quant quant_of(float scale, bool opened) {
    return Quant{scale, __frcp_rn(scale), opened && scale > 1e-24f && scale < 1e30f};
}

// The codes of x / scale, the fp32 quotient.  Markstein's theorem (IBM J. Res. Dev. 34,
// 1990): with a correctly rounded reciprocal, a quotient within a step of the true one
// becomes the correctly rounded one when its remainder, exact in a fused
// multiply-add, times the reciprocal is added.  x times the reciprocal is within one and a
// half steps; one such correction brings it within one, a second is the theorem's.
// (Quotients below 2^-11, whose remainders may underflow, have the code zero anyway.)
// Five operations on two elements at a time, against a division's dozen on one.
__device__ __forceinline__ uint2 encode8(const float *x, const Quant &q) {
    float y[8];
    if (q.quick) {
        const float2 inv = make_float2(q.inv, q.inv), scale = make_float2(-q.scale, -q.scale);
#pragma unroll
        for (int e = 0; e < 8; e += 2) {
            const float2 a = make_float2(x[e], x[e + 1]);
            float2 v = mul2(a, inv);
            v = fma2(fma2(v, scale, a), inv, v);
            v = fma2(fma2(v, scale, a), inv, v);
            y[e] = copysignf(v.x, a.x);  // a negative zero loses its sign in the sums
            y[e + 1] = copysignf(v.y, a.y);
        }
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) y[e] = __fdiv_rn(x[e], q.scale);
    }
    uint32_t w[2] = {0u, 0u};
#pragma unroll
    for (int e = 0; e < 8; e += 2)
        w[e >> 2] |= (uint32_t)__nv_cvt_float2_to_fp8x2(make_float2(y[e], y[e + 1]), __NV_SATFINITE, __NV_E4M3) << (8 * (e & 3));
    return make_uint2(w[0], w[1]);
}

__device__ __forceinline__ float absmax16(const float *x) {
    float m = 0.f;
#pragma unroll
    for (int e = 0; e < 16; ++e) m = fmaxf(m, fabsf(x[e]));
    return m;
}

// Of sixteen bf16 elements as they were loaded.
__device__ __forceinline__ float absmax16(const uint4 &a, const uint4 &b) {
    const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
    __nv_bfloat162 m = __habs2(*reinterpret_cast<const __nv_bfloat162 *>(&w[0]));
#pragma unroll
    for (int i = 1; i < 8; ++i) m = __hmax2(m, __habs2(*reinterpret_cast<const __nv_bfloat162 *>(&w[i])));
    const float2 f = __bfloat1622float2(m);
    return fmaxf(f.x, f.y);
}

__device__ __forceinline__ float warp_max(float m) {
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, off));
    return m;
}

// The query rows of tokens t0 .. t1 - 1 of request b, `first` and `step` in
// groups of rows that a warp takes at once.
template <int D>
__device__ __forceinline__ void turn_queries(const RowsArg &q, const RowsArg &out, int Hq, const TokenArgs &tok,
                                             const TurnArgs &turn, const Span &sp, const Trig &tr, int tlo, int b,
                                             int t0, int t1, int first, int step) {
    constexpr int LANES = D / 16, RPW = 32 / LANES;
    const int lane = threadIdx.x & 31, p = lane % LANES;
    const Share sh = lane_share(turn, p);
    const int rows = (t1 - t0) * Hq;
    // the next group's row is on its way while one is turned
    struct Row {
        uint4 w0, w1;
        uint4 *dst;
        int t;
    };
    auto load = [&](int i, Row &r) {
        if (i >= rows) return;
        const int t = i / Hq, h = i - t * Hq;
        const uint4 *src = reinterpret_cast<const uint4 *>(row_of(q, tok, sp, b, t0 + t, h));
        r.dst = reinterpret_cast<uint4 *>(row_of(out, tok, sp, b, t0 + t, h));
        r.w0 = src[sh.c0];
        r.w1 = src[sh.c1];
        r.t = t0 + t - tlo;
    };
    int i = first * RPW + lane / LANES;
    Row r[kRowsAhead] = {};
#pragma unroll
    for (int u = 0; u < kRowsAhead; ++u) load(i + u * step * RPW, r[u]);
    for (; i < rows; i += kRowsAhead * step * RPW) {
#pragma unroll
        for (int u = 0; u < kRowsAhead; ++u) {
            const int at = i + u * step * RPW;
            if (at >= rows) continue;
            const Row now = r[u];
            load(at + kRowsAhead * step * RPW, r[u]);
            if (!sh.turned) {
                now.dst[sh.c0] = now.w0;
                now.dst[sh.c1] = now.w1;
                continue;
            }
            float x[16];
            unpack8(now.w0, x);
            unpack8(now.w1, x + 8);
            turn16(x, tr.cs[now.t], p, turn.inter);
            now.dst[sh.c0] = pack8(x);
            now.dst[sh.c1] = pack8(x + 8);
        }
    }
}

// What one (request, kv head) writes into its k-th unit: tokens tb .. te - 1
// from slot slot0, or nothing; `bits` says why not.
struct UnitSpan {
    long long lp;
    int tb, te, slot0;
    uint32_t bits;
};

__device__ __forceinline__ UnitSpan unit_span(int p0, int n, int k, int max_pages) {
    UnitSpan u{0, 0, 0, 0, 0u};
    if (n <= 0) return u;
    if (p0 < 0) {
        if (k == 0) u.bits = PFKV_FLAG_BAD_LENGTH;
        return u;
    }
    u.lp = (long long)(p0 / kPage) + k;
    const long long tb = max((long long)p0, u.lp * kPage) - p0;
    const long long te = min((long long)p0 + n, (u.lp + 1) * kPage) - p0;
    if (tb >= te) return u;
    if (u.lp >= max_pages) {
        u.bits = PFKV_FLAG_BAD_LENGTH;
        return u;
    }
    u.tb = (int)tb;
    u.te = (int)te;
    u.slot0 = (int)((p0 + tb) % kPage);
    return u;
}

// --------------------------------------------------------------------------
// pfkv_rope_append: a CTA takes a slice of the heads of one request's k-th
// tile of 16 cache slots.  The angles of its tokens are computed once in shared
// memory and serve every head; then a warp takes a unit (16 tokens of one kv
// head, K or V, its bf16 words held in registers between the absolute maximum and
// the encoding, so that each element is read once) or a group of query rows.
//
// 16,752 tokens, 32 query and 8 kv heads of 128, FP8: 377 MB in 86 us (4.4 TB/s).  The
// queries alone take what a copy of them takes (43 us).  Keys and values alone take 37 us
// for 103 MB: turning, maximum and codes are 23 instructions an element and lane, and half of
// the issue slots are used: 24 warps a multiprocessor leave latencies open, and the CTAs are
// 3.4 rounds of those that fit.  In one call the two parts add up.
// --------------------------------------------------------------------------
template <int D, bool FP8>
__device__ __forceinline__ void append_turned_unit(const RopeAppendArgs &a, const Span &sp, const Trig &tr, int tlo,
                                                   int b, int h, bool is_v, int k) {
    constexpr int LANES = D / 16, RPW = 32 / LANES, PASSES = kPage / RPW;
    const int lane = threadIdx.x & 31, p = lane % LANES, sub = lane / LANES;
    const long long li = (long long)b * a.tok.len_sb + (long long)h * a.tok.len_sh;
    const UnitSpan u = unit_span(a.tok.positions[li], head_tokens(a.tok, sp, li), k, a.ap.max_pages);
    if (u.bits && lane == 0 && a.ap.flags) atomic_or_byte(a.ap.flags, b, u.bits);
    if (u.tb >= u.te) return;
    Share sh = lane_share(a.turn, p);
    if (is_v) sh = Share{2 * p, 2 * p + 1, false};
    const RowsArg &src = is_v ? a.v : a.k;
    uint4 w[PASSES][2];
#pragma unroll
    for (int j = 0; j < PASSES; ++j) {
        const int t = u.tb + j * RPW + sub;
        w[j][0] = w[j][1] = make_uint4(0u, 0u, 0u, 0u);
        if (t < u.te) {
            const uint4 *row = reinterpret_cast<const uint4 *>(row_of(src, a.tok, sp, b, t, h));
            w[j][0] = row[sh.c0];
            w[j][1] = row[sh.c1];
        }
    }
    const long long bi = (long long)b * a.ap.bt_sb + (long long)h * a.ap.bt_sh + u.lp;
    const int phys = a.ap.block_tables[bi];
    uint32_t bits = 0;
    if (phys < 0 || phys >= a.ap.num_pages) bits = PFKV_FLAG_BAD_PAGE;
    else if (a.ap.page_tags && a.ap.page_tags[(long long)phys * a.ap.Hkv + h] != a.ap.expected_tags[bi])
        bits = PFKV_FLAG_TAG_MISMATCH;
    if (bits) {
        if (lane == 0 && a.ap.flags) atomic_or_byte(a.ap.flags, b, bits);
        return;
    }
    const long long unit = (long long)phys * a.ap.Hkv + h;
    const long long dst0 = (unit * kPage + u.slot0) * D;
    // A row is turned once for the absolute maximum and once for its codes: kept in
    // fp32 between, the rows take 120 registers a thread, which halves the warps.
    auto turned = [&](int j, float *x) {
        unpack8(w[j][0], x);
        unpack8(w[j][1], x + 8);
        const int t = u.tb + j * RPW + sub;
        if (sh.turned && t < u.te) turn16(x, tr.cs[t - tlo], p, a.turn.inter);
    };
    if constexpr (FP8) {
        float *scales = is_v ? a.ap.v_scale : a.ap.k_scale;
        float scale;
        if (u.slot0 == 0) {  // this call opens the unit
            float top = 0.f;
#pragma unroll
            for (int j = 0; j < PASSES; ++j) {
                if (!sh.turned) {
                    top = fmaxf(top, absmax16(w[j][0], w[j][1]));
                    continue;
                }
                float x[16];
                turned(j, x);
                top = fmaxf(top, absmax16(x));
            }
            top = warp_max(top);
            scale = top == 0.f ? 1.f : __fdiv_rn(top, 448.f);
            if (lane == 0) scales[unit] = scale;
        } else {
            scale = scales[unit];
        }
        const Quant qn = quant_of(scale, u.slot0 == 0);
        uint8_t *dst = static_cast<uint8_t *>(is_v ? a.ap.v_pages : a.ap.k_pages) + dst0;
#pragma unroll
        for (int j = 0; j < PASSES; ++j) {
            const int r = j * RPW + sub;
            if (u.tb + r >= u.te) continue;
            float x[16];
            turned(j, x);
            uint2 *row = reinterpret_cast<uint2 *>(dst + (long long)r * D);
            row[sh.c0] = encode8(x, qn);
            row[sh.c1] = encode8(x + 8, qn);
        }
    } else {
        __nv_bfloat16 *dst = static_cast<__nv_bfloat16 *>(is_v ? a.ap.v_pages : a.ap.k_pages) + dst0;
#pragma unroll
        for (int j = 0; j < PASSES; ++j) {
            const int r = j * RPW + sub;
            if (u.tb + r >= u.te) continue;
            uint4 *row = reinterpret_cast<uint4 *>(dst + (long long)r * D);
            if (!sh.turned) {
                row[sh.c0] = w[j][0];
                row[sh.c1] = w[j][1];
                continue;
            }
            float x[16];
            turned(j, x);
            row[sh.c0] = pack8(x);
            row[sh.c1] = pack8(x + 8);
        }
    }
}

// The tokens whose angles tile k of request b needs, and the query tokens of
// the tile.  One length a request: the 16 slots of the tile.  A length a head:
// the heads' tiles start up to 15 tokens apart.
struct TileTokens {
    int tlo, t0, t1, q0, q1;
};

__device__ __forceinline__ TileTokens tile_tokens(int p0, int n_all, int n_q, int k, bool per_head) {
    TileTokens r;
    const int o = p0 < 0 ? 0 : p0 % kPage;
    const int first = k * kPage - o;
    r.tlo = per_head ? k * kPage - (kPage - 1) : first;
    r.t0 = max(0, r.tlo);
    r.t1 = max(r.t0, min(n_all, per_head ? k * kPage + kPage : first + kPage));
    r.q0 = max(0, first);
    r.q1 = max(r.q0, min(n_q, first + kPage));
    return r;
}

template <int D, bool FP8>
__global__ void __launch_bounds__(kRopeThreads, 3) rope_append_kernel(RopeAppendArgs a) {
    __shared__ Trig tr;
    pdl_enter();
    const int b = blockIdx.x / a.tiles, k = blockIdx.x - b * a.tiles;
    const Span sp = request_span(a.tok, b);
    if (sp.bad) {
        if (k == 0 && blockIdx.y == 0 && threadIdx.x == 0 && a.ap.flags)
            atomic_or_byte(a.ap.flags, b, PFKV_FLAG_BAD_LENGTH);
        return;
    }
    const long long l0 = (long long)b * a.tok.len_sb;
    const int p0 = a.tok.positions[l0];
    const int nq = head_tokens(a.tok, sp, l0);
    const bool per_head = a.tok.len_sh != 0;
    const TileTokens tt = tile_tokens(p0, per_head ? sp.n : nq, nq, k, per_head);
    if (tt.t0 >= tt.t1) return;  // uniform: no token of the request in this tile
    const int warp = blockIdx.y * kRopeWarps + (threadIdx.x >> 5), warps = gridDim.y * kRopeWarps;
    const int units = 2 * a.ap.Hkv, turns = units > warp ? (units - warp + warps - 1) / warps : 0;  // units of this warp
    const int first = warp + turns * warps - units;  // its first group of query rows
    fill_trig(tr, a.turn, a.tok.rope_pos ? a.tok.rope_pos[b] : p0, tt.tlo, tt.t0, tt.t1);
    for (int item = warp; item < units; item += warps) {
        const bool is_v = item >= a.ap.Hkv;
        append_turned_unit<D, FP8>(a, sp, tr, tt.tlo, b, is_v ? item - a.ap.Hkv : item, is_v, k);
    }
    if (a.Hq > 0) turn_queries<D>(a.q, a.q_out, a.Hq, a.tok, a.turn, sp, tr, tt.tlo, b, tt.q0, tt.q1, first, warps);
}

// --------------------------------------------------------------------------
// pfkv_latent_append: the same for a latent pool.  Four warps of the first
// slice take the tile's latents (128 elements each, one scale), a fifth the
// turned keys; every warp then takes query rows.  28 KB a tile of 16 tokens with 16
// heads: short prompts are bound by the chain of loads (starts, positions, angles,
// rows), 15 us for 61 MB; longer ones by memory.
// --------------------------------------------------------------------------
constexpr int kLatentWarps = PFKV_LATENT_DIM / 128;

template <bool FP8>
__device__ __forceinline__ void append_latents(const LatentAppendArgs &a, const Span &sp, int b, const UnitSpan &u,
                                               int phys, int part, float *red) {
    constexpr int LANES = 8, RPW = 4, PASSES = 4;
    const int lane = threadIdx.x & 31, p = lane % LANES, sub = lane / LANES;
    const int chunk = part * 16 + 2 * p;  // of eight elements
    uint4 w[PASSES][2];
#pragma unroll
    for (int j = 0; j < PASSES; ++j) {
        const int t = u.tb + j * RPW + sub;
        w[j][0] = w[j][1] = make_uint4(0u, 0u, 0u, 0u);
        if (t < u.te) {
            const uint4 *row = reinterpret_cast<const uint4 *>(row_of(a.c, a.tok, sp, b, t, 0));
            w[j][0] = row[chunk];
            w[j][1] = row[chunk + 1];
        }
    }
    const long long dst0 = ((long long)phys * kPage + u.slot0) * PFKV_LATENT_DIM;
    if constexpr (FP8) {
        float scale;
        if (u.slot0 == 0) {
            float top = 0.f;
#pragma unroll
            for (int j = 0; j < PASSES; ++j) top = fmaxf(top, absmax16(w[j][0], w[j][1]));
            top = warp_max(top);
            if (lane == 0) red[part] = top;
            asm volatile("bar.sync 1, %0;" ::"n"(kLatentWarps * 32) : "memory");
#pragma unroll
            for (int i = 0; i < kLatentWarps; ++i) top = fmaxf(top, red[i]);
            scale = top == 0.f ? 1.f : __fdiv_rn(top, 448.f);
            if (lane == 0 && part == 0) a.pool.c_scale[phys] = scale;
        } else {
            scale = a.pool.c_scale[phys];
        }
        const Quant qn = quant_of(scale, u.slot0 == 0);
        uint8_t *dst = static_cast<uint8_t *>(a.pool.c_pages) + dst0;
#pragma unroll
        for (int j = 0; j < PASSES; ++j) {
            const int r = j * RPW + sub;
            if (u.tb + r >= u.te) continue;
            float x[16];
            unpack8(w[j][0], x);
            unpack8(w[j][1], x + 8);
            const uint2 lo = encode8(x, qn), hi = encode8(x + 8, qn);
            reinterpret_cast<uint4 *>(dst + (long long)r * PFKV_LATENT_DIM)[chunk / 2] =
                make_uint4(lo.x, lo.y, hi.x, hi.y);
        }
    } else {
        __nv_bfloat16 *dst = static_cast<__nv_bfloat16 *>(a.pool.c_pages) + dst0;
#pragma unroll
        for (int j = 0; j < PASSES; ++j) {
            const int r = j * RPW + sub;
            if (u.tb + r >= u.te) continue;
            uint4 *row = reinterpret_cast<uint4 *>(dst + (long long)r * PFKV_LATENT_DIM);
            row[chunk] = w[j][0];
            row[chunk + 1] = w[j][1];
        }
    }
}

__device__ __forceinline__ void append_turned_keys(const LatentAppendArgs &a, const Span &sp, const Trig &tr, int tlo,
                                                   int b, const UnitSpan &u, int phys) {
    constexpr int D = PFKV_LATENT_ROPE, LANES = D / 16, RPW = 32 / LANES;
    const int lane = threadIdx.x & 31, p = lane % LANES;
    const Share sh = lane_share(a.turn, p);
    for (int r = lane / LANES; u.tb + r < u.te; r += RPW) {
        const int t = u.tb + r;
        const uint4 *src = reinterpret_cast<const uint4 *>(row_of(a.r, a.tok, sp, b, t, 0));
        uint4 *dst = reinterpret_cast<uint4 *>(a.pool.r_pages + ((long long)phys * kPage + u.slot0 + r) * D);
        const uint4 w0 = src[sh.c0], w1 = src[sh.c1];
        float x[16];
        unpack8(w0, x);
        unpack8(w1, x + 8);
        if (sh.turned) turn16(x, tr.cs[t - tlo], p, a.turn.inter);
        dst[sh.c0] = sh.turned ? pack8(x) : w0;
        dst[sh.c1] = sh.turned ? pack8(x + 8) : w1;
    }
}

template <bool FP8>
__global__ void __launch_bounds__(kRopeThreads, 3) latent_append_kernel(LatentAppendArgs a) {
    __shared__ Trig tr;
    __shared__ float red[kLatentWarps];
    pdl_enter();
    const int b = blockIdx.x / a.tiles, k = blockIdx.x - b * a.tiles;
    const Span sp = request_span(a.tok, b);
    if (sp.bad) {
        if (k == 0 && blockIdx.y == 0 && threadIdx.x == 0 && a.flags) atomic_or_byte(a.flags, b, PFKV_FLAG_BAD_LENGTH);
        return;
    }
    const long long l0 = (long long)b * a.tok.len_sb;
    const int p0 = a.tok.positions[l0];
    const int n = head_tokens(a.tok, sp, l0);
    const TileTokens tt = tile_tokens(p0, n, n, k, false);
    if (tt.t0 >= tt.t1) return;
    const int warp = threadIdx.x >> 5;
    fill_trig(tr, a.turn, a.tok.rope_pos ? a.tok.rope_pos[b] : p0, tt.tlo, tt.t0, tt.t1);
    if (blockIdx.y == 0 && warp <= kLatentWarps) {
        // uniform over these warps, so that the barrier inside is met by all
        const UnitSpan u = unit_span(p0, n, k, a.pool.max_pages);
        uint32_t bits = u.bits;
        int phys = 0;
        if (u.tb < u.te) {
            const long long bi = (long long)b * a.pool.bt_sb + u.lp;
            phys = a.pool.block_tables[bi];
            bits = latent_entry_bits(a.pool, phys, bi);
        }
        if (bits) {
            if (threadIdx.x == 0 && a.flags) atomic_or_byte(a.flags, b, bits);
        } else if (u.tb < u.te) {
            if (warp < kLatentWarps) append_latents<FP8>(a, sp, b, u, phys, warp, red);
            else append_turned_keys(a, sp, tr, tt.tlo, b, u, phys);
        }
    }
    if (a.Hq > 0)
        turn_queries<PFKV_LATENT_ROPE>(a.q, a.q_out, a.Hq, a.tok, a.turn, sp, tr, tt.tlo, b, tt.q0, tt.q1,
                                       blockIdx.y * kRopeWarps + warp, gridDim.y * kRopeWarps);
}

// Slices of one tile's heads: enough CTAs for two a streaming multiprocessor
// when the batch alone gives fewer, and no more than there are warps' items.
unsigned head_slices(long long tiles, long long items, int num_sms) {
    const long long want = (2LL * num_sms + tiles - 1) / tiles;
    const long long most = (items + kRopeWarps - 1) / kRopeWarps;
    return (unsigned)max(1LL, min(min(want, most), 64LL));
}

pfkv_status check_turn(const pfkv_rope *r, int row) {
    if (!r) return PFKV_ERR_INVALID_ARG;
    if (r->rot_dim <= 0 || r->rot_dim % 16 != 0 || r->rot_dim > row) return PFKV_ERR_INVALID_ARG;
    if (r->interleaved != 0 && r->interleaved != 1) return PFKV_ERR_INVALID_ARG;
    if (!std::isfinite(r->scale)) return PFKV_ERR_INVALID_ARG;
    return PFKV_OK;
}

pfkv_status check_tokens(const pfkv_new_tokens *t, const pfkv_pages *p, const pfkv_rope *r) {
    if (!t || t->num_new_tokens <= 0) return PFKV_ERR_INVALID_ARG;
    if (t->num_new_tokens > (1 << 24)) return PFKV_ERR_UNSUPPORTED;  // tile and row counts are 32-bit
    if (p->batch == 0) return PFKV_OK;
    if (!t->positions || !r->inv_freq) return PFKV_ERR_INVALID_ARG;
    if (!t->rope_positions && p->len_stride_h != 0) return PFKV_ERR_INVALID_ARG;
    if (t->row_starts && t->total_rows < 0) return PFKV_ERR_INVALID_ARG;
    const void *four[] = {t->positions, t->new_lens, t->rope_positions, t->row_starts, r->inv_freq};
    for (const void *q : four)
        if (!aligned(q, 4)) return PFKV_ERR_ALIGNMENT;
    return PFKV_OK;
}

// Rows that the arrays of new tokens hold, as far as it is known here.
int64_t new_rows(const pfkv_new_tokens *t) { return t->row_starts ? t->total_rows : 1; }

// Queries: both arrays or neither.
pfkv_status check_queries(const pfkv_rows *q, const pfkv_rows *out, int heads, bool use_b, int64_t rows) {
    if ((q == nullptr) != (out == nullptr)) return PFKV_ERR_INVALID_ARG;
    if (!q) return PFKV_OK;
    if (heads <= 0) return PFKV_ERR_INVALID_ARG;
    pfkv_status st = check_rows(q, use_b, true, rows);
    if (st == PFKV_OK) st = check_rows(out, use_b, true, rows);
    return st;
}

TokenArgs token_args(const pfkv_new_tokens *t, const pfkv_pages *p) {
    return TokenArgs{t->positions, t->new_lens, (long long)p->len_stride_b, (long long)p->len_stride_h,
                     t->rope_positions, t->row_starts, (long long)t->total_rows, t->num_new_tokens};
}

TurnArgs turn_args(const pfkv_rope *r) { return TurnArgs{r->inv_freq, r->rot_dim, r->interleaved, r->scale}; }

}  // namespace

pfkv_status check_rows(const pfkv_rows *r, bool use_b, bool use_h, int64_t rows) {
    if (!r) return PFKV_ERR_INVALID_ARG;
    if (rows == 0) return PFKV_OK;
    if (!r->data) return PFKV_ERR_INVALID_ARG;
    const int64_t sb = use_b ? r->stride_b : 0, sh = use_h ? r->stride_h : 0;
    if (sb < 0 || r->stride_t < 0 || sh < 0) return PFKV_ERR_INVALID_ARG;
    if (!aligned(r->data, 16) || ((sb | r->stride_t | sh) & 7)) return PFKV_ERR_ALIGNMENT;
    return PFKV_OK;
}

cudaError_t preload_rope() {
    cudaError_t e = cudaSuccess;
    auto one = [&](cudaError_t r) { if (e == cudaSuccess) e = r; };
    one(preload_kernel(rope_append_kernel<128, true>));
    one(preload_kernel(rope_append_kernel<64, true>));
    one(preload_kernel(rope_append_kernel<128, false>));
    one(preload_kernel(rope_append_kernel<64, false>));
    one(preload_kernel(latent_append_kernel<true>));
    one(preload_kernel(latent_append_kernel<false>));
    return e;
}

}  // namespace pfkv

using namespace pfkv;

extern "C" {

pfkv_status pfkv_rope_append(const pfkv_cache *cache, const pfkv_pages *pages, const pfkv_rope *rope,
                             const pfkv_new_tokens *tokens, const pfkv_rows *k_new, const pfkv_rows *v_new,
                             const pfkv_rows *q, const pfkv_rows *q_out, int32_t num_q_heads, uint8_t *flags,
                             void *stream) {
    pfkv_status st = check_cache(cache);
    if (st == PFKV_OK) st = check_pages(cache, pages);
    if (st == PFKV_OK) st = check_turn(rope, cache->head_dim);
    if (st == PFKV_OK) st = check_tokens(tokens, pages, rope);
    if (st != PFKV_OK || pages->batch == 0) return st;
    const bool use_b = tokens->row_starts == nullptr;
    const int64_t n = new_rows(tokens);
    st = check_rows(k_new, use_b, true, n);
    if (st == PFKV_OK) st = check_rows(v_new, use_b, true, n);
    if (st == PFKV_OK) st = check_queries(q, q_out, num_q_heads, use_b, n);
    if (st != PFKV_OK) return st;
    if (flags && !aligned(flags, 4)) return PFKV_ERR_ALIGNMENT;
    const long long tiles = ((long long)tokens->num_new_tokens + 30) / kPage;  // ceil((T + 15) / 16)
    const long long grid = (long long)pages->batch * tiles;
    if (grid > 0x7fffffffLL || (q && num_q_heads > 0x7fffffff / kPage)) return PFKV_ERR_UNSUPPORTED;
    int sms = 0;
    st = device_check(&sms);
    if (st != PFKV_OK) return st;
    RopeAppendArgs a{};
    a.ap.k_pages = cache->k_pages;
    a.ap.v_pages = cache->v_pages;
    a.ap.k_scale = cache->k_scale;
    a.ap.v_scale = cache->v_scale;
    a.ap.page_tags = cache->page_tags;
    a.ap.num_pages = cache->num_pages;
    a.ap.Hkv = cache->num_kv_heads;
    a.ap.block_tables = pages->block_tables;
    a.ap.bt_sb = pages->bt_stride_b;
    a.ap.bt_sh = pages->bt_stride_h;
    a.ap.expected_tags = pages->expected_tags;
    a.ap.max_pages = pages->max_pages;
    a.ap.flags = flags;
    a.tok = token_args(tokens, pages);
    a.turn = turn_args(rope);
    a.k = rows_arg(k_new);
    a.v = rows_arg(v_new);
    a.Hq = q ? num_q_heads : 0;
    if (q) {
        a.q = rows_arg(q);
        a.q_out = rows_arg(q_out);
    }
    a.tiles = (int)tiles;
    const int rpw = 512 / cache->head_dim;  // query rows that a warp takes at once
    const long long rows = (long long)min(tokens->num_new_tokens, (int32_t)kPage) * a.Hq;
    const dim3 g((unsigned)grid, head_slices(grid, 2LL * a.ap.Hkv + (rows + rpw - 1) / rpw, sms));
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    const bool fp8 = cache->dtype == PFKV_KV_FP8_E4M3;
    cudaError_t e;
    if (cache->head_dim == 128)
        e = fp8 ? launch_pdl(rope_append_kernel<128, true>, g, dim3(kRopeThreads), 0, s, a)
                : launch_pdl(rope_append_kernel<128, false>, g, dim3(kRopeThreads), 0, s, a);
    else
        e = fp8 ? launch_pdl(rope_append_kernel<64, true>, g, dim3(kRopeThreads), 0, s, a)
                : launch_pdl(rope_append_kernel<64, false>, g, dim3(kRopeThreads), 0, s, a);
    return e == cudaSuccess ? PFKV_OK : PFKV_ERR_CUDA;
}

pfkv_status pfkv_latent_append(const pfkv_latent_cache *cache, const pfkv_pages *pages, const pfkv_rope *rope,
                               const pfkv_new_tokens *tokens, const pfkv_rows *c_new, const pfkv_rows *r_new,
                               const pfkv_rows *q, const pfkv_rows *q_out, int32_t num_q_heads, uint8_t *flags,
                               void *stream) {
    pfkv_status st = check_latent(cache, pages);
    if (st == PFKV_OK) st = check_turn(rope, cache->rope_dim);
    if (st == PFKV_OK) st = check_tokens(tokens, pages, rope);
    if (st != PFKV_OK || pages->batch == 0) return st;
    const bool use_b = tokens->row_starts == nullptr;
    const int64_t n = new_rows(tokens);
    st = check_rows(c_new, use_b, false, n);
    if (st == PFKV_OK) st = check_rows(r_new, use_b, false, n);
    if (st == PFKV_OK) st = check_queries(q, q_out, num_q_heads, use_b, n);
    if (st != PFKV_OK) return st;
    if (flags && !aligned(flags, 4)) return PFKV_ERR_ALIGNMENT;
    const long long tiles = ((long long)tokens->num_new_tokens + 30) / kPage;
    const long long grid = (long long)pages->batch * tiles;
    if (grid > 0x7fffffffLL || (q && num_q_heads > 0x7fffffff / kPage)) return PFKV_ERR_UNSUPPORTED;
    int sms = 0;
    st = device_check(&sms);
    if (st != PFKV_OK) return st;
    LatentAppendArgs a{};
    a.pool = latent_pool(cache, pages);
    a.flags = flags;
    a.tok = token_args(tokens, pages);
    a.turn = turn_args(rope);
    a.c = rows_arg(c_new);
    a.r = rows_arg(r_new);
    a.Hq = q ? num_q_heads : 0;
    if (q) {
        a.q = rows_arg(q);
        a.q_out = rows_arg(q_out);
    }
    a.tiles = (int)tiles;
    const long long rows = (long long)min(tokens->num_new_tokens, (int32_t)kPage) * a.Hq;
    const dim3 g((unsigned)grid, head_slices(grid, kLatentWarps + 1 + (rows + 7) / 8, sms));
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    const cudaError_t e = cache->dtype == PFKV_KV_FP8_E4M3
                              ? launch_pdl(latent_append_kernel<true>, g, dim3(kRopeThreads), 0, s, a)
                              : launch_pdl(latent_append_kernel<false>, g, dim3(kRopeThreads), 0, s, a);
    return e == cudaSuccess ? PFKV_OK : PFKV_ERR_CUDA;
}

}  // extern "C"

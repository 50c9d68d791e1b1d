// prefix_attn.cu -- attention of all query rows of a prefix's requests over the prefix, by
// the fifth-generation tensor cores (the middle part of pfkv_prefix_decode_attn).
//
// Mathematics.  For a prefix and kv head, with the rows of its requests (request, query token,
// head of the group) as one matrix Q of R rows: S = Q K^T, P = softmax weights, O = P V.  A token
// costs 4 R D operations and 2 D bytes an element of the pool: with 128 rows a BF16 pool is still
// bound by memory (128 operations a byte, the machine has 282), with 256 rows both bind.
//
// A CTA takes a range of tiles of 128 tokens (see PrefixSeg) and leaves a partial result (rows
// normalised, with their log2-sum-exp) for every segment that it touches.  Two groups of four
// softmax warps work in turns, so that one's softmax runs under the other's products: on the two
// halves of a block of more than 128 rows, both on every tile; or, with up to 128 rows, on every
// second tile of the same rows, and their results are merged at the end.  Tensor memory holds S of
// both (a group's weights overwrite its scores and are read from there as the A operand) and O of
// both.
//
// A weight enters the second product as a pair of 16-bit values, upper bits and what is left of them, in
// two instructions: rounded once to bf16 or f16 it would be off by 2^-8 or 2^-11 of w |v|, which a sum of
// large values that cancel does not shrink, and the result by more than the library's bound for attention
// (nine times it for BF16 pools where w |v| sums to 50).  The pair costs 2 to 11% of a call.
// BF16 pools: K and V come by TMA as the operands that they are; weights are pairs of bf16.
// FP8 pools: K comes as it is too, and Q enters as a pair of 8-bit values (hi e4m3, lo e5m2: two products of
// half the cost of one in 16 bits); two warps convert V to f16 (exact), and weights times their
// unit's V scale are pairs of f16.  K's scales are applied to the scores, 16 columns at a time.
//
// Roles of the twelve warps: 0-3 and 4-7 softmax; 8 issues the products; 9 finds the segments and
// loads K and the scales; 10 and 11 load the V of four pages of every tile each (FP8: and convert it).  A
// page's slab of 2 KB is a copy, and a warp issues one in 67 cycles whatever its size (measured), so three
// warps share them: one alone would feed 28 bytes a cycle.
//
// Measured (inputs not in L2): BF16, 64 rows, 131,072 tokens of 8 heads: 87 us, 6.1 TB/s, 91% of the copy
// rate.  BF16, blocks of 256 rows, 8,192 tokens, 2,048 rows a head: 78 us, 0.88 PFLOP/s (1.3 with the second
// products); what bounds it are the two groups' chains (scores, 32-column loads, maximum, weights, products),
// with the tensor pipe 60% busy.  FP8, 128 rows, 16,384 tokens of 8 heads: 17 to 24 us, of which the start
// (segment, ids, queries, first copies) and the end of a CTA take as long as four of its seven tiles.
#include "prefix_internal.cuh"
#include "umma.cuh"

namespace pfkv {
namespace {

constexpr int kThreads = 384;
constexpr int kPages = kPrefixTile / kPage;  // pages of a tile
constexpr int kInfo = 4;                     // tiles' scales kept ahead, a softmax group
constexpr int kItems = 3;                    // segments found ahead
constexpr uint32_t kColO = 256;
// Weights are 2^(score - reference).  The reference is set so far above the maximum, and O rescaled once
// the maximum is so far above the reference (log2).  f16 weights have 2^7 below 2^8 of room.  bf16's
// exponents are those of fp32: weights grow from 2^-32, so that O is rescaled as seldom as the maximum
// grows by 2^40 (8,192 tokens, 256 requests: 151 us a call, 156 with 2^8), and never above 2^8, so that
// sums with values up to 2^100 are finite (growing from 1, weights of 2^40 left room for 2^70).
template <bool FP8>
constexpr float kAbove = FP8 ? 0.f : 32.f;
constexpr float kGrowth = 8.f;
constexpr float kMinusInf = -INFINITY;

template <int T>
struct Group {
    static constexpr int value = T;
};

template <int D, bool FP8>
struct Cfg {
    static constexpr int ROWB = D * (FP8 ? 1 : 2);            // a token's row in the pool
    static constexpr uint32_t KB = kPrefixTile * ROWB;        // a tile of K (and of V as loaded)
    static constexpr uint32_t VB = kPrefixTile * D * 2;       // of V as the operand
    static constexpr uint32_t HALF = kPrefixTile * 128;       // 64 16-bit columns of it
    static constexpr uint32_t QB = 128 * D * 2;               // 128 query rows (FP8: hi, then lo)
    static constexpr int NK = FP8 ? (D == 128 ? 4 : 6) : (D == 128 ? 3 : 4);
    static constexpr int NV = FP8 ? (D == 128 ? 2 : 3) : (D == 128 ? 2 : 4);
    static constexpr int NR = FP8 ? (D == 128 ? 2 : 4) : 0;   // V as loaded
    static constexpr uint32_t OFF_K = 2 * QB, OFF_V = OFF_K + NK * KB, OFF_R = OFF_V + NV * VB;
    static constexpr uint32_t OFF_MISC = OFF_R + NR * KB;
    static constexpr int CPP = FP8 || D == 64 ? 1 : 2;        // copies a page (128 bytes of a row at most)
    static constexpr uint32_t COPYB = kPage * ROWB / CPP;
};

struct Item {
    int p, h;            // p < 0: no more
    int row0, rows;      // query rows of the segment
    int t0, nt;          // tiles of this CTA
    int len;             // tokens of the prefix
    int base;            // first row of the partial result
    float vinv, vback;   // weights' factor beside the V scale, and what undoes it
};

// Scales of a tile's pages.
struct alignas(16) Info {
    float ks[kPages], vs[kPages];
};

struct Misc {
    uint64_t kfull[6], kempty[6], vfull[4], vempty[4], rfull[2][4];
    uint64_t qfull, sfull[2], pready[2][2], odone[2], merge, rest;
    uint64_t tfull[2][kInfo], tempty[2][kInfo];
    uint64_t ifull[kItems], iempty[kItems], drain;
    Item item[kItems];
    Info info[2][kInfo];
    union {  // the rows' factors at a segment's start; group 1's softmax at its end
        float qmul[kPrefixBlock];
        struct {
            float ref1[128], sum1[128];
        };
    };
    uint32_t tmem, gave_up;
};
template <int D, bool FP8>
constexpr size_t smem_bytes() {
    return Cfg<D, FP8>::OFF_MISC + sizeof(Misc);
}
static_assert(smem_bytes<128, true>() <= 232448 && smem_bytes<128, false>() <= 232448, "shared memory of one CTA");

// D (+)= A B of 8-bit operands (B e4m3; A e4m3, or e5m2 with this bit of the instruction's descriptor); `up` is
// the descriptors' upper word.
constexpr uint32_t kQueryE5M2 = 1u << 7;
template <uint32_t UP>
__device__ __forceinline__ void umma_ss_f8(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, bool accumulate) {
    asm volatile("{\n\t.reg .pred p;\n\t.reg .b64 a, b;\n\tsetp.ne.b32 p, %4, 0;\n\tmov.b64 a, {%1, %5};\n\t"
                 "mov.b64 b, {%2, %5};\n\ttcgen05.mma.cta_group::1.kind::f8f6f4 [%0], a, b, %3, p;\n\t}" ::"r"(d),
                 "r"(a), "r"(b), "r"(idesc), "r"((uint32_t)accumulate), "n"(UP)
                 : "memory");
}
// Rows of 64 bytes with the 64-byte swizzle: 16-byte chunk c of row r at chunk c ^ (r / 2 & 3),
// eight rows a 512-byte atom.
constexpr uint32_t kDescUpper64 = (512u >> 4) | (1u << 14) | (4u << 29);

__device__ __forceinline__ uint32_t pack16(float a, float b, bool bf16) {
    if (bf16) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
        return *reinterpret_cast<const uint32_t *>(&h);
    }
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&h);
}

// Four e4m3 codes -> two f16 pairs.
__device__ __forceinline__ uint2 e4m3x4_to_half4(uint32_t w) {
    uint2 r;
    asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\t"
        "cvt.rn.f16x2.e4m3x2 %0, l;\n\tcvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
        : "=r"(r.x), "=r"(r.y)
        : "r"(w));
    return r;
}

// Selftest: waits of as many tries as the call says.
template <int D, bool FP8, bool Selftest>
__global__ void __launch_bounds__(kThreads, 1)
    prefix_attn_kernel(const __grid_constant__ CUtensorMap mapk, const __grid_constant__ CUtensorMap mapv, PrefixArgs a,
                       uint32_t idS) {
    using C = Cfg<D, FP8>;
    extern __shared__ __align__(1024) uint8_t psm[];  // no static shared memory: the window's aligned base
    Misc &m = *reinterpret_cast<Misc *>(psm + C::OFF_MISC);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (tid == 0) {
        for (int i = 0; i < C::NK; ++i) {
            mbar_init(&m.kfull[i], 1);
            mbar_init(&m.kempty[i], 1);
        }
        for (int i = 0; i < C::NV; ++i) {
            mbar_init(&m.vfull[i], 2);
            mbar_init(&m.vempty[i], 1);
        }
        for (int i = 0; i < C::NR; ++i) {
            mbar_init(&m.rfull[0][i], 1);
            mbar_init(&m.rfull[1][i], 1);
        }
        mbar_init(&m.qfull, 8);
        mbar_init(&m.merge, 4);
        mbar_init(&m.rest, 8);
        for (int i = 0; i < 2; ++i) {
            mbar_init(&m.sfull[i], 1);
            mbar_init(&m.pready[i][0], 4);
            mbar_init(&m.pready[i][1], 4);
            mbar_init(&m.odone[i], 1);
            for (int j = 0; j < kInfo; ++j) {
                mbar_init(&m.tfull[i][j], 1);
                mbar_init(&m.tempty[i][j], 4);
            }
        }
        for (int i = 0; i < kItems; ++i) {
            mbar_init(&m.ifull[i], 1);
            mbar_init(&m.iempty[i], 11);  // softmax warps, the issuing thread, the warps of V
        }
        mbar_init(&m.drain, 1);
        m.gave_up = (smem_addr(psm) & 1023u) != 0u;  // nothing runs on a base that the swizzle cannot take
        fence_mbar_init();
    }
    if (warp == 8) tmem_alloc512<1>(&m.tmem);
    tmem_fence_before();
    __syncthreads();
    tmem_fence_after();
    // After the own tokens' split kernel, which lets this one start once its own wait for the plan has
    // passed and which this kernel does not read, only the end waits; the merge that follows needs both
    // (the rules are at launch_pdl).
    if (a.after_own) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    else pdl_enter();
    const uint32_t tmem = m.tmem;
    volatile uint32_t *const gave_up = &m.gave_up;
    const int tries = Selftest ? a.tries : kTries, item_tries = Selftest ? a.tries * (kItemTries / kTries) : kItemTries;
    auto item_ready = [&](int i) {
        return bar_wait(&m.ifull[i % kItems], (i / kItems) & 1, gave_up, item_tries) && m.item[i % kItems].p >= 0;
    };
    // Steps of softmax group `g`: every tile, or every second one.
    auto steps_of = [](const Item &it, int g) { return it.rows > 128 ? it.nt : (it.nt + 1 - g) / 2; };

    if (warp < 8) {
        // ----------------------- queries, softmax and results -----------------------
        reg_share_more<208>();
        const int grp = warp >> 2, r = (warp & 3) * 32 + lane;
        const uint32_t lanes = tmem + ((uint32_t)((warp & 3) * 32) << 16);
        const uint32_t cs = lanes + grp * 128, co = lanes + kColO + grp * 128;
        const float a2 = fmaxf(fabsf(a.sm_scale) * 1.4426950408889634f, 1.1754944e-38f);
        uint32_t done = 0, outs = 0, merges = 0, base_pos = 0;
        for (int i = 0; __all_sync(0xffffffffu, item_ready(i)); ++i) {
            const Item &it = m.item[i % kItems];
            const bool wide = it.rows > 128;
            const int steps = steps_of(it, grp), nt = it.nt;
            const int row = wide ? grp * 128 + r : r;
            const bool live = row < it.rows;
            const bool warp_live = (row & ~31) < it.rows;
            bool ok = true;
            // The queries: a warp takes 32 rows, or 16 where both groups have the same; LPR lanes read a
            // row, 16 bytes each.
            {
                constexpr int LPR = D / 8, RPI = 32 / LPR;
                const int rw = wide ? 32 : 16, first = warp * rw;
                const __nv_bfloat16 *mine = nullptr;  // row `lane`
                if (lane < rw && first + lane < it.rows) {
                    const int R = it.row0 + first + lane, per = a.kq * a.G, member = R / per, tg = R - member * per;
                    const int t = tg / a.G, g = tg - t * a.G;
                    const int b = a.members[a.mstart[it.p] + member];
                    mine = a.q.p + (long long)b * a.q.sb + (long long)t * a.q.st + (long long)(it.h * a.G + g) * a.q.sh;
                }
                const int c = lane % LPR;
                uint8_t *const dst = psm + (wide ? grp : 0) * C::QB;
#pragma unroll 1
                for (int n0 = 0; n0 < rw; n0 += 4 * RPI) {
                    uint4 w[4];
#pragma unroll
                    for (int n = 0; n < 4; ++n) {
                        const uint4 *src = reinterpret_cast<const uint4 *>(
                            __shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(mine), (n0 + n * RPI + lane / LPR) & 31));
                        w[n] = src ? src[c] : make_uint4(0u, 0u, 0u, 0u);
                    }
#pragma unroll
                    for (int n = 0; n < 4; ++n) {
                        const int at = first + n0 + n * RPI + lane / LPR, q = at & 127;  // in the block, and in its tile
                        if constexpr (!FP8) {
                            *reinterpret_cast<uint4 *>(dst + (c >> 3) * C::HALF + q * 128 + (((c & 7) ^ (q & 7)) << 4)) = w[n];
                        } else {
                            const uint32_t u[4] = {w[n].x, w[n].y, w[n].z, w[n].w};
                            uint32_t top = __vimax3_u16x2(u[0] & 0x7fff7fffu, u[1] & 0x7fff7fffu, u[2] & 0x7fff7fffu);
                            top = __vimax3_u16x2(top, u[3] & 0x7fff7fffu, 0u);
                            top = max(top << 16, top & 0x7fff0000u);
#pragma unroll
                            for (int off = LPR / 2; off > 0; off >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, off));
                            // The largest element between 128 and 256.  hi (e4m3) is within 2^-4 of an element down
                            // to 2^-6, so what is left is 0 to 8 of the element's last places: three bits, or a power
                            // of two, exact in lo as e5m2, whose steps end at 2^-16.  (As e4m3, whose steps end at
                            // 2^-9, lo rounded elements below 2^-9 of the largest.)  Smaller elements are within
                            // 2^-14.  What is not finite spoils the row.
                            const int e = min(126, max(-119, (int)(top >> 23) - 127));
                            float up = __uint_as_float((uint32_t)(127 + 7 - e) << 23);
                            if (a.sm_scale < 0.f) up = -up;
                            if (c == 0)
                                m.qmul[at] = top >= 0x7f800000u ? __uint_as_float(0x7fffffffu)
                                                                : a2 * __uint_as_float((uint32_t)(127 + e - 7) << 23);
                            uint32_t hi[2], lo[2];
#pragma unroll
                            for (int k = 0; k < 2; ++k) {
                                uint32_t hh[2], ll[2];
#pragma unroll
                                for (int x = 0; x < 2; ++x) {
                                    const float2 y = mul2(bf16x2_to_float2(u[2 * k + x]), make_float2(up, up));
                                    hh[x] = __nv_cvt_float2_to_fp8x2(y, __NV_SATFINITE, __NV_E4M3);
                                    const float2 z = e4m3x2_to_float2((uint16_t)hh[x]);
                                    ll[x] = __nv_cvt_float2_to_fp8x2(make_float2(y.x - z.x, y.y - z.y), __NV_SATFINITE, __NV_E5M2);
                                }
                                hi[k] = hh[0] | (hh[1] << 16);
                                lo[k] = ll[0] | (ll[1] << 16);
                            }
                            const int cc = c >> 1;  // 16-byte chunk of e4m3
                            const int to = (D == 128 ? q * 128 + ((cc ^ (q & 7)) << 4) : q * 64 + ((cc ^ ((q >> 1) & 3)) << 4)) + (c & 1) * 8;
                            *reinterpret_cast<uint2 *>(dst + to) = make_uint2(hi[0], hi[1]);
                            *reinterpret_cast<uint2 *>(dst + C::QB / 2 + to) = make_uint2(lo[0], lo[1]);
                        }
                    }
                }
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) bar_arrive(&m.qfull);
            float mul = a2;
            if constexpr (FP8) {
                ok = bar_wait(&m.qfull, i & 1, gave_up, tries);
                mul = live ? m.qmul[row] : a2;
            }
            const float vinv = it.vinv;

            float ref = kMinusInf, sum = 0.f;
            for (int j = 0; j < steps; ++j, ++done) {
                ok = bar_wait(&m.sfull[grp], done & 1, gave_up, tries);
                if (!__all_sync(0xffffffffu, ok)) break;
                tmem_fence_after();
                const int tile = wide ? j : 2 * j + grp;
                const int seen = it.len - (it.t0 + tile) * kPrefixTile;
                const Info &inf = m.info[grp][done % kInfo];
                if constexpr (FP8) {
                    ok = bar_wait(&m.tfull[grp][done % kInfo], (done / kInfo) & 1, gave_up, tries);
                    if (!__all_sync(0xffffffffu, ok)) break;
                }
                if (!FP8 && seen < kPrefixTile && (!wide || grp == 0)) {
                    // tokens past the last may hold anything, NaN among it, and meet weights of zero: V's
                    // are zeroed where they lie, by the group whose products use the tile first
                    const uint32_t pos = base_pos + tile;
                    ok = bar_wait(&m.vfull[pos % C::NV], (pos / C::NV) & 1, gave_up, tries);
                    uint4 *v = reinterpret_cast<uint4 *>(psm + C::OFF_V + (pos % C::NV) * C::VB);
#pragma unroll 1
                    for (int e = seen * 8 + r; e < kPrefixTile * 8; e += 128) {
                        v[e] = make_uint4(0u, 0u, 0u, 0u);
                        if (D == 128) v[e + C::HALF / 16] = make_uint4(0u, 0u, 0u, 0u);
                    }
                    fence_proxy_async_smem();
                }
                if (warp_live) {
                    float x[4][32];
#pragma unroll
                    for (int g = 0; g < 4; ++g) tmem_ld32(cs + g * 32, x[g]);
                    tmem_wait_ld();
                    float f[kPages];  // factors of 16 columns each
                    if constexpr (FP8) {
                        const float4 k0 = *reinterpret_cast<const float4 *>(inf.ks), k1 = *reinterpret_cast<const float4 *>(inf.ks + 4);
                        const float k[kPages] = {k0.x, k0.y, k0.z, k0.w, k1.x, k1.y, k1.z, k1.w};
                        const float least = fminf(fminf(fminf(k0.x, k0.y), fminf(k0.z, k0.w)), fminf(fminf(k1.x, k1.y), fminf(k1.z, k1.w)));
                        if (least < 0.f) {  // scales below zero: the scores' sign
#pragma unroll
                            for (int p = 0; p < kPages; ++p) {
                                const float sign = k[p] < 0.f ? -1.f : 1.f;
#pragma unroll
                                for (int e = 0; e < 16; ++e) x[p >> 1][(p & 1) * 16 + e] *= sign;
                            }
                        }
#pragma unroll
                        for (int p = 0; p < kPages; ++p) {
                            f[p] = fabsf(k[p]) * mul;
                            if (f[p] < 1.1754944e-38f) f[p] = 1.1754944e-38f;  // hidden scores stay -inf; NaN stays
                        }
                    }
                    if (seen < kPrefixTile) {
#pragma unroll
                        for (int g = 0; g < 4; ++g)
#pragma unroll
                            for (int e = 0; e < 32; ++e)
                                if (g * 32 + e >= seen) x[g][e] = kMinusInf;
                        if constexpr (FP8) {  // what follows the last page has no scale
#pragma unroll
                            for (int p = 0; p < kPages; ++p)
                                if (p * kPage >= seen) f[p] = mul;
                        }
                    }
                    float tops[8];
#pragma unroll
                    for (int p = 0; p < 8; ++p) tops[p] = fmaxf(x[p >> 1][(p & 1) * 16], x[p >> 1][(p & 1) * 16 + 1]);
#pragma unroll
                    for (int e = 2; e < 16; e += 2)
#pragma unroll
                        for (int p = 0; p < 8; ++p)
                            tops[p] = fmaxf(tops[p], fmaxf(x[p >> 1][(p & 1) * 16 + e], x[p >> 1][(p & 1) * 16 + e + 1]));
                    if constexpr (FP8) {
#pragma unroll
                        for (int p = 0; p < 8; ++p) tops[p] *= f[p];
                    }
                    float top = fmaxf(fmaxf(fmaxf(tops[0], tops[1]), fmaxf(tops[2], tops[3])),
                                      fmaxf(fmaxf(tops[4], tops[5]), fmaxf(tops[6], tops[7])));
                    if constexpr (!FP8) top *= a2;
                    float shrink = 1.f;
                    if (top > ref + kGrowth || (ref == kMinusInf && top > kMinusInf)) {
                        top += kAbove<FP8>;
                        shrink = fast_exp2(ref - top);  // 0 when nothing was seen yet
                        sum *= shrink;
                        ref = top;
                    }
                    // the scores are here, so the products before them (O among them) are done
                    if (j > 0 && __any_sync(0xffffffffu, shrink != 1.f)) {
#pragma unroll 1
                        for (int g = 0; g < D / 16; ++g) {
                            float o[16];
                            tmem_ld16(co + g * 16, o);
                            tmem_wait_ld();
#pragma unroll
                            for (int e = 0; e < 16; ++e) o[e] *= shrink;
                            tmem_st16(co + g * 16, o);
                        }
                    }
                    const float base = ref == kMinusInf ? 0.f : -ref;
                    const float2 base2 = make_float2(base, base);
                    float2 sums[4] = {};
                    // the weights of 64 tokens at a time: the products with the first half's V start
                    // while the second half is computed
#pragma unroll
                    for (int half = 0; half < 2; ++half) {
                        // V scales, once in registers: a load in every pair took 2,000 cycles a tile (those of pages
                        // past the last are zero)
                        float vf[4] = {};
                        if constexpr (FP8) {
                            const float4 v = *reinterpret_cast<const float4 *>(inf.vs + 4 * half);
                            vf[0] = v.x * vinv;
                            vf[1] = v.y * vinv;
                            vf[2] = v.z * vinv;
                            vf[3] = v.w * vinv;
                        }
#pragma unroll
                        for (int p = 4 * half; p < 4 * half + 4; ++p) {
                            float w[16];  // packed pairs of 16 weights: upper parts, then what is left of them
#pragma unroll
                            for (int e = 0; e < 16; e += 2) {
                                const float *const s2 = &x[p >> 1][(p & 1) * 16 + e];
                                const float fp = FP8 ? f[p] : a2;
                                float2 y = fma2(make_float2(s2[0], s2[1]), make_float2(fp, fp), base2);
                                y = make_float2(fast_exp2(y.x), fast_exp2(y.y));
                                sums[(e >> 1) & 3] = add2(sums[(e >> 1) & 3], y);
                                if constexpr (FP8) y = mul2(y, make_float2(vf[p - 4 * half], vf[p - 4 * half]));
                                // the bits that f16 or bf16 holds, cut off, so that nothing has to be converted back
                                constexpr uint32_t kUpper = FP8 ? 0xffffe000u : 0xffff0000u;
                                const uint32_t ux = __float_as_uint(y.x) & kUpper, uy = __float_as_uint(y.y) & kUpper;
                                const float hx = __uint_as_float(ux), hy = __uint_as_float(uy);
                                w[e >> 1] = __uint_as_float(FP8 ? pack16(hx, hy, false) : __byte_perm(ux, uy, 0x7632));
                                const float2 rest = add2(y, make_float2(-hx, -hy));
                                w[8 + (e >> 1)] = __uint_as_float(pack16(rest.x, rest.y, !FP8));
                            }
                            tmem_st16(cs + p * 16, w);
                        }
                        tmem_wait_st();
                        tmem_fence_before();
                        __syncwarp();
                        if (lane == 0) bar_arrive(&m.pready[grp][half]);
                    }
                    const float2 s2 = add2(add2(sums[0], sums[1]), add2(sums[2], sums[3]));
                    sum += s2.x + s2.y;
                } else {
                    __syncwarp();
                    if (lane == 0) {
                        bar_arrive(&m.pready[grp][0]);
                        bar_arrive(&m.pready[grp][1]);
                    }
                }
                if constexpr (FP8) {
                    __syncwarp();
                    if (lane == 0) bar_arrive(&m.tempty[grp][done % kInfo]);
                }
            }
            if (steps > 0) {
                ok = bar_wait(&m.odone[grp], outs++ & 1, gave_up, tries) && ok;
                tmem_fence_after();
            }
            ok = __all_sync(0xffffffffu, ok);
            const bool both = !wide && nt > 1;  // two parts to merge
            float4 *part = reinterpret_cast<float4 *>(psm);  // the queries' place: [D / 4][128] of group 1's O
            if (both && grp == 1 && warp_live && ok) {
#pragma unroll 1
                for (int g = 0; g < D / 32; ++g) {
                    float o[32];
                    tmem_ld32(co + g * 32, o);
                    tmem_wait_ld();
#pragma unroll
                    for (int k = 0; k < 8; ++k)
                        part[(g * 8 + k) * 128 + r] = make_float4(o[4 * k], o[4 * k + 1], o[4 * k + 2], o[4 * k + 3]);
                }
                m.ref1[r] = ref;
                m.sum1[r] = sum;
            }
            if (both) {
                if (grp == 1) {
                    __syncwarp();
                    if (lane == 0) bar_arrive(&m.merge);
                } else {
                    ok = bar_wait(&m.merge, merges & 1, gave_up, tries) && ok;
                    ok = __all_sync(0xffffffffu, ok);
                }
                ++merges;
            }
            if ((wide || grp == 0) && warp_live && ok) {
                float f0 = 1.f, f1 = 0.f;
                if (both) {
                    const float ref1 = m.ref1[r], sum1 = m.sum1[r];
                    const float top = fmaxf(ref, ref1);
                    f0 = ref == top ? 1.f : fast_exp2(ref - top);
                    f1 = ref1 == top ? 1.f : fast_exp2(ref1 - top);
                    sum = sum * f0 + sum1 * f1;
                    ref = top;
                }
                const float inv = sum == 0.f ? 0.f : (FP8 ? it.vback : 1.f) / sum;
                const int n8 = rows8(it.rows);
                float4 *dst = reinterpret_cast<float4 *>(a.po + (long long)it.base * D) + row;
                if (live) a.plse[it.base + row] = sum == 0.f ? kMinusInf : ref + log2f(sum);
                f0 *= inv;
                f1 *= inv;
#pragma unroll 1
                for (int g = 0; g < D / 32; ++g) {
                    float o[32];
                    __syncwarp();
                    tmem_ld32(co + g * 32, o);
                    tmem_wait_ld();
                    if (!live) continue;
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        float4 y = make_float4(o[4 * k] * f0, o[4 * k + 1] * f0, o[4 * k + 2] * f0, o[4 * k + 3] * f0);
                        if (both) {
                            const float4 z = part[(g * 8 + k) * 128 + r];
                            y = make_float4(fmaf(z.x, f1, y.x), fmaf(z.y, f1, y.y), fmaf(z.z, f1, y.z), fmaf(z.w, f1, y.w));
                        }
                        dst[(long long)(g * 8 + k) * n8] = y;
                    }
                }
            }
            base_pos += nt;
            tmem_fence_before();
            __syncwarp();
            // Both groups are done with the queries' place and with O.
            if (lane == 0) bar_arrive(&m.rest);
            ok = bar_wait(&m.rest, i & 1, gave_up, tries) && ok;
            if (lane == 0) bar_arrive(&m.iempty[i % kItems]);
            if (!__all_sync(0xffffffffu, ok)) break;
        }
    } else if (warp == 8) {
        // ------------------------------ products ------------------------------
        reg_share_less<88>();
        if (elect_one()) {
            constexpr uint32_t idO = umma_idesc(128, D, !FP8, false, true);
            const uint32_t qa = smem_addr(psm), ka = qa + C::OFF_K, va = qa + C::OFF_V;
            // Straight code, a copy a group: one thread issues all products of the CTA, and what it does
            // between them is time that the tensor cores wait.  So each barrier is asked for while the
            // products before are issued, and waited for only if it has not passed by then.
            uint32_t weighed0 = 0, weighed1 = 0, pos = 0;  // steps whose weights were used, tiles so far
            bool wide = false, ready = false;              // ready: the next group's first weights, asked ahead
            int n0 = 0, n1 = 0;
            // Step j of a group: O of its step j - 1, then S of step j.
            auto step = [&](auto which, int j) {
                constexpr int T = decltype(which)::value;
                const uint32_t cs = tmem + T * 128, co = tmem + kColO + T * 128;
                const int mine = T ? n1 : n0, other = T ? n0 : n1;
                uint32_t &weighed = T ? weighed1 : weighed0;
                const uint32_t at = pos + (wide ? j : 2 * j + T), kslot = at % C::NK, kparity = (at / C::NK) & 1;
                const bool again = wide && T == 1;  // the tile is there already, and this group is done with it last
                bool keys = again;
                if (j > 0 && j <= mine) {
                    const uint32_t vat = pos + (wide ? j - 1 : 2 * j - 2 + T), slot = vat % C::NV, parity = weighed++ & 1;
                    const uint32_t db = umma_desc(va + slot * C::VB, C::HALF);
                    if (!ready && !bar_wait(&m.pready[T][0], parity, gave_up, tries)) return false;
                    if (!again && !bar_wait(&m.vfull[slot], (vat / C::NV) & 1, gave_up, tries)) return false;
                    const bool rest = bar_passed(&m.pready[T][1], parity);
                    tmem_fence_after();
#pragma unroll
                    for (int s = 0; s < 4; ++s) {
                        umma_ts(co, cs + s * 16, db + s * 128, idO, j > 1 || s > 0);
                        umma_ts(co, cs + s * 16 + 8, db + s * 128, idO, true);
                    }
                    if (!rest && !bar_wait(&m.pready[T][1], parity, gave_up, tries)) return false;
                    if (j < mine && !again) keys = bar_passed(&m.kfull[kslot], kparity);
                    tmem_fence_after();
#pragma unroll
                    for (int s = 4; s < 8; ++s) {
                        umma_ts(co, cs + s * 16, db + s * 128, idO, true);
                        umma_ts(co, cs + s * 16 + 8, db + s * 128, idO, true);
                    }
                    if (!wide || T == 1) umma_commit(&m.vempty[slot]);
                    if (j == mine) umma_commit(&m.odone[T]);
                }
                ready = false;
                const int jn = j + T;  // the next group's step
                const bool follows = jn > 0 && jn <= other;
                const uint32_t next_parity = (T ? weighed0 : weighed1) & 1;
                if (j >= mine) {
                    if (follows) ready = bar_passed(&m.pready[T ^ 1][0], next_parity);
                    return true;
                }
                const uint32_t qt = qa + (wide ? T : 0) * C::QB, kt = ka + kslot * C::KB;
                if (!keys && !bar_wait(&m.kfull[kslot], kparity, gave_up, tries)) return false;
                if (follows) ready = bar_passed(&m.pready[T ^ 1][0], next_parity);
                tmem_fence_after();
                if constexpr (!FP8) {
#pragma unroll
                    for (int c = 0; c < D / 64; ++c) {
                        const uint32_t da = umma_desc(qt + c * C::HALF, 16), db = umma_desc(kt + c * C::HALF, 16);
#pragma unroll
                        for (int s = 0; s < 4; ++s) umma_ss<1>(cs, da + 2 * s, db + 2 * s, idS, c > 0 || s > 0);
                    }
                } else {
                    constexpr uint32_t UP = D == 128 ? kDescUpper : kDescUpper64;
                    const uint32_t db = umma_desc(kt, 16);
#pragma unroll
                    for (int part = 0; part < 2; ++part) {
                        const uint32_t da = umma_desc(qt + part * (C::QB / 2), 16);
#pragma unroll
                        for (int s = 0; s < D / 32; ++s)
                            umma_ss_f8<UP>(cs, da + 2 * s, db + 2 * s, part ? idS | kQueryE5M2 : idS, part > 0 || s > 0);
                    }
                }
                if (!wide || T == 1) umma_commit(&m.kempty[kslot]);
                umma_commit(&m.sfull[T]);
                return true;
            };
            bool ok = true;
            for (int i = 0; ok && item_ready(i); ++i) {
                wide = m.item[i % kItems].rows > 128;
                const int nt = m.item[i % kItems].nt;
                n0 = steps_of(m.item[i % kItems], 0);
                n1 = steps_of(m.item[i % kItems], 1);
                bar_arrive(&m.iempty[i % kItems]);
                ok = bar_wait(&m.qfull, i & 1, gave_up, item_tries);
                const int most = max(n0, n1);
                ready = false;
#pragma unroll 1
                for (int j = 0; j <= most && ok; ++j) ok = step(Group<0>{}, j) && step(Group<1>{}, j);
                pos += nt;
            }
            // nothing in flight when the CTA leaves
            umma_commit(&m.drain);
            bar_drain(&m.drain, 0);
        }
        __syncwarp();
    } else if (warp == 9) {
        // --------------------------- segments, scales and K ---------------------------
        reg_share_less<88>();
        const uint64_t pol = l2_policy_evict_normal();
        const PrefixRange range = a.range[blockIdx.x];
        int x = range.x0, k = range.seg;
        const int x1 = range.x1;
        uint32_t pos = 0, info[2] = {0, 0};
        int i = 0;
        bool ok = true;
        auto put = [&](const Item &it) {
            ok = bar_wait(&m.iempty[i % kItems], ((i / kItems) & 1) ^ 1, gave_up, item_tries);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) return;
            if (lane == 0) {
                m.item[i % kItems] = it;
                bar_arrive(&m.ifull[i % kItems]);
            }
            ++i;
        };
        while (ok && x < x1) {
            const PrefixSeg sg = a.seg[k];
            const int end = min(x1, sg.tile0 + sg.ntiles);
            if (end <= x) {  // an empty segment
                ++k;
                continue;
            }
            Item it{};
            it.p = sg.p;
            it.h = sg.h;
            it.row0 = sg.row0;
            it.rows = sg.rows;
            it.t0 = x - sg.tile0;
            it.nt = end - x;
            it.len = sg.len;
            it.base = sg.base + ((int)blockIdx.x - sg.first) * rows8(sg.rows);
            x = end;
            ++k;
            const bool wide = it.rows > 128;
            // 32 pages (four tiles) a round, one a lane; the next round's ids are on their way
            const int32_t *table = a.pre.block_tables + (long long)it.p * a.pre.bt_sb + (long long)it.h * a.pre.bt_sh;
            const int npages = min((it.len + kPage - 1) / kPage, (it.t0 + it.nt) * kPages);
            auto fetch = [&](int t) {
                const int page = (it.t0 + t) * kPages + lane;
                return page < npages ? table[page] : -1;
            };
            int next_id = fetch(0);
            // a prefix that failed a check is not read: its requests are flagged
            const long long words = (long long)sg.p * a.Hkv * a.pre.htiles;
            uint32_t bits = 0u;
            float top = 0.f;
            for (int w = lane; w < a.Hkv * a.pre.htiles; w += 32) bits |= a.pre_bits[words + w];
            if constexpr (FP8)
                for (int w = lane; w < a.pre.htiles; w += 32) top = fmaxf(top, a.pre_vmax[words + (long long)sg.h * a.pre.htiles + w]);
            if (__any_sync(0xffffffffu, bits != 0u)) continue;
            if constexpr (FP8) {
                top = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(top)));  // not negative: ordered as numbers
                // scales over a power of two above the largest, and 2^7: half a step of f16's subnormals, for
                // either of a pair, is 2^-31 of the largest at most.  (The largest of all pages, by the plan: the
                // scales of a tile that is not here yet cannot be asked.)
                const int e = min(120, max(-112, (int)(__float_as_uint(top) >> 23) - 126));
                it.vinv = __uint_as_float((uint32_t)(127 + 7 - e) << 23);
                it.vback = __uint_as_float((uint32_t)(127 + e - 7) << 23);
            }
            put(it);
            for (int t = 0; ok && t < it.nt; t += 4) {
                const int id = next_id;
                const bool there = id >= 0 && id < a.num_pages;
                const int unit = there ? id * a.Hkv + it.h : -1;
                float ks = 1.f, vs = 0.f;
                if (FP8 && there) {
                    ks = a.k_scale[unit];
                    vs = a.v_scale[unit];
                }
                if (t + 4 < it.nt) next_id = fetch(t + 4);
                const int live = min(4, it.nt - t);
                // K of the tile that follows is on its way before the scales of this one are waited for
                for (int q = 0; ok && q < live; ++q, ++pos) {
                    const int copy = lane / kPages;  // of a page
                    const int u = __shfl_sync(0xffffffffu, unit, q * kPages + lane % kPages);
                    const bool mine = copy < C::CPP && u >= 0;
                    const uint32_t bytes = __popc(__ballot_sync(0xffffffffu, mine)) * C::COPYB;
                    const uint32_t slot = pos % C::NK;
                    ok = __all_sync(0xffffffffu, bar_wait(&m.kempty[slot], ((pos / C::NK) & 1) ^ 1, gave_up, tries));
                    if (!ok) break;
                    if (lane == 0) mbar_arrive_expect_tx(&m.kfull[slot], bytes);
                    __syncwarp();
                    if (mine)
                        tma_box3(psm + C::OFF_K + slot * C::KB + copy * C::HALF + lane % kPages * C::COPYB, &mapk, copy * 64, 0, u,
                                 &m.kfull[slot], pol);
                    if constexpr (FP8) {
#pragma unroll 1
                        for (int g = 0; g < 2; ++g) {
                            if (!wide && (q & 1) != g) continue;
                            const uint32_t at = info[g] % kInfo;
                            ok = ok && bar_wait(&m.tempty[g][at], ((info[g] / kInfo) & 1) ^ 1, gave_up, tries);
                            ok = __all_sync(0xffffffffu, ok);
                            if (!ok) break;
                            if (lane / kPages == q) {
                                m.info[g][at].ks[lane % kPages] = ks;
                                m.info[g][at].vs[lane % kPages] = vs;
                            }
                            __syncwarp();
                            if (lane == 0) bar_arrive(&m.tfull[g][at]);
                            ++info[g];
                        }
                    }
                }
            }
        }
        if (ok) {
            Item it{};
            it.p = -1;
            put(it);
        }
        if (*gave_up) {  // copies in flight are left time to land
            const unsigned long long t0 = globaltimer_ns();
            while (globaltimer_ns() - t0 < kWaitLimitNs) {}
        }
        __syncwarp();
    } else {
        // ------------------------------------ V ------------------------------------
        reg_share_less<88>();
        const uint64_t pol = l2_policy_evict_normal();
        const int half = warp - 10;  // pages 4 half .. 4 half + 3 of every tile
        uint32_t pos = 0;
        bool ok = true;
        for (int i = 0; ok && __all_sync(0xffffffffu, item_ready(i)); ++i) {
            const Item it = m.item[i % kItems];
            __syncwarp();
            if (lane == 0) bar_arrive(&m.iempty[i % kItems]);
            const int32_t *table = a.pre.block_tables + (long long)it.p * a.pre.bt_sb + (long long)it.h * a.pre.bt_sh;
            const int npages = min((it.len + kPage - 1) / kPage, (it.t0 + it.nt) * kPages);
            // the units of this half of eight tiles, four a tile; the next eight tiles' ids are on their way
            auto fetch = [&](int t) {
                const int page = (it.t0 + t + lane / 4) * kPages + half * 4 + lane % 4;
                return page < npages ? table[page] : -1;
            };
            int id = fetch(0), next_id = it.nt > 8 ? fetch(8) : -1, batch = 0;
            // copies of tile t (in order): of the item's tile number `at`, `full` counting their bytes
            auto load = [&](int t, uint8_t *dst, uint64_t *full) {
                if (t - batch == 8) {
                    batch += 8;
                    id = next_id;
                    next_id = t + 8 < it.nt ? fetch(t + 8) : -1;
                }
                const int copy = lane / 4;  // of a page
                const int u = __shfl_sync(0xffffffffu, id, (t - batch) * 4 + lane % 4);
                const bool mine = copy < C::CPP && u >= 0 && u < a.num_pages;
                const uint32_t bytes = __popc(__ballot_sync(0xffffffffu, mine)) * C::COPYB;
                if (lane == 0) mbar_arrive_expect_tx(full, bytes);
                __syncwarp();
                if (mine)
                    tma_box3(dst + copy * C::HALF + (half * 4 + lane % 4) * C::COPYB, &mapv, copy * 64, 0, u * a.Hkv + it.h, full, pol);
            };
            if constexpr (!FP8) {
                for (int t = 0; ok && t < it.nt; ++t, ++pos) {
                    const uint32_t slot = pos % C::NV;
                    ok = __all_sync(0xffffffffu, bar_wait(&m.vempty[slot], ((pos / C::NV) & 1) ^ 1, gave_up, tries));
                    if (ok) load(t, psm + C::OFF_V + slot * C::VB, &m.vfull[slot]);
                }
            } else {
                // this half's place of a tile as loaded is written and read by this warp alone
                int ahead = 0;  // tiles whose copies have been issued
                for (; ahead < min(C::NR, it.nt); ++ahead) {
                    const uint32_t slot = (pos + ahead) % C::NR;
                    load(ahead, psm + C::OFF_R + slot * C::KB, &m.rfull[half][slot]);
                }
                for (int t = 0; ok && t < it.nt; ++t, ++pos) {
                    const uint32_t rs = pos % C::NR, vslot = pos % C::NV;
                    ok = bar_wait(&m.rfull[half][rs], (pos / C::NR) & 1, gave_up, tries) &&
                         bar_wait(&m.vempty[vslot], ((pos / C::NV) & 1) ^ 1, gave_up, tries);
                    ok = __all_sync(0xffffffffu, ok);
                    if (!ok) break;
                    const int seen = it.len - (it.t0 + t) * kPrefixTile;
                    const uint8_t *raw = psm + C::OFF_R + rs * C::KB;
                    uint8_t *dst = psm + C::OFF_V + vslot * C::VB;
                    constexpr int CH = D / 16, RP = 32 / CH;  // chunks a row, rows at a time
                    const int ch = lane % CH, r0 = half * 64 + lane / CH, flip = ch >> 2;
                    constexpr int AHEAD = 8;  // loads on their way together
#pragma unroll 1
                    for (int p0 = 0; p0 < 64 / RP; p0 += AHEAD) {
                        uint4 w[AHEAD];
#pragma unroll
                        for (int p = 0; p < AHEAD; ++p) {
                            const int r = (p0 + p) * RP + r0;
                            const int at = D == 128 ? r * 128 + ((ch ^ (r & 7)) << 4) : r * 64 + ((ch ^ ((r >> 1) & 3)) << 4);
                            w[p] = *reinterpret_cast<const uint4 *>(raw + at);
                        }
#pragma unroll
                        for (int p = 0; p < AHEAD; ++p) {
                            const int r = (p0 + p) * RP + r0;
                            if (r >= seen) w[p] = make_uint4(0u, 0u, 0u, 0u);  // whatever follows the last token
                            const uint2 h0 = e4m3x4_to_half4(w[p].x), h1 = e4m3x4_to_half4(w[p].y);
                            const uint2 h2 = e4m3x4_to_half4(w[p].z), h3 = e4m3x4_to_half4(w[p].w);
                            uint8_t *to = dst + (ch >> 2) * C::HALF + r * 128;
                            const int d0 = 2 * (ch & 3);
                            const uint4 lo = make_uint4(h0.x, h0.y, h1.x, h1.y), hi = make_uint4(h2.x, h2.y, h3.x, h3.y);
                            // the two halves' lanes store their chunks in opposite order, on banks of their own
                            *reinterpret_cast<uint4 *>(to + (((d0 + flip) ^ (r & 7)) << 4)) = flip ? hi : lo;
                            *reinterpret_cast<uint4 *>(to + (((d0 + 1 - flip) ^ (r & 7)) << 4)) = flip ? lo : hi;
                        }
                    }
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) bar_arrive(&m.vfull[vslot]);
                    if (ahead < it.nt) {
                        load(ahead, psm + C::OFF_R + rs * C::KB, &m.rfull[half][rs]);
                        ++ahead;
                    }
                }
            }
        }
        if (*gave_up) {  // copies in flight are left time to land
            const unsigned long long t0 = globaltimer_ns();
            while (globaltimer_ns() - t0 < kWaitLimitNs) {}
        }
        __syncwarp();
    }
    __syncthreads();
    if (tid == 0 && *gave_up) atomicOr(&a.head->timeout, PFKV_FLAG_DEVICE_TIMEOUT);
    tmem_fence_after();
    if (warp == 8) tmem_free512<1>(tmem);
    if (a.after_own) asm volatile("griddepcontrol.wait;" ::: "memory");
}

// A pool as [units][16][D], read in boxes of one unit's 16 rows of 128 bytes at most.
cudaError_t pool_map(CUtensorMap *map, const void *pages, long long units, int D, bool fp8) {
    const PFN_cuTensorMapEncodeTiled_v12000 enc = umma_map_encoder();
    if (!enc) return cudaErrorNotSupported;
    const int el = fp8 ? 1 : 2;
    const cuuint64_t dims[3] = {(cuuint64_t)D, kPage, (cuuint64_t)units};
    const cuuint64_t strides[2] = {(cuuint64_t)(D * el), (cuuint64_t)(kPage * D * el)};
    const cuuint32_t box[3] = {(cuuint32_t)(fp8 ? D : 64), kPage, 1};
    const cuuint32_t one[3] = {1, 1, 1};
    const CUresult r = enc(map, fp8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3,
                           const_cast<void *>(pages), dims, strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
                           fp8 && D == 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B,
                           CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

template <int D, bool FP8>
cudaError_t launch_d(const PrefixArgs &a, cudaStream_t s) {
    CUtensorMap mk{}, mv{};
    const long long units = (long long)a.num_pages * a.Hkv;
    cudaError_t e = pool_map(&mk, a.k_pages, units, D, FP8);
    if (e == cudaSuccess) e = pool_map(&mv, a.v_pages, units, D, FP8);
    if (e != cudaSuccess) return e;
    // the first product's instruction: both operands e4m3, or bf16 with A negated for a scale below
    // zero (the softmax works with its magnitude; FP8 queries change sign as they are converted)
    const uint32_t idS = FP8 ? (1u << 4) | ((128u >> 3) << 17) | ((128u >> 4) << 24)
                             : umma_idesc(128, 128, true, false, false) | (a.sm_scale < 0.f ? 1u << 13 : 0u);
    auto *const kernel = a.tries == kTries ? prefix_attn_kernel<D, FP8, false> : prefix_attn_kernel<D, FP8, true>;
    return launch_pdl(kernel, dim3((unsigned)a.ctas), dim3(kThreads), smem_bytes<D, FP8>(), s, mk, mv, a, idS);
}

template <int D, bool FP8>
cudaError_t preload_d() {
    cudaError_t e = cudaSuccess;
    for (auto *const kernel : {prefix_attn_kernel<D, FP8, false>, prefix_attn_kernel<D, FP8, true>}) {
        if (e == cudaSuccess)
            e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem_bytes<D, FP8>());
        if (e == cudaSuccess) e = preload_kernel(kernel);
    }
    return e;
}

}  // namespace

cudaError_t launch_prefix_attn(const PrefixArgs &a, int D, bool fp8, cudaStream_t s) {
    if (D == 128) return fp8 ? launch_d<128, true>(a, s) : launch_d<128, false>(a, s);
    return fp8 ? launch_d<64, true>(a, s) : launch_d<64, false>(a, s);
}

cudaError_t preload_prefix_attn() {
    cudaError_t e = preload_d<128, true>();
    if (e == cudaSuccess) e = preload_d<128, false>();
    if (e == cudaSuccess) e = preload_d<64, true>();
    if (e == cudaSuccess) e = preload_d<64, false>();
    return e;
}

}  // namespace pfkv

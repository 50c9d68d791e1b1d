// latent_prefill.cu -- pfkv_latent_prefill_attn: ragged causal attention of
// prompts in the expanded form (declared in pfkv_latent.h).
//
// Mathematics.  For each request and head S = scale (Qn Kn^T + Qr Kr^T), O =
// softmax(S) V with 128 + 64 and 128 columns: 640 operations a (query, key) pair,
// against 512 bytes of K and V a key and head that a tile of 256 queries shares.
// It is bound by the tensor cores.
//
// A CTA takes 256 queries of one head, as two tiles of 128 that alternate: while
// one tile's softmax runs, the other tile's products do.  A step of 128 keys costs
// the tensor cores 12 products of 128 x 128 x 16 for S (64 cycles each) and 16 of
// 128 x 64 x 16 for O (32 cycles) a tile: 2,560 cycles for both.  Tensor memory
// holds S of both tiles (a tile's weights overwrite its scores, bf16, and are read
// from there as the A operand) and O of both: all 512 columns.  Shared memory holds
// Q of both (96 KB), four slots of 16 KB for K (128 keys x 64 columns; three a step) and
// two of 32 KB for V, each refilled when the second tile's products have used it.
//
// Softmax: one thread a row, one pass, with a running reference that moves only
// when the maximum has grown by 2^8 (O is then rescaled in tensor memory).
//
// What bounds it: one thread issues all products of the CTA, and they need it to be
// quick.  A wait between two groups of them, satisfied or not, costs the tensor cores
// about 140 cycles, and loops and descriptors in 64 bits as much again: 4,096 tokens of
// 128 heads took 704 us with those, 480 us with barriers asked a group ahead and straight
// code.  Then shared memory: S reads 128 bytes a cycle, all there is, and the copies of
// K and V write beside it (1.39 us a pair of steps without them, 1.64 with them; the
// whole kernel 1.75).  That is 1,430 TFLOP/s.
//
// A row that does not see every key and comes out not finite has its item done once more, with
// care for the values that it must not see (below).
//
// The kernel is persistent.  Work items are ordered so that the CTAs at work share
// the K and V of few heads (about two rounds of items a group of heads, or all heads
// where L2 holds most of their K and V), longest first within a group, and dealt out in turns
// that change direction, so that each CTA gets long and short ones.
//
// Roles of a CTA's twelve warps: 0-3 and 4-7 softmax and output of the two tiles; 8
// issues the products; 9 loads K and V, 10 loads Q (TMA); 11 looks up items.  The flags are written by a
// launch before it.
#include "latent_internal.cuh"
#include "umma.cuh"

namespace pfkv {
namespace {

constexpr int kQTile = 128, kItemRows = 2 * kQTile, kKeys = 128;
constexpr uint32_t kSlotB = 128 * 128;  // 128 rows of 128 bytes
constexpr int kKSlots = 4, kKChunks = 3;  // K: chunks 0 and 1, rotated
constexpr int kVSlots = 2;                // V: both chunks
constexpr int kPreThreads = 384;
constexpr int kItems = 3;               // items looked up ahead
constexpr uint32_t kOffK = 2 * kKChunks * kSlotB, kOffV = kOffK + kKSlots * kSlotB;
constexpr uint32_t kOffPre = kOffV + kVSlots * 2 * kSlotB;
constexpr uint32_t kColO = 256;
constexpr float kGrowth = 8.f;
constexpr float kMinusInf = -INFINITY;

template <int T>
struct Tile {
    static constexpr int value = T;
};

struct Item {
    int b, h;        // b < 0: no more
    int q0, nq;      // the request's first query row, and its queries from this item's first on
    int k0, nk;      // the request's first key row and key rows
    int sees0;       // keys that the item's first query sees (each further one sees one more if causal)
    int n0, n1;      // steps of the two tiles
    bool careful;    // done again: values that a row must not see may not be finite
};

struct PreMisc {
    uint64_t kfull[kKSlots], kempty[kKSlots], vfull[kVSlots], vempty[kVSlots];
    uint64_t qfull[2], qempty[2], sfull[2], pready[2][2], odone[2];
    uint64_t ifull[kItems], iempty[kItems], drain;
    Item item[kItems];
    uint32_t redo[kItems];     // a row that does not see every key came out not finite
    uint32_t unsound[kItems];  // careful: values were not finite, and zeroed
    uint32_t tmem, gave_up;
};
constexpr size_t kPreSmem = kOffPre + sizeof(PreMisc);
static_assert(kPreSmem <= 232448, "shared memory of one CTA");

// How the items are numbered: groups of `pairs` (request, head) pairs; within a
// group the last tiles of all pairs first.
struct Deal {
    int tiles;     // items of the longest request allowed
    int pairs;     // pairs a group
    bool dense;    // numbers that stand for an item are dealt out, rather than all numbers
    long long items;
};

// Values that a row must not see meet its weight of zero in the product, which is harmless where
// they are finite.  Looking for others costs 1 to 2 us an item, so it is left to items that are
// done again because they came out not finite: what is not finite from the first hidden key on is
// zeroed by the tile that uses a step first, and given at the end to the rows that see it.  (Calls,
// not inlined: 0.9 us for short prompts.)

// Row r of the V of step number `pos`.
__device__ __noinline__ void zero_odd_values(PreMisc &m, uint8_t *values, uint32_t pos, int r, uint32_t *odd, int tries) {
    if (!bar_wait(&m.vfull[pos % kVSlots], (pos / kVSlots) & 1, &m.gave_up, tries)) return;
    uint32_t *v = reinterpret_cast<uint32_t *>(values + (pos % kVSlots) * 2 * kSlotB) + r * 32;
    bool any = false;
#pragma unroll 1
    for (int c = 0; c < 64; ++c) {  // words; each lane starts at another, or all would read the same bank
        uint32_t *w = v + (c >> 5) * (kSlotB / 4) + ((c + r) & 31);
        const uint32_t bad = not_finite(*w);
        if (bad == 0) continue;
        if (!any) *static_cast<volatile uint32_t *>(odd) = 1u;
        any = true;
        *w &= ~((bad >> 15) * 0xFFFFu);
    }
    if (any) fence_proxy_async_smem();
}

// Adds to a row's results, `o` in tensor memory, what is not finite in the values of keys k0 .. k1 - 1.
__device__ __noinline__ void add_odd_values(const __nv_bfloat16 *v, long long stride, int k0, int k1, uint32_t o) {
#pragma unroll 1
    for (int g = 0; g < 8; ++g) {
        float x[16];
        tmem_ld16(o + g * 16, x);
        tmem_wait_ld();
#pragma unroll 1
        for (int j = k0; j < k1; ++j) {
            const uint4 *src = reinterpret_cast<const uint4 *>(v + j * stride + g * 16);
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                const uint4 w = src[c];
                const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const uint32_t bad = not_finite(u[k]);
                    const float2 y = bf16x2_to_float2(u[k]);
                    if (bad & 0x8000u) x[c * 8 + 2 * k] += y.x;
                    if (bad & 0x80000000u) x[c * 8 + 2 * k + 1] += y.y;
                }
            }
        }
        __syncwarp();
        tmem_st16(o + g * 16, x);
    }
    tmem_wait_st();
}

// The rows of request b; false where they are not within the arrays or the bound.
__device__ __forceinline__ bool request_rows(const LatentPrefillArgs &a, int b, int &q0, int &nq, int &k0, int &nk) {
    q0 = a.q_starts[b];
    const int q1 = a.q_starts[b + 1], k1 = a.k_starts[b + 1];
    k0 = a.k_starts[b];
    nq = q1 - q0;
    nk = k1 - k0;
    return q0 >= 0 && q1 >= q0 && q1 <= a.total_q && k0 >= 0 && k1 >= k0 && k1 <= a.total_k && nq <= a.max_q_len;
}

// The flags that depend on the starts alone: in a launch of its own, so that no CTA that starts
// late writes over the flag of one whose waits gave up.
constexpr int kFlagThreads = 256;
__global__ void __launch_bounds__(kFlagThreads) latent_prefill_flags_kernel(LatentPrefillArgs a) {
    pdl_enter();
    int q0, nq, k0, nk;
    for (long long b = (long long)blockIdx.x * kFlagThreads + threadIdx.x; b < a.B; b += gridDim.x * kFlagThreads)
        a.flags[b] = request_rows(a, (int)b, q0, nq, k0, nk) ? 0 : PFKV_FLAG_BAD_LENGTH;
}

// Selftest: waits of as many tries as the call says (as arguments the limits cost 0.7 us a call).
template <bool Selftest>
__global__ void __launch_bounds__(kPreThreads, 1)
    latent_prefill_kernel(const __grid_constant__ CUtensorMap mapqn, const __grid_constant__ CUtensorMap mapqr,
                          const __grid_constant__ CUtensorMap mapkn, const __grid_constant__ CUtensorMap mapkr,
                          const __grid_constant__ CUtensorMap mapv, LatentPrefillArgs a, Deal deal, uint32_t idS,
                          int qn_h, int qr_h, int kn_h, int v_h) {
    extern __shared__ __align__(1024) uint8_t psm[];  // no static shared memory: the window's aligned base
    PreMisc &m = *reinterpret_cast<PreMisc *>(psm + kOffPre);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (tid == 0) {
        for (int i = 0; i < kKSlots; ++i) {
            mbar_init(&m.kfull[i], 1);
            mbar_init(&m.kempty[i], 1);
        }
        for (int i = 0; i < kVSlots; ++i) {
            mbar_init(&m.vfull[i], 1);
            mbar_init(&m.vempty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&m.qfull[i], 1);
            mbar_init(&m.qempty[i], 1);
            mbar_init(&m.sfull[i], 1);
            mbar_init(&m.pready[i][0], 4);
            mbar_init(&m.pready[i][1], 4);
            mbar_init(&m.odone[i], 1);
        }
        for (int i = 0; i < kItems; ++i) {
            mbar_init(&m.ifull[i], 1);
            mbar_init(&m.iempty[i], 11);  // eight softmax warps and three threads
        }
        mbar_init(&m.drain, 1);
        m.gave_up = (smem_addr(psm) & 1023u) != 0u;  // nothing runs on a base that the swizzle cannot take
        fence_mbar_init();
    }
    if (warp == 8) tmem_alloc512<1>(&m.tmem);
    tmem_fence_before();
    __syncthreads();
    tmem_fence_after();
    pdl_enter();
    const uint32_t tmem = m.tmem;
    volatile uint32_t *const gave_up = &m.gave_up;
    const int tries = Selftest ? a.tries : kTries, item_tries = Selftest ? a.tries * (kItemTries / kTries) : kItemTries;
    // Waits for item number i of this CTA; false when there is none, or a wait has given up.
    auto item_ready = [&](int i) {
        return bar_wait(&m.ifull[i % kItems], (i / kItems) & 1, gave_up, item_tries) && m.item[i % kItems].b >= 0;
    };

    if (warp < 8) {
        // ------------------------- softmax and output -------------------------
        reg_share_more<208>();
        const int tile = warp >> 2, r = (warp & 3) * 32 + lane;
        const uint32_t lanes = tmem + ((uint32_t)((warp & 3) * 32) << 16);
        const uint32_t cs = lanes + tile * 128, co = lanes + kColO + tile * 128;
        const float a2 = fmaxf(fabsf(a.sm_scale) * 1.4426950408889634f, 1.1754944e-38f);
        uint32_t done = 0;   // steps of this tile so far, of all items
        uint32_t outs = 0;   // items that it had steps in
        uint32_t base_pos = 0;
        for (int i = 0; __all_sync(0xffffffffu, item_ready(i)); ++i) {
            const Item &it = m.item[i % kItems];
            const int steps = tile ? it.n1 : it.n0;
            const int nk = it.nk;
            const int sees = a.causal ? min(nk, it.sees0 + tile * kQTile + r) : nk;
            float ref = kMinusInf, sum = 0.f;
            bool ok = true;
            for (int j = 0; j < steps; ++j, ++done) {
                if (it.careful && (j + 1) * kKeys > it.sees0 && (tile == 0 || j >= it.n0) && j * kKeys + r >= it.sees0 &&
                    j * kKeys + r < nk)
                    zero_odd_values(m, psm + kOffV, base_pos + j, r, &m.unsound[i % kItems], tries);
                // an item's first scores come when the other tile is done with the item before it
                ok = bar_wait(&m.sfull[tile], done & 1, gave_up, item_tries);
                if (!__all_sync(0xffffffffu, ok)) break;
                tmem_fence_after();
                float x[4][32];
#pragma unroll
                for (int g = 0; g < 4; ++g) tmem_ld32(cs + g * 32, x[g]);
                tmem_wait_ld();
                const int seen = sees - j * kKeys;
                if (__any_sync(0xffffffffu, seen < kKeys)) {
#pragma unroll
                    for (int g = 0; g < 4; ++g)
#pragma unroll
                        for (int e = 0; e < 32; ++e)
                            if (g * 32 + e >= seen) x[g][e] = kMinusInf;
                }
                float tops[4] = {kMinusInf, kMinusInf, kMinusInf, kMinusInf};  // four chains, not one
#pragma unroll
                for (int e = 0; e < 32; e += 2)
#pragma unroll
                    for (int g = 0; g < 4; ++g) tops[g] = fmaxf(tops[g], fmaxf(x[g][e], x[g][e + 1]));
                const float top = fmaxf(fmaxf(tops[0], tops[1]), fmaxf(tops[2], tops[3])) * a2;
                float shrink = 1.f;
                if (top > ref + kGrowth || (ref == kMinusInf && top > kMinusInf)) {
                    shrink = fast_exp2(ref - top);  // 0 when nothing was seen yet
                    sum *= shrink;
                    ref = top;
                }
                // the scores are here, so the products before them (O among them) are done
                if (j > 0 && __any_sync(0xffffffffu, shrink != 1.f)) {
#pragma unroll 1
                    for (int g = 0; g < 8; ++g) {
                        float o[16];
                        tmem_ld16(co + g * 16, o);
                        tmem_wait_ld();
#pragma unroll
                        for (int e = 0; e < 16; ++e) o[e] *= shrink;
                        tmem_st16(co + g * 16, o);
                    }
                }
                if (nk - j * kKeys < kKeys) {
                    // key rows past the request's last may hold anything, NaN among it, and
                    // meet weights of zero: V's are zeroed where they lie
                    const uint32_t pos = base_pos + j;
                    ok = bar_wait(&m.vfull[pos % kVSlots], (pos / kVSlots) & 1, gave_up, tries);
                    uint4 *v = reinterpret_cast<uint4 *>(psm + kOffV + (pos % kVSlots) * 2 * kSlotB);
#pragma unroll 1
                    for (int e = (nk - j * kKeys) * 8 + r; e < kKeys * 8; e += kQTile) {
                        v[e] = make_uint4(0u, 0u, 0u, 0u);
                        v[e + kSlotB / 16] = make_uint4(0u, 0u, 0u, 0u);
                    }
                    fence_proxy_async_smem();
                }
                const float base = ref == kMinusInf ? 0.f : -ref;
                const float2 scale2 = make_float2(a2, a2), base2 = make_float2(base, base);
                float2 sums[4] = {};
                // the weights of 64 keys at a time: the products with the first half's V start
                // while the second half is computed
#pragma unroll
                for (int half = 0; half < 2; ++half) {
#pragma unroll
                    for (int g = 2 * half; g < 2 * half + 2; ++g) {
                        float w[16];  // packed pairs
#pragma unroll
                        for (int e = 0; e < 32; e += 2) {
                            float2 y = fma2(make_float2(x[g][e], x[g][e + 1]), scale2, base2);
                            y = make_float2(fast_exp2(y.x), fast_exp2(y.y));
                            sums[(e >> 1) & 3] = add2(sums[(e >> 1) & 3], y);
                            const __nv_bfloat162 h = __floats2bfloat162_rn(y.x, y.y);
                            w[e >> 1] = __uint_as_float(*reinterpret_cast<const uint32_t *>(&h));
                        }
                        tmem_st16(cs + g * 16, w);
                    }
                    tmem_wait_st();
                    tmem_fence_before();
                    __syncwarp();
                    if (lane == 0) bar_arrive(&m.pready[tile][half]);
                }
                const float2 s2 = add2(add2(sums[0], sums[1]), add2(sums[2], sums[3]));
                sum += s2.x + s2.y;
            }
            if (steps > 0) {
                ok = bar_wait(&m.odone[tile], outs++ & 1, gave_up, tries) && ok;
                tmem_fence_after();
            }
            ok = __all_sync(0xffffffffu, ok);
            const float inv = sum > 0.f ? __fdiv_rn(1.f, sum) : sum;  // zero and NaN stay
            const int row = tile * kQTile + r;
            const bool live = row < it.nq;
            if (it.careful && __any_sync(0xffffffffu, ok && *static_cast<volatile uint32_t *>(&m.unsound[i % kItems]) != 0u))
                add_odd_values(a.v.p + (long long)it.k0 * a.v.st + (long long)it.h * a.v.sh, a.v.st, max(it.sees0, 0),
                               row < it.nq ? sees : 0, co);
            float2 odd = make_float2(0.f, 0.f);  // NaN once a result was not finite
            __nv_bfloat16 *out = a.out.p + (long long)(it.q0 + row) * a.out.st + (long long)it.h * a.out.sh;
#pragma unroll 1
            for (int g = 0; g < 4; ++g) {
                float o[32];
                if (steps > 0) {
                    tmem_ld32(co + g * 32, o);
                    tmem_wait_ld();
                }
                if (!live || !ok) continue;
#pragma unroll
                for (int e = 0; e < 32; e += 2) odd = fma2(make_float2(o[e], o[e + 1]), make_float2(0.f, 0.f), odd);
#pragma unroll
                for (int e = 0; e < 32; e += 8) {
                    uint32_t u[4];
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        // a row that sees no key is zero
                        const float lo = sum == 0.f ? 0.f : o[e + 2 * k] * inv, hi = sum == 0.f ? 0.f : o[e + 2 * k + 1] * inv;
                        const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
                        u[k] = *reinterpret_cast<const uint32_t *>(&h);
                    }
                    *reinterpret_cast<uint4 *>(out + g * 32 + e) = make_uint4(u[0], u[1], u[2], u[3]);
                }
            }
            base_pos += max(it.n0, it.n1);
            if (sees < nk && sees > 0 && !it.careful && live && odd.x + odd.y != 0.f)
                *static_cast<volatile uint32_t *>(&m.redo[i % kItems]) = 1u;
            tmem_fence_before();
            __syncwarp();
            if (lane == 0) bar_arrive(&m.iempty[i % kItems]);
            if (!ok) break;
        }
    } else if (warp == 8) {
        // ------------------------------ products ------------------------------
        reg_share_less<88>();
        if (elect_one()) {
            constexpr uint32_t idO = umma_idesc(kQTile, 128, true, false, true);
            const uint32_t qa = smem_addr(psm), ka = qa + kOffK, va = qa + kOffV;
            // Straight code, a copy a tile: one thread issues all products of the CTA, and what
            // it does between them is time that the tensor cores wait.
            uint32_t weighed0 = 0, weighed1 = 0;  // steps of the tiles whose weights were used
            uint32_t items0 = 0, items1 = 0, vpos = 0, kpos = 0;
            bool ready = false;                   // the next tile's weights, and V: asked ahead
            int n0 = 0, n1 = 0;
            // Step j of a tile: O of step j - 1, then S of step j.  K and V are waited for
            // where the first tile of the two uses them, and released by the last.
            auto step = [&](auto which, int j) {
                constexpr int T = decltype(which)::value;
                constexpr uint32_t cs = T * 128, co = kColO + T * 128;
                const int mine = T ? n1 : n0, other = T ? n0 : n1;
                uint32_t &weighed = T ? weighed1 : weighed0, &items = T ? items1 : items0;
                const bool first = T == 0 || j >= n0, last = T == 1 || j >= n1;
                const uint32_t kstart = first ? kpos : kpos - kKChunks;
                bool keys = T == 0 && bar_passed(&m.kfull[kstart % kKSlots], (kstart / kKSlots) & 1);
                if (j > 0 && j <= mine) {
                    const uint32_t pos = vpos + j - 1, slot = pos % kVSlots, parity = weighed++ & 1;
                    if (!ready && !bar_wait(&m.pready[T][0], parity, gave_up, tries)) return false;
                    if ((T == 0 ? !ready : j > n0) && !bar_wait(&m.vfull[slot], (pos / kVSlots) & 1, gave_up, tries)) return false;
                    const bool rest = bar_passed(&m.pready[T][1], parity);
                    tmem_fence_after();
                    const uint32_t db = umma_desc(va + slot * 2 * kSlotB, kSlotB);
#pragma unroll
                    for (int s = 0; s < 4; ++s) umma_ts(tmem + co, tmem + cs + s * 8, db + s * 128, idO, j > 1 || s > 0);
                    if (!rest && !bar_wait(&m.pready[T][1], parity, gave_up, tries)) return false;
                    tmem_fence_after();
#pragma unroll
                    for (int s = 4; s < 8; ++s) umma_ts(tmem + co, tmem + cs + s * 8, db + s * 128, idO, true);
                    if (T == 1 || j > n1) umma_commit(&m.vempty[slot]);
                    if (j == mine) umma_commit(&m.odone[T]);
                }
                ready = false;
                if (j >= mine) return true;
                if (j == 0 && !bar_wait(&m.qfull[T], items++ & 1, gave_up, tries)) return false;
                const uint32_t da = umma_desc(qa + T * kKChunks * kSlotB, 16);
#pragma unroll
                for (int c = 0; c < kKChunks; ++c) {
                    const uint32_t at = kstart + c, slot = at % kKSlots;
                    if (first && !keys && !bar_wait(&m.kfull[slot], (at / kKSlots) & 1, gave_up, tries)) return false;
                    if (c + 1 < kKChunks) {
                        keys = T == 0 && bar_passed(&m.kfull[(at + 1) % kKSlots], ((at + 1) / kKSlots) & 1);
                    } else {
                        const int jn = j + T;  // step of the next tile
                        const uint32_t pos = vpos + jn - 1, weights = T ? weighed0 : weighed1;
                        ready = jn > 0 && jn <= other && bar_passed(&m.pready[T ^ 1][0], weights & 1) &&
                                (T == 0 || bar_passed(&m.vfull[pos % kVSlots], (pos / kVSlots) & 1));
                    }
                    const uint32_t db = umma_desc(ka + slot * kSlotB, 16);
#pragma unroll
                    for (int s = 0; s < 4; ++s)
                        umma_ss<1>(tmem + cs, da + c * (kSlotB >> 4) + 2 * s, db + 2 * s, idS, c > 0 || s > 0);
                    if (last) umma_commit(&m.kempty[slot]);
                }
                if (first) kpos += kKChunks;
                umma_commit(&m.sfull[T]);
                if (j + 1 == mine) umma_commit(&m.qempty[T]);
                return true;
            };
            bool ok = true;
            for (int i = 0; ok && item_ready(i); ++i) {
                n0 = m.item[i % kItems].n0;
                n1 = m.item[i % kItems].n1;
                bar_arrive(&m.iempty[i % kItems]);
                const int n = max(n0, n1);
#pragma unroll 1
                for (int j = 0; j <= n && ok; ++j) ok = step(Tile<0>{}, j) && step(Tile<1>{}, j);
                vpos += n;
                ready = false;
            }
            // nothing in flight when the CTA leaves
            umma_commit(&m.drain);
            bar_drain(&m.drain, 0);
        }
        __syncwarp();
    } else if (warp == 9) {
        // ------------------------------ K and V ------------------------------
        reg_share_less<88>();
        if (elect_one()) {
            const uint64_t pol = l2_policy_evict_normal();
            uint32_t kpos = 0, vpos = 0;
            bool ok = true;
            for (int i = 0; ok && item_ready(i); ++i) {
                const int n = max(m.item[i % kItems].n0, m.item[i % kItems].n1);
                const int h = m.item[i % kItems].h, k0 = m.item[i % kItems].k0;
                bar_arrive(&m.iempty[i % kItems]);
                for (int j = 0; ok && j < n; ++j, ++vpos) {
                    const int y = k0 + j * kKeys;
#pragma unroll 1
                    for (int c = 0; ok && c < kKChunks; ++c, ++kpos) {
                        const uint32_t slot = kpos % kKSlots;
                        ok = bar_wait(&m.kempty[slot], ((kpos / kKSlots) & 1) ^ 1, gave_up, tries);
                        if (!ok) break;
                        uint8_t *dst = psm + kOffK + slot * kSlotB;
                        mbar_arrive_expect_tx(&m.kfull[slot], kSlotB);
                        if (c < 2) tma_box3(dst, &mapkn, c * 64, kn_h ? h : 0, y, &m.kfull[slot], pol);
                        else tma_box3(dst, &mapkr, 0, 0, y, &m.kfull[slot], pol);
                    }
                    const uint32_t slot = vpos % kVSlots;
                    ok = ok && bar_wait(&m.vempty[slot], ((vpos / kVSlots) & 1) ^ 1, gave_up, tries);
                    if (!ok) break;
                    uint8_t *dst = psm + kOffV + slot * 2 * kSlotB;
                    mbar_arrive_expect_tx(&m.vfull[slot], 2 * kSlotB);
                    tma_box3(dst, &mapv, 0, v_h ? h : 0, y, &m.vfull[slot], pol);
                    tma_box3(dst + kSlotB, &mapv, 64, v_h ? h : 0, y, &m.vfull[slot], pol);
                }
            }
            if (*gave_up) {  // copies in flight are left time to land
                const unsigned long long t0 = globaltimer_ns();
                while (globaltimer_ns() - t0 < kWaitLimitNs) {}
            }
        }
        __syncwarp();
    } else if (warp == 10) {
        // --------------------------------- Q ---------------------------------
        reg_share_less<88>();
        if (elect_one()) {
            const uint64_t pol = l2_policy_evict_first();
            uint32_t used = 0;  // parities: bit `tile`
            bool ok = true;
            for (int i = 0; ok && item_ready(i); ++i) {
                const int n0 = m.item[i % kItems].n0, n1 = m.item[i % kItems].n1;
                const int h = m.item[i % kItems].h, q0 = m.item[i % kItems].q0;
                bar_arrive(&m.iempty[i % kItems]);
#pragma unroll 1
                for (int tile = 0; tile < 2; ++tile) {
                    if ((tile ? n1 : n0) == 0 || !ok) continue;
                    ok = bar_wait(&m.qempty[tile], ((used >> tile) & 1) ^ 1, gave_up, item_tries);
                    used ^= 1u << tile;
                    if (!ok) continue;
                    uint64_t *full = &m.qfull[tile];
                    uint8_t *dst = psm + tile * kKChunks * kSlotB;
                    const int y = q0 + tile * kQTile;
                    mbar_arrive_expect_tx(full, kKChunks * kSlotB);
                    tma_box3(dst, &mapqn, 0, qn_h ? h : 0, y, full, pol);
                    tma_box3(dst + kSlotB, &mapqn, 64, qn_h ? h : 0, y, full, pol);
                    tma_box3(dst + 2 * kSlotB, &mapqr, 0, qr_h ? h : 0, y, full, pol);
                }
            }
            if (*gave_up) {
                const unsigned long long t0 = globaltimer_ns();
                while (globaltimer_ns() - t0 < kWaitLimitNs) {}
            }
        }
        __syncwarp();
    } else {
        // -------------------------------- items --------------------------------
        reg_share_less<88>();
        int q0, nq, k0, nk;
        // A lane a number (dense), or a number of the CTA's own turns: with a max_q_len far above
        // the lengths most numbers stand for no item.
        int i = 0;
        // Waits until the place of number n is free; then its last item's redo flag stands.
        auto is_free = [&](int n) { return bar_wait(&m.iempty[n % kItems], ((n / kItems) & 1) ^ 1, gave_up, item_tries); };
        auto put = [&](const Item &it) {
            m.item[i % kItems] = it;
            m.redo[i % kItems] = m.unsound[i % kItems] = 0u;
            bar_arrive(&m.ifull[i % kItems]);
            ++i;
        };
        // Done by one lane: numbers i, and the item in the place of number n (free, as is that of i)
        // once more before it if it came out not finite.
        auto again = [&](int n) {
            if (n < kItems || !*static_cast<volatile uint32_t *>(&m.redo[n % kItems])) return false;
            Item it = m.item[n % kItems];
            it.careful = true;
            m.redo[n % kItems] = 0u;
            put(it);
            return true;
        };
        auto publish = [&](const Item &it) {
            do {
                if (!is_free(i)) return false;
            } while (again(i));
            put(it);
            return true;
        };
        bool ok = true;
        Item it{};
        const long long turns = (deal.items + gridDim.x - 1) / gridDim.x;
        uint32_t dealt = 0;  // items so far (dense)
        for (long long at = 0; ok && at < (deal.dense ? deal.items : turns); at += 32) {
            const long long turn = at + lane;
            const long long x = deal.dense ? turn : turn * gridDim.x + ((turn & 1) ? gridDim.x - 1 - blockIdx.x : blockIdx.x);
            const long long group = x / ((long long)deal.pairs * deal.tiles);
            const int in_group = (int)(x - group * deal.pairs * deal.tiles);
            const int t = deal.tiles - 1 - in_group / deal.pairs;
            const long long pair = group * deal.pairs + in_group % deal.pairs;
            bool there = x < deal.items && pair < (long long)a.B * a.H;
            if (there) {
                it.b = (int)(pair / a.H);
                it.h = (int)(pair - (long long)it.b * a.H);
                there = request_rows(a, it.b, q0, nq, k0, nk) && t * kItemRows < nq;
            }
            if (there) {
                it.q0 = q0 + t * kItemRows;
                it.nq = nq - t * kItemRows;
                it.k0 = k0;
                it.nk = nk;
                it.sees0 = nk - nq + 1 + t * kItemRows;
                auto steps = [&](int tile) {
                    const int rows = min(kQTile, it.nq - tile * kQTile);
                    const int most = a.causal ? min(nk, it.sees0 + tile * kQTile + rows - 1) : nk;
                    return rows > 0 && most > 0 ? (most + kKeys - 1) / kKeys : 0;
                };
                it.n0 = steps(0);
                it.n1 = steps(1);
            }
            if (deal.dense) {
                const uint32_t all = __ballot_sync(0xffffffffu, there);
                const uint32_t rank = dealt + __popc(all & ((1u << lane) - 1u)), round = rank / gridDim.x;
                const uint32_t place = rank - round * gridDim.x;
                there = there && ((round & 1) ? gridDim.x - 1 - place : place) == blockIdx.x;
                dealt += __popc(all);
            }
            for (uint32_t left = __ballot_sync(0xffffffffu, there); ok && left; left &= left - 1) {
                const int from = __ffs(left) - 1;
                ok = __all_sync(0xffffffffu, lane != from || publish(it));
                i = __shfl_sync(0xffffffffu, i, from);
            }
        }
        if (lane == 0 && ok) {
            it.b = -1;
            // no more, once no item is to be done again
            for (int n = i; a.causal && ok && n < i + kItems; ++n) {
                ok = is_free(n);
                if (ok && again(n)) n = i - 1;
            }
            if (ok) publish(it);
        }
        __syncwarp();
    }
    __syncthreads();
    // After a wait gave up, items of this CTA are left unwritten; which ones is not kept, and
    // every request of the call is flagged.
    if (*gave_up && a.flags)
        for (int b = tid; b < a.B; b += kPreThreads) atomic_or_byte(a.flags, b, PFKV_FLAG_DEVICE_TIMEOUT);
    tmem_fence_after();
    if (warp == 8) tmem_free512<1>(tmem);
}

}  // namespace

cudaError_t launch_latent_prefill(const LatentPrefillArgs &a, int num_sms, cudaStream_t s) {
    CUtensorMap qn{}, qr{}, kn{}, kr{}, v{};
    // [rows][heads][width]; heads that share a row (stride 0), and a single head, are one
    auto map = [](CUtensorMap *m, const RowsArg &r, int width, int heads, long long rows, int *per_head) {
        *per_head = heads > 1 && r.sh > 0;
        const uint64_t h = *per_head ? heads : 1;
        return bf16_map3(m, r.p, width, h, rows, *per_head ? r.sh : 8, r.st > 0 ? r.st : 8, 1, 128);
    };
    int qn_h = 0, qr_h = 0, kn_h = 0, v_h = 0, one = 0;
    cudaError_t e = cudaSuccess;
    if (a.total_q > 0 && a.total_k > 0) {
        e = map(&qn, a.qn, PFKV_LATENT_NOPE, a.H, a.total_q, &qn_h);
        if (e == cudaSuccess) e = map(&qr, a.qr, PFKV_LATENT_ROPE, a.H, a.total_q, &qr_h);
        if (e == cudaSuccess) e = map(&kn, a.kn, PFKV_LATENT_NOPE, a.H, a.total_k, &kn_h);
        if (e == cudaSuccess) e = map(&kr, a.kr, PFKV_LATENT_ROPE, 1, a.total_k, &one);
        if (e == cudaSuccess) e = map(&v, a.v, PFKV_LATENT_VDIM, a.H, a.total_k, &v_h);
        if (e != cudaSuccess) return e;
    }
    Deal d;
    d.tiles = (int)((min((long long)a.max_q_len, a.total_q) + kItemRows - 1) / kItemRows);
    const long long pairs = (long long)a.B * a.H;
    // One group, all items in order of their length, while K and V of all heads are at most 1.5
    // times L2 (causal items of one length read them at different times).  Prompts of 3,000,
    // 2,000 and 1,000 tokens, 64 heads (188 MiB): 242 us, 278 in groups; one of 4,096, 128
    // heads (256 MiB): 502 us, 438 in groups.
    // Where there are few numbers, every CTA can look through all of them (32 a step of the
    // looking warp) and items alone are dealt out, which evens out ragged lengths: 5 prompts
    // of up to 777 tokens, 16 heads, 26.5 us, 33.9 with all numbers dealt (29.6 now, with the
    // flags' launch and the list's end behind the last result).
    const bool fits = a.total_k * a.H * (PFKV_LATENT_NOPE + PFKV_LATENT_VDIM) * 2 <= (192LL << 20) &&
                      pairs <= (1LL << 30) / max(1, d.tiles);  // numbers within a group are 32-bit
    d.pairs = (int)min(pairs, fits ? pairs : (2LL * num_sms + d.tiles - 1) / max(1, d.tiles));
    d.items = (pairs + d.pairs - 1) / d.pairs * d.pairs * d.tiles;
    d.dense = d.items <= 16LL * num_sms;
    const unsigned grid = (unsigned)max(1LL, min(d.items, (long long)num_sms));
    if (a.flags) {
        const unsigned ctas = (unsigned)min((a.B + kFlagThreads - 1LL) / kFlagThreads, 4LL * num_sms);
        e = launch_pdl(latent_prefill_flags_kernel, dim3(ctas), dim3(kFlagThreads), 0, s, a);
        if (e != cudaSuccess) return e;
    }
    // a negative scale is the operands' sign: the softmax works with its magnitude
    const uint32_t idS = umma_idesc(kQTile, kKeys, true, false, false) | (a.sm_scale < 0.f ? 1u << 13 : 0u);
    auto *const kernel = a.tries == kTries ? latent_prefill_kernel<false> : latent_prefill_kernel<true>;
    return launch_pdl(kernel, dim3(grid), dim3(kPreThreads), kPreSmem, s, qn, qr, kn, kr, v, a, d, idS,
                      qn_h, qr_h, kn_h, v_h);
}

cudaError_t preload_latent_prefill() {
    cudaError_t e = preload_kernel(latent_prefill_flags_kernel);
    for (auto *const kernel : {latent_prefill_kernel<false>, latent_prefill_kernel<true>}) {
        if (e == cudaSuccess) e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kPreSmem);
        if (e == cudaSuccess) e = preload_kernel(kernel);
    }
    return e;
}

}  // namespace pfkv

// latent_prefill.cu -- pfkv_latent_prefill_attn: ragged causal attention of
// prompts in the expanded form (declared in pfkv_latent.h).
//
// First form: one warp a query row and head, a running maximum and sum over the
// keys one at a time.
#include "latent_internal.cuh"

namespace pfkv {
namespace {

constexpr int kSimpleRows = 8;

__device__ __forceinline__ void load4(const __nv_bfloat16 *p, float *x) {
    const uint2 w = *reinterpret_cast<const uint2 *>(p);
    const float2 a = bf16x2_to_float2(w.x), b = bf16x2_to_float2(w.y);
    x[0] = a.x;
    x[1] = a.y;
    x[2] = b.x;
    x[3] = b.y;
}

__global__ void __launch_bounds__(kSimpleRows * 32) latent_prefill_kernel(LatentPrefillArgs a) {
    pdl_enter();
    const int b = blockIdx.z, h = blockIdx.y, lane = threadIdx.x & 31;
    const int q0 = a.q_starts[b], q1 = a.q_starts[b + 1], k0 = a.k_starts[b], k1 = a.k_starts[b + 1];
    const bool bad = q0 < 0 || q1 < q0 || q1 > a.total_q || k0 < 0 || k1 < k0 || k1 > a.total_k || q1 - q0 > a.max_q_len;
    if (blockIdx.x == 0 && h == 0 && threadIdx.x == 0 && a.flags) a.flags[b] = bad ? PFKV_FLAG_BAD_LENGTH : 0;
    if (bad) return;
    const int i = blockIdx.x * kSimpleRows + (threadIdx.x >> 5);
    if (i >= q1 - q0) return;
    const int nk = k1 - k0;
    const int sees = a.causal ? min(nk, i + 1 + nk - (q1 - q0)) : nk;
    float q[4], o[4] = {};
    load4(a.qn.p + (long long)(q0 + i) * a.qn.st + (long long)h * a.qn.sh + lane * 4, q);
    const __nv_bfloat16 *qr = a.qr.p + (long long)(q0 + i) * a.qr.st + (long long)h * a.qr.sh + 2 * lane;
    const float r0 = __bfloat162float(qr[0]), r1 = __bfloat162float(qr[1]);
    float m = -INFINITY, l = 0.f;
    for (int j = 0; j < sees; ++j) {
        float k[4], v[4];
        load4(a.kn.p + (long long)(k0 + j) * a.kn.st + (long long)h * a.kn.sh + lane * 4, k);
        load4(a.v.p + (long long)(k0 + j) * a.v.st + (long long)h * a.v.sh + lane * 4, v);
        const __nv_bfloat16 *kr = a.kr.p + (long long)(k0 + j) * a.kr.st + 2 * lane;
        float s = r0 * __bfloat162float(kr[0]) + r1 * __bfloat162float(kr[1]);
#pragma unroll
        for (int e = 0; e < 4; ++e) s += q[e] * k[e];
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
        s *= a.sm_scale;
        const float mn = fmaxf(m, s), f = __expf(m - mn), w = __expf(s - mn);
        m = mn;
        l = l * f + w;
#pragma unroll
        for (int e = 0; e < 4; ++e) o[e] = o[e] * f + w * v[e];
    }
    __nv_bfloat16 *out = a.out.p + (long long)(q0 + i) * a.out.st + (long long)h * a.out.sh + lane * 4;
#pragma unroll
    for (int e = 0; e < 4; ++e) out[e] = __float2bfloat16(sees > 0 ? o[e] / l : 0.f);
}

}  // namespace

cudaError_t launch_latent_prefill(const LatentPrefillArgs &a, int, cudaStream_t s) {
    if (a.B > 65535) return cudaErrorInvalidValue;
    const unsigned tiles = (unsigned)max(1, (a.max_q_len + kSimpleRows - 1) / kSimpleRows);
    return launch_pdl(latent_prefill_kernel, dim3(tiles, a.H, a.B), dim3(kSimpleRows * 32), 0, s, a);
}

cudaError_t preload_latent_prefill() { return preload_kernel(latent_prefill_kernel); }

}  // namespace pfkv

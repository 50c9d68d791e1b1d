// latent_decode.cu -- pfkv_latent_decode_attn: attention in the absorbed form
// over a paged latent cache (declared in pfkv_latent.h).
//
// First form: one CTA a query row.  Each of its warps takes every eighth token,
// keeps a running maximum, sum and weighted latent in registers, and the warps
// meet in shared memory.  Every row reads the request's whole cache, so this is
// bound by L2 traffic (rows x tokens x 1,152 bytes).
#include "latent_internal.cuh"

namespace pfkv {
namespace {

constexpr int kSimpleWarps = 8;

__device__ __forceinline__ void load16(const __nv_bfloat16 *p, float *x) {
    const uint4 *w = reinterpret_cast<const uint4 *>(p);
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        const uint4 v = w[k];
        const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 f = bf16x2_to_float2(u[i]);
            x[8 * k + 2 * i] = f.x;
            x[8 * k + 2 * i + 1] = f.y;
        }
    }
}

__global__ void __launch_bounds__(kSimpleWarps * 32) latent_decode_kernel(LatentDecodeArgs a) {
    __shared__ float so[kSimpleWarps][PFKV_LATENT_DIM];
    __shared__ float sm[kSimpleWarps], sl[kSimpleWarps];
    pdl_enter();
    const int row = blockIdx.x, b = blockIdx.y;
    const int t = row / a.H, h = row - t * a.H;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const LatentPool &p = a.pool;
    const int n = p.seq_lens[(long long)b * p.len_sb];
    uint32_t bits = 0;
    if (n < 0 || (long long)n > (long long)p.max_pages * kPage || n > a.max_seq_len) bits = PFKV_FLAG_BAD_LENGTH;
    else
        for (int i = threadIdx.x; i < (n + kPage - 1) / kPage; i += blockDim.x) {
            const long long bi = (long long)b * p.bt_sb + i;
            bits |= latent_entry_bits(p, p.block_tables[bi], bi);
        }
    uint32_t all = 0;
    for (uint32_t f = 1; f < 8; f <<= 1)
        if (__syncthreads_or(bits & f)) all |= f;
    if (row == 0 && threadIdx.x == 0 && a.flags) a.flags[b] = (uint8_t)all;
    const int sees = all ? 0 : n - a.kq + 1 + t;
    float q[16], qr[2], o[16] = {};
    load16(a.qc.p + (long long)b * a.qc.sb + (long long)t * a.qc.st + (long long)h * a.qc.sh + lane * 16, q);
    const __nv_bfloat16 *pr = a.qr.p + (long long)b * a.qr.sb + (long long)t * a.qr.st + (long long)h * a.qr.sh;
    qr[0] = __bfloat162float(pr[2 * lane]);
    qr[1] = __bfloat162float(pr[2 * lane + 1]);
    float m = -INFINITY, l = 0.f;
    for (int j = warp; j < sees; j += kSimpleWarps) {
        const int phys = p.block_tables[(long long)b * p.bt_sb + j / kPage];
        const long long r = (long long)phys * kPage + j % kPage;
        float c[16];
        if (p.fp8) {
            const uint4 w = reinterpret_cast<const uint4 *>(static_cast<const uint8_t *>(p.c_pages) + r * PFKV_LATENT_DIM)[lane];
            const uint32_t u[4] = {w.x, w.y, w.z, w.w};
            const float z = p.c_scale[phys];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float2 f = e4m3x2_to_float2((uint16_t)(u[i >> 1] >> (16 * (i & 1))));
                c[2 * i] = f.x * z;
                c[2 * i + 1] = f.y * z;
            }
        } else {
            load16(static_cast<const __nv_bfloat16 *>(p.c_pages) + r * PFKV_LATENT_DIM + lane * 16, c);
        }
        const __nv_bfloat16 *rr = p.r_pages + r * PFKV_LATENT_ROPE + 2 * lane;
        float s = qr[0] * __bfloat162float(rr[0]) + qr[1] * __bfloat162float(rr[1]);
#pragma unroll
        for (int i = 0; i < 16; ++i) s += q[i] * c[i];
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
        s *= a.sm_scale;
        const float mn = fmaxf(m, s), f = __expf(m - mn), w = __expf(s - mn);
        m = mn;
        l = l * f + w;
#pragma unroll
        for (int i = 0; i < 16; ++i) o[i] = o[i] * f + w * c[i];
    }
#pragma unroll
    for (int i = 0; i < 16; ++i) so[warp][lane * 16 + i] = o[i];
    if (lane == 0) {
        sm[warp] = m;
        sl[warp] = l;
    }
    __syncthreads();
    float top = -INFINITY, sum = 0.f;
    for (int w = 0; w < kSimpleWarps; ++w) top = fmaxf(top, sm[w]);
    for (int w = 0; w < kSimpleWarps; ++w)
        if (sl[w] != 0.f) sum += sl[w] * __expf(sm[w] - top);
    __nv_bfloat16 *out = a.out.p + (long long)b * a.out.sb + (long long)t * a.out.st + (long long)h * a.out.sh;
    for (int i = threadIdx.x; i < PFKV_LATENT_DIM; i += blockDim.x) {
        float x = 0.f;
        for (int w = 0; w < kSimpleWarps; ++w)
            if (sl[w] != 0.f) x += so[w][i] * __expf(sm[w] - top);
        out[i] = __float2bfloat16(sees > 0 ? x / sum : 0.f);
    }
}

}  // namespace

size_t latent_decode_workspace(int, int, int, int, int) { return 256; }

cudaError_t launch_latent_decode(const LatentDecodeArgs &a, int, cudaStream_t s) {
    if (a.B > 65535) return cudaErrorInvalidValue;
    return launch_pdl(latent_decode_kernel, dim3(a.H * a.kq, a.B), dim3(kSimpleWarps * 32), 0, s, a);
}

cudaError_t preload_latent_decode() { return preload_kernel(latent_decode_kernel); }

}  // namespace pfkv

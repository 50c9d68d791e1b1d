// latent_internal.cuh -- arguments and launchers shared by the rotary-append and
// latent-attention sources (declared to callers in pfkv_rope.h and
// pfkv_latent.h), and the host checks that they share with api.cu.
#pragma once

#include "../../include/pfkv_latent.h"
#include "pfkv_internal.cuh"

namespace pfkv {

// host checks (api.cu)
bool aligned(const void *p, uintptr_t a);
pfkv_status device_check(int *num_sms);
pfkv_status check_cache(const pfkv_cache *c);
pfkv_status check_pages(const pfkv_cache *c, const pfkv_pages *p);
// host checks (rope.cu)
// A pfkv_rows of so many rows: data, alignment, strides (those in use); without rows it is not read.
pfkv_status check_rows(const pfkv_rows *r, bool use_b, bool use_h, int64_t rows = 1);
// host checks (latent.cu)
pfkv_status check_latent(const pfkv_latent_cache *c, const pfkv_pages *p);

// Tries of a wait inside the attention kernels (umma.cuh), unless a self-test asks for fewer.
constexpr int kTries = 100000;
// Of one that lasts as long as an item of a prompt (436 million keys, all that memory holds, take
// 6 s): 20 s at least.  It ends as soon as another wait of its CTA gives up.
constexpr int kItemTries = 1000 * kTries;

struct RowsArg {
    __nv_bfloat16 *p;
    long long sb, st, sh;
};

inline RowsArg rows_arg(const pfkv_rows *r) {
    return RowsArg{static_cast<__nv_bfloat16 *>(r->data), (long long)r->stride_b, (long long)r->stride_t,
                   (long long)r->stride_h};
}

// The pool and tables of a latent call (kernels' copy of the two structs).
struct LatentPool {
    void *c_pages;
    __nv_bfloat16 *r_pages;
    float *c_scale;
    const uint32_t *page_tags;
    int num_pages;
    int fp8;
    const int32_t *block_tables;
    long long bt_sb;
    const uint32_t *expected_tags;
    int max_pages;
    const int32_t *seq_lens;
    long long len_sb;
};

LatentPool latent_pool(const pfkv_latent_cache *c, const pfkv_pages *p);

// Status bits of live table entry `bi` naming page `id` of a latent pool.
__device__ __forceinline__ uint32_t latent_entry_bits(const LatentPool &a, int id, long long bi) {
    if (id < 0 || id >= a.num_pages) return PFKV_FLAG_BAD_PAGE;
    if (a.page_tags && a.page_tags[id] != a.expected_tags[bi]) return PFKV_FLAG_TAG_MISMATCH;
    return 0u;
}

// Which of two bf16 values are not finite: the upper bit of each.
__device__ __forceinline__ uint32_t not_finite(uint32_t w) { return ((w & 0x7F807F80u) + 0x00800080u) & 0x80008000u; }
// Which of four e4m3 codes are NaN (the format has no infinities): the upper bit of each.
__device__ __forceinline__ uint32_t e4m3_nan(uint32_t w) { return ((w & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u; }

// Two fp32 operations an instruction.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    float2 d;
    asm("{\n\t.reg .b64 a, b, c, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\tmov.b64 c, {%6, %7};\n\t"
        "fma.rn.f32x2 d, a, b, c;\n\tmov.b64 {%0, %1}, d;\n\t}"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
    return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
    float2 d;
    asm("{\n\t.reg .b64 a, b, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
        "add.rn.f32x2 d, a, b;\n\tmov.b64 {%0, %1}, d;\n\t}"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return d;
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
    float2 d;
    asm("{\n\t.reg .b64 a, b, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
        "mul.rn.f32x2 d, a, b;\n\tmov.b64 {%0, %1}, d;\n\t}"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return d;
}

struct LatentDecodeArgs {
    LatentPool pool;
    RowsArg qc, qr, out;
    uint8_t *flags;
    int B, H, kq, max_seq_len;
    float sm_scale;
    void *workspace;
    int tries;  // of a wait
};

struct LatentPrefillArgs {
    RowsArg qn, qr, kn, kr, v, out;
    const int32_t *q_starts, *k_starts;
    long long total_q, total_k;
    uint8_t *flags;
    int B, H, max_q_len, causal;
    float sm_scale;
    int tries;  // of a wait
};

size_t latent_decode_workspace(int B, int H, int kq, int max_seq_len, int num_sms);
cudaError_t launch_latent_decode(const LatentDecodeArgs &a, int num_sms, cudaStream_t s);
cudaError_t launch_latent_prefill(const LatentPrefillArgs &a, int num_sms, cudaStream_t s);

cudaError_t preload_rope();
cudaError_t preload_latent();
cudaError_t preload_latent_decode();
cudaError_t preload_latent_prefill();

}  // namespace pfkv

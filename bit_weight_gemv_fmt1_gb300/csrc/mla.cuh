// mla.cuh -- arguments of the latent-attention kernels (mla_cache.cu,
// mla_attend.cu, mla_prefill.cu; entry points in mla_api.cu).
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "coli_internal.cuh"

namespace coli {

// Device view of a coli_mla_cache.
struct MlaCache {
    uint8_t *rows;
    float *scales;      // NULL for bf16
    int e4m3;
    int L, R;           // latent and rope dims
    int page;           // tokens per page
    int n_pages;
    int row_bytes;
};

struct MlaQueryArgs {
    const float *q;
    long long q_stride;
    int T, H, nope, rope;
    const int32_t *pos;
    const float *rot;
    int n_pos, interleaved;
    void *out_nope, *out_rope;
    long long ld_nope, ld_rope;
    int *err;
};

struct MlaAppendArgs {
    MlaCache c;
    const float *kv;
    long long kv_stride;
    int T;
    const float *norm;
    float eps;
    const int32_t *pos;
    const float *rot;
    int n_pos, interleaved;
    const int64_t *slots;
    int *err;
};

struct MlaReadArgs {
    MlaCache c;
    const int32_t *pages;
    long long pages_stride;
    int n_seq;
    const int32_t *cu;
    int T;
    void *out;
    long long out_stride;
    int *err;
};

struct MlaAttendArgs {
    MlaCache c;
    const void *q_latent, *q_rope;
    int q_bf16, out_bf16;
    int n_seq, n_q, H;
    const int32_t *pages;
    long long pages_stride;
    const int32_t *lens;
    float scale;
    void *out;
    float *lse;
    int *err;
};

struct MlaPrefillArgs {
    const void *q, *kv, *k_rope;
    long long q_stride, kv_stride, kr_stride;   // elements
    int in_f32, out_bf16;
    int Tq, Tk, n_seq;
    const int32_t *cu_q, *cu_k;
    int H, nope, rope, v;
    float scale;
    void *out;
    float *lse;
    int *err;
};

cudaError_t launch_mla_query(const MlaQueryArgs &a, bool nope_bf16, bool rope_bf16, int n_sm, cudaStream_t st);
cudaError_t launch_mla_append(const MlaAppendArgs &a, cudaStream_t st);
cudaError_t launch_mla_read(const MlaReadArgs &a, bool out_bf16, cudaStream_t st);
// Scratch of a call, and the call (d.scratch: that many bytes, NULL if none).
size_t mla_attend_scratch(const MlaAttendArgs &a, int n_sm);
cudaError_t launch_mla_attend(const MlaAttendArgs &a, const DevInfo &d, cudaStream_t st, int *n_launch);
size_t mla_prefill_scratch(const MlaPrefillArgs &a);
cudaError_t launch_mla_prefill(const MlaPrefillArgs &a, const DevInfo &d, cudaStream_t st, int *n_launch);

__device__ __forceinline__ void mla_bad_index(int *err) { atomicCAS(err, 0, (int)DEV_ERR_BAD_INDEX); }

// Two f32 -> two bf16 in one register, the first in the low half; to nearest.
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
// Two f32 -> two f16 in one register, the first in the low half; to nearest.
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
// Two f32 -> two E4M3 bytes, the first in the low one; to nearest, saturating, NaN kept.
__device__ __forceinline__ uint32_t pack_e4m3(float lo, float hi) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}
// The same to E5M2.
__device__ __forceinline__ uint32_t pack_e5m2(float lo, float hi) {
    uint16_t r;
    asm("cvt.rn.satfinite.e5m2x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}
// Two E4M3 bytes -> two f16 in one register (exact).
__device__ __forceinline__ uint32_t e4m3x2_f16x2(uint32_t two) {
    uint32_t r;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"((uint16_t)two));
    return r;
}
__device__ __forceinline__ float2 bf16x2_f32x2(uint32_t w) {
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
}

// Byte address of a cached row.
__device__ __forceinline__ const uint8_t *mla_row(const MlaCache &c, long long slot) {
    return c.rows + slot * c.row_bytes;
}

}  // namespace coli

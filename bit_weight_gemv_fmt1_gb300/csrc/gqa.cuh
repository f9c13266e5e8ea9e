// gqa.cuh -- arguments of the grouped-head attention kernels (gqa_cache.cu,
// gqa_evict.cu, gqa_attend.cu, gqa_prefill.cu; entry points in gqa_api.cu).
#pragma once

#include "mla.cuh"

namespace coli {

// Device view of a coli_gqa_cache.
struct GqaCache {
    uint8_t *k, *v;
    __nv_bfloat16 *ks, *vs;
    float *w;           // NULL: none
    int n_kv, dim, gs;
    int page;           // tokens per page
    int n_pages;
};

struct GqaAppendArgs {
    GqaCache c;
    const void *k, *v;
    long long k_stride, v_stride;   // elements
    int T;
    const int64_t *slots;
    int *err;
};

struct GqaReadArgs {
    GqaCache c;
    const int32_t *pages;
    long long pages_stride;
    int n_seq;
    const int32_t *cu;
    int T;
    void *k, *v;
    long long k_stride, v_stride;
    int *err;
};

struct GqaAttendArgs {
    GqaCache c;
    int longest;            // length allowed
    const void *q;
    int q_bf16, out_bf16, weigh;
    int n_seq, n_q, H;
    const int32_t *pages;
    long long pages_stride;
    const int32_t *lens;
    float scale;
    void *out;
    float *lse;
    int *err;
};

struct GqaEvictArgs {
    GqaCache c;
    int longest;            // length allowed
    const int32_t *pages;
    long long pages_stride;
    int n_seq;
    const int32_t *lens;
    int keep, recent;
    const int32_t *dst;
    long long dst_stride;
    int32_t *kept, *new_lens;
    int *err;
};

struct GqaPrefillArgs {
    const void *q, *k, *v;
    long long q_stride, k_stride, v_stride;     // elements
    int in_f32, out_bf16;
    int Tq, Tk, n_seq;
    const int32_t *cu_q, *cu_k;
    int heads;          // query heads
    int H;              // key / value heads: units of one pair of query tiles
    int group;          // query heads of one
    int tokens;         // tokens of a query tile: rows token * group + head, 128 at most
    int dim;
    float scale;
    void *out;
    float *lse;
    // f16 inputs made from f32: what takes each row of q back [Tq][heads], and two bf16 factors for each key and its value [H][Tk]
    const float *q_power;
    const uint32_t *kv_power;
    int *err;
};

cudaError_t launch_gqa_append(const GqaAppendArgs &a, bool in_bf16, int n_sm, cudaStream_t st);
cudaError_t launch_gqa_read(const GqaReadArgs &a, bool out_bf16, cudaStream_t st);
cudaError_t launch_gqa_evict(const GqaEvictArgs &a, const DevInfo &d, cudaStream_t st, int *n_launch);
// Scratch of a call, and the call (d.scratch: that many bytes, NULL if none).
size_t gqa_attend_scratch(const GqaAttendArgs &a, int n_sm);
cudaError_t launch_gqa_attend(const GqaAttendArgs &a, const DevInfo &d, cudaStream_t st, int *n_launch);
size_t gqa_prefill_scratch(const GqaPrefillArgs &a);
cudaError_t launch_gqa_prefill(const GqaPrefillArgs &a, const DevInfo &d, cudaStream_t st, int *n_launch);

// Row of the arrays of a cache that holds head h of a page's first token.
__device__ __forceinline__ long long gqa_row(const GqaCache &c, int page, int h) {
    return ((long long)page * c.n_kv + h) * c.page;
}

}  // namespace coli

// mla_prefill.cu -- causal attention of packed sequences in the expanded form.
//
// One warp per (query row, head): lanes over the dims, one warp-wide dot
// product a key, the running maximum and sum of the softmax, the weighted sum
// of the values in registers.  Everything is f32.
#include "mla.cuh"

namespace coli {

namespace {

template <bool F32>
__device__ __forceinline__ float ld(const void *p, long long e) {
    if constexpr (F32) return reinterpret_cast<const float *>(p)[e];
    else return __bfloat162float(reinterpret_cast<const __nv_bfloat16 *>(p)[e]);
}

template <bool F32>
__global__ void __launch_bounds__(128) mla_prefill_kernel(const MlaPrefillArgs a) {
    const int lane = threadIdx.x & 31;
    const long long row = (long long)blockIdx.x * 4 + (threadIdx.x >> 5);   // query * H + head
    pdl_wait();
    pdl_trigger();
    if (row >= (long long)a.Tq * a.H) return;
    const int i = (int)(row / a.H), h = (int)(row - (long long)i * a.H);
    int lo = 0, hi = a.n_seq;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (a.cu_q[mid] <= i) lo = mid;
        else hi = mid;
    }
    const int k0 = a.cu_k[lo], nk = a.cu_k[lo + 1] - k0, nq = a.cu_q[lo + 1] - a.cu_q[lo];
    if (k0 < 0 || nk < 0 || k0 > a.Tk - nk) {
        if (lane == 0) mla_bad_index(a.err);
        return;
    }
    const int limit = i - a.cu_q[lo] + nk - nq + 1;
    const int dk = a.nope + a.rope;
    float q[6], o[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int k = 0; k < 6; k++) q[k] = 32 * k + lane < dk ? ld<F32>(a.q, i * a.q_stride + (long long)h * dk + 32 * k + lane) : 0.f;
    float m = -INFINITY, l = 0.f;
    for (int j = 0; j < limit; j++) {
        const long long kb = (k0 + j) * a.kv_stride + (long long)h * (a.nope + a.v);
        float dot = 0.f;
#pragma unroll
        for (int k = 0; k < 6; k++) {
            const int d = 32 * k + lane;
            if (d < a.nope) dot = fmaf(q[k], ld<F32>(a.kv, kb + d), dot);
            else if (d < dk) dot = fmaf(q[k], ld<F32>(a.k_rope, (k0 + j) * a.kr_stride + d - a.nope), dot);
        }
        const float s = warp_sum(dot) * a.scale;
        const float mn = fmaxf(m, s);
        const float f = mn == -INFINITY ? 1.f : expf(m - mn), p = mn == -INFINITY ? 0.f : expf(s - mn);
        l = fmaf(l, f, p);
#pragma unroll
        for (int k = 0; k < 4; k++)
            if (32 * k + lane < a.v) o[k] = fmaf(o[k], f, p * ld<F32>(a.kv, kb + a.nope + 32 * k + lane));
        m = mn;
    }
#pragma unroll
    for (int k = 0; k < 4; k++) {
        const int d = 32 * k + lane;
        if (d >= a.v) continue;
        const float r = l != 0.f ? o[k] / l : 0.f;
        if (a.out_bf16) reinterpret_cast<__nv_bfloat16 *>(a.out)[row * a.v + d] = __float2bfloat16_rn(r);
        else reinterpret_cast<float *>(a.out)[row * a.v + d] = r;
    }
    if (a.lse && lane == 0) a.lse[row] = l != 0.f ? m + logf(l) : -INFINITY;
}

}  // namespace

cudaError_t launch_mla_prefill(const MlaPrefillArgs &a, cudaStream_t st) {
    const dim3 grid((unsigned)(((long long)a.Tq * a.H + 3) / 4));
    return a.in_f32 ? launch_pdl(mla_prefill_kernel<true>, grid, dim3(128), 0, st, a)
                    : launch_pdl(mla_prefill_kernel<false>, grid, dim3(128), 0, st, a);
}

}  // namespace coli

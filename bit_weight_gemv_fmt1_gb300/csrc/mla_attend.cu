// mla_attend.cu -- attention over the paged latent cache (absorbed form).
//
// One CTA per (sequence, query token, head).  Each of the 8 warps takes every
// eighth token: lanes over the dims, one warp-wide dot product, the running
// maximum and sum of the softmax, and the weighted sum of the latent parts in
// registers; the warps' results are joined at the end.  Everything is f32.
#include "mla.cuh"

namespace coli {

namespace {

constexpr int kWarps = 8;

__device__ __forceinline__ float cached(const MlaCache &c, const uint8_t *row, int d) {
    if (c.e4m3) {
        const uint32_t h = e4m3x2_f16x2(row[d]);
        return __half22float2(*reinterpret_cast<const __half2 *>(&h)).x;
    }
    return __bfloat162float(reinterpret_cast<const __nv_bfloat16 *>(row)[d]);
}

__device__ __forceinline__ float load_q(const void *p, int bf16, long long e) {
    return bf16 ? __bfloat162float(reinterpret_cast<const __nv_bfloat16 *>(p)[e]) : reinterpret_cast<const float *>(p)[e];
}

__global__ void __launch_bounds__(kWarps * 32) mla_attend_kernel(const MlaAttendArgs a) {
    __shared__ float s_o[512], s_m[kWarps], s_l[kWarps];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const long long row = blockIdx.x;   // (b * n_q + j) * H + h
    pdl_wait();
    pdl_trigger();
    const int b = (int)(row / ((long long)a.n_q * a.H));
    const int j = (int)(row / a.H - (long long)b * a.n_q);
    const int L = a.c.L, R = a.c.R;
    int len = a.lens[b];
    if (len < 0 || len > a.pages_stride * a.c.page) {
        if (threadIdx.x == 0) mla_bad_index(a.err);
        len = 0;
    }
    const int limit = len - (a.n_q - 1 - j);
    float q[18], o[16];
#pragma unroll
    for (int k = 0; k < 16; k++) {
        q[k] = 32 * k + lane < L ? load_q(a.q_latent, a.q_bf16, row * L + 32 * k + lane) : 0.f;
        o[k] = 0.f;
    }
#pragma unroll
    for (int k = 0; k < 2; k++) q[16 + k] = 32 * k + lane < R ? load_q(a.q_rope, a.q_bf16, row * R + 32 * k + lane) : 0.f;
    float m = -INFINITY, l = 0.f;
    for (int t = warp; t < limit; t += kWarps) {
        const int pi = t / a.c.page, id = a.pages[b * a.pages_stride + pi];
        if (id < 0 || id >= a.c.n_pages) {
            if (lane == 0) mla_bad_index(a.err);
            continue;
        }
        const long long slot = (long long)id * a.c.page + (t - pi * a.c.page);
        const uint8_t *src = mla_row(a.c, slot);
        const float sc = a.c.e4m3 ? a.c.scales[slot] : 1.f;
        float v[16], dot = 0.f;
#pragma unroll
        for (int k = 0; k < 16; k++) {
            v[k] = 32 * k + lane < L ? cached(a.c, src, 32 * k + lane) : 0.f;
            dot = fmaf(q[k], v[k], dot);
        }
#pragma unroll
        for (int k = 0; k < 2; k++)
            if (32 * k + lane < R) dot = fmaf(q[16 + k], cached(a.c, src, L + 32 * k + lane), dot);
        const float s = warp_sum(dot) * sc * a.scale;
        const float mn = fmaxf(m, s);
        const float f = mn == -INFINITY ? 1.f : expf(m - mn), p = mn == -INFINITY ? 0.f : expf(s - mn);
        l = fmaf(l, f, p);
#pragma unroll
        for (int k = 0; k < 16; k++) o[k] = fmaf(o[k], f, p * sc * v[k]);
        m = mn;
    }
    if (lane == 0) {
        s_m[warp] = m;
        s_l[warp] = l;
    }
    for (int d = threadIdx.x; d < 512; d += kWarps * 32) s_o[d] = 0.f;
    __syncthreads();
    float M = -INFINITY, Z = 0.f;
    for (int w = 0; w < kWarps; w++) M = fmaxf(M, s_m[w]);
    if (M == -INFINITY) M = 0.f;
    for (int w = 0; w < kWarps; w++) Z += s_l[w] * expf(s_m[w] - M);
    for (int w = 0; w < kWarps; w++) {
        if (w == warp) {
            const float f = expf(m - M);
#pragma unroll
            for (int k = 0; k < 16; k++) s_o[32 * k + lane] = fmaf(o[k], f, s_o[32 * k + lane]);
        }
        __syncthreads();
    }
    for (int d = threadIdx.x; d < L; d += kWarps * 32) {
        const float r = Z != 0.f ? s_o[d] / Z : 0.f;
        if (a.out_bf16) reinterpret_cast<__nv_bfloat16 *>(a.out)[row * L + d] = __float2bfloat16_rn(r);
        else reinterpret_cast<float *>(a.out)[row * L + d] = r;
    }
    if (a.lse && threadIdx.x == 0) a.lse[row] = Z != 0.f ? M + logf(Z) : -INFINITY;
}

}  // namespace

cudaError_t launch_mla_attend(const MlaAttendArgs &a, cudaStream_t st) {
    return launch_pdl(mla_attend_kernel, dim3((unsigned)((long long)a.n_seq * a.n_q * a.H)), dim3(kWarps * 32), 0, st, a);
}

}  // namespace coli

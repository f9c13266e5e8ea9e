// gqa_cache.cu -- writing keys and values into the paged 4-bit cache and reading
// them back.  Both touch every input and output once and are bound by HBM on
// long inputs, by launch and two memory round trips on short ones.
//
// Group of gs elements: scale = bf16(max|x| / 7), code = clamp(rint(x / scale)).
// Codes are taken against the scale as it is stored, so its rounding to 8 bits
// moves the steps and adds no error of its own.
#include "gqa.cuh"

namespace coli {

namespace {

constexpr int kThreads = 256;

// 8 consecutive elements as f32.
template <bool BF16>
__device__ __forceinline__ void load8(const void *base, long long e, float (&x)[8]) {
    if constexpr (BF16) {
        const uint4 w = *reinterpret_cast<const uint4 *>(reinterpret_cast<const __nv_bfloat16 *>(base) + e);
        const uint32_t v[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int i = 0; i < 4; i++) {
            const float2 p = bf16x2_f32x2(v[i]);
            x[2 * i] = p.x;
            x[2 * i + 1] = p.y;
        }
    } else {
        const float4 p = *reinterpret_cast<const float4 *>(reinterpret_cast<const float *>(base) + e);
        const float4 q = *reinterpret_cast<const float4 *>(reinterpret_cast<const float *>(base) + e + 4);
        x[0] = p.x, x[1] = p.y, x[2] = p.z, x[3] = p.w, x[4] = q.x, x[5] = q.y, x[6] = q.z, x[7] = q.w;
    }
}

// One thread per 8 elements of a token's key or value row, gs / 8 neighbouring threads per group.
template <bool BF16, int GS>
__global__ void __launch_bounds__(kThreads) gqa_append_kernel(const GqaAppendArgs a) {
    const int upr = a.c.dim / 8;                         // 8 or 16
    const uint32_t row = blockIdx.x * (kThreads / upr) + threadIdx.x / upr, heads = 2 * a.c.n_kv;
    const int u = threadIdx.x & (upr - 1);
    const uint32_t t = row / heads, h2 = row - t * heads;
    const bool value = h2 >= (uint32_t)a.c.n_kv;
    const int h = value ? h2 - a.c.n_kv : h2;
    const bool live = t < (uint32_t)a.T;
    pdl_wait();
    pdl_trigger();
    float x[8];
    long long slot = -1;
    if (live) {
        slot = a.slots[t];
        load8<BF16>(value ? a.v : a.k, t * (value ? a.v_stride : a.k_stride) + h * a.c.dim + 8 * u, x);
    } else {
#pragma unroll
        for (int i = 0; i < 8; i++) x[i] = 0.f;
    }
    float m = 0.f;
    bool fine = true;
#pragma unroll
    for (int i = 0; i < 8; i++) {
        m = fmaxf(m, fabsf(x[i]));
        fine = fine && fabsf(x[i]) <= 3.402823466e38f;   // neither NaN nor infinite
    }
    if (!fine) m = INFINITY;
#pragma unroll
    for (int o = 1; o < GS / 8; o <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    if (!live || slot == -1) return;
    if (slot < 0 || slot >= (long long)a.c.n_pages * a.c.page) {
        mla_bad_index(a.err);
        return;
    }
    fine = m < INFINITY;
    const __nv_bfloat16 stored = __float2bfloat16_rn(fine ? __fdiv_rn(m, 7.f) : __uint_as_float(0x7FC00000u));
    const float scale = __bfloat162float(stored), by = scale > 0.f ? scale : 1.f;
    uint32_t w = 0x88888888u;
    if (fine) {
        w = 0;
#pragma unroll
        for (int i = 0; i < 8; i++) {
            const int c = __float2int_rn(fminf(fmaxf(__fdiv_rn(x[i], by), -8.f), 7.f)) + 8;
            w |= (uint32_t)c << (4 * i);
        }
    }
    const int page = (int)(slot / a.c.page);
    const long long r = gqa_row(a.c, page, h) + (slot - (long long)page * a.c.page);
    reinterpret_cast<uint32_t *>(value ? a.c.v : a.c.k)[r * upr + u] = w;
    if (u % (GS / 8) == 0) (value ? a.c.vs : a.c.ks)[r * (a.c.dim / GS) + u / (GS / 8)] = stored;
    if (u == 0 && !value && a.c.w) a.c.w[r] = 0.f;
}

// kReadRows tokens of one head per CTA: as many threads find the tokens' rows, then every thread moves units of 8 elements,
// keys first.
constexpr int kReadRows = 32;

template <bool OB>
__device__ __forceinline__ void store8(void *base, long long e, uint32_t w, float scale) {
    float x[8];
#pragma unroll
    for (int i = 0; i < 8; i++) x[i] = (__uint_as_float(0x4B000000u | ((w >> (4 * i)) & 15u)) - 8388616.f) * scale;   // 2^23 + code
    if constexpr (OB) {
        *reinterpret_cast<uint4 *>(reinterpret_cast<__nv_bfloat16 *>(base) + e) =
            make_uint4(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4], x[5]), pack_bf16(x[6], x[7]));
    } else {
        float4 *d = reinterpret_cast<float4 *>(reinterpret_cast<float *>(base) + e);
        d[0] = make_float4(x[0], x[1], x[2], x[3]);
        d[1] = make_float4(x[4], x[5], x[6], x[7]);
    }
}

template <bool OB, int D>
__global__ void __launch_bounds__(kThreads) gqa_read_kernel(const GqaReadArgs a) {
    constexpr int kUnits = D / 8, kEach = 2 * kReadRows * kUnits / kThreads;
    __shared__ long long s_row[kReadRows];    // -1: a zero row, -2: not to be written
    const int r0 = blockIdx.x * kReadRows, h = blockIdx.y;
    pdl_wait();
    pdl_trigger();
    if (threadIdx.x < kReadRows) {
        const int r = r0 + threadIdx.x;
        long long row = -2;
        if (r < a.T && r < a.cu[a.n_seq] && r >= a.cu[0]) {
            int lo = 0, hi = a.n_seq;         // cu[lo] <= r < cu[hi]
            while (hi - lo > 1) {
                const int m = (lo + hi) >> 1;
                if (a.cu[m] <= r) lo = m;
                else hi = m;
            }
            const int i = r - a.cu[lo];
            const int pi = i / a.c.page;
            const int id = i >= 0 && pi < a.pages_stride ? a.pages[lo * a.pages_stride + pi] : -1;
            if (id < 0 || id >= a.c.n_pages) {
                mla_bad_index(a.err);
                row = -1;
            } else {
                row = gqa_row(a.c, id, h) + (i - pi * a.c.page);
            }
        }
        s_row[threadIdx.x] = row;
    }
    __syncthreads();
    const int ng = D / a.c.gs, per = a.c.gs / 8;
    uint32_t w[kEach];
    float sc[kEach];
#pragma unroll
    for (int k = 0; k < kEach; k++) {
        const int i = threadIdx.x + k * kThreads, u = i % kUnits, r = i / kUnits % kReadRows;
        const bool value = i >= kReadRows * kUnits;
        const long long row = s_row[r];
        w[k] = 0x88888888u;
        sc[k] = 0.f;
        if (row >= 0) {
            w[k] = reinterpret_cast<const uint32_t *>(value ? a.c.v : a.c.k)[row * kUnits + u];
            sc[k] = __bfloat162float((value ? a.c.vs : a.c.ks)[row * ng + u / per]);
        }
    }
#pragma unroll
    for (int k = 0; k < kEach; k++) {
        const int i = threadIdx.x + k * kThreads, u = i % kUnits, r = i / kUnits % kReadRows;
        const bool value = i >= kReadRows * kUnits;
        if (s_row[r] == -2) continue;
        store8<OB>(value ? a.v : a.k, (r0 + r) * (value ? a.v_stride : a.k_stride) + h * D + 8 * u, w[k], sc[k]);
    }
}

template <bool BF16>
cudaError_t append(const GqaAppendArgs &a, cudaStream_t st) {
    const long long rows = 2LL * a.T * a.c.n_kv, per = kThreads / (a.c.dim / 8);
    const dim3 grid((unsigned)((rows + per - 1) / per)), block(kThreads);
    switch (a.c.gs) {
        case 32: return launch_pdl(gqa_append_kernel<BF16, 32>, grid, block, 0, st, a);
        case 64: return launch_pdl(gqa_append_kernel<BF16, 64>, grid, block, 0, st, a);
        default: return launch_pdl(gqa_append_kernel<BF16, 128>, grid, block, 0, st, a);
    }
}

}  // namespace

cudaError_t launch_gqa_append(const GqaAppendArgs &a, bool in_bf16, cudaStream_t st) {
    return in_bf16 ? append<true>(a, st) : append<false>(a, st);
}

cudaError_t launch_gqa_read(const GqaReadArgs &a, bool out_bf16, cudaStream_t st) {
    const dim3 grid((a.T + kReadRows - 1) / kReadRows, a.c.n_kv), block(kThreads);
    if (a.c.dim == 64)
        return out_bf16 ? launch_pdl(gqa_read_kernel<true, 64>, grid, block, 0, st, a)
                        : launch_pdl(gqa_read_kernel<false, 64>, grid, block, 0, st, a);
    return out_bf16 ? launch_pdl(gqa_read_kernel<true, 128>, grid, block, 0, st, a)
                    : launch_pdl(gqa_read_kernel<false, 128>, grid, block, 0, st, a);
}

}  // namespace coli

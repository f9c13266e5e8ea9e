// gqa_cache.cu -- writing keys and values into the paged 4-bit cache and reading
// them back.  Both touch every input and output once.  16384 tokens x 8 heads of 128, gs 32, inputs and outputs rotated through four sets:
// write of f32 25 us (153 MB: 6.1 TB/s, 0.90 of the measured copy rate: HBM), of bf16 25 us, too (86 MB: 3.5 TB/s, 0.51: the issue slots,
// 70 % of them taken, some 17 instructions an element); read to bf16 18 us (4.8 TB/s), to f32 38 (4.1); 48000 tokens to bf16 45 (5.6).
// Short inputs are bound by launch and two memory round trips: 8 tokens, both, 3.3 us on the device.
//
// Group of gs elements: scale = bf16(max|x| / 7), code = clamp(rint(x / scale)).
// Codes are taken against the scale as it is stored, so its rounding to 8 bits
// moves the steps and adds no error of its own.
#include "gqa.cuh"

namespace coli {

namespace {

constexpr int kThreads = 256;

// 8 consecutive elements as they stand in memory.
template <bool BF16>
struct Raw {
    uint4 w[BF16 ? 1 : 2];
    __device__ __forceinline__ void load(const void *base, long long e) {
        const uint4 *at = reinterpret_cast<const uint4 *>(reinterpret_cast<const char *>(base) + e * (BF16 ? 2 : 4));
#pragma unroll
        for (int i = 0; i < (BF16 ? 1 : 2); i++) w[i] = at[i];
    }
    // The values in f32, and the largest magnitude among them as an integer: above infinity for a NaN.
    __device__ __forceinline__ uint32_t values(float (&x)[8]) const {
        uint32_t m = 0;
        if constexpr (BF16) {
            const uint32_t v[4] = {w[0].x, w[0].y, w[0].z, w[0].w};
#pragma unroll
            for (int i = 0; i < 4; i++) {
                const float2 two = bf16x2_f32x2(v[i]);
                x[2 * i] = two.x;
                x[2 * i + 1] = two.y;
                m = __vmaxu2(m, v[i] & 0x7FFF7FFFu);
            }
            return max(m << 16, m & 0xFFFF0000u);
        } else {
            const uint32_t v[8] = {w[0].x, w[0].y, w[0].z, w[0].w, w[1].x, w[1].y, w[1].z, w[1].w};
#pragma unroll
            for (int i = 0; i < 8; i++) {
                x[i] = __uint_as_float(v[i]);
                m = max(m, v[i] & 0x7FFFFFFFu);
            }
            return m;
        }
    }
};

// x / b to nearest from r, the reciprocal of b to nearest, by a step with the exact remainder (Markstein, IBM J. Res. Dev. 1990): 3
// instructions where a division has about 20.  The theorem wants x r within an ulp of the quotient; for b = 7 and every b of 8 bits
// the result was compared with the quotient for all x of seven binades, as far from overflow and underflow as its caller sees to.
__device__ __forceinline__ float divide(float x, float b, float r) {
    const float q = x * r;
    return fmaf(fmaf(-q, b, x), r, q);
}

// 8 elements, of magnitudes up to m, of a group that GS / 8 neighbouring threads have: their codes, and the group's scale.
template <int GS>
__device__ __forceinline__ uint32_t quantise(const float (&x)[8], uint32_t m, __nv_bfloat16 &stored) {
#pragma unroll
    for (int o = 1; o < GS / 8; o <<= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
    const float amax = __uint_as_float(m);
    uint32_t w = 0;
    if (amax >= 1e-30f && m < 0x7F800000u) {
        // max|x| / scale <= 7 (1 + 2^-8): no code needs the clamp.  q + 1.5 2^23 + 8 has rint(q) + 8 in its low bits.
        stored = __float2bfloat16_rn(divide(amax, 7.f, 1.f / 7.f));
        const float b = __bfloat162float(stored), r = __frcp_rn(b);
#pragma unroll
        for (int i = 7; i >= 0; i--) w = 16 * w + __float_as_uint(divide(x[i], b, r) + 12582920.f);
        return w - 0x11111111u * 0x4B400000u;            // the float's own bits, added up as the codes
    }
    if (m >= 0x7F800000u) {
        stored = __float2bfloat16_rn(__uint_as_float(0x7FC00000u));
        return 0x88888888u;
    }
    stored = __float2bfloat16_rn(__fdiv_rn(amax, 7.f));
    const float b = __bfloat162float(stored), by = b > 0.f ? b : 1.f;
#pragma unroll
    for (int i = 7; i >= 0; i--) w = 16 * w + (uint32_t)(__float2int_rn(fminf(fmaxf(__fdiv_rn(x[i], by), -8.f), 7.f)) + 8);
    return w;
}

// One thread per 8 elements of a token's key and of its value; a CTA has tokens of one head, and asks for the next ones before it works
// on those that have come.
template <bool BF16, int D, int GS>
__global__ void __launch_bounds__(kThreads) gqa_append_kernel(const GqaAppendArgs a) {
    constexpr int kUnits = D / 8, kTokens = kThreads / kUnits;
    const int h = blockIdx.y, u = threadIdx.x % kUnits, step = gridDim.x * kTokens;
    int t = blockIdx.x * kTokens + threadIdx.x / kUnits;
    pdl_wait();
    Raw<BF16> k, v;
    long long slot = -1;
    auto load = [&](int t) {
        if (t < a.T) {
            slot = a.slots[t];
            k.load(a.k, t * a.k_stride + h * D + 8 * u);
            v.load(a.v, t * a.v_stride + h * D + 8 * u);
        }
    };
    load(t);
    for (int t0 = blockIdx.x * kTokens; t0 < a.T; t0 += step, t += step) {   // the warp stays together
        float kx[8], vx[8];
        const uint32_t km = k.values(kx), vm = v.values(vx);
        const long long at = t < a.T ? slot : -1;
        if (t0 + step < a.T) load(t + step);
        __nv_bfloat16 ks, vs;
        const uint32_t kw = quantise<GS>(kx, km, ks), vw = quantise<GS>(vx, vm, vs);
        if (at == -1) continue;
        if (at < 0 || at >= (long long)a.c.n_pages * a.c.page) {
            mla_bad_index(a.err);
            continue;
        }
        const int place = (int)at, page = place / a.c.page;   // n_pages * page_size < 2^31, rows too
        const int r = (page * a.c.n_kv + h) * a.c.page + (place - page * a.c.page);
        reinterpret_cast<uint32_t *>(a.c.k)[(long long)r * kUnits + u] = kw;
        reinterpret_cast<uint32_t *>(a.c.v)[(long long)r * kUnits + u] = vw;
        if (u % (GS / 8) == 0) {
            a.c.ks[(long long)r * (D / GS) + u / (GS / 8)] = ks;
            a.c.vs[(long long)r * (D / GS) + u / (GS / 8)] = vs;
        }
        if (u == 0 && a.c.w) a.c.w[r] = 0.f;
    }
    pdl_trigger();
}

// The values of a word of codes.  bf16: 128 + code by an OR, minus 136 exactly, times the scale to nearest: the same as the f32
// product, which is exact, rounded.
template <bool OB>
__device__ __forceinline__ void store8(void *base, long long e, uint32_t w, uint32_t scale) {
    if constexpr (OB) {
        const uint32_t up = w >> 4;
        uint32_t x[4];
#pragma unroll
        for (int i = 0; i < 4; i++) {
            x[i] = (__byte_perm(w, up, (4 + i) << 8 | i) & 0x000F000Fu) | 0x43004300u;   // codes 2 i, 2 i + 1
            asm("sub.rn.bf16x2 %0, %0, %1;\n mul.rn.bf16x2 %0, %0, %2;" : "+r"(x[i]) : "r"(0x43084308u), "r"(scale * 0x10001u));
        }
        *reinterpret_cast<uint4 *>(reinterpret_cast<__nv_bfloat16 *>(base) + e) = make_uint4(x[0], x[1], x[2], x[3]);
    } else {
        float x[8];
#pragma unroll
        for (int i = 0; i < 8; i++) x[i] = (__uint_as_float(0x4B000000u | ((w >> (4 * i)) & 15u)) - 8388616.f) * __uint_as_float(scale << 16);
        float4 *d = reinterpret_cast<float4 *>(reinterpret_cast<float *>(base) + e);
        d[0] = make_float4(x[0], x[1], x[2], x[3]);
        d[1] = make_float4(x[4], x[5], x[6], x[7]);
    }
}

// kReadRows tokens of one head per CTA: as many threads find the tokens' rows, then every thread moves units of 8 elements.  (Every
// thread of a row finding it by itself, without the barrier: slower, 21 us where this takes 16.5.)
constexpr int kReadRows = 32;

template <bool OB, int D>
__global__ void __launch_bounds__(kThreads) gqa_read_kernel(const GqaReadArgs a) {
    constexpr int kUnits = D / 8, kStep = kThreads / kUnits, kEach = kReadRows / kStep;   // a thread's unit, every kStep-th row
    __shared__ int s_row[kReadRows];          // -1: a zero row, -2: not to be written
    const int r0 = blockIdx.x * kReadRows, h = blockIdx.y;
    pdl_wait();
    if (threadIdx.x < kReadRows) {
        const int r = r0 + threadIdx.x;
        int row = -2;
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
                row = (id * a.c.n_kv + h) * a.c.page + (i - pi * a.c.page);
            }
        }
        s_row[threadIdx.x] = row;
    }
    __syncthreads();
    const int u = threadIdx.x % kUnits, r1 = threadIdx.x / kUnits, ng = D / a.c.gs, g = 8 * u / a.c.gs;
    uint32_t kw[kEach], vw[kEach], ks[kEach], vs[kEach];
#pragma unroll
    for (int i = 0; i < kEach; i++) {
        const int row = s_row[r1 + i * kStep];
        kw[i] = vw[i] = 0x88888888u;
        ks[i] = vs[i] = 0;
        if (row >= 0) {
            kw[i] = reinterpret_cast<const uint32_t *>(a.c.k)[(long long)row * kUnits + u];
            vw[i] = reinterpret_cast<const uint32_t *>(a.c.v)[(long long)row * kUnits + u];
            ks[i] = reinterpret_cast<const uint16_t *>(a.c.ks)[(long long)row * ng + g];
            vs[i] = reinterpret_cast<const uint16_t *>(a.c.vs)[(long long)row * ng + g];
        }
    }
#pragma unroll
    for (int i = 0; i < kEach; i++) {
        const int r = r1 + i * kStep;
        if (s_row[r] == -2) continue;
        store8<OB>(a.k, (r0 + r) * a.k_stride + h * D + 8 * u, kw[i], ks[i]);
        store8<OB>(a.v, (r0 + r) * a.v_stride + h * D + 8 * u, vw[i], vs[i]);
    }
    pdl_trigger();
}

template <bool BF16, int D, int GS>
cudaError_t append_by(const GqaAppendArgs &a, int n_sm, cudaStream_t st) {
    constexpr int kTokens = kThreads / (D / 8);
    const int want = (a.T + kTokens - 1) / kTokens, most = (4 * n_sm + a.c.n_kv - 1) / a.c.n_kv;   // 4 CTAs an SM
    return launch_pdl(gqa_append_kernel<BF16, D, GS>, dim3(want < most ? want : most, a.c.n_kv), dim3(kThreads), 0, st, a);
}
template <bool BF16, int D>
cudaError_t append(const GqaAppendArgs &a, int n_sm, cudaStream_t st) {
    if (a.c.gs == 32) return append_by<BF16, D, 32>(a, n_sm, st);
    if (a.c.gs == 64) return append_by<BF16, D, 64>(a, n_sm, st);
    return append_by<BF16, D, D>(a, n_sm, st);           // 128: dim is 128 then
}
template <bool OB, int D>
cudaError_t read(const GqaReadArgs &a, cudaStream_t st) {
    return launch_pdl(gqa_read_kernel<OB, D>, dim3((a.T + kReadRows - 1) / kReadRows, a.c.n_kv), dim3(kThreads), 0, st, a);
}

}  // namespace

cudaError_t launch_gqa_append(const GqaAppendArgs &a, bool in_bf16, int n_sm, cudaStream_t st) {
    if (a.c.dim == 64) return in_bf16 ? append<true, 64>(a, n_sm, st) : append<false, 64>(a, n_sm, st);
    return in_bf16 ? append<true, 128>(a, n_sm, st) : append<false, 128>(a, n_sm, st);
}

cudaError_t launch_gqa_read(const GqaReadArgs &a, bool out_bf16, cudaStream_t st) {
    if (a.c.dim == 64) return out_bf16 ? read<true, 64>(a, st) : read<false, 64>(a, st);
    return out_bf16 ? read<true, 128>(a, st) : read<false, 128>(a, st);
}

}  // namespace coli

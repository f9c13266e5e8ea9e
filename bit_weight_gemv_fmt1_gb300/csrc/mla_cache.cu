// mla_cache.cu -- the memory-bound kernels of the latent attention: the
// queries' split and rotation, the write of new tokens into the paged cache
// (norm, rotation, quantisation) and the read back.  Each touches every input
// and output once, with 16-byte accesses where the types allow, and is bound by
// HBM on long inputs and by launch plus one or two memory round trips on short
// ones.
//
// Rotation: pair (a, b) at angle with (cos, sin) -> (a cos - b sin, a sin + b cos).
#include "mla.cuh"

namespace coli {

namespace {

constexpr int kThreads = 256;

// Store 4 consecutive f32 as f32 or bf16.
template <bool BF16>
__device__ __forceinline__ void store4(void *base, long long e, float4 v) {
    if constexpr (BF16) {
        *reinterpret_cast<uint2 *>(reinterpret_cast<__nv_bfloat16 *>(base) + e) =
            make_uint2(pack_bf16(v.x, v.y), pack_bf16(v.z, v.w));
    } else {
        *reinterpret_cast<float4 *>(reinterpret_cast<float *>(base) + e) = v;
    }
}

__device__ __forceinline__ float2 turn(float a, float b, float c, float s) {
    return make_float2(fmaf(a, c, -(b * s)), fmaf(a, s, b * c));
}

// One thread per unit of 8 query elements: a nope unit is copied, a rope unit
// holds 4 pairs (8 neighbours when interleaved, 4 + 4 elements half a row apart
// otherwise).  Two float4 in, two stores out.  6001 tokens x 64 heads x 192, f32 -> bf16: 75 us, 5.9 TB/s (0.87 of the
// measured copy rate); one token x 128 heads: 2.4 us on the device, its two round trips.
template <bool NB, bool RB>
__global__ void __launch_bounds__(kThreads) mla_query_kernel(const MlaQueryArgs a) {
    const int un = a.nope / 8, upr = un + a.rope / 8, half = a.rope / 2;
    const long long total = (long long)a.T * a.H * upr;
    pdl_wait();
    pdl_trigger();
    for (long long i = (long long)blockIdx.x * kThreads + threadIdx.x; i < total; i += (long long)gridDim.x * kThreads) {
        const long long row = i / upr;
        const int u = (int)(i - row * upr);
        const int t = (int)(row / a.H), h = (int)(row - (long long)t * a.H);
        const float *src = a.q + t * a.q_stride + (long long)h * (a.nope + a.rope);
        if (u < un) {
            const float4 x = *reinterpret_cast<const float4 *>(src + 8 * u);
            const float4 y = *reinterpret_cast<const float4 *>(src + 8 * u + 4);
            store4<NB>(a.out_nope, row * a.ld_nope + 8 * u, x);
            store4<NB>(a.out_nope, row * a.ld_nope + 8 * u + 4, y);
            continue;
        }
        const int k = 4 * (u - un);   // first pair of the unit
        const int p = a.pos[t];
        const bool ok = p >= 0 && p < a.n_pos;
        if (!ok) mla_bad_index(a.err);
        const float *rot = a.rot + (long long)(ok ? p : 0) * a.rope;
        const float z = ok ? 1.f : 0.f;
        float4 c = *reinterpret_cast<const float4 *>(rot + k);
        float4 s = *reinterpret_cast<const float4 *>(rot + half + k);
        src += a.nope;
        const int e0 = a.interleaved ? 2 * k : k, e1 = a.interleaved ? 2 * k + 4 : half + k;
        const float4 x = *reinterpret_cast<const float4 *>(src + e0);
        const float4 y = *reinterpret_cast<const float4 *>(src + e1);
        float4 o0, o1;
        if (a.interleaved) {
            const float2 r0 = turn(x.x, x.y, c.x, s.x), r1 = turn(x.z, x.w, c.y, s.y);
            const float2 r2 = turn(y.x, y.y, c.z, s.z), r3 = turn(y.z, y.w, c.w, s.w);
            o0 = make_float4(r0.x, r0.y, r1.x, r1.y);
            o1 = make_float4(r2.x, r2.y, r3.x, r3.y);
        } else {
            const float2 r0 = turn(x.x, y.x, c.x, s.x), r1 = turn(x.y, y.y, c.y, s.y);
            const float2 r2 = turn(x.z, y.z, c.z, s.z), r3 = turn(x.w, y.w, c.w, s.w);
            o0 = make_float4(r0.x, r1.x, r2.x, r3.x);
            o1 = make_float4(r0.y, r1.y, r2.y, r3.y);
        }
        if (!ok) o0 = o1 = make_float4(z, z, z, z);
        store4<RB>(a.out_rope, row * a.ld_rope + e0, o0);
        store4<RB>(a.out_rope, row * a.ld_rope + e1, o1);
    }
}

__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
    return v;
}

// One warp per token: lane l holds elements 128k + 4l .. +3 of the latent part
// (k < L/128 <= 4) and pair l of the rope part, all loads in flight together; the
// mean square and the largest magnitude are warp reductions in f32.  16384 tokens -> E4M3: 11.4 us, 4.5 TB/s; 65536:
// 47 us, 4.0 TB/s.  A warp waits for two dependent round trips (input, rotation) and then reduces and stores, and 54
// registers hold 9 CTAs, 36 tokens, on an SM: its loads pause meanwhile.
__global__ void __launch_bounds__(128) mla_append_kernel(const MlaAppendArgs a) {
    const int lane = threadIdx.x & 31;
    const int t = blockIdx.x * 4 + (threadIdx.x >> 5);
    pdl_wait();
    pdl_trigger();
    if (t >= a.T) return;
    const int L = a.c.L, R = a.c.R, half = R / 2, nk = L / 128;
    const float *src = a.kv + t * a.kv_stride;
    const bool pair = lane < half;
    const int e0 = a.interleaved ? 2 * lane : lane, e1 = a.interleaved ? 2 * lane + 1 : half + lane;
    // everything that needs no index first: one round trip, then one for the rotation
    const long long slot = a.slots[t];
    const int p = a.pos[t];
    float4 x[4], wn[4];
#pragma unroll
    for (int k = 0; k < 4; k++) {
        x[k] = k < nk ? __ldcs(reinterpret_cast<const float4 *>(src + 128 * k + 4 * lane)) : make_float4(0.f, 0.f, 0.f, 0.f);
        wn[k] = k < nk && a.norm ? *reinterpret_cast<const float4 *>(a.norm + 128 * k + 4 * lane) : make_float4(0.f, 0.f, 0.f, 0.f);
    }
    const float xa = pair ? src[L + e0] : 0.f, xb = pair ? src[L + e1] : 0.f;
    if (slot == -1) return;
    if (slot < -1 || slot >= (long long)a.c.n_pages * a.c.page || p < 0 || p >= a.n_pos) {
        if (lane == 0) mla_bad_index(a.err);
        return;
    }
    const float *rot = a.rot + (long long)p * R;
    const float2 r = pair ? turn(xa, xb, rot[lane], rot[half + lane]) : make_float2(0.f, 0.f);
    if (a.norm) {
        float ss = 0.f;
#pragma unroll
        for (int k = 0; k < 4; k++) ss += x[k].x * x[k].x + x[k].y * x[k].y + x[k].z * x[k].z + x[k].w * x[k].w;
        const float f = rsqrtf(warp_sum(ss) / (float)L + a.eps);
#pragma unroll
        for (int k = 0; k < 4; k++) {
            if (k >= nk) break;
            x[k] = make_float4(x[k].x * f * wn[k].x, x[k].y * f * wn[k].y, x[k].z * f * wn[k].z, x[k].w * f * wn[k].w);
        }
    }
    uint8_t *dst = a.c.rows + slot * a.c.row_bytes;
    if (!a.c.e4m3) {
        __nv_bfloat16 *d = reinterpret_cast<__nv_bfloat16 *>(dst);
#pragma unroll
        for (int k = 0; k < 4; k++)
            if (k < nk) store4<true>(d, 128 * k + 4 * lane, x[k]);
        if (pair) {
            if (a.interleaved) {
                *reinterpret_cast<uint32_t *>(d + L + e0) = pack_bf16(r.x, r.y);
            } else {
                d[L + e0] = __float2bfloat16_rn(r.x);
                d[L + e1] = __float2bfloat16_rn(r.y);
            }
        }
        return;
    }
    float m = fmaxf(fabsf(r.x), fabsf(r.y));
#pragma unroll
    for (int k = 0; k < 4; k++)
        m = fmaxf(fmaxf(fmaxf(m, fabsf(x[k].x)), fmaxf(fabsf(x[k].y), fabsf(x[k].z))), fabsf(x[k].w));
    const float scale = warp_max(m) / 448.f;
    // A row of scale 0 holds zeros, magnitudes that vanish as codes, and NaN, which the maximum passes over: it is divided by
    // 1 (a choice for each element instead costs 0.7 of 12 us).
    const float by = scale > 0.f ? scale : 1.f;
    auto q = [&](float v) { return __fdiv_rn(v, by); };
#pragma unroll
    for (int k = 0; k < 4; k++)
        if (k < nk)
            *reinterpret_cast<uint32_t *>(dst + 128 * k + 4 * lane) =
                pack_e4m3(q(x[k].x), q(x[k].y)) | (pack_e4m3(q(x[k].z), q(x[k].w)) << 16);
    if (pair) {
        const uint32_t two = pack_e4m3(q(r.x), q(r.y));
        if (a.interleaved) {
            *reinterpret_cast<uint16_t *>(dst + L + e0) = (uint16_t)two;
        } else {
            dst[L + e0] = (uint8_t)two;
            dst[L + e1] = (uint8_t)(two >> 8);
        }
    }
    if (lane == 0) a.c.scales[slot] = scale;
}

// 32 rows per CTA: 32 threads find the rows' slots and scales, then every
// thread moves units of 8 elements (8 or 16 bytes in, 16 or 32 out).  7 sequences of up to 20000 rows, bf16 -> bf16: 42 us,
// 5.9 TB/s (0.87 of the measured copy rate).
constexpr int kReadRows = 32;

template <bool E4M3, bool OB>
__global__ void __launch_bounds__(kThreads) mla_read_kernel(const MlaReadArgs a) {
    __shared__ long long s_slot[kReadRows];   // -1: a zero row, -2: not to be written
    __shared__ float s_scale[kReadRows];
    const int r0 = blockIdx.x * kReadRows;
    pdl_wait();
    pdl_trigger();
    if (threadIdx.x < kReadRows) {
        const int r = r0 + threadIdx.x;
        long long slot = -2;
        float sc = 0.f;
        if (r < a.T && r < a.cu[a.n_seq] && r >= a.cu[0]) {
            int lo = 0, hi = a.n_seq;   // cu[lo] <= r < cu[hi]
            while (hi - lo > 1) {
                const int m = (lo + hi) >> 1;
                if (a.cu[m] <= r) lo = m;
                else hi = m;
            }
            const int i = r - a.cu[lo];
            const int pi = i / a.c.page;
            const int id = pi < a.pages_stride ? a.pages[lo * a.pages_stride + pi] : -1;
            if (id < 0 || id >= a.c.n_pages) {
                mla_bad_index(a.err);
                slot = -1;
            } else {
                slot = (long long)id * a.c.page + (i - pi * a.c.page);
                if (E4M3) sc = a.c.scales[slot];
            }
        }
        s_slot[threadIdx.x] = slot;
        s_scale[threadIdx.x] = sc;
    }
    __syncthreads();
    const int upr = (a.c.L + a.c.R) / 8;
    for (int i = threadIdx.x; i < kReadRows * upr; i += kThreads) {
        const int r = i / upr, u = i - r * upr;
        const long long slot = s_slot[r];
        if (slot == -2) continue;
        float4 x = make_float4(0.f, 0.f, 0.f, 0.f), y = x;
        const long long o = (r0 + r) * a.out_stride + 8 * u;
        if (slot >= 0) {
            const uint8_t *src = mla_row(a.c, slot);
            if constexpr (E4M3) {
                const uint2 w = *reinterpret_cast<const uint2 *>(src + 8 * u);
                const float f = s_scale[r];
                auto two = [](uint32_t b) {
                    const uint32_t h = e4m3x2_f16x2(b & 0xFFFFu);
                    return __half22float2(*reinterpret_cast<const __half2 *>(&h));
                };
                const float2 p0 = two(w.x), p1 = two(w.x >> 16), p2 = two(w.y), p3 = two(w.y >> 16);
                x = make_float4(p0.x * f, p0.y * f, p1.x * f, p1.y * f);
                y = make_float4(p2.x * f, p2.y * f, p3.x * f, p3.y * f);
            } else {
                const uint4 w = *reinterpret_cast<const uint4 *>(src + 16 * u);
                if constexpr (OB) {
                    *reinterpret_cast<uint4 *>(reinterpret_cast<__nv_bfloat16 *>(a.out) + o) = w;
                    continue;
                }
                const float2 p0 = bf16x2_f32x2(w.x), p1 = bf16x2_f32x2(w.y), p2 = bf16x2_f32x2(w.z), p3 = bf16x2_f32x2(w.w);
                x = make_float4(p0.x, p0.y, p1.x, p1.y);
                y = make_float4(p2.x, p2.y, p3.x, p3.y);
            }
        }
        if constexpr (OB) {
            *reinterpret_cast<uint4 *>(reinterpret_cast<__nv_bfloat16 *>(a.out) + o) =
                make_uint4(pack_bf16(x.x, x.y), pack_bf16(x.z, x.w), pack_bf16(y.x, y.y), pack_bf16(y.z, y.w));
        } else {
            store4<false>(a.out, o, x);
            store4<false>(a.out, o + 4, y);
        }
    }
}

}  // namespace

cudaError_t launch_mla_query(const MlaQueryArgs &a, bool nope_bf16, bool rope_bf16, int n_sm, cudaStream_t st) {
    const long long units = (long long)a.T * a.H * ((a.nope + a.rope) / 8);
    const long long want = (units + kThreads - 1) / kThreads;
    const dim3 grid((unsigned)(want < 64LL * n_sm ? want : 64LL * n_sm)), block(kThreads);
    if (nope_bf16)
        return rope_bf16 ? launch_pdl(mla_query_kernel<true, true>, grid, block, 0, st, a)
                         : launch_pdl(mla_query_kernel<true, false>, grid, block, 0, st, a);
    return rope_bf16 ? launch_pdl(mla_query_kernel<false, true>, grid, block, 0, st, a)
                     : launch_pdl(mla_query_kernel<false, false>, grid, block, 0, st, a);
}

cudaError_t launch_mla_append(const MlaAppendArgs &a, cudaStream_t st) {
    return launch_pdl(mla_append_kernel, dim3((a.T + 3) / 4), dim3(128), 0, st, a);
}

cudaError_t launch_mla_read(const MlaReadArgs &a, bool out_bf16, cudaStream_t st) {
    const dim3 grid((a.T + kReadRows - 1) / kReadRows), block(kThreads);
    if (a.c.e4m3)
        return out_bf16 ? launch_pdl(mla_read_kernel<true, true>, grid, block, 0, st, a)
                        : launch_pdl(mla_read_kernel<true, false>, grid, block, 0, st, a);
    return out_bf16 ? launch_pdl(mla_read_kernel<false, true>, grid, block, 0, st, a)
                    : launch_pdl(mla_read_kernel<false, false>, grid, block, 0, st, a);
}

}  // namespace coli

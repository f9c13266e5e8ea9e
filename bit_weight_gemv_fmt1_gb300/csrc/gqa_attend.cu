// gqa_attend.cu -- attention of the newest tokens over the paged 4-bit cache, and
// the weights that its rows get.
//
// A unit of work is a tile of 32 cached tokens of one sequence and key / value
// head, for 8 or 16 query rows (n_q tokens x the group's heads).  The units of
// all sequences stand in one row; every CTA takes an equal share of it and walks
// it by segments (the tiles of one sequence, head and set of rows).  A segment's
// tiles go round the CTA's 8 warps, each with a running maximum, sum and output of its own
// and a ring of tiles that bulk copies fill; the warps join at the segment's end.
// A segment that several CTAs have is joined by a second kernel.
//
// Per warp and 16 tokens (mma.sync m16n8k16, tokens or dims as M, query rows as N):
//   S^T = K q^T   codes AND-ed out of the words are f16 subnormals n 2^-24 (odd nibbles
//                 16 times that, q a 16th there); accumulators begin at -8 sum q, one
//                 chain per scale group, whose f32 result takes the scale
//   O^T += V^T P^T  codes OR-ed into bf16 as 128 + n; p times the row's scale rounded to
//                 bf16, transposed in registers; -136 sum P comes from one more product
// so no code is converted one by one and nothing is rounded but q and p * scale.
// Softmax: x = log2(e) scale score, m moves (and O, l with it) only when a tile's
// maximum passes it by 8.
//
// Rows past a length are masked by selection, of scores and of p * scale: their codes are
// always finite numbers, their scales need not be.
// Weights need the final maximum and sum, so a third kernel goes over the keys again: keeping the
// scores instead would need scratch for every token that the page tables could hold.
// Every wait is bounded, by a limit that each segment renews.
#include <algorithm>

#include "encode_tiled.cuh"
#include "gqa.cuh"
#include "tcgen05.cuh"

namespace coli {

namespace {

constexpr int kTile = 32, kWarps = 8, kThreads = 32 * kWarps;
constexpr float kGrow = 8.f;             // log2 of the weight that moves the reference
constexpr float kNone = -3e38f;          // reference of a row that has seen no key

template <int D_, int NG_, int NT_>
struct Shape {
    static constexpr int D = D_, NG = NG_, NT = NT_;    // dims, scale groups of a row, sets of 8 query rows
    static constexpr int kParts = D / 32, kPer = kParts / NG, kRow = D / 2, kRows = 8 * NT;
    static constexpr uint32_t kCodes = kTile * kRow, kScales = kTile * NG * 2;
    static constexpr uint32_t kStage = (2 * kCodes + 2 * kScales + 511) / 512 * 512;
    static constexpr int kCtas = NT == 1 ? 2 : 1;       // on an SM
    static constexpr int kDepth = std::min(8u, (kCtas == 2 ? 110u : 222u) * 1024u / (kWarps * kStage));
    static constexpr uint32_t kSmem = kWarps * kDepth * kStage + 1024;
    static_assert(kDepth * kStage >= kRows * D * 4, "a warp's output fits its ring");
};

struct AttendPlan {
    int n_cta, rg, boxes;                // CTAs, sets of query rows per head, copies per tile (pages of 16, 48, ... tokens: 2)
    float *part;                         // [n_cta][2][kRows][D + 2]: O, m, l
    float2 *stat;                        // [n_seq][n_kv][rg][kRows]: m and 1 / l, for the weights
};

__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_bf16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
    uint32_t y;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}
__device__ __forceinline__ float low_bf16(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float high_bf16(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

__device__ __forceinline__ int length_of(const GqaAttendArgs &a, int b, bool report) {
    const int n = a.lens[b];
    if (n >= 0 && n <= a.pages_stride * a.c.page) return n;
    if (report) mla_bad_index(a.err);
    return 0;
}
__device__ __forceinline__ int tiles_of(const GqaAttendArgs &a, int b) { return (length_of(a, b, false) + kTile - 1) / kTile; }

// The whole CTA: the tiles of the sequences before `upto`.
__device__ __forceinline__ long long tiles_before(const GqaAttendArgs &a, int upto, long long *red) {
    long long n = 0;
    for (int b = threadIdx.x; b < upto; b += blockDim.x) n += tiles_of(a, b);
#pragma unroll
    for (int o = 16; o; o >>= 1) n += __shfl_xor_sync(0xffffffffu, n, o);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = n;
    __syncthreads();
    n = 0;
    for (int w = 0; w < (int)blockDim.x / 32; w++) n += red[w];
    return n;
}
// The whole CTA: the sequence that holds tile x / per (x < tiles of all * per), and the tiles before it.
__device__ __forceinline__ int find_sequence(const GqaAttendArgs &a, long long x, int per, long long &first, long long *red) {
    __shared__ int s_seq;
    __shared__ long long s_first;
    long long run = 0;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    for (int b0 = 0;; b0 += kThreads) {
        const int b = b0 + threadIdx.x;
        const long long n = b < a.n_seq ? tiles_of(a, b) : 0;
        long long incl = n;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long v = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += v;
        }
        __syncthreads();
        if (threadIdx.x == 0) s_seq = -1;
        if (lane == 31) red[warp] = incl;
        __syncthreads();
        long long before = run, all = run;
        for (int w = 0; w < kWarps; w++) {
            if (w < warp) before += red[w];
            all += red[w];
        }
        before += incl - n;
        if (before * per <= x && x < (before + n) * per) {
            s_seq = b;
            s_first = before;
        }
        __syncthreads();
        if (s_seq >= 0 || b0 + kThreads >= a.n_seq) break;
        run = all;
    }
    first = s_first;
    return s_seq;
}

// A warp's query rows as the B operand of the key product, and what its scores need.
template <class S>
struct Query {
    uint32_t q[S::NT][S::kParts][4];     // rows lane / 4, dims 8 (lane % 4) + {0,4}, {1,5}/16, {2,6}, {3,7}/16 of each 32
    float off[S::NT][S::NG][2];          // -8 sum q of rows 2 (lane % 4) + {0, 1}
    float f[S::NT][2];                   // log2(e) * scale * 2^24 / the row's power of two
};

template <class S>
__device__ __forceinline__ void load_query(const GqaAttendArgs &a, int b, int h, int r0, int lane, Query<S> &y) {
    const int G = a.H / a.c.n_kv, n = a.n_q * G, c = lane & 3;
#pragma unroll
    for (int t = 0; t < S::NT; t++) {
        const int row = r0 + 8 * t + (lane >> 2);
        float x[S::kParts][8];
        if (row < n) {
            const int j = row / G;
            const long long e = ((long long)(b * (long long)a.n_q + j) * a.H + h * G + row - j * G) * S::D + 8 * c;
#pragma unroll
            for (int p = 0; p < S::kParts; p++) {
                if (a.q_bf16) {
                    const uint4 w = *reinterpret_cast<const uint4 *>(reinterpret_cast<const __nv_bfloat16 *>(a.q) + e + 32 * p);
                    const uint32_t v[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                    for (int i = 0; i < 4; i++) {
                        x[p][2 * i] = low_bf16(v[i]);
                        x[p][2 * i + 1] = high_bf16(v[i]);
                    }
                } else {
                    const float4 u = *reinterpret_cast<const float4 *>(reinterpret_cast<const float *>(a.q) + e + 32 * p);
                    const float4 v = *reinterpret_cast<const float4 *>(reinterpret_cast<const float *>(a.q) + e + 32 * p + 4);
                    x[p][0] = u.x, x[p][1] = u.y, x[p][2] = u.z, x[p][3] = u.w, x[p][4] = v.x, x[p][5] = v.y, x[p][6] = v.z, x[p][7] = v.w;
                }
            }
        } else {
#pragma unroll
            for (int p = 0; p < S::kParts; p++)
#pragma unroll
                for (int i = 0; i < 8; i++) x[p][i] = 0.f;
        }
        float m = 0.f;
#pragma unroll
        for (int p = 0; p < S::kParts; p++)
#pragma unroll
            for (int i = 0; i < 8; i++) m = fmaxf(m, fabsf(x[p][i]));
        m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
        m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 2));
        int e = 0;                                       // the row times 2^e has its largest magnitude in 2^14 .. 2^15
        if (m > 0.f && m < INFINITY) e = 14 - ilogbf(m);
        float sum[S::NG];
#pragma unroll
        for (int g = 0; g < S::NG; g++) sum[g] = 0.f;
#pragma unroll
        for (int p = 0; p < S::kParts; p++)
#pragma unroll
            for (int i = 0; i < 4; i++) {
                const int odd = i & 1;
                const uint32_t w = pack_f16(ldexpf(x[p][i], e - 4 * odd), ldexpf(x[p][i + 4], e - 4 * odd));
                y.q[t][p][i] = w;
                const float2 back = __half22float2(*reinterpret_cast<const __half2 *>(&w));
                sum[p / S::kPer] += (back.x + back.y) * (odd ? 16.f : 1.f);
            }
        float f = ldexpf(a.scale * 1.4426950408889634f, 24 - e);
#pragma unroll
        for (int g = 0; g < S::NG; g++) {
            sum[g] += __shfl_xor_sync(0xffffffffu, sum[g], 1);
            sum[g] += __shfl_xor_sync(0xffffffffu, sum[g], 2);
            sum[g] *= -8.f / 16777216.f;
        }
#pragma unroll
        for (int i = 0; i < 2; i++) {
            const int src = 4 * (2 * c + i);
            y.f[t][i] = __shfl_sync(0xffffffffu, f, src);
#pragma unroll
            for (int g = 0; g < S::NG; g++) y.off[t][g][i] = __shfl_sync(0xffffffffu, sum[g], src);
        }
    }
}

// Byte of part p of row `key` (whose swizzle bits are x) in a tile of codes.
template <class S>
__device__ __forceinline__ int code_at(int key, int p, int x) {
    return key * S::kRow + ((p ^ x) << 4);
}
// The scales of row `key`.
template <class S>
__device__ __forceinline__ void load_scales(const uint8_t *sm, int key, float (&s)[S::NG]) {
    if constexpr (S::NG == 4) {
        const uint2 w = *reinterpret_cast<const uint2 *>(sm + key * 8);
        s[0] = low_bf16(w.x), s[1] = high_bf16(w.x), s[2] = low_bf16(w.y), s[3] = high_bf16(w.y);
    } else if constexpr (S::NG == 2) {
        const uint32_t w = *reinterpret_cast<const uint32_t *>(sm + key * 4);
        s[0] = low_bf16(w), s[1] = high_bf16(w);
    } else {
        s[0] = low_bf16(*reinterpret_cast<const uint16_t *>(sm + key * 2));
    }
}

// x of the tile's scores: [k][t][i] is token 16 k + lane / 4 + 8 (i / 2) and row 8 t + 2 (lane % 4) + i % 2.
template <class S>
__device__ __forceinline__ void scores(const uint8_t *codes, const uint8_t *scales, const Query<S> &y, int lane, float (&s)[2][S::NT][4]) {
    const int r = lane >> 2, c = lane & 3, x = S::D == 128 ? (r >> 1) & 3 : r >> 2;
#pragma unroll
    for (int k = 0; k < 2; k++) {
        float lo[S::NG], hi[S::NG];
        load_scales<S>(scales, 16 * k + r, lo);
        load_scales<S>(scales, 16 * k + r + 8, hi);
#pragma unroll
        for (int t = 0; t < S::NT; t++)
#pragma unroll
            for (int i = 0; i < 4; i++) s[k][t][i] = 0.f;
#pragma unroll
        for (int g = 0; g < S::NG; g++) {
            float d[S::NT][4];
#pragma unroll
            for (int t = 0; t < S::NT; t++)
#pragma unroll
                for (int i = 0; i < 4; i++) d[t][i] = y.off[t][g][i & 1];
#pragma unroll
            for (int p = g * S::kPer; p < (g + 1) * S::kPer; p++) {
                const uint32_t u = *reinterpret_cast<const uint32_t *>(codes + code_at<S>(16 * k + r, p, x) + 4 * c);
                const uint32_t v = *reinterpret_cast<const uint32_t *>(codes + code_at<S>(16 * k + r + 8, p, x) + 4 * c);
                const uint32_t u8 = u >> 8, v8 = v >> 8;
#pragma unroll
                for (int t = 0; t < S::NT; t++) {
                    mma_f16(d[t], u & 0x000F000Fu, v & 0x000F000Fu, u & 0x00F000F0u, v & 0x00F000F0u, y.q[t][p][0], y.q[t][p][1]);
                    mma_f16(d[t], u8 & 0x000F000Fu, v8 & 0x000F000Fu, u8 & 0x00F000F0u, v8 & 0x00F000F0u, y.q[t][p][2], y.q[t][p][3]);
                }
            }
#pragma unroll
            for (int t = 0; t < S::NT; t++)
#pragma unroll
                for (int i = 0; i < 4; i++) s[k][t][i] = fmaf(d[t][i], i < 2 ? lo[g] : hi[g], s[k][t][i]);
        }
#pragma unroll
        for (int t = 0; t < S::NT; t++)
#pragma unroll
            for (int i = 0; i < 4; i++) s[k][t][i] *= y.f[t][i & 1];
    }
}

// What a warp has added up of a segment: rows 8 t + 2 (lane % 4) + i % 2, dims 32 p + 8 (r % 4) + 4 (r / 4) + {0..3} with r = lane / 4
// ([2 e + i / 2] is dim 2 e + i / 2: m-tile e, its rows r and r + 8).
template <class S>
struct Sums {
    float o[S::NT][S::kParts][2][4], corr[S::NT][S::NG][4], m[S::NT][2], l[S::NT][2];
};

template <class S, bool EDGE>
__device__ __forceinline__ void tile(const GqaAttendArgs &a, const uint8_t *sm, const Query<S> &y, Sums<S> &z, int lane, int r0, int t0, int len) {
    const int r = lane >> 2, c = lane & 3;
    float s[2][S::NT][4];
    scores<S>(sm, sm + 2 * S::kCodes, y, lane, s);
    uint32_t seen = 0xFFFFFFFFu;                         // bit (k * NT + t) * 4 + i
    if constexpr (EDGE) {
        const int G = a.H / a.c.n_kv;
#pragma unroll
        for (int t = 0; t < S::NT; t++)
#pragma unroll
            for (int i = 0; i < 2; i++) {
                const int limit = len - (a.n_q - 1 - (r0 + 8 * t + 2 * c + i) / G);
#pragma unroll
                for (int k = 0; k < 2; k++)
#pragma unroll
                    for (int e = 0; e < 2; e++)
                        if (t0 + 16 * k + r + 8 * e >= min(limit, len)) {
                            s[k][t][2 * e + i] = -INFINITY;
                            seen &= ~(1u << ((k * S::NT + t) * 4 + 2 * e + i));
                        }
            }
    }
    bool move = false;
    float now[S::NT][2];
#pragma unroll
    for (int t = 0; t < S::NT; t++)
#pragma unroll
        for (int i = 0; i < 2; i++) {
            float m = fmaxf(fmaxf(s[0][t][i], s[0][t][2 + i]), fmaxf(s[1][t][i], s[1][t][2 + i]));
            m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 4));
            m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 8));
            m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 16));
            now[t][i] = m;
            move |= m > z.m[t][i] + kGrow;
        }
    if (__any_sync(0xffffffffu, move)) {
#pragma unroll
        for (int t = 0; t < S::NT; t++)
#pragma unroll
            for (int i = 0; i < 2; i++) {
                if (!(now[t][i] > z.m[t][i] + kGrow)) continue;
                const float f = ex2(z.m[t][i] - now[t][i]);
                z.m[t][i] = now[t][i];
                z.l[t][i] *= f;
#pragma unroll
                for (int p = 0; p < S::kParts; p++)
#pragma unroll
                    for (int e = 0; e < 2; e++) z.o[t][p][e][i] *= f, z.o[t][p][e][2 + i] *= f;
#pragma unroll
                for (int g = 0; g < S::NG; g++) z.corr[t][g][i] *= f, z.corr[t][g][2 + i] *= f;
            }
    }
    const uint8_t *codes = sm + S::kCodes, *scales = sm + 2 * S::kCodes + S::kScales;
    const int x = S::D == 128 ? c : c >> 1;
    const uint32_t sel = r >> 2 ? 0x7632u : 0x5410u;
#pragma unroll
    for (int k = 0; k < 2; k++) {
#pragma unroll
        for (int t = 0; t < S::NT; t++)
#pragma unroll
            for (int i = 0; i < 4; i++) {
                const float p = ex2(s[k][t][i] - z.m[t][i & 1]);
                s[k][t][i] = p;
                z.l[t][i & 1] += p;
            }
        float lo[S::NG], hi[S::NG];
        load_scales<S>(scales, 16 * k + r, lo);
        load_scales<S>(scales, 16 * k + r + 8, hi);
        const uint8_t *at = codes + (16 * k + 2 * c) * S::kRow + 4 * (r & 3);
#pragma unroll
        for (int g = 0; g < S::NG; g++) {
            uint32_t b[S::NT][2];
#pragma unroll
            for (int t = 0; t < S::NT; t++) {
                float v[4];
#pragma unroll
                for (int i = 0; i < 4; i++) {
                    v[i] = s[k][t][i] * (i < 2 ? lo[g] : hi[g]);
                    if (EDGE && !(seen >> ((k * S::NT + t) * 4 + i) & 1)) v[i] = 0.f;
                }
                b[t][0] = transpose8(pack_bf16(v[0], v[1]));
                b[t][1] = transpose8(pack_bf16(v[2], v[3]));
                mma_bf16(z.corr[t][g], 0xC308C308u, 0xC308C308u, 0xC308C308u, 0xC308C308u, b[t][0], b[t][1]);
            }
#pragma unroll
            for (int p = g * S::kPer; p < (g + 1) * S::kPer; p++) {
                const int o = (p ^ x) << 4;
                const uint32_t u = __byte_perm(*reinterpret_cast<const uint32_t *>(at + o), *reinterpret_cast<const uint32_t *>(at + S::kRow + o), sel);
                const uint32_t v = __byte_perm(*reinterpret_cast<const uint32_t *>(at + 8 * S::kRow + o),
                                               *reinterpret_cast<const uint32_t *>(at + 9 * S::kRow + o), sel);
                uint32_t n[2][4];
#pragma unroll
                for (int i = 0; i < 4; i++) {
                    n[0][i] = ((u >> (4 * i)) & 0x000F000Fu) | 0x43004300u;
                    n[1][i] = ((v >> (4 * i)) & 0x000F000Fu) | 0x43004300u;
                }
#pragma unroll
                for (int t = 0; t < S::NT; t++)
#pragma unroll
                    for (int e = 0; e < 2; e++)
                        mma_bf16(z.o[t][p][e], n[0][2 * e], n[0][2 * e + 1], n[1][2 * e], n[1][2 * e + 1], b[t][0], b[t][1]);
            }
        }
    }
}

template <class S, bool WEIGH>
__global__ void __launch_bounds__(kThreads, S::kCtas)
    gqa_attend_kernel(const __grid_constant__ CUtensorMap k_map, const __grid_constant__ CUtensorMap v_map, const GqaAttendArgs a,
                      const AttendPlan plan, long long wait_ns) {
    extern __shared__ uint8_t raw[];
    __shared__ uint64_t full[kWarps][S::kDepth];
    __shared__ long long red[kWarps];
    __shared__ float2 ml[kWarps][S::kRows];
    __shared__ int s_abort;
    uint8_t *base = raw + (((smem_addr(raw) + 1023u) & ~1023u) - smem_addr(raw));
    const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
    uint8_t *ring = base + warp * S::kDepth * S::kStage;
    if (lane == 0)
        for (int i = 0; i < S::kDepth; i++) mbar_init(&full[warp][i], 1);
    if (tid == 0) s_abort = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    pdl_wait();
    pdl_trigger();
    __syncthreads();
    volatile int *abort = &s_abort;
    const int n_kv = a.c.n_kv, G = a.H / n_kv, n_rows = a.n_q * G;
    const int per = WEIGH ? n_kv : n_kv * plan.rg;       // segments of a sequence
    const long long units = tiles_before(a, a.n_seq, red) * per;
    if (blockIdx.x == 0)
        for (int b = tid; b < a.n_seq; b += kThreads) length_of(a, b, !WEIGH);
    const long long n_cta = min((long long)gridDim.x, units);   // every one of them has a unit
    if (blockIdx.x >= n_cta) return;
    const long long u1 = units * (blockIdx.x + 1) / n_cta;
    long long u = units * blockIdx.x / n_cta;
    long long first;
    int b = find_sequence(a, u, per, first, red);
    int slot = 0, par = 0;                               // next stage to be read, parity of its use
    bool ok = true;
    while (u < u1) {
        const int len = length_of(a, b, false), nt = (len + kTile - 1) / kTile;
        const long long at = u - first * per;
        const int seg = (int)(at / nt), t0 = (int)(at - (long long)seg * nt), t1 = (int)min((long long)nt, t0 + (u1 - u));
        const int h = WEIGH ? seg : seg / plan.rg;
        const int32_t *pages = a.pages + b * a.pages_stride;
        const int mine = (t1 - t0 - warp + kWarps - 1) / kWarps;   // tiles t0 + warp, t0 + warp + 8, ...
        const uint64_t deadline = deadline_after(wait_ns, max(mine, 0));
        for (int set = WEIGH ? 0 : seg - h * plan.rg, sets = WEIGH ? plan.rg : set + 1; set < sets; set++) {
            const int r0 = set * S::kRows;
            // copies: lane i holds the page of the i-th box from `base_tile` on
            int ids = 0, base_tile = 0;
            const int per_load = 32 / plan.boxes;
            auto look_up = [&](int i) {                  // whole warp, tiles i, i + 1, ... of this warp
                base_tile = i;
                const int t = t0 + warp + kWarps * (i + lane / plan.boxes), tok = t * kTile + (plan.boxes == 2 ? 16 * (lane & 1) : 0);
                ids = 0;
                if (tok < len && i + lane / plan.boxes < mine) {
                    ids = pages[tok / a.c.page];
                    if (ids < 0 || ids >= a.c.n_pages) {
                        mla_bad_index(a.err);
                        ids = 0;                         // that page's rows: the output is unspecified
                    }
                }
            };
            auto ask = [&](int i, int stage) {           // whole warp
                if (i - base_tile >= per_load) look_up(i);
                const int tok = (t0 + warp + kWarps * i) * kTile;
                const uint32_t dst = smem_addr(ring + stage * S::kStage);
                uint64_t *bar = &full[warp][stage];
                const int n = plan.boxes == 1 || tok + 16 < len ? plan.boxes : 1, rows = kTile / plan.boxes;
                expect_bytes(bar, (uint32_t)(n * rows) * (WEIGH ? S::kRow + S::NG * 2 : 2 * (S::kRow + S::NG * 2)));
                for (int k = 0; k < n; k++) {
                    const int id = __shfl_sync(0xffffffffu, ids, (i - base_tile) * plan.boxes + k);
                    const long long row = gqa_row(a.c, id, h) + (tok + 16 * k) % a.c.page;
                    const uint32_t o = dst + k * 16 * S::kRow, so = dst + 2 * S::kCodes + k * 16 * S::NG * 2;
                    tma_box(o, &k_map, 0, (int)row, bar);
                    bulk_copy(so, a.c.ks + row * S::NG, rows * S::NG * 2, bar);
                    if (!WEIGH) {
                        tma_box(o + S::kCodes, &v_map, 0, (int)row, bar);
                        bulk_copy(so + S::kScales, a.c.vs + row * S::NG, rows * S::NG * 2, bar);
                    }
                }
            };
            if (mine > 0) look_up(0);
            for (int i = 0; i < S::kDepth && i < mine; i++) {
                int st = slot + i;
                if (st >= S::kDepth) st -= S::kDepth;
                ask(i, st);
            }
            Query<S> y;
            load_query<S>(a, b, h, r0, lane, y);
            Sums<S> z;
            float2 stat[S::NT][2];
            if constexpr (WEIGH) {
#pragma unroll
                for (int t = 0; t < S::NT; t++)
#pragma unroll
                    for (int i = 0; i < 2; i++)
                        stat[t][i] = plan.stat[((long long)(b * (long long)n_kv + h) * plan.rg + set) * S::kRows + 8 * t + 2 * (lane & 3) + i];
            } else {
#pragma unroll
                for (int t = 0; t < S::NT; t++) {
#pragma unroll
                    for (int i = 0; i < 2; i++) z.m[t][i] = kNone, z.l[t][i] = 0.f;
#pragma unroll
                    for (int i = 0; i < 4; i++) {
#pragma unroll
                        for (int p = 0; p < S::kParts; p++) z.o[t][p][0][i] = z.o[t][p][1][i] = 0.f;
#pragma unroll
                        for (int g = 0; g < S::NG; g++) z.corr[t][g][i] = 0.f;
                    }
                }
            }
            for (int i = 0; i < mine; i++) {
                if (ok && !warp_wait_now(&full[warp][slot], par, deadline, abort, lane)) {
                    ok = false;
                    *abort = 1;
                    atomicCAS(a.err, 0, (int)DEV_ERR_TIMEOUT);
                }
                if (!ok) break;
                const uint8_t *sm = ring + slot * S::kStage;
                const int tok = (t0 + warp + kWarps * i) * kTile;
                const bool edge = tok + kTile > len - (a.n_q - 1);
                if constexpr (WEIGH) {
                    float s[2][S::NT][4];
                    scores<S>(sm, sm + 2 * S::kCodes, y, lane, s);
#pragma unroll
                    for (int k = 0; k < 2; k++)
#pragma unroll
                        for (int e = 0; e < 2; e++) {
                            const int t = tok + 16 * k + (lane >> 2) + 8 * e;
                            float w = 0.f;
#pragma unroll
                            for (int n = 0; n < S::NT; n++)
#pragma unroll
                                for (int i = 0; i < 2; i++) {
                                    const int row = r0 + 8 * n + 2 * (lane & 3) + i;
                                    if (row < n_rows && t < len - (a.n_q - 1 - row / G))
                                        w += ex2(s[k][n][2 * e + i] - stat[n][i].x) * stat[n][i].y;
                                }
                            w += __shfl_xor_sync(0xffffffffu, w, 1);
                            w += __shfl_xor_sync(0xffffffffu, w, 2);
                            if ((lane & 3) == 0 && t < len) {
                                const int page = pages[t / a.c.page];
                                if (page >= 0 && page < a.c.n_pages) atomicAdd(a.c.w + gqa_row(a.c, page, h) + t % a.c.page, w);
                            }
                        }
                } else if (edge) {
                    tile<S, true>(a, sm, y, z, lane, r0, tok, len);
                } else {
                    tile<S, false>(a, sm, y, z, lane, r0, tok, len);
                }
                __syncwarp();
                if (i + S::kDepth < mine) ask(i + S::kDepth, slot);
                if (++slot == S::kDepth) {
                    slot = 0;
                    par ^= 1;
                }
            }
            if constexpr (!WEIGH) {
                // ------------------------------------------------------ the warps' sums become the segment's
#pragma unroll
                for (int t = 0; t < S::NT; t++)
#pragma unroll
                    for (int i = 0; i < 2; i++) {
                        float l = z.l[t][i];
                        l += __shfl_xor_sync(0xffffffffu, l, 4);
                        l += __shfl_xor_sync(0xffffffffu, l, 8);
                        l += __shfl_xor_sync(0xffffffffu, l, 16);
                        if (lane < 4) ml[warp][8 * t + 2 * lane + i] = make_float2(z.m[t][i], l);
                    }
                __syncthreads();
                float *mine_o = reinterpret_cast<float *>(ring);
#pragma unroll
                for (int t = 0; t < S::NT; t++)
#pragma unroll
                    for (int i = 0; i < 2; i++) {
                        const int row = 8 * t + 2 * (lane & 3) + i;
                        float m = ml[0][row].x;
#pragma unroll
                        for (int w = 1; w < kWarps; w++) m = fmaxf(m, ml[w][row].x);
                        const float f = ex2(z.m[t][i] - m);
#pragma unroll
                        for (int p = 0; p < S::kParts; p++) {
                            const float *cr = z.corr[t][p / S::kPer];
                            const int r = lane >> 2;
                            *reinterpret_cast<float4 *>(mine_o + row * S::D + 32 * p + 8 * (r & 3) + 4 * (r >> 2)) =
                                make_float4((z.o[t][p][0][i] + cr[i]) * f, (z.o[t][p][0][2 + i] + cr[2 + i]) * f,
                                            (z.o[t][p][1][i] + cr[i]) * f, (z.o[t][p][1][2 + i] + cr[2 + i]) * f);
                        }
                    }
                __syncthreads();
                const bool whole = t0 == 0 && t1 == nt;
                float *part = plan.part + ((long long)blockIdx.x * 2 + (t0 == 0)) * S::kRows * (S::D + 2);
                for (int i = tid; i < S::kRows * (S::D / 4); i += kThreads) {
                    const int row = i / (S::D / 4), d = 4 * (i % (S::D / 4));
                    float m = ml[0][row].x, l = 0.f;
#pragma unroll
                    for (int w = 1; w < kWarps; w++) m = fmaxf(m, ml[w][row].x);
#pragma unroll
                    for (int w = 0; w < kWarps; w++) l += ml[w][row].y * ex2(ml[w][row].x - m);
                    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                    for (int w = 0; w < kWarps; w++) {
                        const float4 x = *reinterpret_cast<const float4 *>(base + w * S::kDepth * S::kStage + (row * S::D + d) * 4);
                        o.x += x.x, o.y += x.y, o.z += x.z, o.w += x.w;
                    }
                    if (!whole) {
                        *reinterpret_cast<float4 *>(part + row * S::D + d) = o;
                        if (d == 0) *reinterpret_cast<float2 *>(part + S::kRows * S::D + 2 * row) = make_float2(m, l);
                        continue;
                    }
                    const int at = r0 + row;
                    if (at >= n_rows) continue;
                    const float inv = l != 0.f ? 1.f / l : 0.f;
                    const long long orow = (long long)(b * (long long)a.n_q + at / G) * a.H + h * G + at % G;
                    if (a.out_bf16)
                        *reinterpret_cast<uint2 *>(reinterpret_cast<__nv_bfloat16 *>(a.out) + orow * S::D + d) =
                            make_uint2(pack_bf16(o.x * inv, o.y * inv), pack_bf16(o.z * inv, o.w * inv));
                    else
                        *reinterpret_cast<float4 *>(reinterpret_cast<float *>(a.out) + orow * S::D + d) =
                            make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv);
                    if (d == 0 && a.lse) a.lse[orow] = l != 0.f ? (m + log2f(l)) * 0.6931471805599453f : -INFINITY;
                    if (d == 0 && a.weigh)
                        plan.stat[((long long)(b * (long long)n_kv + h) * plan.rg + set) * S::kRows + row] = make_float2(m, inv);
                }
                fence_async_smem();
                __syncthreads();
                ok = ok && !*abort;
            }
        }
        u += t1 - t0;
        if (u < u1 && at + (t1 - t0) == (long long)nt * per) {
            first += nt;
            do b++;
            while (tiles_of(a, b) == 0);
        }
        if (!ok) break;
    }
    if (*abort) settle();
}

// One CTA per segment: joins the parts of one that several CTAs had, fills one without tokens.
template <class S>
__global__ void __launch_bounds__(kThreads) gqa_join_kernel(const GqaAttendArgs a, const AttendPlan plan) {
    __shared__ long long red[kWarps];
    const int n_kv = a.c.n_kv, G = a.H / n_kv, n_rows = a.n_q * G, per = n_kv * plan.rg;
    const int b = blockIdx.x / per, seg = blockIdx.x - b * per, h = seg / plan.rg, set = seg - h * plan.rg;
    pdl_wait();
    pdl_trigger();
    const int nt = tiles_of(a, b);
    const long long units = tiles_before(a, a.n_seq, red) * per;
    const long long u0 = tiles_before(a, b, red) * per + (long long)seg * nt;
    int c0 = 0, c1 = -1;
    if (nt > 0) {
        // the CTA of unit u is the largest c with units * c / n <= u, of the n that have units
        const long long n = min((long long)plan.n_cta, units);
        c0 = (int)(((u0 + 1) * n - 1) / units);
        c1 = (int)(((u0 + nt) * n - 1) / units);
        if (c0 == c1) return;
    }
    constexpr int kPart = S::kRows * (S::D + 2);
    for (int i = threadIdx.x; i < S::kRows * (S::D / 4); i += kThreads) {
        const int row = i / (S::D / 4), d = 4 * (i % (S::D / 4)), at = set * S::kRows + row;
        if (at >= n_rows) continue;
        float m = kNone, l = 0.f;
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int c = c0; c <= c1; c++) {
            const float *part = plan.part + ((long long)c * 2 + (c == c0)) * kPart;
            const float2 ml = *reinterpret_cast<const float2 *>(part + S::kRows * S::D + 2 * row);
            const float4 x = *reinterpret_cast<const float4 *>(part + row * S::D + d);
            const float now = fmaxf(m, ml.x), f = ex2(m - now), g = ex2(ml.x - now);
            m = now;
            l = l * f + ml.y * g;
            o = make_float4(o.x * f + x.x * g, o.y * f + x.y * g, o.z * f + x.z * g, o.w * f + x.w * g);
        }
        const float inv = l != 0.f ? 1.f / l : 0.f;
        const long long orow = (long long)(b * (long long)a.n_q + at / G) * a.H + h * G + at % G;
        if (a.out_bf16)
            *reinterpret_cast<uint2 *>(reinterpret_cast<__nv_bfloat16 *>(a.out) + orow * S::D + d) =
                make_uint2(pack_bf16(o.x * inv, o.y * inv), pack_bf16(o.z * inv, o.w * inv));
        else
            *reinterpret_cast<float4 *>(reinterpret_cast<float *>(a.out) + orow * S::D + d) = make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv);
        if (d == 0 && a.lse) a.lse[orow] = l != 0.f ? (m + log2f(l)) * 0.6931471805599453f : -INFINITY;
        if (d == 0 && a.weigh) plan.stat[(long long)blockIdx.x * S::kRows + row] = make_float2(m, inv);
    }
}

// Rows of `bytes` codes; boxes of box_rows of them, swizzled by their length.
cudaError_t code_map(const void *p, int bytes, long long rows, int box_rows, CUtensorMap *out) {
    const PFN_cuTensorMapEncodeTiled_v12000 fn = encode_tiled();
    if (!fn) return cudaErrorNotSupported;
    const cuuint64_t dims[2] = {(cuuint64_t)bytes, (cuuint64_t)rows}, strides[1] = {(cuuint64_t)bytes};
    const cuuint32_t box[2] = {(cuuint32_t)bytes, (cuuint32_t)box_rows}, estr[2] = {1, 1};
    return fn(out, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void *>(p), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
              bytes == 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_32B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS
               ? cudaSuccess
               : cudaErrorInvalidValue;
}

size_t round256(size_t n) { return (n + 255) / 256 * 256; }

// Sets of 8 query rows that a CTA has: 2 where the group's rows need them.
int sets_of(const GqaAttendArgs &a) { return (long long)a.n_q * (a.H / a.c.n_kv) > 8 ? 2 : 1; }
int row_groups(const GqaAttendArgs &a) {
    const int rows = a.n_q * (a.H / a.c.n_kv), each = 8 * sets_of(a);
    return (rows + each - 1) / each;
}
// CTAs: all that fit, no more than units that the page tables could hold.
int grid_of(const GqaAttendArgs &a, int n_sm, int ctas) {
    const double most = (double)a.n_seq * (a.pages_stride * a.c.page / kTile + 1) * a.c.n_kv * row_groups(a);
    return (int)std::min((double)(ctas * n_sm), most);
}
size_t part_bytes(const GqaAttendArgs &a, int n_cta) {
    return round256((size_t)n_cta * 2 * 8 * sets_of(a) * (a.c.dim + 2) * sizeof(float));
}

template <class S>
cudaError_t run(const GqaAttendArgs &a, const DevInfo &d, cudaStream_t st, int *n_launch) {
    AttendPlan plan;
    plan.rg = row_groups(a);
    plan.boxes = a.c.page % kTile ? 2 : 1;
    plan.n_cta = grid_of(a, d.n_sm, S::kCtas);
    plan.part = (float *)d.scratch;
    plan.stat = (float2 *)((char *)d.scratch + part_bytes(a, plan.n_cta));
    CUtensorMap k, v;
    const long long rows = (long long)a.c.n_pages * a.c.n_kv * a.c.page;
    if (cudaError_t e = code_map(a.c.k, S::kRow, rows, kTile / plan.boxes, &k)) return e;
    if (cudaError_t e = code_map(a.c.v, S::kRow, rows, kTile / plan.boxes, &v)) return e;
    static std::atomic<uint64_t> done{0}, done_weigh{0};
    if (cudaError_t e = allow_smem(gqa_attend_kernel<S, false>, S::kSmem, d.device, done)) return e;
    if (cudaError_t e = launch_pdl(gqa_attend_kernel<S, false>, dim3(plan.n_cta), dim3(kThreads), S::kSmem, st, k, v, a, plan, d.wait_ns)) return e;
    *n_launch = 2;
    if (cudaError_t e = launch_pdl(gqa_join_kernel<S>, dim3((unsigned)a.n_seq * a.c.n_kv * plan.rg), dim3(kThreads), 0, st, a, plan)) return e;
    if (!a.weigh) return cudaSuccess;
    *n_launch = 3;
    if (cudaError_t e = allow_smem(gqa_attend_kernel<S, true>, S::kSmem, d.device, done_weigh)) return e;
    return launch_pdl(gqa_attend_kernel<S, true>, dim3(plan.n_cta), dim3(kThreads), S::kSmem, st, k, v, a, plan, d.wait_ns);
}

template <int D, int NG>
cudaError_t by_rows(const GqaAttendArgs &a, const DevInfo &d, cudaStream_t st, int *n_launch) {
    return sets_of(a) == 1 ? run<Shape<D, NG, 1>>(a, d, st, n_launch) : run<Shape<D, NG, 2>>(a, d, st, n_launch);
}

}  // namespace

size_t gqa_attend_scratch(const GqaAttendArgs &a, int n_sm) {
    const int n_cta = grid_of(a, n_sm, sets_of(a) == 1 ? 2 : 1);
    return part_bytes(a, n_cta) + (a.weigh ? (size_t)a.n_seq * a.c.n_kv * row_groups(a) * 8 * sets_of(a) * sizeof(float2) : 0);
}

cudaError_t launch_gqa_attend(const GqaAttendArgs &a, const DevInfo &d, cudaStream_t st, int *n_launch) {
    switch (a.c.dim * 8 + a.c.dim / a.c.gs) {
        case 64 * 8 + 1: return by_rows<64, 1>(a, d, st, n_launch);
        case 64 * 8 + 2: return by_rows<64, 2>(a, d, st, n_launch);
        case 128 * 8 + 1: return by_rows<128, 1>(a, d, st, n_launch);
        case 128 * 8 + 2: return by_rows<128, 2>(a, d, st, n_launch);
        default: return by_rows<128, 4>(a, d, st, n_launch);
    }
}

}  // namespace coli

// gqa_attend.cu -- attention of the newest tokens over the paged 4-bit cache, and
// the weights that its rows get.
//
// A unit of work is a tile of 32 cached tokens of one sequence and key / value head, for 8 query rows (n_q tokens x the
// group's heads).  A segment is the tiles of one sequence, head and set of rows; CTAs have a piece of one each, or, where segments
// are many, an equal share of all units in a row, which they walk by segments.  A segment's tiles go round the CTA's 8 warps, each
// with a running maximum, sum and output of its own and a ring of tiles that bulk copies fill; the warps join at the
// segment's end.  A segment that several CTAs have is joined by a second kernel.  Short calls (cluster_of) have a cluster of 8, 4, 2 or
// 1 CTAs for each segment instead, which hand one another their sums through shared memory: one kernel in all.
//
// Per warp and 16 tokens (mma.sync m16n8k16, tokens or dims as M, query rows as N):
//   S^T = K q^T   codes AND-ed out of the words are f16 subnormals n 2^-24 (odd nibbles
//                 16 times that, q a 16th there); accumulators begin at -8 sum q, one
//                 chain per scale group, whose f32 result takes the scale
//   O^T += V^T P^T  codes AND-ed out are bf16 subnormals n 2^-133 (odd nibbles 16 times that, taken back at the end); p times
//                 2^80 rounded to bf16, transposed in registers, its product with the row's scale rounded to bf16; -8 sum P comes from
//                 one more product.  2^80 keeps products and sums within f32 for scales from 2^-60 to 2^38.  (Codes as
//                 128 + n need an OR and two more shifts a word: 48x12000 3 us more.)
// so no code is converted one by one.  ldmatrix, transposing for the values, deals the words out as the products want them:
// its 16-bit elements are 4 codes of one token.  N = 8 is what few query rows need; 5th-generation products would want the codes
// as bytes in shared memory, M = 128 tokens, and N = 8 as well.
// Softmax: x = log2(e) scale score, m moves (and O, l with it) only when a tile's
// maximum passes it by 8.
//
// Rows past a length are masked by selection, of scores and of p * scale: their codes are
// always finite numbers, their scales need not be.
// Weights need the final maximum and sum, so a third kernel goes over the keys again: keeping the
// scores instead would need scratch for every token that the page tables could hold.
// Every wait is bounded, by a limit that each segment and set of rows renews.
//
// Bound: HBM once a call is long.  A tile takes 480 instructions of a warp, 215 of them ANDs, shifts and the like on the ALU pipe (430
// cycles of a quarter of an SM, which HBM gives a tile in 790); measured, 100000 more tokens of 8 heads, gs 32, take 17 us,
// 6.7 TB/s.  Some 14 us of a call that fills the GPU are start (lengths, pages, first copies), last tiles and join: 48x12000 (64 heads on
// 8) 80.9 us = 4.6 TB/s, 1x100000 (32 on 8, gs 128) 28.6, 4x9000 of 3 tokens (28 on 4) 18.4, 16x8000 with weights 49; 1x1000, a cluster a head, 7.2.
// 16 warps an SM with 128 registers each; 12 with 168 or 20 with 96 are 14 to 17 % slower.
#include <algorithm>

#include "encode_tiled.cuh"
#include "gqa.cuh"
#include "tcgen05.cuh"

namespace coli {

namespace {

constexpr int kTile = 32, kWarps = 8, kThreads = 32 * kWarps;
constexpr int kJoin = 256, kGroup = 64;  // threads of the join, parts at a time
constexpr float kGrow = 8.f;             // log2 of the weight that moves the reference
constexpr float kUp = 80.f, kScale = 0x1p80f;   // log2 of what p is held times, and that: references are lower by it
constexpr float kDown = 0x1p53f;         // codes' 2^133 without it: outputs without factors
constexpr float kNone = -3e38f;          // reference of a row that has seen no key
constexpr int kRows = 8;                 // query rows of a unit: N of the products
constexpr int kRounds = 4;               // tiles of a warp, at the most that page tables could hold, for which clusters are taken

template <int D_, int NG_>
struct Shape {
    static constexpr int D = D_, NG = NG_;              // dims, scale groups of a row
    static constexpr int kParts = D / 32, kPer = kParts / NG, kRow = D / 2;
    static constexpr uint32_t kCodes = kTile * kRow, kScales = kTile * NG * 2;
};
// A warp's ring of tiles: keys' codes, values' codes, keys' scales, values' scales; the keys' alone for the weights.
template <class S, bool WEIGH>
struct Ring {
    static constexpr uint32_t kScaleAt = (WEIGH ? 1 : 2) * S::kCodes;
    static constexpr uint32_t kStage = (kScaleAt + (WEIGH ? 1 : 2) * S::kScales + 511) / 512 * 512;
    // Two CTAs on an SM, 74 KB each for 128 dims: what the rings hold when the last copies have come is worked on with HBM idle (3 tiles a
    // warp: 48x12000 84.2 us, 2: 82.4).
    static constexpr int kDepth = WEIGH ? 4 : 2;
    static constexpr uint32_t kSmem = kWarps * kDepth * kStage + 1024;
    static_assert(WEIGH || kDepth * kStage >= kRows * S::D * 4, "a warp's output fits its ring");
};

struct AttendPlan {
    int n_cta, rg, boxes;                // CTAs, sets of query rows per head, copies per tile (pages of 16, 48, ... tokens: 2)
    int cluster;                         // CTAs of a cluster, which share a segment; 0: no clusters
    float *part;                         // [n_cta][2][kRows][D + 2]: O, m, l
    float2 *stat;                        // [n_seq][n_kv][rg][kRows]: m and 1 / l without 2^80, for the weights: exponents near 80 would
                                         // be rounded to 2^-18, 1e-6 of a weight
    long long *before;                   // [n_seq + 2]: tiles (or pieces) of the sequences before each and of all, tiles of a piece
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
// Four 8 x 8 matrices of 16-bit elements, rows of 16 bytes at the addresses of lanes 0-7, 8-15, ...: of each a thread gets elements
// 2 (lane % 4) and the next of row lane / 4, or (transposed) of column lane / 4.
__device__ __forceinline__ void load_matrices(uint32_t at, uint32_t (&x)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];" : "=r"(x[0]), "=r"(x[1]), "=r"(x[2]), "=r"(x[3]) : "r"(at));
}
__device__ __forceinline__ void load_matrices_t(uint32_t at, uint32_t (&x)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];" : "=r"(x[0]), "=r"(x[1]), "=r"(x[2]), "=r"(x[3]) : "r"(at));
}
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
    uint32_t y;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}
// Two bf16 products, to nearest.
__device__ __forceinline__ uint32_t mul_bf16(uint32_t a, uint32_t b) {
    uint32_t c;
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(c) : "r"(a), "r"(b));
    return c;
}
// Fills a stage, or the second half of one: a box of either codes and their scales, counted on `bar`, which the first call tells
// of all the bytes.  Whole warp, uniform arguments, one thread issues.
template <bool VALUES, bool FIRST>
__device__ __forceinline__ void fill(uint32_t dst, uint32_t v_off, uint32_t scales, uint32_t vs_off, const CUtensorMap *k, const CUtensorMap *v, int row,
                                     const void *ks, const void *vs, uint32_t scale_bytes, uint64_t *bar, uint32_t bytes) {
    if constexpr (FIRST) expect_bytes(bar, bytes);
    if constexpr (VALUES)
        asm volatile(
            "{\n .reg .pred q;\n .reg .b32 z;\n mov.b32 z, 0;\n elect.sync _|q, 0xffffffff;\n"
            " @q cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes [%1], [%3, {z, %5}], [%0];\n"
            " @q cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%6], [%8], %10, [%0];\n"
            " @q cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes [%2], [%4, {z, %5}], [%0];\n"
            " @q cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%7], [%9], %10, [%0];\n}\n" ::"r"(smem_addr(bar)),
            "r"(dst), "r"(dst + v_off), "l"(k), "l"(v), "r"(row), "r"(scales), "r"(scales + vs_off), "l"(ks), "l"(vs), "r"(scale_bytes)
            : "memory");
    else
        asm volatile(
            "{\n .reg .pred q;\n .reg .b32 z;\n mov.b32 z, 0;\n elect.sync _|q, 0xffffffff;\n"
            " @q cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes [%1], [%2, {z, %3}], [%0];\n"
            " @q cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%4], [%5], %6, [%0];\n}\n" ::"r"(smem_addr(bar)),
            "r"(dst), "l"(k), "r"(row), "r"(scales), "l"(ks), "r"(scale_bytes)
            : "memory");
}
__device__ __forceinline__ float low_bf16(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float high_bf16(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

__device__ __forceinline__ int length_of(const GqaAttendArgs &a, int b, bool report) {
    const int n = a.lens[b];
    if (n >= 0 && n <= a.longest) return n;
    if (report) mla_bad_index(a.err);
    return 0;
}
__device__ __forceinline__ int tiles_of(const GqaAttendArgs &a, int b) { return (length_of(a, b, false) + kTile - 1) / kTile; }

// A CTA's work.
struct Share {
    int piece;                           // tiles of a piece at most; 0: a share of the row of units
    long long u, u1;                     // the CTA's units, or its own number
    long long first;                     // units (or pieces) of the sequences before `seq`, by segment
    int seq;                             // -1: no work
};
// The whole CTA: how the tiles of all sequences, `per` segments each, are dealt out.
// Pieces: every segment is cut into pieces of at most 8 r tiles, r for each warp, a CTA each.  r is the rounds of an even
// share, or up to 2 more: what a CTA pays whose share spans two segments (look-ups, first copies, two joins: 3 to 4 us, a round takes
// 1.7).  Where no such pieces fit the grid, every CTA has an even share of the units in a row.
// The first CTA writes `before`, if there is one: the sums, and `piece`.
__device__ __forceinline__ Share find_share(const GqaAttendArgs &a, int per, long long *before) {
    __shared__ long long sums[kWarps];
    __shared__ int counts[kWarps][3];
    __shared__ long long s_first;
    __shared__ int s_seq;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int mine = tid < a.n_seq ? tiles_of(a, tid) : 0;
    long long n = mine;
    for (int b = tid + kThreads; b < a.n_seq; b += kThreads) n += tiles_of(a, b);
#pragma unroll
    for (int o = 16; o; o >>= 1) n += __shfl_xor_sync(0xffffffffu, n, o);
    if (tid == 0) s_seq = -1;
    if (lane == 0) sums[warp] = n;
    __syncthreads();
    long long tiles = 0;
    for (int w = 0; w < kWarps; w++) tiles += sums[w];
    const long long units = tiles * per;
    const int grid = gridDim.x;
    // pieces of 8 r, 8 (r + 1) and 8 (r + 2) tiles
    const int least = (int)min((units + 8LL * grid - 1) / (8LL * grid), 1LL << 27) * 8;
    int k[3] = {0, 0, 0};
    for (int b = tid; b < a.n_seq; b += kThreads) {
        const int t = b == tid ? mine : tiles_of(a, b);
#pragma unroll
        for (int i = 0; i < 3; i++) k[i] += t ? (t - 1) / max(least + 8 * i, 1) + 1 : 0;
    }
#pragma unroll
    for (int i = 0; i < 3; i++) {
        k[i] = __reduce_add_sync(0xffffffffu, k[i]);
        if (lane == 0) counts[warp][i] = k[i];
    }
    __syncthreads();
    Share z;
    z.piece = 0;
    long long pieces = 0;
#pragma unroll
    for (int i = 2; i >= 0; i--) {
        long long all = 0;
        for (int w = 0; w < kWarps; w++) all += counts[w][i];
        if (all * per <= grid) {
            z.piece = max(least + 8 * i, 1);
            pieces = all * per;
        }
    }
    z.seq = -1;
    const bool work = z.piece ? blockIdx.x < pieces : blockIdx.x < units, writes = before && blockIdx.x == 0;
    if (!work && !writes) return z;
    const long long n_cta = min((long long)grid, units);
    z.u = z.piece ? (long long)blockIdx.x : work ? units * blockIdx.x / n_cta : 0;
    z.u1 = z.piece ? z.u + 1 : work ? units * (blockIdx.x + 1) / n_cta : 0;
    long long run = 0;
    for (int b0 = 0; b0 < a.n_seq; b0 += kThreads) {
        const int b = b0 + tid;
        n = b0 == 0 ? mine : b < a.n_seq ? tiles_of(a, b) : 0;
        if (z.piece && n) n = ((int)n - 1) / z.piece + 1;
        long long incl = n;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long v = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += v;
        }
        __syncthreads();
        if (lane == 31) sums[warp] = incl;
        __syncthreads();
        long long at = run + incl - n;
        for (int w = 0; w < kWarps; w++) {
            if (w < warp) at += sums[w];
            run += sums[w];
        }
        if (writes && b < a.n_seq) before[b] = at;
        if (work && at * per <= z.u && z.u < (at + n) * per) {
            s_seq = b;
            s_first = at;
        }
        __syncthreads();
        if (s_seq >= 0 && !writes) break;
    }
    if (writes && tid == 0) {
        before[a.n_seq] = run;
        before[a.n_seq + 1] = z.piece;
    }
    z.seq = s_seq;
    z.first = s_first;
    return z;
}

// 2^e, -126 <= e <= 127.
__device__ __forceinline__ float exp2i(int e) { return __uint_as_float((uint32_t)(127 + e) << 23); }

// A warp's query rows as the B operand of the key product, and what its scores need.
template <class S>
struct Query {
    uint32_t q[S::kParts][4];            // row lane / 4, dims 8 (lane % 4) + {0,4}, {1,5}/16, {2,6}, {3,7}/16 of each 32
    float f[2];                          // rows 2 (lane % 4) + {0, 1}: log2(e) * |scale| * 2^24 / the row's power of two; q has the scale's sign
};

// `off`: what the accumulators of lane % 4 begin with, -8 sum q of its two rows, twice.
template <class S>
__device__ __forceinline__ void load_query(const GqaAttendArgs &a, int b, int h, int r0, int lane, Query<S> &y, float4 (*off)[4]) {
    const int G = a.H / a.c.n_kv, n = a.n_q * G, c = lane & 3, row = r0 + (lane >> 2);
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
        for (int i = 0; i < 8; i++) {
            m = fmaxf(m, fabsf(x[p][i]));
            if (a.scale < 0.f) x[p][i] = -x[p][i];
        }
    m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
    m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 2));
    int e = 0;                                           // the row times 2^e has its largest magnitude in 2^14 .. 2^15
    if (m > 0.f && m < INFINITY) e = 14 - ilogbf(m);
    const float up = exp2i(e / 2), even = exp2i(e - e / 2), odd = even * 0.0625f;   // 2^e in two factors: it may pass the range
    float sum[S::NG];
#pragma unroll
    for (int g = 0; g < S::NG; g++) sum[g] = 0.f;
#pragma unroll
    for (int p = 0; p < S::kParts; p++)
#pragma unroll
        for (int i = 0; i < 4; i++) {
            const uint32_t w = pack_f16(x[p][i] * up * (i & 1 ? odd : even), x[p][i + 4] * up * (i & 1 ? odd : even));
            y.q[p][i] = w;
            const float2 back = __half22float2(*reinterpret_cast<const __half2 *>(&w));
            sum[p / S::kPer] += (back.x + back.y) * (i & 1 ? 16.f : 1.f);
        }
    // a scale of zero must still send masked scores (-infinity) to -infinity
    const float f = fmaxf(ldexpf(fabsf(a.scale) * 1.4426950408889634f, 24 - e), 1e-37f);
#pragma unroll
    for (int i = 0; i < 2; i++) y.f[i] = __shfl_sync(0xffffffffu, f, 4 * (2 * c + i));
#pragma unroll
    for (int g = 0; g < S::NG; g++) {
        sum[g] += __shfl_xor_sync(0xffffffffu, sum[g], 1);
        sum[g] += __shfl_xor_sync(0xffffffffu, sum[g], 2);
        sum[g] *= -8.f / 16777216.f;
        const float u = __shfl_sync(0xffffffffu, sum[g], 8 * c), v = __shfl_sync(0xffffffffu, sum[g], 8 * c + 4);
        if (lane < 4) off[g][lane] = make_float4(u, v, u, v);
    }
    __syncwarp();
}

// Part p of row `key` of a tile of codes stands at 16-byte piece p ^ swizzle(key) of it (64- and 32-byte swizzles of the copies).
template <class S>
__device__ __forceinline__ int swizzle(int key) {
    return S::D == 128 ? (key >> 1) & 3 : (key >> 2) & 1;
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

// The scales of rows `key` (low halves) and `key` + 1, bf16; key is even.
template <class S>
__device__ __forceinline__ void pair_scales(const uint8_t *sm, int key, uint32_t (&s)[S::NG]) {
    if constexpr (S::NG == 4) {
        const uint4 w = *reinterpret_cast<const uint4 *>(sm + key * 8);
        s[0] = __byte_perm(w.x, w.z, 0x5410), s[1] = __byte_perm(w.x, w.z, 0x7632);
        s[2] = __byte_perm(w.y, w.w, 0x5410), s[3] = __byte_perm(w.y, w.w, 0x7632);
    } else if constexpr (S::NG == 2) {
        const uint2 w = *reinterpret_cast<const uint2 *>(sm + key * 4);
        s[0] = __byte_perm(w.x, w.y, 0x5410), s[1] = __byte_perm(w.x, w.y, 0x7632);
    } else {
        s[0] = *reinterpret_cast<const uint32_t *>(sm + key * 2);
    }
}

// Adds part p of a tile's key product: d[k] is of tokens 16 k + lane / 4 + 8 (i / 2), rows 2 (lane % 4) + i % 2.
template <class S>
__device__ __forceinline__ void key_part(uint32_t at, int p, const Query<S> &y, float (&d)[2][4]) {
    uint32_t w[4];                                       // 8 codes of tokens r, r + 8, r + 16, r + 24, r = lane / 4
    load_matrices(at, w);
#pragma unroll
    for (int k = 0; k < 2; k++) {
        const uint32_t u = w[2 * k], v = w[2 * k + 1], u8 = u >> 8, v8 = v >> 8;
        mma_f16(d[k], u & 0x000F000Fu, v & 0x000F000Fu, u & 0x00F000F0u, v & 0x00F000F0u, y.q[p][0], y.q[p][1]);
        mma_f16(d[k], u8 & 0x000F000Fu, v8 & 0x000F000Fu, u8 & 0x00F000F0u, v8 & 0x00F000F0u, y.q[p][2], y.q[p][3]);
    }
}
// The scores of a scale group: s (+)= d times the tokens' scales.
template <class S>
__device__ __forceinline__ void add_scores(const float (&d)[2][4], const float (&sc)[4][S::NG], int g, float (&s)[2][4]) {
#pragma unroll
    for (int k = 0; k < 2; k++)
#pragma unroll
        for (int i = 0; i < 4; i++) {
            const float by = sc[2 * k + i / 2][g];
            s[k][i] = g ? fmaf(d[k][i], by, s[k][i]) : d[k][i] * by;
        }
}
__device__ __forceinline__ void begin(const float4 &c, float (&d)[2][4]) {
#pragma unroll
    for (int k = 0; k < 2; k++) d[k][0] = c.x, d[k][1] = c.y, d[k][2] = c.z, d[k][3] = c.w;
}

// What a warp has added up of a segment: rows 2 (lane % 4) + i % 2, dims 32 p + 4 (lane / 4) + 2 e + i / 2 (m-tile e, its rows
// lane / 4 and 8 more).
template <class S>
struct Sums {
    float o[S::kParts][2][4], corr[S::NG][4], m[2], l[2];
};

// Adds the outputs of the tile at `sm`, whose scores (before the factor f) are s and which the references have been moved for.
// EDGE: some row does not see all of the tile's tokens; `seen` is how many of them row lane / 4 sees.
template <class S, bool EDGE>
__device__ __forceinline__ void outputs(const uint8_t *sm, const Query<S> &y, Sums<S> &z, int lane, int seen, const float (&s)[2][4]) {
    const int c = lane & 3, x = swizzle<S>(lane);
    const uint8_t *scales = sm + 2 * S::kCodes + S::kScales;
    uint32_t b[2][S::NG][2];                             // P^T times the scales: row lane / 4, tokens 16 k + 8 e + 2 c + {0, 1}
#pragma unroll
    for (int k = 0; k < 2; k++) {
        float p[4];
#pragma unroll
        for (int i = 0; i < 4; i++) {
            p[i] = ex2(fmaf(s[k][i], y.f[i & 1], -z.m[i & 1]));
            z.l[i & 1] += p[i];
        }
#pragma unroll
        for (int e = 0; e < 2; e++) {
            const uint32_t pt = transpose8(pack_bf16(p[2 * e], p[2 * e + 1]));
            uint32_t sc[S::NG], mask = 0xFFFFFFFFu;
            pair_scales<S>(scales, 16 * k + 8 * e + 2 * c, sc);
            if constexpr (EDGE) {
                const int n = seen - (16 * k + 8 * e + 2 * c);   // of this pair
                mask = (n > 0 ? 0x0000FFFFu : 0u) | (n > 1 ? 0xFFFF0000u : 0u);
            }
#pragma unroll
            for (int g = 0; g < S::NG; g++) b[k][g][e] = mul_bf16(pt, sc[g]) & mask;
        }
    }
    const uint32_t at = smem_addr(sm) + S::kCodes + lane * S::kRow;
#pragma unroll
    for (int g = 0; g < S::NG; g++) {
#pragma unroll
        for (int k = 0; k < 2; k++) mma_bf16(z.corr[g], 0x80088008u, 0x80088008u, 0x80088008u, 0x80088008u, b[k][g][0], b[k][g][1]);
#pragma unroll
        for (int p = g * S::kPer; p < (g + 1) * S::kPer; p++) {
            uint32_t w[4];                               // 4 codes of tokens 2 c, 2 c + 1 (low and high half), 8, 16 and 24 more
            load_matrices_t(at + ((p ^ x) << 4), w);
#pragma unroll
            for (int k = 0; k < 2; k++) {
                const uint32_t u = w[2 * k], v = w[2 * k + 1];
                const uint32_t u8 = u >> 8, v8 = v >> 8;
                const uint32_t n[2][4] = {{u & 0x000F000Fu, u & 0x00F000F0u, u8 & 0x000F000Fu, u8 & 0x00F000F0u},
                                          {v & 0x000F000Fu, v & 0x00F000F0u, v8 & 0x000F000Fu, v8 & 0x00F000F0u}};
#pragma unroll
                for (int e = 0; e < 2; e++) mma_bf16(z.o[p][e], n[0][2 * e], n[0][2 * e + 1], n[1][2 * e], n[1][2 * e + 1], b[k][g][0], b[k][g][1]);
            }
        }
    }
}
template <class S>
__device__ __forceinline__ void scores(const uint8_t *sm, const uint8_t *scales, const Query<S> &y, const float4 (*off)[4], int lane, float (&s)[2][4]) {
    float sc[4][S::NG];
#pragma unroll
    for (int e = 0; e < 4; e++) load_scales<S>(scales, 8 * e + (lane >> 2), sc[e]);
    const uint32_t at = smem_addr(sm) + lane * S::kRow;
    const int x = swizzle<S>(lane);
#pragma unroll
    for (int g = 0; g < S::NG; g++) {
        float d[2][4];
        begin(off[g][lane & 3], d);
#pragma unroll
        for (int p = g * S::kPer; p < (g + 1) * S::kPer; p++) key_part<S>(at + ((p ^ x) << 4), p, y, d);
        add_scores<S>(d, sc, g, s);
    }
}

__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire;" ::: "memory"); }
// The address of a place in the shared memory of the cluster's CTA `rank`.
__device__ __forceinline__ uint32_t of_rank(const void *p, int rank) {
    uint32_t at;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(smem_addr(p)), "r"(rank));
    return at;
}

// Output, lse and what the weights need (`stat`), of a head's row `at` = token * G + head of the group and its dims d .. d + 3.
template <int D>
__device__ __forceinline__ void finish(const GqaAttendArgs &a, float2 *stat, int b, int h, int G, int at, int d, const float4 &o, float m, float l) {
    const float inv = l != 0.f ? 1.f / l * kScale : 0.f;
    const long long orow = (long long)(b * (long long)a.n_q + at / G) * a.H + h * G + at % G;
    if (a.out_bf16)
        *reinterpret_cast<uint2 *>(reinterpret_cast<__nv_bfloat16 *>(a.out) + orow * D + d) = make_uint2(pack_bf16(o.x * inv, o.y * inv), pack_bf16(o.z * inv, o.w * inv));
    else
        *reinterpret_cast<float4 *>(reinterpret_cast<float *>(a.out) + orow * D + d) = make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv);
    if (d == 0 && a.lse) a.lse[orow] = l != 0.f ? (m + kUp + log2f(l * 0x1p-80f)) * 0.6931471805599453f : -INFINITY;
    if (d == 0 && a.weigh) *stat = make_float2(m + kUp, inv);
}

// Moves the references, and what has been added up, if some score of the tile is 8 above: that much is seen without a look at the other
// lanes.
template <class S>
__device__ __forceinline__ void move_references(const Query<S> &y, Sums<S> &z, const float (&s)[2][4]) {
    bool move = false;
    float now[2];
#pragma unroll
    for (int i = 0; i < 2; i++) {
        now[i] = fmaxf(fmaxf(s[0][i], s[0][2 + i]), fmaxf(s[1][i], s[1][2 + i]));
        move |= fmaf(now[i], y.f[i], -z.m[i]) > kUp + kGrow;
    }
    if (!__any_sync(0xffffffffu, move)) return;
#pragma unroll
    for (int i = 0; i < 2; i++) {
        float m = now[i];
        m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 4));
        m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 8));
        m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 16)) * y.f[i];
        if (!(m - z.m[i] > kUp + kGrow)) continue;
        m -= kUp;
        const float f = ex2(z.m[i] - m);
        z.m[i] = m;
        z.l[i] *= f;
#pragma unroll
        for (int p = 0; p < S::kParts; p++)
#pragma unroll
            for (int e = 0; e < 2; e++) z.o[p][e][i] *= f, z.o[p][e][2 + i] *= f;
#pragma unroll
        for (int g = 0; g < S::NG; g++) z.corr[g][i] *= f, z.corr[g][2 + i] *= f;
    }
}

template <class S, bool WEIGH, bool CLUSTER>
__global__ void __launch_bounds__(kThreads, 2)
    gqa_attend_kernel(const __grid_constant__ CUtensorMap k_map, const __grid_constant__ CUtensorMap v_map, const GqaAttendArgs a,
                      const AttendPlan plan, long long wait_ns) {
    using R = Ring<S, WEIGH>;
    extern __shared__ uint8_t raw[];
    __shared__ uint64_t full[kWarps][R::kDepth];
    __shared__ float2 ml[kWarps][kRows];
    __shared__ float4 s_off[kWarps][S::NG][4];
    __shared__ int s_row[kWarps][R::kDepth][2];          // WEIGH: the cache rows that a stage's halves come from, -1: none
    __shared__ int s_abort;
    uint8_t *base = raw + (((smem_addr(raw) + 1023u) & ~1023u) - smem_addr(raw));
    const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
    uint8_t *ring = base + warp * R::kDepth * R::kStage;
    if (lane == 0)
        for (int i = 0; i < R::kDepth; i++) mbar_init(&full[warp][i], 1);
    if (tid == 0) s_abort = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    if constexpr (CLUSTER) cluster_arrive();             // the CTAs have begun
    pdl_wait();
    __syncthreads();
    volatile int *abort = &s_abort;
    const int n_kv = a.c.n_kv, G = a.H / n_kv, n_rows = a.n_q * G;
    const int per = WEIGH ? n_kv : n_kv * plan.rg;       // segments of a sequence
    if (!WEIGH && blockIdx.x == 0)
        for (int b = tid; b < a.n_seq; b += kThreads) length_of(a, b, true);
    Share share;
    int rank = 0;
    if constexpr (CLUSTER) {
        const int place = blockIdx.x / plan.cluster;     // a segment each
        rank = blockIdx.x - place * plan.cluster;
        share.seq = place / per;
        share.first = 0;
        share.u = place - share.seq * per;
        share.u1 = share.u + 1;
        share.piece = 1;
    } else {
        share = find_share(a, per, WEIGH ? nullptr : plan.before);
        if (share.seq < 0) return;
    }
    const long long u1 = share.u1;
    long long u = share.u, first = share.first;
    int b = share.seq;
    int slot = 0, par = 0;                               // next stage to be read, parity of its use
    bool ok = true;
    while (u < u1) {
        const int len = length_of(a, b, false), nt = (len + kTile - 1) / kTile;
        const long long at = u - first * per;
        const int each = CLUSTER ? plan.cluster : share.piece ? (nt - 1) / share.piece + 1 : nt;   // pieces or tiles of a segment
        const int seg = CLUSTER ? (int)at : (int)(at / each), k = CLUSTER ? rank : (int)(at - (long long)seg * each);
        const int t0 = share.piece ? (int)((long long)nt * k / each) : k;
        const int t1 = share.piece ? (int)((long long)nt * (k + 1) / each) : (int)min((long long)nt, t0 + (u1 - u));
        const int h = WEIGH ? seg : seg / plan.rg;
        const int32_t *pages = a.pages + b * a.pages_stride;
        const int mine = (t1 - t0 - warp + kWarps - 1) / kWarps;   // tiles t0 + warp, t0 + warp + 8, ...
        for (int set = WEIGH ? 0 : seg - h * plan.rg, sets = WEIGH ? plan.rg : set + 1; set < sets && (!WEIGH || ok); set++) {   // after a wait that ran out, no copies into a stage that has some
            const int r0 = set * kRows;
            const uint64_t deadline = deadline_after(wait_ns, max(mine, 0));
            // copies: lane i holds the first row of the i-th box from `base_tile` on
            int first_row = 0, base_tile = 0;
            const int per_load = 32 / plan.boxes, box_rows = kTile / plan.boxes;
            auto look_up = [&](int i) {                  // whole warp, tiles i, i + 1, ... of this warp
                base_tile = i;
                const int t = t0 + warp + kWarps * (i + lane / plan.boxes), tok = t * kTile + (plan.boxes == 2 ? 16 * (lane & 1) : 0);
                first_row = -1;
                if (tok < len && i + lane / plan.boxes < mine) {
                    const int p = tok / a.c.page, id = pages[p];
                    if (id < 0 || id >= a.c.n_pages) mla_bad_index(a.err);   // the cache's first rows instead: the output is unspecified
                    else first_row = (int)gqa_row(a.c, id, h) + (tok - p * a.c.page);   // rows < 2^31, a row plus a token need not be
                }
            };
            auto ask = [&](int i, int stage) {           // whole warp
                if (i - base_tile >= per_load) look_up(i);
                const uint32_t dst = smem_addr(ring + stage * R::kStage);
                const bool two = plan.boxes == 2 && (t0 + warp + kWarps * i) * kTile + 16 < len;
                const uint32_t bytes = (two ? kTile : box_rows) * (WEIGH ? 1 : 2) * (S::kRow + S::NG * 2);
                const int found = __shfl_sync(0xffffffffu, first_row, (i - base_tile) * plan.boxes), row = max(found, 0);
                if (WEIGH && lane == 0) {
                    s_row[warp][stage][0] = found;
                    s_row[warp][stage][1] = found < 0 ? -1 : found + 16;
                }
                fill<!WEIGH, true>(dst, S::kCodes, dst + R::kScaleAt, S::kScales, &k_map, &v_map, row, a.c.ks + (long long)row * S::NG,
                             a.c.vs + (long long)row * S::NG, box_rows * S::NG * 2, &full[warp][stage], bytes);
                if (two) {
                    const int found2 = __shfl_sync(0xffffffffu, first_row, (i - base_tile) * 2 + 1), next = max(found2, 0);
                    if (WEIGH && lane == 0) s_row[warp][stage][1] = found2;
                    fill<!WEIGH, false>(dst + 16 * S::kRow, S::kCodes, dst + R::kScaleAt + 16 * S::NG * 2, S::kScales, &k_map, &v_map, next,
                                   a.c.ks + (long long)next * S::NG, a.c.vs + (long long)next * S::NG, 16 * S::NG * 2, &full[warp][stage], 0);
                }
            };
            if (mine > 0) look_up(0);
            for (int i = 0; i < R::kDepth && i < mine; i++) {
                int st = slot + i;
                if (st >= R::kDepth) st -= R::kDepth;
                ask(i, st);
            }
            Query<S> y;
            float4(*off)[4] = s_off[warp];
            load_query<S>(a, b, h, r0, lane, y, off);
            Sums<S> z;
            float2 stat[2];
            if constexpr (WEIGH) {
                // a row that is none has scores of 0 and no weight
#pragma unroll
                for (int i = 0; i < 2; i++) {
                    const int row = 2 * (lane & 3) + i;
                    stat[i] = make_float2(0.f, 0.f);
                    if (r0 + row < n_rows) stat[i] = plan.stat[((long long)(b * (long long)n_kv + h) * plan.rg + set) * kRows + row];
                }
            } else {
#pragma unroll
                for (int i = 0; i < 2; i++) z.m[i] = kNone, z.l[i] = 0.f;
#pragma unroll
                for (int i = 0; i < 4; i++) {
#pragma unroll
                    for (int p = 0; p < S::kParts; p++) z.o[p][0][i] = z.o[p][1][i] = 0.f;
#pragma unroll
                    for (int g = 0; g < S::NG; g++) z.corr[g][i] = 0.f;
                }
            }
            // the stage that comes next, when it has come
            auto arrived = [&]() {
                if (ok && !warp_wait_now(&full[warp][slot], par, deadline, abort, lane)) {
                    ok = false;
                    *abort = 1;
                    atomicCAS(a.err, 0, (int)DEV_ERR_TIMEOUT);
                }
                const uint8_t *sm = ring + slot * R::kStage;
                if (++slot == R::kDepth) {
                    slot = 0;
                    par ^= 1;
                }
                return sm;
            };
            auto limit_of = [&](int row) { return min(len - (a.n_q - 1 - (r0 + row) / G), len); };   // tokens that a row sees
            auto token_of = [&](int i) { return (t0 + warp + kWarps * i) * kTile; };
            if constexpr (WEIGH) {
                const int limit[2] = {limit_of(2 * (lane & 3)), limit_of(2 * (lane & 3) + 1)};
                for (int i = 0; i < mine; i++) {
                    const uint8_t *sm = arrived();
                    if (!ok) break;
                    const int tok = token_of(i), stage = (int)(sm - ring) / (int)R::kStage;
                    float s[2][4];
                    scores<S>(sm, sm + R::kScaleAt, y, off, lane, s);
                    if (tok + kTile > len - (a.n_q - 1))
#pragma unroll
                        for (int k = 0; k < 2; k++)
#pragma unroll
                            for (int j = 0; j < 4; j++)
                                if (tok + 16 * k + (lane >> 2) + 8 * (j / 2) >= limit[j & 1]) s[k][j] = -INFINITY;
                    // of token 16 k + 8 e + lane / 4: this thread's two rows, then all eight
                    float w[2][2];
#pragma unroll
                    for (int k = 0; k < 2; k++)
#pragma unroll
                        for (int e = 0; e < 2; e++) {
                            w[k][e] = 0.f;
#pragma unroll
                            for (int j = 0; j < 2; j++) {
                                const float x = s[k][2 * e + j];
                                const float p = ex2(fmaf(x, y.f[j], -stat[j].x)) * stat[j].y;
                                w[k][e] += x == -INFINITY ? 0.f : p;   // a row that sees nothing has no reference
                            }
                            w[k][e] += __shfl_xor_sync(0xffffffffu, w[k][e], 1);
                            w[k][e] += __shfl_xor_sync(0xffffffffu, w[k][e], 2);
                        }
                    // lane 4 r + c adds token 8 c + r
                    const int c = lane & 3, t = 8 * c + (lane >> 2), at = s_row[warp][stage][c >> 1];
                    const float mine_w = c & 2 ? (c & 1 ? w[1][1] : w[1][0]) : (c & 1 ? w[0][1] : w[0][0]);
                    if (tok + t < len && at >= 0) atomicAdd(a.c.w + at + (t & 15), mine_w);
                    __syncwarp();
                    if (i + R::kDepth < mine) ask(i + R::kDepth, stage);
                }
            } else {
                for (int i = 0; i < mine; i++) {
                    const uint8_t *sm = arrived();
                    if (!ok) break;
                    float s[2][4];
                    scores<S>(sm, sm + R::kScaleAt, y, off, lane, s);
                    const bool edge = token_of(i) + kTile > len - (a.n_q - 1);
                    if (edge)
#pragma unroll
                        for (int k = 0; k < 2; k++)
#pragma unroll
                            for (int j = 0; j < 4; j++)
                                if (token_of(i) + 16 * k + (lane >> 2) + 8 * (j / 2) >= limit_of(2 * (lane & 3) + j % 2)) s[k][j] = -INFINITY;
                    move_references<S>(y, z, s);
                    if (edge) outputs<S, true>(sm, y, z, lane, limit_of(lane >> 2) - token_of(i), s);
                    else outputs<S, false>(sm, y, z, lane, kTile, s);
                    __syncwarp();
                    if (i + R::kDepth < mine) ask(i + R::kDepth, (int)(sm - ring) / (int)R::kStage);
                }
            }
            if constexpr (!WEIGH) {
                // ------------------------------------------------------ the warps' sums become the segment's
#pragma unroll
                for (int i = 0; i < 2; i++) {
                    float l = z.l[i];
                    l += __shfl_xor_sync(0xffffffffu, l, 4);
                    l += __shfl_xor_sync(0xffffffffu, l, 8);
                    l += __shfl_xor_sync(0xffffffffu, l, 16);
                    if (lane < 4) ml[warp][2 * lane + i] = make_float2(z.m[i], l);
                }
                __syncthreads();
                float *mine_o = reinterpret_cast<float *>(ring);
#pragma unroll
                for (int i = 0; i < 2; i++) {
                    const int row = 2 * (lane & 3) + i;
                    float m = ml[0][row].x;
#pragma unroll
                    for (int w = 1; w < kWarps; w++) m = fmaxf(m, ml[w][row].x);
                    const float f = ex2(z.m[i] - m);
#pragma unroll
                    for (int p = 0; p < S::kParts; p++) {
                        const float *cr = z.corr[p / S::kPer];
                        *reinterpret_cast<float4 *>(mine_o + row * S::D + 32 * p + 4 * (lane >> 2)) =
                            make_float4((z.o[p][0][i] + cr[i]) * kDown * f, fmaf(z.o[p][0][2 + i], 0.0625f, cr[2 + i]) * kDown * f, (z.o[p][1][i] + cr[i]) * kDown * f,
                                        fmaf(z.o[p][1][2 + i], 0.0625f, cr[2 + i]) * kDown * f);
                    }
                }
                __syncthreads();
                __shared__ float4 c_o[CLUSTER ? kRows : 1][S::D / 4];   // of each CTA of the cluster, the rows that this one joins
                __shared__ float2 c_ml[kRows];
                const int rows = CLUSTER ? kRows / plan.cluster : kRows;
                if constexpr (CLUSTER) cluster_wait();
                const bool whole = t0 == 0 && t1 == nt;
                float *part = plan.part + ((long long)blockIdx.x * 2 + (t0 == 0)) * kRows * (S::D + 2);
                for (int i = tid; i < kRows * (S::D / 4); i += kThreads) {
                    const int row = i / (S::D / 4), d = 4 * (i % (S::D / 4));
                    float m = ml[0][row].x, l = 0.f;
#pragma unroll
                    for (int w = 1; w < kWarps; w++) m = fmaxf(m, ml[w][row].x);
#pragma unroll
                    for (int w = 0; w < kWarps; w++) l += ml[w][row].y * ex2(ml[w][row].x - m);
                    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                    for (int w = 0; w < kWarps; w++) {
                        const float4 x = *reinterpret_cast<const float4 *>(base + w * R::kDepth * R::kStage + (row * S::D + d) * 4);
                        o.x += x.x, o.y += x.y, o.z += x.z, o.w += x.w;
                    }
                    if constexpr (CLUSTER) {
                        const int to = row / rows, place = rank * rows + row - to * rows;
                        asm volatile("st.shared::cluster.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(of_rank(&c_o[place][d / 4], to)), "f"(o.x), "f"(o.y), "f"(o.z),
                                     "f"(o.w)
                                     : "memory");
                        if (d == 0) asm volatile("st.shared::cluster.v2.f32 [%0], {%1, %2};" ::"r"(of_rank(&c_ml[place], to)), "f"(m), "f"(l) : "memory");
                        continue;
                    }
                    if (!whole) {
                        *reinterpret_cast<float4 *>(part + row * S::D + d) = o;
                        if (d == 0) *reinterpret_cast<float2 *>(part + kRows * S::D + 2 * row) = make_float2(m, l);
                        continue;
                    }
                    if (r0 + row < n_rows)
                        finish<S::D>(a, plan.stat + ((long long)(b * (long long)n_kv + h) * plan.rg + set) * kRows + row, b, h, G, r0 + row, d, o, m, l);
                }
                if constexpr (CLUSTER) {
                    cluster_arrive();
                    cluster_wait();
                    if (tid < rows * (S::D / 4)) {
                        const int row = tid / (S::D / 4), col = tid % (S::D / 4);
                        float m = kNone, l = 0.f;
                        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                        for (int c = 0; c < kRows; c++)
                            if (c < plan.cluster) m = fmaxf(m, c_ml[c * rows + row].x);
#pragma unroll
                        for (int c = 0; c < kRows; c++)
                            if (c < plan.cluster) {
                                const float2 ml1 = c_ml[c * rows + row];
                                const float4 x = c_o[c * rows + row][col];
                                const float f = ex2(ml1.x - m);
                                l = fmaf(ml1.y, f, l);
                                o = make_float4(fmaf(x.x, f, o.x), fmaf(x.y, f, o.y), fmaf(x.z, f, o.z), fmaf(x.w, f, o.w));
                            }
                        if (const int r = rank * rows + row; r0 + r < n_rows)
                            finish<S::D>(a, plan.stat + ((long long)(b * (long long)n_kv + h) * plan.rg + set) * kRows + r, b, h, G, r0 + r, 4 * col, o, m, l);
                    }
                }
                fence_async_smem();
                __syncthreads();
                ok = ok && !*abort;
            }
        }
        u += share.piece ? 1 : t1 - t0;
        if (u < u1 && at + (t1 - t0) == (long long)nt * per) {
            first += nt;
            do b++;
            while (tiles_of(a, b) == 0);
        }
        if (!ok) break;
    }
    pdl_trigger();                       // not before: the next kernel's CTAs would take room that these want (4x9000: 21 us, this way 19)
    if (*abort) settle();
}

// Joins the parts of a segment that several CTAs had, fills one without tokens.  A CTA has ROWS rows of one: all 8 where a segment
// has few parts, a single one where it has many, whose loads then spread over 8 times as many SMs (1x100000, 38 parts: 5.5 us less).
template <class S, int ROWS>
__global__ void __launch_bounds__(kJoin) gqa_join_kernel(const GqaAttendArgs a, const AttendPlan plan) {
    constexpr int kSets = kRows / ROWS;
    const int n_kv = a.c.n_kv, G = a.H / n_kv, n_rows = a.n_q * G, per = n_kv * plan.rg;
    const int place = blockIdx.x / kSets, row0 = (blockIdx.x - place * kSets) * ROWS;
    const int b = place / per, seg = place - b * per, h = seg / plan.rg, set = seg - h * plan.rg;
    pdl_wait();
    const long long before = plan.before[b], units = plan.before[a.n_seq] * per;
    const int nt = (int)(plan.before[b + 1] - before);   // tiles, or pieces
    const long long u0 = before * per + (long long)seg * nt;
    int c0 = 0, c1 = -1;
    if (plan.before[a.n_seq + 1]) {                      // a CTA per piece
        c0 = (int)u0;
        c1 = c0 + nt - 1;
        if (nt == 1) return;
    } else if (nt > 0) {
        // the CTA of unit u is the largest c with units * c / n <= u, of the n that have units
        const long long n = min((long long)plan.n_cta, units);
        c0 = (int)(((u0 + 1) * n - 1) / units);
        c1 = (int)(((u0 + nt) * n - 1) / units);
        if (c0 == c1) return;
    }
    // Part c's factor per row in shared memory (parts in groups of kGroup), then the sums: threads of a row's dims take every kSplit-th
    // part with kAhead of them in flight, in a fixed order.
    constexpr int kPart = kRows * (S::D + 2), kCols = S::D / 4, kSplit = kJoin / (ROWS * kCols), kAhead = 4;
    __shared__ float factor[kGroup][ROWS];
    __shared__ float4 sum[kSplit][ROWS][kCols];
    __shared__ float s_m[ROWS], s_l[ROWS];
    const int tid = threadIdx.x, row = tid / kCols % ROWS, d = 4 * (tid % kCols), lot = tid / (kCols * ROWS);
    if (tid < ROWS) s_m[tid] = kNone, s_l[tid] = 0.f;
    auto part = [&](int c) { return plan.part + ((long long)c * 2 + (c == c0)) * kPart; };
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int g0 = c0; g0 <= c1; g0 += kGroup) {
        const int n = min(kGroup, c1 - g0 + 1);
        __syncthreads();
        const float old = s_m[row];
        __syncthreads();
        // a warp per row, its lanes the parts
        for (int r = tid >> 5; r < ROWS; r += kJoin / 32) {
            float m = kNone, l = 0.f;
            float2 ml[kGroup / 32];
#pragma unroll
            for (int k = 0; k < kGroup / 32; k++) {
                const int c = (tid & 31) + 32 * k;
                ml[k] = c < n ? *reinterpret_cast<const float2 *>(part(g0 + c) + kRows * S::D + 2 * (row0 + r)) : make_float2(kNone, 0.f);
                m = fmaxf(m, ml[k].x);
            }
            m = fmaxf(m, s_m[r]);
#pragma unroll
            for (int k = 16; k; k >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, k));
#pragma unroll
            for (int k = 0; k < kGroup / 32; k++) {
                const float f = ex2(ml[k].x - m);
                factor[(tid & 31) + 32 * k][r] = f;
                l += ml[k].y * f;
            }
#pragma unroll
            for (int k = 16; k; k >>= 1) l += __shfl_xor_sync(0xffffffffu, l, k);
            __syncwarp();
            if ((tid & 31) == 0) {
                s_l[r] = s_l[r] * ex2(s_m[r] - m) + l;
                s_m[r] = m;
            }
        }
        __syncthreads();
        const float f0 = ex2(old - s_m[row]);
        o = make_float4(o.x * f0, o.y * f0, o.z * f0, o.w * f0);
        for (int i = lot; i < n; i += kSplit * kAhead) {
            float4 x[kAhead];
#pragma unroll
            for (int k = 0; k < kAhead; k++)
                x[k] = i + k * kSplit < n ? *reinterpret_cast<const float4 *>(part(g0 + i + k * kSplit) + (row0 + row) * S::D + d) : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int k = 0; k < kAhead; k++) {
                const float f = i + k * kSplit < n ? factor[i + k * kSplit][row] : 0.f;
                o = make_float4(fmaf(x[k].x, f, o.x), fmaf(x[k].y, f, o.y), fmaf(x[k].z, f, o.z), fmaf(x[k].w, f, o.w));
            }
        }
    }
    sum[lot][row][d / 4] = o;
    __syncthreads();
    const int at = set * kRows + row0 + row;
    if (lot == 0 && at < n_rows) {
        const float m = s_m[row], l = s_l[row];
#pragma unroll
        for (int k = 1; k < kSplit; k++) {
            const float4 x = sum[k][row][d / 4];
            o = make_float4(o.x + x.x, o.y + x.y, o.z + x.z, o.w + x.w);
        }
        finish<S::D>(a, plan.stat + (long long)place * kRows + row0 + row, b, h, G, at, d, o, m, l);
    }
    pdl_trigger();
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

// Sets of 8 query rows of a head.
int row_groups(const GqaAttendArgs &a) { return (a.n_q * (a.H / a.c.n_kv) + kRows - 1) / kRows; }
// CTAs: all that fit, no more than units that the page tables could hold.
int grid_of(const GqaAttendArgs &a, int n_sm) {
    const double most = (double)a.n_seq * (a.pages_stride * a.c.page / kTile + 1) * a.c.n_kv * row_groups(a);
    return (int)std::min(2.0 * n_sm, most);
}
size_t part_bytes(const GqaAttendArgs &a, int n_cta) {
    return round256((size_t)n_cta * 2 * kRows * (a.c.dim + 2) * sizeof(float));
}

// CTAs of a cluster that shares a segment, 0: segments are dealt out by find_share and joined by a second kernel.  Clusters
// need neither the one nor the other, but leave SMs idle where 8 CTAs a segment do not fill the GPU, and go by the longest sequence: what
// counts is the rounds of tiles a warp would go through, by the page tables' width, since lengths are known on the device alone.
// Device time, this way / that: 1x1000 (8 heads) 7.3 / 10.0 us, 4x4000 11.4 / 14.0, 16x500 9.8 / 12.5, at 4 rounds 1x8000 11.9 / 12.5, 32x1000
// 14.8 / 15.2; at 5 4x10000 17.7 / 17.6, at 6 to 8 8x6000 18.7 / 17.6, 1x16000 16.5 / 14.8.  More segments than CTAs fit at once come one
// after another, two on an SM beside each other: 48x300 17.7 / 25.5, 100x1000 39.6 / 48.9, 45x165 of 5 tokens (96 heads on 8) 61 / 77.
int cluster_of(const GqaAttendArgs &a, int n_sm) {
    const long long segments = (long long)a.n_seq * a.c.n_kv * row_groups(a), tiles = (a.longest + kTile - 1) / kTile;
    for (int c = kRows; c; c /= 2)
        if (segments * c <= 2 * n_sm || c == 1) return (tiles + c - 1) / c <= kRounds * kWarps ? c : 0;
    return 0;
}

template <class... P, class... A>
cudaError_t launch_clusters(void (*kern)(P...), int n_cta, int size, size_t smem, cudaStream_t st, A &&...args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(n_cta);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = size;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, kern, std::forward<A>(args)...);
}

template <class S>
cudaError_t run(const GqaAttendArgs &a, const DevInfo &d, cudaStream_t st, int *n_launch) {
    AttendPlan plan;
    plan.rg = row_groups(a);
    plan.boxes = a.c.page % kTile ? 2 : 1;
    plan.n_cta = grid_of(a, d.n_sm);
    plan.part = (float *)d.scratch;
    plan.before = (long long *)((char *)d.scratch + part_bytes(a, plan.n_cta));
    plan.stat = (float2 *)((char *)plan.before + round256((size_t)(a.n_seq + 2) * sizeof(long long)));
    CUtensorMap k, v;
    const long long rows = (long long)a.c.n_pages * a.c.n_kv * a.c.page;
    if (cudaError_t e = code_map(a.c.k, S::kRow, rows, kTile / plan.boxes, &k)) return e;
    if (cudaError_t e = code_map(a.c.v, S::kRow, rows, kTile / plan.boxes, &v)) return e;
    static std::atomic<uint64_t> done{0}, done_cluster{0}, done_weigh{0};
    const long long segments = (long long)a.n_seq * a.c.n_kv * plan.rg;
    plan.cluster = cluster_of(a, d.n_sm);
    if (plan.cluster) {
        if (cudaError_t e = allow_smem(gqa_attend_kernel<S, false, true>, Ring<S, false>::kSmem, d.device, done_cluster)) return e;
        if (cudaError_t e = launch_clusters(gqa_attend_kernel<S, false, true>, (int)segments * plan.cluster, plan.cluster, Ring<S, false>::kSmem, st, k, v, a, plan, d.wait_ns))
            return e;
        *n_launch = 1;
    } else {
        if (cudaError_t e = allow_smem(gqa_attend_kernel<S, false, false>, Ring<S, false>::kSmem, d.device, done)) return e;
        if (cudaError_t e = launch_pdl(gqa_attend_kernel<S, false, false>, dim3(plan.n_cta), dim3(kThreads), Ring<S, false>::kSmem, st, k, v, a, plan, d.wait_ns))
            return e;
        *n_launch = 2;
        if (plan.n_cta > 4 * segments) {      // 4 parts a segment or more
            if (cudaError_t e = launch_pdl(gqa_join_kernel<S, 1>, dim3((unsigned)segments * kRows), dim3(kJoin), 0, st, a, plan)) return e;
        } else {
            if (cudaError_t e = launch_pdl(gqa_join_kernel<S, kRows>, dim3((unsigned)segments), dim3(kJoin), 0, st, a, plan)) return e;
        }
    }
    if (!a.weigh) return cudaSuccess;
    ++*n_launch;
    if (cudaError_t e = allow_smem(gqa_attend_kernel<S, true, false>, Ring<S, true>::kSmem, d.device, done_weigh)) return e;
    return launch_pdl(gqa_attend_kernel<S, true, false>, dim3(plan.n_cta), dim3(kThreads), Ring<S, true>::kSmem, st, k, v, a, plan, d.wait_ns);
}

}  // namespace

size_t gqa_attend_scratch(const GqaAttendArgs &a, int n_sm) {
    const int n_cta = grid_of(a, n_sm);
    return part_bytes(a, n_cta) + round256((size_t)(a.n_seq + 2) * sizeof(long long)) + (a.weigh ? (size_t)a.n_seq * a.c.n_kv * row_groups(a) * kRows * sizeof(float2) : 0);
}

cudaError_t launch_gqa_attend(const GqaAttendArgs &a, const DevInfo &d, cudaStream_t st, int *n_launch) {
    switch (a.c.dim * 8 + a.c.dim / a.c.gs) {
        case 64 * 8 + 1: return run<Shape<64, 1>>(a, d, st, n_launch);
        case 64 * 8 + 2: return run<Shape<64, 2>>(a, d, st, n_launch);
        case 128 * 8 + 1: return run<Shape<128, 1>>(a, d, st, n_launch);
        case 128 * 8 + 2: return run<Shape<128, 2>>(a, d, st, n_launch);
        default: return run<Shape<128, 4>>(a, d, st, n_launch);
    }
}

}  // namespace coli

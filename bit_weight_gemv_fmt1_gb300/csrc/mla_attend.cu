// mla_attend.cu -- attention over the paged latent cache (absorbed form), on
// the 5th-generation tensor cores.
//
// All heads of a token read the same cached rows, so the rows [t][L + R] of a
// tile of 128 tokens are brought into shared memory once, as 16-bit values, and
// serve both products of every head:
//   S^T[t][c] = sum_d row[t][d] q[c][d]      M = 128 tokens, N = columns, K = L + R
//   O^T[d][c] += sum_t row[t][d] P^T[t][c]   M = 128 dims (L/128 times), N = columns, K = 128 tokens
// The rows are the A operand of both: K-major (a token's dims along a row) for S,
// MN-major (the same bytes read across) for O.  A column c is one query row
// (query token j, head h); a CTA has N = 16, 32 or 64 of them.  Tokens are the
// lanes of S^T in TMEM, so one thread holds one token's scores of all columns.
//
// Softmax.  With x = log2(e) * scale * score, m_c a running reference and s_t
// the row's scale (1 for bf16): e = 2^(x - m_c), l_c += e, P = 16-bit(e * s_t).
// m_c starts 6 below the first tile's maximum of x + log2(s_t) and moves only
// when some e * s_t passes 2^14 (f16 holds 65504): most tiles need no maximum
// and no rescaling of O, and weights down to 2^-20 of the largest keep f16's full
// precision.  l and O are f32; P is rounded to the cache's 16-bit type (E4M3 codes
// are exact in f16, the row scale rides on P), q to the same type.
//
// Work.  The tiles of all sequences form one line that is cut into equal
// contiguous pieces, one for each group of CTAs; the CTAs of a group take the
// piece's row blocks side by side, so each row comes from HBM once.  Pieces that
// hold part of a sequence leave (O, m, l) in f32 in scratch, and
// mla_join_kernel adds them up; the rest is written directly.
//
// Warps: 0-7 softmax and output (two threads per token, each half the columns;
// warp 0 issues the MMAs, which alternate with the softmax anyway), then for E4M3 eight warps that load codes into registers one
// whole tile ahead, convert and store them; for bf16 one warp of tiled bulk copies.
// Every wait is bounded; after one has run out all waits return at once, no
// further MMA or copy is issued, and the kernel records DEV_ERR_TIMEOUT.
#include <cudaTypedefs.h>

#include "mla.cuh"
#include "tcgen05.cuh"

namespace coli {

namespace {

constexpr int kTile = 128;
constexpr uint32_t kBlk = kTile * 128;   // 128 tokens x 64 dims of 16 bits, 128-byte swizzle
constexpr int kSoft = 256;               // softmax threads
constexpr int kMaxPairs = 4;             // pairs of blocks: L / 128
constexpr float kHead = 6.f;             // log2 of the largest weight of a fresh reference
constexpr float kLimit = 16384.f;        // weights past this move the reference

struct Geometry {
    int n_rows;            // query rows of a sequence: n_q * H
    int nrb;               // row blocks of N columns
    int n_groups, n_slots; // pieces of the line of tiles; CTAs of a group
    float *part;           // [n_groups * nrb * 2][N][L] partial O, then [..][N][2] m, l
    float *part_ml;
    int *prefix;           // [n_seq + 1] tiles before each sequence
    int pbox;              // tokens per copy box (bf16)
    long long timeout_ns;
};

struct Shared {
    uint64_t full[kMaxPairs + 1], empty[kMaxPairs + 1], s_full, o_full;
    uint32_t tmem;
    int abort;
    int u0, u1, b0, p0;               // this group's piece, its first sequence, the tiles before that
    alignas(16) float f[64];
    alignas(16) float m[2][64];       // read as float4, like f
    float linv[64];
    int limit[64];
    float red[4][64];
    int slot[2][kTile];
    float scale[2][kTile];
};

__device__ __forceinline__ int seq_len(const MlaAttendArgs &a, int b) {
    const int n = a.lens[b];
    return n < 0 || n > a.pages_stride * a.c.page ? 0 : n;
}
__device__ __forceinline__ int tiles_of(int len) { return len > 0 ? (len + kTile - 1) / kTile : 1; }

// The tiles of a CTA's piece, for each of its row blocks, in order.
struct Walk {
    const MlaAttendArgs &a;
    const Geometry &g;
    const Shared &s;
    int rb, u, b, p, T, len;
    __device__ Walk(const MlaAttendArgs &a_, const Geometry &g_, const Shared &s_, int slot) : a(a_), g(g_), s(s_), rb(slot) { start(); }
    __device__ void start() {
        u = s.u0;
        b = s.b0;
        p = s.p0;
        if (u < s.u1) {
            len = seq_len(a, b);
            T = tiles_of(len);
        }
    }
    __device__ bool valid() const { return rb < g.nrb && u < s.u1; }
    __device__ int tile() const { return u - p; }
    __device__ bool first() const { return u == s.u0 || u == p; }              // of this CTA's part of the sequence
    __device__ bool last() const { return u + 1 == s.u1 || u + 1 == p + T; }
    __device__ bool whole() const { return p >= s.u0 && p + T <= s.u1; }       // the piece holds all of the sequence
    __device__ int which() const { return p < s.u0 ? 0 : 1; }                  // which of the piece's two partial results
    __device__ void next() {
        if (++u == s.u1) {
            rb += g.n_slots;
            start();
        } else if (u == p + T) {
            p += T;
            len = seq_len(a, ++b);
            T = tiles_of(len);
        }
    }
};

// Slot of a token, -1 past the length or for a bad page.
__device__ __forceinline__ int token_slot(const MlaAttendArgs &a, int b, int t, int len) {
    if (t >= len) return -1;
    const int pi = t / a.c.page;
    const int id = a.pages[(long long)b * a.pages_stride + pi];
    if (id < 0 || id >= a.c.n_pages) {
        mla_bad_index(a.err);
        return -1;
    }
    return id * a.c.page + (t - pi * a.c.page);
}

// Order-preserving map of floats to ints (its own inverse up to the sign rule).
__device__ __forceinline__ int float_key(float f) {
    const int i = __float_as_int(f);
    return i ^ ((i >> 31) & 0x7FFFFFFF);
}

// One round of query rows: loads, scale (f16 operands), conversion, swizzled store.
template <int N, bool E4M3, bool QB>
__device__ __forceinline__ void load_queries(const MlaAttendArgs &a, const Geometry &g, Shared &s, uint8_t *qsm, int b, int rb, int len,
                                             int warp, int lane) {
    constexpr int RB = QB ? 4 : 2;         // rows in flight per warp
    constexpr int W = QB ? 1 : 2;          // 16-byte words per unit of 8 elements
    const int nu = a.c.L / 8, nr = a.c.R / 8;
    for (int c0 = warp; c0 < N; c0 += 8 * RB) {
        uint4 x[RB][3][W];
#pragma unroll
        for (int i = 0; i < RB; i++) {
            const int c = c0 + 8 * i, r = rb * N + c;
            const bool live = c < N && r < g.n_rows;
            const long long row = (long long)b * g.n_rows + r;
#pragma unroll
            for (int k = 0; k < 3; k++) {
                const int u = lane + 32 * (k == 1);
                const bool ok = live && (k < 2 ? u < nu : lane < nr);
                const long long e = k < 2 ? row * a.c.L + 8 * u : row * a.c.R + 8 * lane;
                const uint8_t *src = reinterpret_cast<const uint8_t *>(k < 2 ? a.q_latent : a.q_rope) + e * (QB ? 2 : 4);
#pragma unroll
                for (int w = 0; w < W; w++) x[i][k][w] = ok ? __ldg(reinterpret_cast<const uint4 *>(src) + w) : make_uint4(0u, 0u, 0u, 0u);
            }
        }
#pragma unroll
        for (int i = 0; i < RB; i++) {
            const int c = c0 + 8 * i, r = rb * N + c;
            if (c >= N) break;
            float v[3][8], f = a.scale * 1.4426950408889634f;
#pragma unroll
            for (int k = 0; k < 3; k++) {
                if constexpr (QB) {
                    const uint32_t w[4] = {x[i][k][0].x, x[i][k][0].y, x[i][k][0].z, x[i][k][0].w};
#pragma unroll
                    for (int q = 0; q < 4; q++) {
                        const float2 t = bf16x2_f32x2(w[q]);
                        v[k][2 * q] = t.x;
                        v[k][2 * q + 1] = t.y;
                    }
                } else {
#pragma unroll
                    for (int q = 0; q < 2; q++) {
                        const uint4 w = x[i][k][q % W];
                        v[k][4 * q] = __uint_as_float(w.x);
                        v[k][4 * q + 1] = __uint_as_float(w.y);
                        v[k][4 * q + 2] = __uint_as_float(w.z);
                        v[k][4 * q + 3] = __uint_as_float(w.w);
                    }
                }
            }
            if constexpr (E4M3) {
                // f16 operand: times 2^k so that the largest magnitude lies in [2^14, 2^15)
                float mx = 0.f;
#pragma unroll
                for (int k = 0; k < 3; k++)
#pragma unroll
                    for (int q = 0; q < 8; q++) mx = fmaxf(mx, fabsf(v[k][q]));
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
                const int ex = (int)((__float_as_uint(mx) >> 23) & 0xFF) - 127;
                const int k2 = mx > 0.f && ex < 128 ? min(14 - ex, 120) : 0;
                const float up = __int_as_float((k2 + 127) << 23);
                f *= __int_as_float((127 - k2) << 23);
#pragma unroll
                for (int k = 0; k < 3; k++)
#pragma unroll
                    for (int q = 0; q < 8; q++) v[k][q] *= up;
            }
#pragma unroll
            for (int k = 0; k < 3; k++) {
                const int u = k < 2 ? lane + 32 * k : nu + lane;
                if (k < 2 ? u >= nu : lane >= nr) continue;
                uint4 w;
                if constexpr (E4M3) w = make_uint4(pack_f16(v[k][0], v[k][1]), pack_f16(v[k][2], v[k][3]), pack_f16(v[k][4], v[k][5]), pack_f16(v[k][6], v[k][7]));
                else w = make_uint4(pack_bf16(v[k][0], v[k][1]), pack_bf16(v[k][2], v[k][3]), pack_bf16(v[k][4], v[k][5]), pack_bf16(v[k][6], v[k][7]));
                *reinterpret_cast<uint4 *>(qsm + (u >> 3) * (N * 128) + c * 128 + (((u & 7) ^ (c & 7)) << 4)) = w;
            }
            if (lane == 0) {
                s.f[c] = f;
                s.limit[c] = r < g.n_rows ? len - (a.n_q - 1 - r / a.H) : 0;
            }
        }
    }
}

template <int N, bool E4M3>
__global__ void __launch_bounds__(E4M3 ? 512 : 288)
    mla_attend_kernel(const __grid_constant__ CUtensorMap map, const MlaAttendArgs a, const Geometry g) {
    constexpr int NC = N / 2;              // columns per softmax thread
    extern __shared__ uint8_t raw[];
    __shared__ Shared s;
    const uint32_t base = (smem_addr(raw) + 1023u) & ~1023u;
    uint8_t *sm = raw + (base - smem_addr(raw));
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int npair = a.c.L / 128, nblk = 2 * npair + 1;
    const uint32_t q_off = nblk * kBlk;    // queries [nblk][N][64]
    const uint32_t p_off = (nblk - 1) * kBlk;   // P^T [128][64], in the rope block's place once S is done
    constexpr uint32_t kCols = N == 64 ? 512 : N == 32 ? 256 : 128;   // S, then O: (1 + L/128) * N <= 5 N
    pdl_wait();
    pdl_trigger();

    if (warp == 0) tmem_alloc(&s.tmem, kCols);
    if (tid == 0) {
        for (int p = 0; p <= kMaxPairs; p++) {
            mbar_init(&s.full[p], E4M3 ? 8 : 1);
            mbar_init(&s.empty[p], 1);
        }
        mbar_init(&s.s_full, 1);
        mbar_init(&s.o_full, 1);
        s.abort = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    const int group = blockIdx.x / g.n_slots, slot = blockIdx.x - group * g.n_slots;
    if (warp == 0) {
        // tiles of all sequences, then the sequence this group's piece begins in
        int total = 0;
        for (int b = lane; b < a.n_seq; b += 32) {
            const int n = a.lens[b];
            if (n < 0 || n > a.pages_stride * a.c.page) mla_bad_index(a.err);
            total += tiles_of(seq_len(a, b));
        }
        total = __reduce_add_sync(0xffffffffu, total);
        const int chunk = (total + g.n_groups - 1) / g.n_groups;
        const int u0 = min(total, group * chunk), u1 = min(total, u0 + chunk);
        int run = 0;
        for (int b0 = 0; b0 < a.n_seq; b0 += 32) {
            const int b = b0 + lane;
            const int T = b < a.n_seq ? tiles_of(seq_len(a, b)) : 0;
            int incl = T;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int v = __shfl_up_sync(0xffffffffu, incl, o);
                if (lane >= o) incl += v;
            }
            const int p = run + incl - T;
            if (b < a.n_seq && p <= u0 && u0 < p + T) {
                s.b0 = b;
                s.p0 = p;
            }
            if (g.prefix && blockIdx.x == 0 && b < a.n_seq) g.prefix[b] = p;
            run += __shfl_sync(0xffffffffu, incl, 31);
        }
        if (lane == 0) {
            s.u0 = u0;
            s.u1 = u1;
            if (g.prefix && blockIdx.x == 0) g.prefix[a.n_seq] = total;
        }
    }
    tc_before_sync();
    __syncthreads();
    tc_after_sync();
    const uint32_t tmem = s.tmem;
    const uint64_t deadline = global_ns() + (uint64_t)g.timeout_ns;
    volatile int *abort = &s.abort;
    bool ok = true;                        // this thread's waits have all ended well
    auto wait = [&](uint64_t *bar, uint32_t parity) {
        if (!ok) return;
        if (!warp_wait(bar, parity, deadline, abort, lane)) {
            ok = false;
            *abort = 1;
            atomicCAS(a.err, 0, (int)DEV_ERR_TIMEOUT);
        }
    };

    if (warp < 8) {
        // ---------------------------------------------------------- softmax and output; warp 0 also issues the MMAs
        constexpr int kType = E4M3 ? 0 : 1;
        constexpr uint32_t id_s = f16_idesc(kType, false, false, kTile, N), id_o = f16_idesc(kType, true, true, 128, N);
        const uint64_t dk = sw128_desc(base, 16, 1024), dq = sw128_desc(base + q_off, 16, 1024);
        const uint64_t dv = sw128_desc(base, kBlk, 1024), dp = sw128_desc(base + p_off, kBlk, 1024);
        const int wq = warp & 3, grp = warp >> 2;
        const int t = 32 * wq + lane;                                   // token of the tile, and dim of an O block
        const uint32_t lanes = tmem + ((uint32_t)(32 * wq) << 16);
        const uint32_t col0 = grp * NC;
        float l[NC];
        int it = 0, seg = 0, cur = 0;
        for (Walk w(a, g, s, slot); w.valid(); w.next(), it++) {
            if (w.first()) {
                if (a.q_bf16) load_queries<N, E4M3, true>(a, g, s, sm + q_off, w.b, w.rb, w.len, warp, lane);
                else load_queries<N, E4M3, false>(a, g, s, sm + q_off, w.b, w.rb, w.len, warp, lane);
                if (tid < N) s.m[cur][tid] = -INFINITY;
#pragma unroll
                for (int c = 0; c < NC; c++) l[c] = 0.f;
                fence_async_smem();
                named_sync(1, kSoft);
            }
            if (warp == 0) {
                for (int p = 0; p <= npair; p++) {
                    wait(&s.full[p], it & 1);
                    tc_after_sync();
                    if (lane == 0 && ok) {
                        const int nk = p < npair ? 8 : a.c.R / 16;
                        for (int k = 0; k < nk; k++) {
                            const int blk = 2 * p + (k >> 2);
                            mma_ss(tmem, dk + ((blk * kBlk + (k & 3) * 32) >> 4), dq + ((blk * (N * 128) + (k & 3) * 32) >> 4), id_s, p | k);
                        }
                    }
                }
                if (lane == 0 && ok) tc_commit(&s.s_full);
                __syncwarp();
            }
            const int tok = w.tile() * kTile + t;
            // every column sees the whole tile: the first query's limit is the lowest
            const bool full = (w.tile() + 1) * kTile <= w.len - (a.n_q - 1) && (w.rb + 1) * N <= g.n_rows;
            if (E4M3) wait(&s.full[npair], it & 1);                     // the loaders' scales
            wait(&s.s_full, it & 1);
            tc_after_sync();
            const float st = E4M3 ? s.scale[it & 1][t] : 1.f;
            if (!E4M3 && (w.tile() + 1) * kTile > w.len && tok >= w.len) {
                // rows past the length may hold anything, and 0 * NaN is NaN
                for (int k = grp; k < 2 * npair; k += 2)
#pragma unroll
                    for (int u = 0; u < 8; u++) *reinterpret_cast<uint4 *>(sm + k * kBlk + t * 128 + 16 * u) = make_uint4(0u, 0u, 0u, 0u);
            }
            uint32_t e[NC];
            // the weights 2^(x - reference) of this thread's token; true if one is too large for P
            auto weigh = [&](bool set) {
                tmem_ld(lanes + col0, e);
                tmem_ld_wait();
                float top = 0.f;
#pragma unroll
                for (int c = 0; c < NC; c += 4) {
                    const float4 f4 = *reinterpret_cast<const float4 *>(&s.f[col0 + c]);
                    const float4 m4 = *reinterpret_cast<const float4 *>(&s.m[cur][col0 + c]);
                    const float f[4] = {f4.x, f4.y, f4.z, f4.w}, m[4] = {m4.x, m4.y, m4.z, m4.w};
#pragma unroll
                    for (int k = 0; k < 4; k++) {
                        // no reference (-inf): once the maximum was taken, all that is unmasked is -inf too
                        const float ref = set && m[k] == -INFINITY ? 0.f : m[k];
                        const float x = E4M3 ? __uint_as_float(e[c + k]) * st : __uint_as_float(e[c + k]);
                        float v = ex2(fmaf(x, f[k], -ref));
                        if (!full && tok >= s.limit[col0 + c + k]) v = 0.f;
                        e[c + k] = __float_as_uint(v);
                        top = fmaxf(top, v);
                    }
                }
                return (E4M3 ? top * st : top) > kLimit || top > 1e37f;
            };
            bool move = w.first();
            if (!move) move = named_or(1, kSoft, weigh(false));
            if (move) {
                const float lg = E4M3 ? __log2f(st) : 0.f;
                tmem_ld(lanes + col0, e);
                tmem_ld_wait();
#pragma unroll
                for (int c = 0; c < NC; c++) {
                    const float y = E4M3 ? __uint_as_float(e[c]) * st : __uint_as_float(e[c]);
                    float x = fmaf(y, s.f[col0 + c], lg);
                    if (!full && tok >= s.limit[col0 + c]) x = -INFINITY;
                    const int k = __reduce_max_sync(0xffffffffu, float_key(x));
                    if (lane == 0) s.red[wq][col0 + c] = __int_as_float(k ^ ((k >> 31) & 0x7FFFFFFF));
                }
                named_sync(1, kSoft);
                float r[NC];
#pragma unroll
                for (int c = 0; c < NC; c++) {
                    const float old = s.m[cur][col0 + c];
                    const float x = fmaxf(fmaxf(s.red[0][col0 + c], s.red[1][col0 + c]), fmaxf(s.red[2][col0 + c], s.red[3][col0 + c]));
                    const float now = fmaxf(old, x - kHead);
                    // -inf (only rows of scale 0 so far, whose weights were taken against 0): O is 0
                    r[c] = now == -INFINITY ? 1.f : ex2(old - now);
                    if (t == 0) s.m[cur ^ 1][col0 + c] = now;
                    if (l[c] != 0.f && now != -INFINITY) l[c] *= ex2((old == -INFINITY ? 0.f : old) - now);
                }
                if (!w.first()) {
                    for (int k = 0; k < npair; k++) {
                        tmem_ld(lanes + N * (1 + k) + col0, e);
                        tmem_ld_wait();
#pragma unroll
                        for (int c = 0; c < NC; c++) e[c] = __float_as_uint(__uint_as_float(e[c]) * r[c]);
                        tmem_st(lanes + N * (1 + k) + col0, e);
                    }
                    tmem_st_wait();
                }
                named_sync(1, kSoft);
                cur ^= 1;
                weigh(true);
            }
#pragma unroll
            for (int c = 0; c < NC; c++) l[c] += __uint_as_float(e[c]);
#pragma unroll
            for (int u = 0; u < NC / 8; u++) {
                uint32_t pk[4];
#pragma unroll
                for (int k = 0; k < 4; k++) {
                    const float x = __uint_as_float(e[8 * u + 2 * k]), y = __uint_as_float(e[8 * u + 2 * k + 1]);
                    pk[k] = E4M3 ? pack_f16(x * st, y * st) : pack_bf16(x, y);
                }
                *reinterpret_cast<uint4 *>(sm + p_off + t * 128 + (((grp * (NC / 8) + u) ^ (t & 7)) << 4)) =
                    make_uint4(pk[0], pk[1], pk[2], pk[3]);
            }
            fence_async_smem();
            tc_before_sync();
            named_sync(1, kSoft);
            if (warp == 0) {
                tc_after_sync();
                if (lane == 0 && ok) {
                    for (int p = 0; p < npair; p++) {
#pragma unroll
                        for (int k = 0; k < 8; k++)
                            mma_ss(tmem + N * (1 + p), dv + ((2 * p * kBlk + k * 2048) >> 4), dp + ((k * 2048) >> 4), id_o, k || !w.first());
                        tc_commit(&s.empty[p]);
                    }
                    tc_commit(&s.empty[npair]);
                    if (w.last()) tc_commit(&s.o_full);
                }
                __syncwarp();
            }
            if (!w.last()) continue;

            // ------------------------------------------------------ this part of the sequence is done
#pragma unroll
            for (int c = 0; c < NC; c++) {
                const float z = warp_sum(l[c]);
                if (lane == 0) s.red[wq][col0 + c] = z;
            }
            named_sync(1, kSoft);
            const bool whole = w.whole();
            const long long pidx = ((long long)group * g.nrb + w.rb) * 2 + w.which();
            if (tid < N) {
                const float z = s.red[0][tid] + s.red[1][tid] + s.red[2][tid] + s.red[3][tid];
                const float m = s.m[cur][tid] == -INFINITY && z != 0.f ? 0.f : s.m[cur][tid];
                s.linv[tid] = whole ? (z != 0.f ? 1.f / z : 0.f) : 1.f;
                const int r = w.rb * N + tid;
                if (!whole) {
                    g.part_ml[(pidx * N + tid) * 2] = m;
                    g.part_ml[(pidx * N + tid) * 2 + 1] = z;
                } else if (a.lse && r < g.n_rows) {
                    a.lse[(long long)w.b * g.n_rows + r] = z != 0.f ? (m + log2f(z)) * 0.6931471805599453f : -INFINITY;
                }
            }
            named_sync(1, kSoft);
            wait(&s.o_full, seg & 1);
            tc_after_sync();
            for (int k = 0; k < npair; k++) {
                tmem_ld(lanes + N * (1 + k) + col0, e);
                tmem_ld_wait();
                const int d = 128 * k + t;
#pragma unroll
                for (int c = 0; c < NC; c++) {
                    const int r = w.rb * N + col0 + c;
                    if (r >= g.n_rows) break;
                    const float v = __uint_as_float(e[c]) * s.linv[col0 + c];
                    const long long o = ((long long)w.b * g.n_rows + r) * a.c.L + d;
                    if (!whole) g.part[(pidx * N + col0 + c) * a.c.L + d] = v;
                    else if (a.out_bf16) reinterpret_cast<__nv_bfloat16 *>(a.out)[o] = __float2bfloat16_rn(v);
                    else reinterpret_cast<float *>(a.out)[o] = v;
                }
            }
            tc_before_sync();
            named_sync(1, kSoft);
            seg++;
        }
    } else if constexpr (E4M3) {
        // ---------------------------------------------------------- loaders: codes -> f16
        const int lt = tid - kSoft, col = lt & 7, row = lt >> 3, rcol = lt & 3, rrow = lt >> 2;
        const bool rope_live = rcol < a.c.R / 16;
        uint4 x[kMaxPairs][4], xr[2];
        Walk w(a, g, s, slot);             // the tile whose slots are looked up next
        int my_slot = -1;
        float my_scale = 0.f;
        auto look_up = [&] {
            my_slot = -1;
            if (lt < kTile && w.valid()) my_slot = token_slot(a, w.b, w.tile() * kTile + lt, w.len);
        };
        auto load = [&](const int *slots, int p) {
#pragma unroll
            for (int i = 0; i < 4; i++) {
                const int sl = slots[row + 32 * i];
                x[p][i] = sl >= 0 ? ld_stream(mla_row(a.c, sl) + 128 * p + 16 * col) : make_uint4(0u, 0u, 0u, 0u);
            }
        };
        auto load_rope = [&](const int *slots) {
#pragma unroll
            for (int i = 0; i < 2; i++) {
                const int sl = slots[rrow + 64 * i];
                xr[i] = sl >= 0 && rope_live ? ld_stream(mla_row(a.c, sl) + a.c.L + 16 * rcol) : make_uint4(0u, 0u, 0u, 0u);
            }
        };
        // 16 codes of token r -> units u, u + 1 of the block; `odd` swaps the two stores' order so that the
        // eight lanes of a store phase, which hit two blocks, use all banks once
        auto put = [&](uint32_t blk, int r, int u, uint4 c, bool odd) {
            const uint4 lo = make_uint4(e4m3x2_f16x2(c.x & 0xFFFF), e4m3x2_f16x2(c.x >> 16), e4m3x2_f16x2(c.y & 0xFFFF), e4m3x2_f16x2(c.y >> 16));
            const uint4 hi = make_uint4(e4m3x2_f16x2(c.z & 0xFFFF), e4m3x2_f16x2(c.z >> 16), e4m3x2_f16x2(c.w & 0xFFFF), e4m3x2_f16x2(c.w >> 16));
            uint8_t *d = sm + blk * kBlk + r * 128;
            *reinterpret_cast<uint4 *>(d + (((u + odd) ^ (r & 7)) << 4)) = odd ? hi : lo;
            *reinterpret_cast<uint4 *>(d + (((u + !odd) ^ (r & 7)) << 4)) = odd ? lo : hi;
        };
        look_up();
        if (lt < kTile) {
            s.slot[0][lt] = my_slot;
            my_scale = my_slot >= 0 ? a.c.scales[my_slot] : 0.f;
        }
        named_sync(2, 256);
        bool more = w.valid();
        if (more) {
#pragma unroll
            for (int p = 0; p < kMaxPairs; p++)
                if (p < npair) load(s.slot[0], p);
            load_rope(s.slot[0]);
            w.next();
            look_up();
        }
        for (int it = 0; more; it++) {
            const int *next = s.slot[(it + 1) & 1];
            more = w.valid();
            if (lt < kTile) {
                s.scale[it & 1][lt] = my_scale;
                s.slot[(it + 1) & 1][lt] = my_slot;
                my_scale = my_slot >= 0 ? a.c.scales[my_slot] : 0.f;
            }
            named_sync(2, 256);
            if (more) {
                w.next();
                look_up();
            }
#pragma unroll
            for (int p = 0; p <= kMaxPairs; p++) {
                if (p < kMaxPairs && p >= npair) continue;
                const int bar = p < kMaxPairs ? p : npair;
                if (it > 0) wait(&s.empty[bar], (it - 1) & 1);
                if (p < kMaxPairs) {
#pragma unroll
                    for (int i = 0; i < 4; i++) put(2 * p + (col >> 2), row + 32 * i, 2 * (col & 3), x[p % kMaxPairs][i], col >= 4);
                } else {
#pragma unroll
                    for (int i = 0; i < 2; i++) put(nblk - 1, rrow + 64 * i, 2 * rcol, xr[i], false);
                }
                fence_async_smem();
                __syncwarp();
                if (lane == 0 && ok) mbar_arrive(&s.full[bar]);
                if (more) {
                    if (p < kMaxPairs) load(next, p % kMaxPairs);
                    else load_rope(next);
                }
            }
        }
    } else {
        // ---------------------------------------------------------- bulk copies of bf16 rows
        const int nbox = kTile / g.pbox;
        int it = 0;
        for (Walk w(a, g, s, slot); w.valid(); w.next(), it++) {
            const int tk = w.tile() * kTile + lane * g.pbox;
            const int sl = lane < nbox ? token_slot(a, w.b, tk, w.len) : -1;
            const uint32_t boxes = __popc(__ballot_sync(0xffffffffu, sl >= 0));
            for (int p = 0; p <= npair; p++) {
                if (it > 0) wait(&s.empty[p], (it - 1) & 1);
                const int nb = p < npair ? 2 : 1;
                if (lane == 0 && ok) mbar_expect_tx(&s.full[p], boxes * g.pbox * 128 * nb);
                __syncwarp();
                if (sl >= 0 && ok)
                    for (int k = 0; k < nb; k++)
                        tma_box(base + (2 * p + k) * kBlk + lane * g.pbox * 128, &map, 64 * (2 * p + k), sl, &s.full[p]);
            }
        }
        // every copy has landed before the CTA may end
        if (it > 0) {
            const uint64_t late = global_ns() + 200000000ull;
            volatile int none = 0;
            for (int p = 0; p <= npair; p++) warp_wait(&s.full[p], (it - 1) & 1, late, &none, lane);
        }
    }
    tc_before_sync();
    __syncthreads();
    if (warp == 0) {
        tc_after_sync();
        tmem_free(tmem, kCols);
    }
}

// Joins the partial results of the sequences that more than one group worked on:
// weights 2^(m - max m), four slices of the parts per row, in a fixed order.
template <int N>
__global__ void __launch_bounds__(512) mla_join_kernel(const MlaAttendArgs a, const Geometry g) {
    __shared__ float s_w[512];
    __shared__ float4 s_o[4][128];
    __shared__ float s_m[16], s_l[16];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    pdl_wait();
    pdl_trigger();
    const int total = g.prefix[a.n_seq], chunk = (total + g.n_groups - 1) / g.n_groups;
    for (long long row = blockIdx.x; row < (long long)a.n_seq * g.n_rows; row += gridDim.x) {
        const int b = (int)(row / g.n_rows), r = (int)(row - (long long)b * g.n_rows);
        const int p = g.prefix[b], g0 = p / chunk, g1 = (g.prefix[b + 1] - 1) / chunk;
        if (g0 == g1) continue;
        const int rb = r / N, c = r - rb * N, n = g1 - g0 + 1;
        auto part = [&](int k) { return (((long long)(g0 + k) * g.nrb + rb) * 2 + (k == 0 ? 1 : 0)) * N + c; };
        float m = -INFINITY, z = 0.f;
        if (tid < n) {
            const float2 ml = *reinterpret_cast<const float2 *>(g.part_ml + part(tid) * 2);
            m = ml.x;
            z = ml.y;
        }
        float M = m;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
        if (lane == 0) s_m[warp] = M;
        __syncthreads();
        M = s_m[0];
        for (int w = 1; w < 16; w++) M = fmaxf(M, s_m[w]);
        const float f = m == -INFINITY ? 0.f : ex2(m - M);
        s_w[tid] = f;
        z = warp_sum(z * f);
        if (lane == 0) s_l[warp] = z;
        __syncthreads();
        z = 0.f;
        for (int w = 0; w < 16; w++) z += s_l[w];
        const int slice = tid >> 7, q = tid & 127;
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
        if (4 * q < a.c.L) {
#pragma unroll 8
            for (int k = slice; k < n; k += 4) {
                const float4 v = *reinterpret_cast<const float4 *>(g.part + part(k) * a.c.L + 4 * q);
                const float f = s_w[k];
                o = make_float4(fmaf(v.x, f, o.x), fmaf(v.y, f, o.y), fmaf(v.z, f, o.z), fmaf(v.w, f, o.w));
            }
        }
        s_o[slice][q] = o;
        __syncthreads();
        if (slice == 0 && 4 * q < a.c.L) {
            const float inv = z != 0.f ? 1.f / z : 0.f;
            for (int k = 1; k < 4; k++) {
                const float4 v = s_o[k][q];
                o = make_float4(o.x + v.x, o.y + v.y, o.z + v.z, o.w + v.w);
            }
            o = make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv);
            if (a.out_bf16)
                *reinterpret_cast<uint2 *>(reinterpret_cast<__nv_bfloat16 *>(a.out) + row * a.c.L + 4 * q) =
                    make_uint2(pack_bf16(o.x, o.y), pack_bf16(o.z, o.w));
            else
                *reinterpret_cast<float4 *>(reinterpret_cast<float *>(a.out) + row * a.c.L + 4 * q) = o;
        }
        if (a.lse && tid == 0) a.lse[row] = z != 0.f ? (M + log2f(z)) * 0.6931471805599453f : -INFINITY;
        __syncthreads();
    }
}

int columns_of(int n_rows) { return n_rows <= 16 ? 16 : n_rows <= 32 ? 32 : 64; }

// The pieces and scratch of a call: part, part_ml and prefix are offsets from NULL until placed.
Geometry plan(const MlaAttendArgs &a, int n_sm, size_t *bytes) {
    Geometry g{};
    const int N = columns_of(a.n_q * a.H);
    g.n_rows = a.n_q * a.H;
    g.nrb = (g.n_rows + N - 1) / N;
    g.n_slots = g.nrb < n_sm ? g.nrb : n_sm;
    const long long cap = a.pages_stride * a.c.page;
    const long long tiles = (long long)a.n_seq * ((cap < (1LL << 31) ? cap : (1LL << 31)) / kTile + 1);
    long long ng = n_sm / g.n_slots;
    if (ng > tiles) ng = tiles;
    g.n_groups = (int)ng;
    size_t at = 0;
    if (g.n_groups > 1) {
        const size_t parts = (size_t)g.n_groups * g.nrb * 2 * N;
        g.part = (float *)at;
        at += parts * a.c.L * sizeof(float);
        g.part_ml = (float *)at;
        at += parts * 2 * sizeof(float);
        g.prefix = (int *)at;
        at += ((size_t)a.n_seq + 1) * sizeof(int);
    }
    g.pbox = 128;
    while (a.c.page % g.pbox) g.pbox /= 2;
    g.timeout_ns = 2000000000LL;
    *bytes = at;
    return g;
}

cudaError_t row_map(const MlaCache &c, int pbox, CUtensorMap *out) {
    static PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
        void *p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) != cudaSuccess ||
            q != cudaDriverEntryPointSuccess)
            p = nullptr;
        return (PFN_cuTensorMapEncodeTiled_v12000)p;
    }();
    if (!fn) return cudaErrorNotSupported;
    const cuuint64_t dims[2] = {(cuuint64_t)(c.L + c.R), (cuuint64_t)c.n_pages * c.page};
    const cuuint64_t strides[1] = {(cuuint64_t)c.row_bytes};
    const cuuint32_t box[2] = {64, (cuuint32_t)pbox}, estr[2] = {1, 1};
    return fn(out, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, c.rows, dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
              CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS
               ? cudaSuccess
               : cudaErrorInvalidValue;
}

template <int N, bool E4M3>
cudaError_t run(const MlaAttendArgs &a, const Geometry &g, int n_sm, cudaStream_t st) {
    CUtensorMap map{};
    if (!E4M3)
        if (cudaError_t e = row_map(a.c, g.pbox, &map)) return e;
    const int nblk = a.c.L / 64 + 1;
    const size_t smem = (size_t)nblk * kBlk + (size_t)nblk * N * 128 + 1024;
    auto kern = mla_attend_kernel<N, E4M3>;
    if (cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem)) return e;
    if (cudaError_t e = launch_pdl(kern, dim3(g.n_groups * g.n_slots), dim3(E4M3 ? 512 : 288), smem, st, map, a, g)) return e;
    if (g.n_groups == 1) return cudaSuccess;
    const long long rows = (long long)a.n_seq * g.n_rows;
    return launch_pdl(mla_join_kernel<N>, dim3((unsigned)(rows < 4LL * n_sm ? rows : 4LL * n_sm)), dim3(512), 0, st, a, g);
}

template <bool E4M3>
cudaError_t run_columns(const MlaAttendArgs &a, const Geometry &g, int n_sm, cudaStream_t st) {
    switch (columns_of(g.n_rows)) {
    case 16: return run<16, E4M3>(a, g, n_sm, st);
    case 32: return run<32, E4M3>(a, g, n_sm, st);
    default: return run<64, E4M3>(a, g, n_sm, st);
    }
}

}  // namespace

size_t mla_attend_scratch(const MlaAttendArgs &a, int n_sm) {
    size_t bytes;
    plan(a, n_sm, &bytes);
    return bytes;
}

cudaError_t launch_mla_attend(const MlaAttendArgs &a, void *scratch, int n_sm, cudaStream_t st, int *n_launch) {
    size_t bytes;
    Geometry g = plan(a, n_sm, &bytes);
    if (bytes) {
        g.part = (float *)((char *)scratch + (size_t)g.part);
        g.part_ml = (float *)((char *)scratch + (size_t)g.part_ml);
        g.prefix = (int *)((char *)scratch + (size_t)g.prefix);
    }
    *n_launch = g.n_groups > 1 ? 2 : 1;
    return a.c.e4m3 ? run_columns<true>(a, g, n_sm, st) : run_columns<false>(a, g, n_sm, st);
}

}  // namespace coli

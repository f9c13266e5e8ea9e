// mla_attend.cu -- attention over the paged latent cache (absorbed form), on
// the 5th-generation tensor cores: the kernel for bf16 caches, the join of partial
// results, and the plan for both kinds of cache (E4M3: mla_attend_e4m3.cu).
//
// All heads of a token read the same cached rows, so the rows [t][L + R] of a
// tile of 128 tokens are brought into shared memory once and serve both products of
// every head:
//   S^T[t][c] = sum_d row[t][d] q[c][d]      M = 128 tokens, N = columns, K = L + R
//   O^T[d][c] += sum_t row[t][d] P^T[t][c]   M = 128 dims (L/128 times), N = columns, K = 128 tokens
// The rows are the A operand of both: K-major (a token's dims along a row) for S,
// MN-major (the same bytes read across) for O.  A column c is one query row
// (query token j, head h); a CTA has N = 16, 32 or 64 of them.  Tokens are the
// lanes of S^T in TMEM, so one thread holds one token's scores of half the columns.
//
// Softmax.  With x = log2(e) * scale * score and m_c a running reference:
// e = 2^(x - m_c), l_c += e, P = bf16(e).  m_c starts 6 below the first tile's
// maximum and moves only when some e passes 2^14: most tiles need no maximum over
// the lanes and no rescaling of O, and bf16 has its full 8 bits at every e down to
// 2^-126.  A NaN score makes e, and with it l and O, NaN; a score of +infinity does
// so by x - m.  l, m and O are f32.  P and q are rounded to bf16, as the cached rows
// are, because the tensor cores multiply equal types.
//
// Work.  The tiles of all sequences form one line that is cut into
// contiguous pieces, one for each group of CTAs; the CTAs of a group take the
// piece's row blocks side by side, so each row comes from HBM once.  Pieces that
// hold part of a sequence leave (O, m, l) in f32 in scratch, and
// mla_join_kernel adds them up; the rest is written directly.
//
// Bound, L + R = 576, 64 columns: a tile's MMAs read 4 KB of rows each whatever N is, 68 of 45 cycles, 3060 (N = 128: 59
// each, but O would fill TMEM and leave no room for S).  One tile is in shared memory at a time (147 KB beside 74 KB of
// queries), so its scores (2000 cycles), softmax (1240) and outputs (1760) follow one another, 5500 cycles a tile with the
// hand-overs; the copies are hidden, each block of 64 dims being asked for again when its last product is done.
// Measured: 48 sequences of up to 12000 tokens (320000 in all), 128 heads: 137 us, 0.65 PFLOP/s, 2.7 TB/s of the cache; 1 x
// 100000: 55 us with the join's 7; 4 x 9000, 16 heads x 3 queries: 28 us, of which launch, first copies and join are 17.
//
// Warps: 0-7 softmax and output (two threads per token, each half the columns), 8
// MMA issue, 9-11 tiled bulk copies.
// Every wait for another role is bounded, by a limit that each part of a sequence
// renews; after one has run out all of them return at once, no further MMA or copy is
// issued, and the kernel records DEV_ERR_TIMEOUT.  Named barriers join the softmax warps
// alone, which pass the same ones whatever has run out.
#include <cudaTypedefs.h>

#include "mla_attend.cuh"

namespace coli {

namespace {

constexpr uint32_t kBlk = kTile * 128;   // 128 tokens x 64 dims of 16 bits, 128-byte swizzle
constexpr int kCopyWarps = 3;            // a warp's copy takes some 500 cycles to issue, so several share a tile
constexpr int kThreads = 32 * (9 + kCopyWarps);
constexpr int kMaxPairs = 4;             // pairs of blocks: L / 128
constexpr float kHead = 6.f;             // log2 of the largest weight of a fresh reference
constexpr float kLimit = 14.f;           // log2 of the weight that moves the reference

struct Shared {
    uint64_t full[kMaxPairs + 1], empty[kMaxPairs + 1], s_full, p_full, o_full, q_full, q_empty;   // q_full: by copies or by a softmax thread
    uint32_t tmem;
    int abort;
    Piece piece;
    alignas(16) float f[64];
    alignas(16) float m[2][64];       // minus the reference; read as float4, like f
    float linv[64], r[64];
    int limit[64];
    float red[4][64];
};

// f32 query rows of a block of N -> bf16 operand [L/64 + 1][N][64], 128-byte swizzle (bf16 ones are copied as boxes).
// The softmax threads share the block's units of 8 elements, five in flight each.
template <int N>
__device__ __forceinline__ void load_queries(const MlaAttendArgs &a, const AttendPlan &g, uint8_t *qsm, int b, int rb, int tid) {
    constexpr int F = 5;
    const int upr = (a.c.L + a.c.R) / 8, total = N * upr;
#pragma unroll 1
    for (int i0 = tid; i0 < total; i0 += F * kSoft) {
        uint4 x[F][2];
#pragma unroll
        for (int f = 0; f < F; f++) {
            const int i = i0 + f * kSoft, c = i / upr, u = i - c * upr, r = rb * N + c;
            const bool live = i < total && r < g.n_rows;
            const uint4 *src = query_unit<false>(a, (long long)b * g.n_rows + (live ? r : 0), live ? u : 0);
#pragma unroll
            for (int w = 0; w < 2; w++) x[f][w] = live ? __ldg(src + w) : make_uint4(0u, 0u, 0u, 0u);
        }
#pragma unroll
        for (int f = 0; f < F; f++) {
            const int i = i0 + f * kSoft, c = i / upr, u = i - c * upr;
            if (i >= total) break;
            auto pack = [](uint32_t lo, uint32_t hi) { return pack_bf16(__uint_as_float(lo), __uint_as_float(hi)); };
            *reinterpret_cast<uint4 *>(qsm + (u >> 3) * (N * 128) + c * 128 + (((u & 7) ^ (c & 7)) << 4)) =
                make_uint4(pack(x[f][0].x, x[f][0].y), pack(x[f][0].z, x[f][0].w), pack(x[f][1].x, x[f][1].y), pack(x[f][1].z, x[f][1].w));
        }
    }
}

template <int N>
__global__ void __launch_bounds__(kThreads, 1) mla_attend_bf16_kernel(const __grid_constant__ CUtensorMap map, const __grid_constant__ CUtensorMap q_map,
                                                                              const __grid_constant__ CUtensorMap qr_map, const MlaAttendArgs a, const AttendPlan g) {
    constexpr int NC = N / 2;              // columns per softmax thread
    extern __shared__ uint8_t raw[];
    __shared__ Shared s;
    const uint32_t base = (smem_addr(raw) + 1023u) & ~1023u;
    uint8_t *sm = raw + (base - smem_addr(raw));
    // the shuffles tell the compiler that these are the same in a whole warp, so that MMA operands live in uniform registers
    const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
    const int npair = a.c.L / 128, nblk = 2 * npair + 1;
    const uint32_t q_off = nblk * kBlk;    // queries [nblk][N][64]
    const uint32_t p_off = (nblk - 1) * kBlk;   // P^T [128][64], in the rope block's place once S is done
    constexpr uint32_t kCols = N == 64 ? 512 : N == 32 ? 256 : 128;   // S, then O: (1 + L/128) * N <= 5 N
    pdl_wait();
    pdl_trigger();

    if (warp == 0) tmem_alloc(&s.tmem, kCols);
    if (tid == 0) {
        for (int p = 0; p <= kMaxPairs; p++) {
            mbar_init(&s.full[p], 1);
            mbar_init(&s.empty[p], 1);
        }
        mbar_init(&s.s_full, 1);
        mbar_init(&s.p_full, 1);
        mbar_init(&s.o_full, 1);
        mbar_init(&s.q_full, 1);
        mbar_init(&s.q_empty, 1);
        s.abort = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    const int group = blockIdx.x / g.n_slots, slot = blockIdx.x - group * g.n_slots;
    if (warp == 0) find_piece(a, g, group, lane, s.piece);
    tc_before_sync();
    __syncthreads();
    tc_after_sync();
    const uint32_t tmem = __shfl_sync(0xffffffffu, s.tmem, 0);
    volatile int *abort = &s.abort;
    uint64_t deadline = deadline_after(g.wait_ns, 0);
    bool ok = true;                        // this thread's waits have all ended well
    auto wait = [&](uint64_t *bar, uint32_t parity) {
        if (!ok) return;
        if (!warp_wait_now(bar, parity, deadline, abort, lane)) {
            ok = false;
            *abort = 1;
            atomicCAS(a.err, 0, (int)DEV_ERR_TIMEOUT);
        }
    };

    // the MMAs of a tile, issued by one warp
    constexpr int kMmaWarp = 8;
    constexpr uint32_t id_s = f16_idesc(1, false, false, kTile, N), id_o = f16_idesc(1, true, true, 128, N);
    const uint64_t dk = sw128_desc(base, 16, 1024), dq = sw128_desc(base + q_off, 16, 1024);
    const uint64_t dv = sw128_desc(base, kBlk, 1024), dp = sw128_desc(base + p_off, kBlk, 1024);
    auto issue_scores = [&](int it) {
        for (int p = 0; p < npair; p++) {
            wait(&s.full[p], it & 1);
            tc_after_sync();
            if (ok) {
#pragma unroll
                for (int k = 0; k < 8; k++)
                    mma_ss(tmem, dk + ((2 * p * kBlk) >> 4) + (((k >> 2) * kBlk + (k & 3) * 32) >> 4),
                           dq + ((2 * p * N * 128) >> 4) + (((k >> 2) * (N * 128) + (k & 3) * 32) >> 4), id_s, k || p);
            }
        }
        wait(&s.full[npair], it & 1);
        tc_after_sync();
        if (ok) {
#pragma unroll
            for (int k = 0; k < 4; k++)
                if (k < a.c.R / 16)
                    mma_ss(tmem, dk + (((nblk - 1) * kBlk) >> 4) + ((k * 32) >> 4), dq + (((nblk - 1) * N * 128) >> 4) + ((k * 32) >> 4), id_s, true);
            tc_commit(&s.s_full);
        }
    };
    auto issue_output = [&](bool first, bool last) {
        tc_after_sync();
        if (ok) {
            for (int p = 0; p < npair; p++) {
#pragma unroll
                for (int k = 0; k < 8; k++)
                    mma_ss(tmem + N * (1 + p), dv + ((2 * p * kBlk + k * 2048) >> 4), dp + ((k * 2048) >> 4), id_o, k || !first);
                tc_commit(&s.empty[p]);
            }
            tc_commit(&s.empty[npair]);
            if (last) tc_commit(&s.o_full);
        }
        __syncwarp();
    };

    if (warp < 8) {
        // ---------------------------------------------------------- softmax and output
        const int wq = warp & 3, grp = warp >> 2;
        const int t = 32 * wq + lane;                                   // token of the tile, and dim of an O block
        const uint32_t lanes = tmem + ((uint32_t)(32 * wq) << 16);
        const uint32_t col0 = grp * NC;
        float2 l[NC / 2];
        int it = 0, seg = 0, cur = 0;
        for (Walk w(a, g, s.piece, slot); w.valid(); w.next(), it++) {
            if (w.first()) {
                deadline = deadline_after(g.wait_ns, w.rest());
                if (!a.q_bf16) load_queries<N>(a, g, sm + q_off, w.b, w.rb, tid);
                if (tid < N) {
                    const int r = w.rb * N + tid;
                    s.f[tid] = a.scale * 1.4426950408889634f;
                    s.limit[tid] = r < g.n_rows ? w.len - (a.n_q - 1 - r / a.H) : 0;
                }
                if (tid < N) s.m[cur][tid] = -kNone;
#pragma unroll
                for (int c = 0; c < NC / 2; c++) l[c] = make_float2(0.f, 0.f);
                fence_async_smem();
                named_sync(1, kSoft);
                if (!a.q_bf16 && tid == 0 && ok) mbar_arrive(&s.q_full);   // behind the barrier: for all of them
            }
            const int tok = w.tile() * kTile + t;
            // every column sees the whole tile: the first query's limit is the lowest
            const bool full = (w.tile() + 1) * kTile <= w.len - (a.n_q - 1) && (w.rb + 1) * N <= g.n_rows;
            wait(&s.s_full, it & 1);
            tc_after_sync();
            if ((w.tile() + 1) * kTile > w.len - a.n_q + 1) {
                // 0 * NaN is NaN.  Rows past the length may hold anything: zero.  Of the newest tokens' rows, which not every
                // query sees, what is not finite: the queries that see it have it in their scores.  Every score of such a row
                // is not finite, so one tells (looking at the rows of 4 x 9000 tokens, 3 queries each, costs 1.1 of 29 us).
                bool clear = false;
                if (a.n_q > 1) {
                    uint32_t v[8];
                    tmem_ld(lanes + col0, v);
                    tmem_ld_wait();
                    clear = tok > w.len - a.n_q && !finite_bits(v[0]);
                }
                if (tok >= w.len) {
                    for (int k = grp; k < 2 * npair; k += 2)
#pragma unroll
                        for (int u = 0; u < 8; u++) *reinterpret_cast<uint4 *>(sm + k * kBlk + t * 128 + 16 * u) = make_uint4(0u, 0u, 0u, 0u);
                } else if (clear) {
#pragma unroll 1
                    for (int i = 0; i < 8 * npair; i++) {
                        uint4 *at = reinterpret_cast<uint4 *>(sm + (grp + 2 * (i >> 3)) * kBlk + t * 128 + 16 * (i & 7));
                        uint4 x = *at;
                        for (uint32_t *e : {&x.x, &x.y, &x.z, &x.w}) *e &= ~__vcmpeq2(*e & 0x7F807F80u, 0x7F807F80u);
                        *at = x;
                    }
                }
            }
            // Columns in chunks: a thread's 32 scores and 32 sums at once would not fit its registers.
            constexpr int CH = NC < 16 ? NC : 16;
            // Weights of a chunk against the current reference, 2^min(x - m, 100), and the largest x - m (before the clamp).
            auto weigh = [&](int c0, float2 (&x)[CH / 2], float &top) {
                uint32_t v[CH];
                tmem_ld(lanes + col0 + c0, v);
                tmem_ld_wait();
#pragma unroll
                for (int c = 0; c < CH; c += 4) {
                    const float4 f = *reinterpret_cast<const float4 *>(&s.f[col0 + c0 + c]);
                    const float4 m = *reinterpret_cast<const float4 *>(&s.m[cur][col0 + c0 + c]);   // minus the reference
                    float2 y0 = make_float2(__uint_as_float(v[c]), __uint_as_float(v[c + 1]));
                    float2 y1 = make_float2(__uint_as_float(v[c + 2]), __uint_as_float(v[c + 3]));
                    x[c / 2] = make_float2(m.x, m.y);
                    x[c / 2 + 1] = make_float2(m.z, m.w);
                    ffma2(x[c / 2], y0, make_float2(f.x, f.y));
                    ffma2(x[c / 2 + 1], y1, make_float2(f.z, f.w));
                }
                if (!full)
#pragma unroll
                    for (int c = 0; c < CH; c += 2) {
                        if (tok >= s.limit[col0 + c0 + c]) x[c / 2].x = -INFINITY;
                        if (tok >= s.limit[col0 + c0 + c + 1]) x[c / 2].y = -INFINITY;
                    }
#pragma unroll
                for (int c = 0; c < CH / 2; c++) {
                    top = fmaxf(top, fmaxf(x[c].x, x[c].y));
                    x[c] = make_float2(ex2(min_nan(x[c].x, 100.f)), ex2(min_nan(x[c].y, 100.f)));
                }
            };
            auto add = [&](float sign) {       // l += sign * weights, and P for sign > 0; true if a weight has outgrown P
                float top = -INFINITY;
#pragma unroll
                for (int c0 = 0; c0 < NC; c0 += CH) {
                    float2 x[CH / 2];
                    weigh(c0, x, top);
#pragma unroll
                    for (int c = 0; c < CH / 2; c++) l[c0 / 2 + c] = sign > 0.f ? fadd2(l[c0 / 2 + c], x[c]) : fadd2(l[c0 / 2 + c], make_float2(-x[c].x, -x[c].y));
                    if (sign < 0.f) continue;
#pragma unroll
                    for (int u = 0; u < CH / 8; u++) {
                        uint32_t pk[4];
#pragma unroll
                        for (int k = 0; k < 4; k++) {
                            const float2 y = x[4 * u + k];
                            pk[k] = pack_bf16(y.x, y.y);
                        }
                        *reinterpret_cast<uint4 *>(sm + p_off + t * 128 + (((grp * (NC / 8) + c0 / 8 + u) ^ (t & 7)) << 4)) =
                            make_uint4(pk[0], pk[1], pk[2], pk[3]);
                    }
                }
                return top > kLimit;
            };
            bool move = w.first();
            if (!move) {
                const bool big = add(1.f);
                fence_async_smem();
                tc_before_sync();
                move = named_or(1, kSoft, big);
                // taking the weights off again is exact to an ulp of the sums with them, which the new reference
                // scales to 2^-24 of its own weights or less
                if (move) add(-1.f);
            }
            if (move) {
                uint32_t v[NC];
                float x[NC];
                tmem_ld(lanes + col0, v);
                tmem_ld_wait();
#pragma unroll
                for (int c = 0; c < NC; c++) {
                    x[c] = __uint_as_float(v[c]) * s.f[col0 + c];
                    if (!full && tok >= s.limit[col0 + c]) x[c] = -INFINITY;
                }
                const float top = reduce_columns(x, lane, [](float p, float q) { return fmaxf(p, q); });
                if (lane % (32 / NC) == 0) s.red[wq][col0 + lane / (32 / NC)] = top;
                named_sync(1, kSoft);
                if (tid < N) {
                    // s.m holds minus the reference
                    const float old = -s.m[cur][tid];
                    const float x = fmaxf(fmaxf(s.red[0][tid], s.red[1][tid]), fmaxf(s.red[2][tid], s.red[3][tid]));
                    const float now = x > old + kLimit ? x - kHead : old;   // only the columns that need it
                    s.m[cur ^ 1][tid] = -now;
                    s.r[tid] = ex2(old - now);
                }
                named_sync(1, kSoft);
                cur ^= 1;
                if (!w.first()) {
#pragma unroll
                    for (int c = 0; c < NC / 2; c++) l[c] = fmul2(l[c], make_float2(s.r[col0 + 2 * c], s.r[col0 + 2 * c + 1]));
#pragma unroll 1
                    for (int k = 0; k < npair * (NC / 8); k++) {
                        const uint32_t at = lanes + N * (1 + k / (NC / 8)) + col0 + 8 * (k % (NC / 8));
                        float r[8];
                        bool same = true;
#pragma unroll
                        for (int c = 0; c < 8; c++) {
                            r[c] = s.r[col0 + 8 * (k % (NC / 8)) + c];
                            same = same && r[c] == 1.f;
                        }
                        if (same) continue;
                        uint32_t o[8];
                        tmem_ld(at, o);
                        tmem_ld_wait();
#pragma unroll
                        for (int c = 0; c < 8; c++) o[c] = __float_as_uint(__uint_as_float(o[c]) * r[c]);
                        tmem_st(at, o);
                    }
                    tmem_st_wait();
                }
                add(1.f);
                fence_async_smem();
                tc_before_sync();
                named_sync(1, kSoft);
            }
            if (tid == 0 && ok) mbar_arrive(&s.p_full);                    // likewise
            if (!w.last()) continue;

            // ------------------------------------------------------ this part of the sequence is done
            {
                float z[NC];
#pragma unroll
                for (int c = 0; c < NC; c++) z[c] = c & 1 ? l[c / 2].y : l[c / 2].x;
                const float sum = reduce_columns(z, lane, [](float p, float q) { return p + q; });
                if (lane % (32 / NC) == 0) s.red[wq][col0 + lane / (32 / NC)] = sum;
            }
            named_sync(1, kSoft);
            const bool whole = w.whole();
            const long long pidx = ((long long)group * g.nrb + w.rb) * 2 + w.which();
            if (tid < N) {
                const float z = s.red[0][tid] + s.red[1][tid] + s.red[2][tid] + s.red[3][tid];
                const float m = -s.m[cur][tid];
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
            const long long row = (long long)w.b * g.n_rows + w.rb * N + col0;
            const int rows = min(NC, g.n_rows - w.rb * N - (int)col0);
#pragma unroll 1
            for (int k = 0; k < npair; k++) {
                uint32_t o[NC];
                tmem_ld(lanes + N * (1 + k) + col0, o);
                tmem_ld_wait();
                const int d = 128 * k + t;
                if (!whole) {
                    float *dst = g.part + (pidx * N + col0) * a.c.L + d;
#pragma unroll
                    for (int c = 0; c < NC; c++)
                        if (c < rows) dst[c * a.c.L] = __uint_as_float(o[c]);
                } else {
#pragma unroll
                    for (int c = 0; c < NC; c++)
                        if (c < rows) store_out(a, (row + c) * a.c.L + d, __uint_as_float(o[c]) * s.linv[col0 + c]);
                }
            }
            tc_before_sync();
            named_sync(1, kSoft);
            seg++;
        }
    } else if (warp == kMmaWarp) {
        // ---------------------------------------------------------- MMA issue
        int it = 0, seg = 0;
        for (Walk w(a, g, s.piece, slot); w.valid(); w.next(), it++) {
            if (w.first()) {
                deadline = deadline_after(g.wait_ns, w.rest());
                wait(&s.q_full, seg++ & 1);
            }
            issue_scores(it);
            if (w.last() && ok) tc_commit(&s.q_empty);
            wait(&s.p_full, it & 1);
            issue_output(w.first(), w.last());
        }
    } else {
        // ---------------------------------------------------------- bulk copies of bf16 rows
        const int who = warp - kMmaWarp - 1;
        BoxAhead box(a, g, s.piece, slot, lane, who == 1);
        int it = 0, seg = 0;
        for (Walk w(a, g, s.piece, slot); w.valid(); w.next(), box.next(), it++) {
            if (w.first()) deadline = deadline_after(g.wait_ns, w.rest());
            const int sl = box.slot[0], nbox = kTile / g.pbox;
            const uint32_t live = __ballot_sync(0xffffffffu, sl >= 0), n = __popc(live) * g.pbox;
            const int y0 = __shfl_sync(0xffffffffu, sl, 0);
            if (who == kCopyWarps - 1 && a.q_bf16 && w.first()) {
                // the block's queries; rows past the sequence's are its neighbour's or zero, and masked
                if (seg > 0) wait(&s.q_empty, (seg - 1) & 1);
                seg++;
                if (ok) {
                    const int y = w.b * g.n_rows + w.rb * N;
                    expect_bytes(&s.q_full, nblk * N * 128);
                    for (int k = 0; k < nblk - 1; k++) tma_box(base + q_off + k * (N * 128), &q_map, 64 * k, y, &s.q_full);
                    tma_box(base + q_off + (nblk - 1) * (N * 128), &qr_map, 0, y, &s.q_full);
                }
            }
            for (int p = who; p <= npair; p += kCopyWarps) {
                const uint32_t dst = base + 2 * p * kBlk;
                if (it > 0) wait(&s.empty[p], (it - 1) & 1);
                if (!ok) continue;
                const bool two = p < npair;
                expect_bytes(&s.full[p], n * (two ? 256 : 128));
                if (live & 1) {
                    tma_box(dst, &map, 128 * p, y0, &s.full[p]);
                    if (two) tma_box(dst + kBlk, &map, 128 * p + 64, y0, &s.full[p]);
                }
                for (int j = 1; j < nbox; j++) {
                    const int y = __shfl_sync(0xffffffffu, sl, j);
                    if (!(live >> j & 1)) continue;
                    tma_box(dst + j * g.pbox * 128, &map, 128 * p, y, &s.full[p]);
                    if (two) tma_box(dst + kBlk + j * g.pbox * 128, &map, 128 * p + 64, y, &s.full[p]);
                }
            }
            __syncwarp();
        }
        // every copy has landed before the CTA may end
        if (it > 0) {
            const uint64_t late = global_ns() + 200000000ull;
            volatile int none = 0;
            if (seg > 0) warp_wait(&s.q_full, (seg - 1) & 1, late, &none, lane);
            for (int p = who; p <= npair; p += kCopyWarps) warp_wait(&s.full[p], (it - 1) & 1, late, &none, lane);
        }
    }
    tc_before_sync();
    __syncthreads();
    if (warp == 0) {
        if (*abort) settle();
        tc_after_sync();
        tmem_free(tmem, kCols);
    }
}

// Joins the partial results of the sequences that more than one group worked on, with weights 2^(m - max m).
// wpr warps (a power of two up to 16) share a row's parts, each lane with 4 dims of every 128; their sums meet in
// shared memory in a fixed order.  Many rows (a batch): one warp each; few rows of many parts (a long context): 16.
__global__ void __launch_bounds__(512) mla_join_kernel(const MlaAttendArgs a, const AttendPlan g, int wpr) {
    __shared__ float4 s_o[16][128];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, sub = warp & (wpr - 1), rpb = 16 / wpr;
    pdl_wait();
    pdl_trigger();
    const int nd = a.c.L / 128;
    const int rows = a.n_seq * g.n_rows;
    for (int row0 = blockIdx.x * rpb; row0 < rows; row0 += gridDim.x * rpb) {
        const int row = row0 + warp / wpr;
        int r = 0;
        int2 piece = make_int2(0, 1);
        if (row < rows) {
            const int b = row / g.n_rows;
            r = row - b * g.n_rows;
            piece = g.pieces[b];
        }
        const int g0 = piece.x, n = piece.y, rb = r / g.cols, c = r - rb * g.cols;
        auto part = [&](int k) { return (((long long)(g0 + k) * g.nrb + rb) * 2 + (k == 0 ? 1 : 0)) * g.cols + c; };
        float4 o[4];
        float M = -INFINITY, z = 0.f;
#pragma unroll
        for (int d = 0; d < 4; d++) o[d] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (n > 1) {
            // the first two parts are asked for before the maxima are known: one round trip for both (four: the same times)
            constexpr int F = 2;
            float4 v[F][4];
            float mk[F];
            auto load = [&](int k, float4 (&x)[4], float &m) {
                const float *src = g.part + part(k) * a.c.L + 4 * lane;
                m = g.part_ml[part(k) * 2];
#pragma unroll
                for (int d = 0; d < 4; d++)
                    if (d < nd) x[d] = __ldcs(reinterpret_cast<const float4 *>(src + 128 * d));
            };
#pragma unroll
            for (int i = 0; i < F; i++)
                if (sub + i * wpr < n) load(sub + i * wpr, v[i], mk[i]);
            float2 ml = make_float2(-INFINITY, 0.f);
            if (lane < n) ml = *reinterpret_cast<const float2 *>(g.part_ml + part(lane) * 2);
            M = ml.x;
            for (int k = lane + 32; k < n; k += 32) M = fmaxf(M, g.part_ml[part(k) * 2]);
#pragma unroll
            for (int s = 16; s > 0; s >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, s));
            z = lane < n ? ml.y * ex2(ml.x - M) : 0.f;
            for (int k = lane + 32; k < n; k += 32) {
                ml = *reinterpret_cast<const float2 *>(g.part_ml + part(k) * 2);
                z = fmaf(ml.y, ex2(ml.x - M), z);
            }
            z = warp_sum(z);
            for (int k0 = sub; k0 < n; k0 += F * wpr) {
#pragma unroll
                for (int i = 0; i < F; i++) {
                    const int k = k0 + i * wpr;
                    if (k >= n) break;
                    if (k0 != sub) load(k, v[i], mk[i]);
                }
#pragma unroll
                for (int i = 0; i < F; i++) {
                    if (k0 + i * wpr >= n) break;
                    const float f = ex2(mk[i] - M);
#pragma unroll
                    for (int d = 0; d < 4; d++)
                        if (d < nd) o[d] = make_float4(fmaf(v[i][d].x, f, o[d].x), fmaf(v[i][d].y, f, o[d].y), fmaf(v[i][d].z, f, o[d].z), fmaf(v[i][d].w, f, o[d].w));
                }
            }
        }
        if (wpr > 1) {
#pragma unroll
            for (int d = 0; d < 4; d++) s_o[warp][32 * d + lane] = o[d];
            __syncthreads();
            if (sub == 0)
                for (int w = 1; w < wpr; w++)
#pragma unroll
                    for (int d = 0; d < 4; d++) {
                        const float4 v = s_o[warp + w][32 * d + lane];
                        o[d] = make_float4(o[d].x + v.x, o[d].y + v.y, o[d].z + v.z, o[d].w + v.w);
                    }
            __syncthreads();
        }
        if (n == 1 || sub != 0) continue;
        const float inv = z != 0.f ? 1.f / z : 0.f;
#pragma unroll
        for (int d = 0; d < 4; d++) {
            if (d >= nd) break;
            const long long e = (long long)row * a.c.L + 128 * d + 4 * lane;
            const float4 v = make_float4(o[d].x * inv, o[d].y * inv, o[d].z * inv, o[d].w * inv);
            if (a.out_bf16)
                *reinterpret_cast<uint2 *>(reinterpret_cast<__nv_bfloat16 *>(a.out) + e) = make_uint2(pack_bf16(v.x, v.y), pack_bf16(v.z, v.w));
            else
                *reinterpret_cast<float4 *>(reinterpret_cast<float *>(a.out) + e) = v;
        }
        if (a.lse && lane == 0) a.lse[row] = z != 0.f ? (M + log2f(z)) * 0.6931471805599453f : -INFINITY;
    }
}

// Columns of a CTA: the fewest that hold the sequence's rows, up to what TMEM and shared memory allow (64, E4M3 with its
// terms 32), as a tile costs nearly the same for any N; and half as many while the tiles that there can be leave half
// the SMs without work (1 x 1000 tokens, 128 heads, E4M3: 32 CTAs of 32 columns 14.8 us, 64 of 16 columns 12.4 us).
int columns_of(bool e4m3, int n_rows, long long tiles, int n_sm) {
    int n = n_rows <= 16 ? 16 : n_rows <= 32 || e4m3 ? 32 : 64;
    while (n > 16 && tiles * ((n_rows + n - 1) / n) * 2 <= n_sm) n /= 2;
    return n;
}

// The pieces and scratch of a call: part, part_ml and pieces are offsets from NULL until placed.
AttendPlan plan(const MlaAttendArgs &a, int n_sm, size_t *bytes) {
    AttendPlan g{};
    g.n_rows = a.n_q * a.H;
    const long long tiles = (long long)a.n_seq * ((a.pages_stride * a.c.page + kTile - 1) / kTile);
    g.cols = columns_of(a.c.e4m3, g.n_rows, tiles, n_sm);
    g.nrb = (g.n_rows + g.cols - 1) / g.cols;
    g.n_slots = g.nrb < n_sm ? g.nrb : n_sm;
    const long long ng = n_sm / g.n_slots;
    g.n_groups = (int)(ng < tiles ? ng : tiles);
    size_t at = 0;
    // sequences of one tile at most are never split
    if (g.n_groups > 1 && a.pages_stride * a.c.page > kTile) {
        const size_t parts = (size_t)g.n_groups * g.nrb * 2 * g.cols;
        g.part = (float *)at;
        at += parts * a.c.L * sizeof(float);
        g.part_ml = (float *)at;
        at += parts * 2 * sizeof(float);
        g.pieces = (int2 *)at;
        at += (size_t)a.n_seq * sizeof(int2);
    }
    g.pbox = kTile;
    while (a.c.page % g.pbox) g.pbox /= 2;
    *bytes = at;
    return g;
}

// Tensor map of packed rows: boxes of `inner` elements x `box_rows`.
cudaError_t encode(const void *p, CUtensorMapDataType type, long long cols, long long rows, long long row_bytes, int inner, int box_rows,
                   CUtensorMapSwizzle swizzle, CUtensorMap *out) {
    static PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
        void *f = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) != cudaSuccess ||
            q != cudaDriverEntryPointSuccess)
            f = nullptr;
        return (PFN_cuTensorMapEncodeTiled_v12000)f;
    }();
    if (!fn) return cudaErrorNotSupported;
    const cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows}, strides[1] = {(cuuint64_t)row_bytes};
    const cuuint32_t box[2] = {(cuuint32_t)inner, (cuuint32_t)box_rows}, estr[2] = {1, 1};
    return fn(out, type, 2, const_cast<void *>(p), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle,
              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS
               ? cudaSuccess
               : cudaErrorInvalidValue;
}
cudaError_t bf16_map(const void *p, int cols, long long rows, int box_rows, CUtensorMap *out) {
    return encode(p, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, cols, rows, 2LL * cols, 64, box_rows, CU_TENSOR_MAP_SWIZZLE_128B, out);
}

template <int N>
cudaError_t run_bf16(const MlaAttendArgs &a, const AttendPlan &g, int device, cudaStream_t st) {
    CUtensorMap map, q, qr;
    if (cudaError_t e = mla_row_map(a.c, 64, g.pbox, CU_TENSOR_MAP_SWIZZLE_128B, &map)) return e;
    q = qr = map;                        // f32 queries: never read
    if (a.q_bf16) {
        const long long rows = (long long)a.n_seq * g.n_rows;
        if (cudaError_t e = bf16_map(a.q_latent, a.c.L, rows, N, &q)) return e;
        if (cudaError_t e = bf16_map(a.q_rope, a.c.R, rows, N, &qr)) return e;
    }
    const int nblk = a.c.L / 64 + 1;
    const size_t smem = (size_t)nblk * kBlk + (size_t)nblk * N * 128 + 1024;
    auto kern = mla_attend_bf16_kernel<N>;
    static std::atomic<uint64_t> done{0};
    if (cudaError_t e = allow_smem(kern, (size_t)9 * (kBlk + N * 128) + 1024, device, done)) return e;   // the largest latent's
    return launch_pdl(kern, dim3(g.n_groups * g.n_slots), dim3(kThreads), smem, st, map, q, qr, a, g);
}

}  // namespace

cudaError_t mla_row_map(const MlaCache &c, int inner, int pbox, CUtensorMapSwizzle swizzle, CUtensorMap *out) {
    return encode(c.rows, c.e4m3 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, c.L + c.R, (long long)c.n_pages * c.page,
                  c.row_bytes, inner, pbox, swizzle, out);
}

size_t mla_attend_scratch(const MlaAttendArgs &a, int n_sm) {
    size_t bytes;
    plan(a, n_sm, &bytes);
    return bytes;
}

cudaError_t launch_mla_attend(const MlaAttendArgs &a, const DevInfo &d, cudaStream_t st, int *n_launch) {
    size_t bytes;
    const int n_sm = d.n_sm;
    AttendPlan g = plan(a, n_sm, &bytes);
    g.wait_ns = d.wait_ns;
    void *scratch = d.scratch;
    if (bytes) {
        g.part = (float *)((char *)scratch + (size_t)g.part);
        g.part_ml = (float *)((char *)scratch + (size_t)g.part_ml);
        g.pieces = (int2 *)((char *)scratch + (size_t)g.pieces);
    }
    *n_launch = g.pieces ? 2 : 1;
    cudaError_t e;
    if (a.c.e4m3) e = launch_mla_attend_e4m3(a, g, d.device, st);
    else e = g.cols == 16 ? run_bf16<16>(a, g, d.device, st) : g.cols == 32 ? run_bf16<32>(a, g, d.device, st) : run_bf16<64>(a, g, d.device, st);
    if (e != cudaSuccess || !g.pieces) return e;
    // enough warps for the device, a block of 16 at a time
    const int rows = a.n_seq * g.n_rows;
    int wpr = 16;
    while (wpr > 1 && (long long)rows * wpr > 32LL * n_sm) wpr /= 2;
    const int blocks = (rows + 16 / wpr - 1) / (16 / wpr);
    return launch_pdl(mla_join_kernel, dim3(blocks < 4 * n_sm ? blocks : 4 * n_sm), dim3(512), 0, st, a, g, wpr);
}

}  // namespace coli

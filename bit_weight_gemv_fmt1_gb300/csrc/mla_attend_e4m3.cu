// mla_attend_e4m3.cu -- attention over a paged E4M3 latent cache (absorbed
// form).  mla_attend.cu explains the products, the softmax with its running
// reference and how the work is cut; this kernel differs in that the codes are
// never converted.
//
// The tensor cores multiply 8-bit floats exactly into f32.  What faces the codes
// is split into 8-bit terms:
//   q  (times a power of two per row)  = q0 + 2^-5 q1             E4M3 (8 bits, but no finer than 2^-22 of the row's largest)
//   P  = weight * row scale            = p0 + 2^-3 p1 + 2^-7 p2   E5M2 (to 2^-11, as f16 has it)
// P's terms are E5M2 for its range: the reference starts 6 below the first tile's maximum and
// weights may grow by 2^8 before it has to move, while those down to 2^-18 of the
// largest keep all 11 bits.  (Three E4M3 terms have 14 bits but a 2^-20 floor under
// a 2^8 ceiling: the reference moved every second tile, 6000 cycles each time.)
// Terms are columns side by side, S^T [128 tokens][2 NH] and O^T [128 dims][3 NH]
// for NH = 16 or 32 query rows, and are added in f32 when they leave TMEM.  An
// MMA reads 4 KB of codes for 128 x 32 values whatever its N, so the terms cost
// little: at NH = 32 a tile takes 18 MMAs of N = 64 (45 cycles) and 16 of N = 96 (52), 1640
// cycles, and its bytes enter shared memory once (converting to f16 instead read
// and wrote them twice more and was bound by that: 10400 cycles for 64 rows).
//
// Bound: tiles are 73 KB, so two fit beside q and P: the scores of tile i + 1 are computed while the
// softmax of tile i runs.  What a buffer goes through in turn is longer than two tiles' MMAs: scores 1150 cycles, softmax
// 1250, the wait for the other tile's MMAs 1200, outputs 1100 to 1450, release to next copy's arrival 2000 (issue 600,
// L2 700), 7300 in all, so a tile takes 3650 to 4400.  What shortened it: one barrier for all blocks of a
// tile and one look at it and at P's (162 -> 157 us), bytes announced ahead of the release (-> 155).
// Measured: 48 sequences of up to 12000 tokens (320000 in all), 128 heads: 154 us, 0.58 PFLOP/s of the formula's work;
// 1 x 1000: 13 us, of which two thirds are launch, the first copies and the join.
//
// Warps: 0-7 softmax and output (two threads per token, each half the rows), 8 MMA issue, 9-13 bulk
// copies of codes and scales.
#include "mla_attend.cuh"

namespace coli {

namespace {

constexpr uint32_t kBlk8 = kTile * 128;  // 128 tokens x 128 codes, 128-byte swizzle
constexpr uint32_t kRope8 = kTile * 64;  // 128 tokens x 64 codes, 64-byte swizzle
constexpr uint32_t kP8 = kTile * 128;    // P [128 tokens][3 NH], rows of 128 bytes
constexpr int kCopyWarps = 5;            // one for each block of a tile
constexpr int kThreads = 32 * (9 + kCopyWarps);
constexpr float kHead8 = 6.f;            // log2 of the largest weight of a fresh reference
constexpr float kLimit8 = 14.f;          // log2 of the weight that moves the reference (E5M2 ends at 57344)
constexpr float kFloor8 = -90.f;         // log2 of a row's scale, at least
constexpr float kQ1 = 32.f;              // q's second term against the first
constexpr float kP1 = 8.f, kP2 = 16.f;   // P's second term against the first, third against the second

struct Shared8 {
    uint64_t k_full[2], k_empty[2][5];      // all of a tile; its blocks of 128 dims, last the rope part
    uint64_t sc_full[4];                    // row scales
    uint64_t s_full[2], p_full[2], q_full;
    uint32_t tmem;
    int abort;
    Piece piece;
    alignas(16) float scale[4][kTile];   // of tile it & 3: a row's codes are freed by the scores, its scale is used after them
    alignas(16) float f[32];
    alignas(16) float m[2][32];          // minus the reference
    float linv[32], r[32];
    int limit[32];
    float red[4][32];
};

// Instruction descriptor of kind::f8f6f4 with f32 accumulators; types: 0 = E4M3, 1 = E5M2.
__host__ __device__ constexpr uint32_t f8_idesc(int a_type, int b_type, bool a_mn_major, bool b_mn_major, int M, int N) {
    return (1u << 4) | ((uint32_t)a_type << 7) | ((uint32_t)b_type << 10) | ((uint32_t)a_mn_major << 15) | ((uint32_t)b_mn_major << 16) |
           ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}
// 64-byte swizzled K-major operand: atoms of 8 rows x 64 bytes.
__device__ __forceinline__ uint64_t sw64_desc(uint32_t saddr) {
    return (uint64_t)((saddr & 0x3FFFF) >> 4) | (uint64_t)1 << 16 | (uint64_t)(512 >> 4) << 32 | (uint64_t)1 << 46 | (uint64_t)4 << 61;
}
__device__ __forceinline__ void mma8_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool acc) {
    asm volatile(
        "{\n .reg .pred p, q;\n elect.sync _|q, 0xffffffff;\n setp.ne.b32 p, %4, 0;\n"
        " @q tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n}\n" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)acc)
        : "memory");
}
// v -> its 8-bit pair; v becomes the remainder times `step`.
template <bool E5M2>
__device__ __forceinline__ uint32_t take_term(float2 &v, float step) {
    const uint32_t u = E5M2 ? pack_e5m2(v.x, v.y) : pack_e4m3(v.x, v.y);
    const uint32_t h = E5M2 ? __byte_perm(u, 0u, 0x1404) : e4m3x2_f16x2(u);   // E5M2 is the high byte of f16
    float2 r = fmul2(v, make_float2(step, step));
    ffma2(r, __half22float2(*reinterpret_cast<const __half2 *>(&h)), make_float2(-step, -step));
    v = r;
    return u;
}

// A unit of 8 query elements times `up` -> its two E4M3 terms, in f16 pairs (of f32 or bf16 input; f16 holds the
// scaled values' 8 and the remainders' 4 bits exactly).
template <bool QB>
__device__ __forceinline__ void query_terms(const uint4 (&x)[QB ? 1 : 2], float up, uint2 (&t)[2]) {
    const uint32_t w[8] = {x[0].x, x[0].y, x[0].z, x[0].w, x[QB ? 0 : 1].x, x[QB ? 0 : 1].y, x[QB ? 0 : 1].z, x[QB ? 0 : 1].w};
    uint32_t hi[4], lo[4];
#pragma unroll
    for (int q = 0; q < 4; q++) {
        float2 y = QB ? bf16x2_f32x2(w[q]) : make_float2(__uint_as_float(w[2 * q]), __uint_as_float(w[2 * q + 1]));
        y = fmul2(y, make_float2(up, up));
        const uint32_t h = pack_f16(y.x, y.y);
        uint16_t e;
        asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(e) : "r"(h));
        const uint32_t b = e4m3x2_f16x2(e);
        const __half2 r = __hmul2(__hsub2(*reinterpret_cast<const __half2 *>(&h), *reinterpret_cast<const __half2 *>(&b)), __float2half2_rn(kQ1));
        uint16_t f;
        asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(f) : "r"(*reinterpret_cast<const uint32_t *>(&r)));
        hi[q] = e;
        lo[q] = f;
    }
    t[0] = make_uint2(hi[0] | hi[1] << 16, hi[2] | hi[3] << 16);
    t[1] = make_uint2(lo[0] | lo[1] << 16, lo[2] | lo[3] << 16);
}
template <bool QB>
__device__ __forceinline__ float largest(const uint4 (&x)[QB ? 1 : 2]) {
    const uint32_t w[8] = {x[0].x, x[0].y, x[0].z, x[0].w, x[QB ? 0 : 1].x, x[QB ? 0 : 1].y, x[QB ? 0 : 1].z, x[QB ? 0 : 1].w};
    float m = 0.f;
#pragma unroll
    for (int q = 0; q < (QB ? 4 : 8); q++) {
        if constexpr (QB) {
            const float2 y = bf16x2_f32x2(w[q]);
            m = fmaxf(m, fmaxf(fabsf(y.x), fabsf(y.y)));
        } else {
            m = fmaxf(m, fabsf(__uint_as_float(w[q])));
        }
    }
    return m;
}

// The query rows of a block -> E4M3 terms [L/128 blocks][2 NH][128], then [2 NH][64] (rope).  A warp takes NH / 8
// rows: lane l holds units l and l + 32 of each, and unit l % 8 of the rope part of row l / 8.
template <int NH, bool QB>
__device__ __forceinline__ void load_queries8(const MlaAttendArgs &a, const AttendPlan &g, Shared8 &s, uint8_t *qsm, int b, int rb,
                                              int len, int warp, int lane) {
    constexpr int W = QB ? 1 : 2, RW = NH / 8;
    const int nu = a.c.L / 8, nr = a.c.R / 8, nru = (a.c.R + 31) / 32 * 4;
    uint8_t *rope = qsm + (a.c.L / 128) * (2 * NH * 128);
    const int c0 = RW * warp;
    {
        uint4 x[RW][2][W], xr[W];
        auto fetch = [&](int c, int u, bool ok, uint4 (&v)[W]) {
            const int r = rb * NH + c;
            ok = ok && r < g.n_rows;
            const uint4 *src = query_unit<QB>(a, (long long)b * g.n_rows + (ok ? r : 0), ok ? u : 0);
#pragma unroll
            for (int w = 0; w < W; w++) v[w] = ok ? __ldg(src + w) : make_uint4(0u, 0u, 0u, 0u);
        };
#pragma unroll
        for (int i = 0; i < RW; i++)
#pragma unroll
            for (int k = 0; k < 2; k++) fetch(c0 + i, lane + 32 * k, lane + 32 * k < nu, x[i][k]);
        fetch(c0 + lane / 8, nu + lane % 8, lane / 8 < RW && lane % 8 < nr, xr);
        float mr = largest<QB>(xr), up_r = 0.f;
#pragma unroll
        for (int o = 4; o > 0; o >>= 1) mr = fmaxf(mr, __shfl_xor_sync(0xffffffffu, mr, o));
#pragma unroll
        for (int i = 0; i < RW; i++) {
            const int c = c0 + i, r = rb * NH + c;
            float mx = fmaxf(largest<QB>(x[i][0]), largest<QB>(x[i][1]));
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
            mx = fmaxf(mx, __shfl_sync(0xffffffffu, mr, 8 * i));
            // times 2^k2: the largest magnitude in [2^7, 2^8); E4M3 has no infinity, so a row with one has NaN for its factor
            const int ex = (int)((__float_as_uint(mx) >> 23) & 0xFF) - 127;
            const int k2 = mx > 0.f && ex < 128 ? min(7 - ex, 120) : 0;
            const float up = __int_as_float((k2 + 127) << 23);
            if (lane / 8 == i) up_r = up;
#pragma unroll
            for (int k = 0; k < 2; k++) {
                const int u = lane + 32 * k;
                uint2 t[2];
                query_terms<QB>(x[i][k], up, t);
                if (u >= nu) continue;
#pragma unroll
                for (int j = 0; j < 2; j++) {
                    const int row = j * NH + c;
                    *reinterpret_cast<uint2 *>(qsm + (u >> 4) * (2 * NH * 128) + row * 128 + ((((u & 15) >> 1) ^ (row & 7)) << 4) + 8 * (u & 1)) = t[j];
                }
            }
            if (lane == 0) {
                s.f[c] = ex < 128 ? a.scale * 1.4426950408889634f * __int_as_float((127 - k2) << 23) : __int_as_float(0x7FC00000);
                s.limit[c] = r < g.n_rows ? len - (a.n_q - 1 - r / a.H) : 0;
            }
        }
        uint2 t[2];
        query_terms<QB>(xr, up_r, t);
        const int u = lane % 8;
        if (u < nru && lane / 8 < RW)
#pragma unroll
            for (int j = 0; j < 2; j++) {
                const int row = j * NH + c0 + lane / 8;
                *reinterpret_cast<uint2 *>(rope + row * 64 + (((u >> 1) ^ ((row >> 1) & 3)) << 4) + 8 * (u & 1)) = t[j];
            }
    }
}

template <int NH>
__global__ void __launch_bounds__(kThreads, 1)
    mla_attend_e4m3_kernel(const __grid_constant__ CUtensorMap map, const __grid_constant__ CUtensorMap rope_map, const MlaAttendArgs a,
                           const AttendPlan g) {
    constexpr int HC = NH / 2;             // rows per softmax thread
    extern __shared__ uint8_t raw[];
    __shared__ Shared8 s;
    const uint32_t base = (smem_addr(raw) + 1023u) & ~1023u;
    uint8_t *sm = raw + (base - smem_addr(raw));
    // the shuffles tell the compiler that these are the same in a whole warp, so that MMA operands live in uniform registers
    const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
    const int np = a.c.L / 128;
    const uint32_t stage = np * kBlk8 + kRope8;
    const uint32_t q_off = 2 * stage, p_off = q_off + np * (2 * NH * 128) + 2 * NH * 64;
    constexpr uint32_t kCols = 16 * NH, kO = 4 * NH;   // TMEM: two S of 2 NH columns, L/128 O of 3 NH
    pdl_wait();
    pdl_trigger();
    if (warp == 0) tmem_alloc(&s.tmem, kCols);
    if (tid == 0) {
        for (int i = 0; i < 4; i++) mbar_init(&s.sc_full[i], 1);
        mbar_init(&s.q_full, 1);
        for (int i = 0; i < 2; i++) {
            mbar_init(&s.k_full[i], np + 1);
            for (int p = 0; p < 5; p++) mbar_init(&s.k_empty[i][p], 1);
            mbar_init(&s.s_full[i], 1);
            mbar_init(&s.p_full[i], 8);
        }
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

    if (warp < 8) {
        // ---------------------------------------------------------- softmax and output
        const int wq = warp & 3, grp = warp >> 2;
        const int t = 32 * wq + lane;                                   // token of the tile, and dim of an O block
        const uint32_t lanes = tmem + ((uint32_t)(32 * wq) << 16);
        const int col0 = grp * HC;
        float2 l[HC / 2];
        int it = 0, cur = 0;
        for (Walk w(a, g, s.piece, slot); w.valid(); w.next(), it++) {
            const int buf = it & 1;
            if (w.first()) {
                deadline = deadline_after(g.wait_ns, w.rest());
                if (a.q_bf16) load_queries8<NH, true>(a, g, s, sm + q_off, w.b, w.rb, w.len, warp, lane);
                else load_queries8<NH, false>(a, g, s, sm + q_off, w.b, w.rb, w.len, warp, lane);
                if (tid < NH) s.m[cur][tid] = -kNone;
#pragma unroll
                for (int c = 0; c < HC / 2; c++) l[c] = make_float2(0.f, 0.f);
                fence_async_smem();
                named_sync(1, kSoft);
                if (tid == 0 && ok) mbar_arrive(&s.q_full);             // behind the barrier: for all of them
            }
            const int tok = w.tile() * kTile + t;
            // every row sees the whole tile: the first query's limit is the lowest
            const bool full = (w.tile() + 1) * kTile <= w.len - (a.n_q - 1) && (w.rb + 1) * NH <= g.n_rows;
            wait(&s.sc_full[it & 3], (it >> 2) & 1);
            wait(&s.s_full[buf], (it >> 1) & 1);
            tc_after_sync();
            const float st = tok < w.len ? s.scale[it & 3][t] : 0.f;
            // what P takes of it: a row with no finite scale has it in its scores, and 0 * NaN is NaN
            const float sp = fabsf(st) < INFINITY ? st : 0.f;
            if ((w.tile() + 1) * kTile > w.len - a.n_q + 1) {
                // Likewise the codes.  Rows past the length may hold anything: zero.  Of the newest tokens' rows, which not
                // every query sees, the NaN: the queries that see it have it in their scores, so one score tells.
                bool clear = false;
                if (a.n_q > 1) {
                    uint32_t v[8];
                    tmem_ld(lanes + buf * (2 * NH) + col0, v);
                    tmem_ld_wait();
                    clear = tok > w.len - a.n_q && !finite_bits(v[0]);
                }
                if (tok >= w.len) {
                    for (int k = grp; k < np; k += 2)
#pragma unroll
                        for (int u = 0; u < 8; u++) *reinterpret_cast<uint4 *>(sm + buf * stage + k * kBlk8 + t * 128 + 16 * u) = make_uint4(0u, 0u, 0u, 0u);
                } else if (clear) {
#pragma unroll 1
                    for (int i = 0; grp + 2 * (i >> 3) < np; i++) {
                        uint4 *at = reinterpret_cast<uint4 *>(sm + buf * stage + (grp + 2 * (i >> 3)) * kBlk8 + t * 128 + 16 * (i & 7));
                        uint4 x = *at;
                        for (uint32_t *e : {&x.x, &x.y, &x.z, &x.w}) *e &= ~__vcmpeq4(*e & 0x7F7F7F7Fu, 0x7F7F7F7Fu);
                        *at = x;
                    }
                }
            }
            // log2 of the row's scale; the floor gives rows of scale 0, which weigh in l alone, a reference too
            const float lg = fmaxf(__log2f(st), kFloor8);
            const uint32_t s_at = lanes + buf * (2 * NH) + col0;
            // l += sign * weights 2^min(x - m, kLimit8 - kFloor8), which the largest that moves no reference reaches, and P for
            // sign > 0; true if a weight has outgrown P
            auto add = [&](float sign) {
                uint32_t v0[HC], v1[HC], pk[3][HC / 4];
                tmem_ld(s_at, v0);
                tmem_ld(s_at + NH, v1);
                tmem_ld_wait();
                float top = -INFINITY;
#pragma unroll
                for (int c = 0; c < HC; c += 2) {
                    const float2 f = *reinterpret_cast<const float2 *>(&s.f[col0 + c]);
                    float2 x = *reinterpret_cast<const float2 *>(&s.m[cur][col0 + c]);
                    float2 y = make_float2(__uint_as_float(v0[c]), __uint_as_float(v0[c + 1]));
                    ffma2(y, make_float2(__uint_as_float(v1[c]), __uint_as_float(v1[c + 1])), make_float2(1.f / kQ1, 1.f / kQ1));
                    ffma2(x, fmul2(y, make_float2(st, st)), f);
                    if (!full) {
                        if (tok >= s.limit[col0 + c]) x.x = -INFINITY;
                        if (tok >= s.limit[col0 + c + 1]) x.y = -INFINITY;
                    }
                    top = fmaxf(top, fmaxf(x.x, x.y));
                    x = make_float2(ex2(min_nan(x.x, kLimit8 - kFloor8)), ex2(min_nan(x.y, kLimit8 - kFloor8)));
                    l[c / 2] = fadd2(l[c / 2], sign > 0.f ? x : make_float2(-x.x, -x.y));
                    if (sign > 0.f) {
                        float2 p = fmul2(x, make_float2(sp, sp));
                        const uint32_t p0 = take_term<true>(p, kP1), p1 = take_term<true>(p, kP2), p2 = pack_e5m2(p.x, p.y);
                        const int sh = 8 * (c & 2), i = c / 4;
                        pk[0][i] = c & 2 ? pk[0][i] | p0 << sh : p0;
                        pk[1][i] = c & 2 ? pk[1][i] | p1 << sh : p1;
                        pk[2][i] = c & 2 ? pk[2][i] | p2 << sh : p2;
                    }
                }
                if (sign > 0.f)
#pragma unroll
                    for (int j = 0; j < 3; j++) {
                        uint8_t *d = sm + p_off + buf * kP8 + t * 128;
                        if constexpr (HC == 16)
                            *reinterpret_cast<uint4 *>(d + (((2 * j + grp) ^ (t & 7)) << 4)) = make_uint4(pk[j][0], pk[j][1], pk[j][2], pk[j][3]);
                        else
                            *reinterpret_cast<uint2 *>(d + ((j ^ (t & 7)) << 4) + 8 * grp) = make_uint2(pk[j][0], pk[j][1]);
                    }
                return top + lg > kLimit8;
            };
            bool move = w.first();
            if (!move) {
                move = named_or(1, kSoft, add(1.f));
                // taking the weights off again is exact to an ulp of the sums with them, which the new reference
                // scales to 2^-24 of its own weights or less
                if (move) add(-1.f);
            }
            if (move) {
                uint32_t v0[HC], v1[HC];
                float x[HC];
                tmem_ld(s_at, v0);
                tmem_ld(s_at + NH, v1);
                tmem_ld_wait();
#pragma unroll
                for (int c = 0; c < HC; c++) {
                    x[c] = fmaf(fmaf(__uint_as_float(v1[c]), 1.f / kQ1, __uint_as_float(v0[c])) * st, s.f[col0 + c], lg);
                    if (!full && tok >= s.limit[col0 + c]) x[c] = -INFINITY;
                }
                const float top = reduce_columns(x, lane, [](float p, float q) { return fmaxf(p, q); });
                if (lane % (32 / HC) == 0) s.red[wq][col0 + lane / (32 / HC)] = top;
                named_sync(1, kSoft);
                if (tid < NH) {
                    const float old = -s.m[cur][tid];
                    const float x = fmaxf(fmaxf(s.red[0][tid], s.red[1][tid]), fmaxf(s.red[2][tid], s.red[3][tid]));
                    const float now = x > old + kLimit8 ? x - kHead8 : old;   // only the columns that need it
                    s.m[cur ^ 1][tid] = -now;
                    s.r[tid] = ex2(old - now);
                }
                named_sync(1, kSoft);
                cur ^= 1;
                if (!w.first()) {
#pragma unroll
                    for (int c = 0; c < HC / 2; c++) l[c] = fmul2(l[c], make_float2(s.r[col0 + 2 * c], s.r[col0 + 2 * c + 1]));
                    wait(&s.k_empty[buf ^ 1][np - 1], ((it - 1) >> 1) & 1);      // the products of the tile before are in O
                    tc_after_sync();
#pragma unroll 1
                    for (int k = 0; k < np * 3 * (HC / 8); k++) {
                        const int c0 = col0 + 8 * (k % (HC / 8));
                        const uint32_t at = lanes + kO + NH * (k / (HC / 8)) + c0;
                        float r[8];
                        bool same = true;
#pragma unroll
                        for (int c = 0; c < 8; c++) {
                            r[c] = s.r[c0 + c];
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
            }
            fence_async_smem();
            tc_before_sync();
            __syncwarp();
            if (lane == 0 && ok) mbar_arrive(&s.p_full[buf]);
            if (!w.last()) continue;

            // ------------------------------------------------------ this part of the sequence is done
            {
                float z[HC];
#pragma unroll
                for (int c = 0; c < HC; c++) z[c] = c & 1 ? l[c / 2].y : l[c / 2].x;
                const float sum = reduce_columns(z, lane, [](float p, float q) { return p + q; });
                if (lane % (32 / HC) == 0) s.red[wq][col0 + lane / (32 / HC)] = sum;
            }
            named_sync(1, kSoft);
            const bool whole = w.whole();
            const long long pidx = ((long long)group * g.nrb + w.rb) * 2 + w.which();
            if (tid < NH) {
                const float z = s.red[0][tid] + s.red[1][tid] + s.red[2][tid] + s.red[3][tid];
                const float m = -s.m[cur][tid];
                s.linv[tid] = whole ? (z != 0.f ? 1.f / z : 0.f) : 1.f;
                const int r = w.rb * NH + tid;
                if (!whole) {
                    g.part_ml[(pidx * NH + tid) * 2] = m;
                    g.part_ml[(pidx * NH + tid) * 2 + 1] = z;
                } else if (a.lse && r < g.n_rows) {
                    a.lse[(long long)w.b * g.n_rows + r] = z != 0.f ? (m + log2f(z)) * 0.6931471805599453f : -INFINITY;
                }
            }
            named_sync(1, kSoft);
            wait(&s.k_empty[buf][np - 1], (it >> 1) & 1);
            tc_after_sync();
            const long long row = (long long)w.b * g.n_rows + w.rb * NH + col0;
            const int rows = min(HC, g.n_rows - w.rb * NH - col0);
#pragma unroll 1
            for (int k = 0; k < np; k++) {
                uint32_t o0[HC], o1[HC], o2[HC];
                tmem_ld(lanes + kO + 3 * NH * k + col0, o0);
                tmem_ld(lanes + kO + 3 * NH * k + NH + col0, o1);
                tmem_ld(lanes + kO + 3 * NH * k + 2 * NH + col0, o2);
                tmem_ld_wait();
                const int d = 128 * k + t;
                float *dst = g.part + (pidx * NH + col0) * a.c.L + d;
#pragma unroll
                for (int c = 0; c < HC; c++) {
                    if (c >= rows) continue;
                    const float v = fmaf(fmaf(__uint_as_float(o2[c]), 1.f / kP2, __uint_as_float(o1[c])), 1.f / kP1, __uint_as_float(o0[c]));
                    if (!whole) dst[c * a.c.L] = v;
                    else store_out(a, (row + c) * a.c.L + d, v * s.linv[col0 + c]);
                }
            }
            tc_before_sync();
            named_sync(1, kSoft);
        }
    } else if (warp == 8) {
        // ---------------------------------------------------------- MMA issue
        constexpr uint32_t id_s = f8_idesc(0, 0, false, false, kTile, 2 * NH), id_o = f8_idesc(0, 1, true, true, 128, 3 * NH);
        const uint64_t dk = sw128_desc(base, 16, 1024), dr = sw64_desc(base + np * kBlk8);
        const uint64_t dq = sw128_desc(base + q_off, 16, 1024), dqr = sw64_desc(base + q_off + np * (2 * NH * 128));
        const uint64_t dv = sw128_desc(base, 16, 1024), dp = sw128_desc(base + p_off, 16, 1024);
        auto scores = [&](int it) {
            const uint32_t buf = __shfl_sync(0xffffffffu, it & 1, 0), so = (buf * stage) >> 4, d = tmem + buf * (2 * NH);
            tc_after_sync();
            for (int p = 0; p < np; p++)
#pragma unroll
                for (int k = 0; k < 4; k++)
                    mma8_ss(d, dk + so + ((p * kBlk8) >> 4) + 2 * k, dq + ((p * 2 * NH * 128) >> 4) + 2 * k, id_s, p || k);
#pragma unroll
            for (int k = 0; k < 2; k++)
                if (32 * k < a.c.R) mma8_ss(d, dr + so + 2 * k, dqr + 2 * k, id_s, true);
            tc_commit(&s.s_full[buf]);
            tc_commit(&s.k_empty[buf][np]);
        };
        auto output = [&](int it, bool first) {
            const uint32_t buf = __shfl_sync(0xffffffffu, it & 1, 0), so = (buf * stage) >> 4, po = (buf * kP8) >> 4;
            const uint32_t more = __shfl_sync(0xffffffffu, first ? 0u : 1u, 0);
            tc_after_sync();
            for (int p = 0; p < np; p++) {
#pragma unroll
                for (int k = 0; k < 4; k++)
                    mma8_ss(tmem + kO + 3 * NH * p, dv + so + ((p * kBlk8 + k * 4096) >> 4), dp + po + ((k * 4096) >> 4), id_o, k || more);
                tc_commit(&s.k_empty[buf][p]);
            }
        };
        // Scores of tile q and outputs of tile v, in whichever order their inputs come, scores first, as the softmax
        // would run dry.  A look at a barrier takes some 250 cycles while the MMAs read shared memory at its full rate, so
        // a tile has one for all of its blocks, and one instruction looks at both: odd lanes at tile q, even ones at P of v.
        int it = 0, seg = 0;
        for (Walk w(a, g, s.piece, slot); w.valid(); w.next()) {
            const int n = w.rest();
            deadline = deadline_after(g.wait_ns, n);
            wait(&s.q_full, seg++ & 1);
            int q = 0, v = 0, spins = 0;
            while (v < n && ok) {
                const int i = lane & 1 ? it + q : it + v;
                const uint32_t ready = __ballot_sync(0xffffffffu, mbar_test(lane & 1 ? &s.k_full[i & 1] : &s.p_full[i & 1], (i >> 1) & 1));
                __syncwarp();                                          // passes on what the other lanes have seen
                if (q < n && q <= v + 1 && (ready & 2)) {
                    scores(it + q++);
                } else if (q > v && (ready & 1)) {
                    output(it + v, v == 0);
                    v++;
                } else if ((++spins & 63) == 0 && __any_sync(0xffffffffu, *abort || global_ns() > deadline)) {
                    ok = false;
                    *abort = 1;
                    atomicCAS(a.err, 0, (int)DEV_ERR_TIMEOUT);
                }
            }
            it += n;
            w.skip(n - 1);
        }
    } else {
        // ---------------------------------------------------------- bulk copies
        // A block's buffer is asked for as soon as it is free, so what stands between the wait and the copies is kept
        // short: each warp has one block of the tile (the last one: rope part and scales).
        const int who = warp - 9, nbox = kTile / g.pbox;
        const int p = who < 4 ? who : np;
        const bool mine = who == 4 || who < np;
        BoxAhead box(a, g, s.piece, slot, lane, who == 4);
        int it = 0;
        for (Walk w(a, g, s.piece, slot); w.valid(); w.next(), box.next(), it++) {
            if (!mine) continue;
            if (w.first()) deadline = deadline_after(g.wait_ns, w.rest());
            const int buf = it & 1, sl = box.slot[0];
            const uint32_t live = __ballot_sync(0xffffffffu, sl >= 0), n = __popc(live) * g.pbox;
            const int y0 = __shfl_sync(0xffffffffu, sl, 0);
            const uint32_t dst = base + buf * stage + p * kBlk8;
            uint64_t *bar = &s.k_full[buf];
            // the bytes are announced once the tile before in this buffer has landed, ahead of the buffer's release
            if (it > 1) wait(bar, ((it - 2) >> 1) & 1);
            if (ok) expect_bytes(bar, n * (who < 4 ? 128 : 64));
            if (it > 1) wait(&s.k_empty[buf][p], ((it - 2) >> 1) & 1);
            if (!ok) continue;
            if (who < 4) {
                if (live & 1) tma_box(dst, &map, 128 * p, y0, bar);
                for (int j = 1; j < nbox; j++) {
                    const int y = __shfl_sync(0xffffffffu, sl, j);
                    if (live >> j & 1) tma_box(dst + j * g.pbox * 128, &map, 128 * p, y, bar);
                }
            } else {
                expect_bytes(&s.sc_full[it & 3], n * 4);
                for (int j = 0; j < nbox; j++) {
                    const int y = __shfl_sync(0xffffffffu, sl, j);
                    if (!(live >> j & 1)) continue;
                    tma_box(dst + j * g.pbox * 64, &rope_map, a.c.L, y, bar);
                    bulk_copy(smem_addr(&s.scale[it & 3][j * g.pbox]), a.c.scales + y, g.pbox * 4, &s.sc_full[it & 3]);
                }
            }
        }
        // every copy has landed before the CTA may end
        const uint64_t late = global_ns() + 200000000ull;
        volatile int none = 0;
        for (int k = it > 1 ? it - 2 : 0; k < it && mine; k++) {
            warp_wait(&s.k_full[k & 1], (k >> 1) & 1, late, &none, lane);
            if (who == 4) warp_wait(&s.sc_full[k & 3], (k >> 2) & 1, late, &none, lane);
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

constexpr size_t smem_bytes(size_t np, size_t cols) {
    return 2 * (np * kBlk8 + kRope8) + np * (2 * cols * 128) + 2 * cols * 64 + 2 * kP8 + 1024;
}

template <int NH>
cudaError_t run(const MlaAttendArgs &a, const AttendPlan &g, int device, cudaStream_t st) {
    CUtensorMap map, rope;
    if (cudaError_t e = mla_row_map(a.c, 128, g.pbox, CU_TENSOR_MAP_SWIZZLE_128B, &map)) return e;
    if (cudaError_t e = mla_row_map(a.c, 64, g.pbox, CU_TENSOR_MAP_SWIZZLE_64B, &rope)) return e;
    const size_t smem = smem_bytes(a.c.L / 128, NH);
    auto kern = mla_attend_e4m3_kernel<NH>;
    static std::atomic<uint64_t> done{0};
    if (cudaError_t e = allow_smem(kern, smem_bytes(4, NH), device, done)) return e;   // the largest latent's
    return launch_pdl(kern, dim3(g.n_groups * g.n_slots), dim3(kThreads), smem, st, map, rope, a, g);
}

}  // namespace

cudaError_t launch_mla_attend_e4m3(const MlaAttendArgs &a, const AttendPlan &g, int device, cudaStream_t st) {
    return g.cols == 16 ? run<16>(a, g, device, st) : run<32>(a, g, device, st);
}

}  // namespace coli

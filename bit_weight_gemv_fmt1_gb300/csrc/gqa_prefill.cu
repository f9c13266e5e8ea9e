// gqa_prefill.cu -- causal attention of packed sequences whose query heads share
// key and value heads, on the 5th-generation tensor cores.
//
// A unit of work is one key / value head and two tiles A and B of 128 query rows of one sequence, and a walk over the
// keys in tiles of 128.  A query tile's rows are tokens x the group's heads (row = token * group + head; 128 / group tokens, rounded
// down), brought by one box over (dims, heads, tokens): a sequence of few tokens fills a tile with its heads, and a group's
// keys and values are read once for all of them.  The grid has a CTA per unit, longest first; a CTA that nears its
// unit's end takes over one that has not started (cluster launch control), so that the next queries, keys and
// scores come while the last output is written.  (A CTA per SM and units dealt out there and back
// measures the same within 2 %.)
//   S = Q K^T   M = 128 queries, N = 128 keys, K = dim (K-major operands in shared memory)
//   O += P V    M = 128 queries, N = dim, K = 128 keys (P in TMEM, V as stored: N-major)
// The two tiles alternate: while the softmax of one runs, the tensor cores work
// on the other.  One thread holds one query row; P overwrites S in TMEM.
//
// Softmax: x = log2(e) * scale * score, e = 2^(x - m), l += e, P = bf16(e).  m is
// the row's running maximum, moved (and O and l rescaled) only when a tile's
// maximum passes it by 8: weights up to 2^8 lose nothing in bf16.  m, l and O are
// f32; rounding P to bf16 is within 2^-8 of each weight, as the values' own.
//
// Bound: the chain of a tile.  A round (128 keys for both tiles) is 32 MMAs of 64 cycles, 2048; measured 2860: either tile's softmax
// takes about 1250 (scores out of TMEM 200, maxima 180, 128 exponentials at 4 cycles and what goes with them 600, P and the
// hand-overs 250), longer than the 1024 of the other tile's products.  P is handed over in halves of 64 keys and the arithmetic on
// pairs is packed (1x8192, 32 heads on 8: 376 us, 370 with halves, 366 packed, 355 once the next unit is asked for late); half a row per
// thread, two warps a tile and SM quarter, is slower (384).  1.54 PFLOP/s, 0.80 of the measured bf16 rate; 1x2048 33 us, 6 ragged up
// to 700 behind 333 cached 47.
//
// f32 inputs become f16, which keeps 3 bits more than bf16: every row (token and head) of q, k and v times a power of two that follows
// from that row alone, so that what a query does not see cannot change its result.  Keys of ordinary size (the largest magnitude in
// 2^-5 .. 2^11) share one, others and queries get the one that takes their largest magnitude to 2^14 .. 2^15; values whose largest
// magnitudes lie between the same two of 2^-4, 2^6, 2^16 and so on share one, which takes the upper end to 2^15.  The powers come out
// again by a factor of the scores, a thread's own for q, and two factors per key, which every softmax warp copies to shared memory a
// tile ahead: the scores', and that of a key's weight in P, which is f16 then, too.  With U the largest weight times factor of a row so
// far, P is held times a power of two B that keeps B U in 100 .. 2^15; O is rescaled when B moves.  A tile of ordinary keys whose
// values' factors are all 1 / B needs neither multiplication, and the bits are the same: 1x8192, 32 heads on 8, 453 us (D 64: 369), with
// values of many sizes 769 (621), keys, too, 869 (743).  Exponents rather than tf32 operands: those would be twice the bytes in
// shared memory, which two query tiles of 128 dims fill, and twice the products' cycles.  24 prompts of up to 301 tokens (16 heads on 2,
// D 64) 24 us, with the launch that makes f16 (10 us by the profiler, its inputs from DRAM: 21 MB and what it works out for each row).
//
// Keys past a causal row's limit are masked by selection; value rows past the
// sequence's end belong to its neighbours and are zeroed in shared memory.
// Warps: 0-3 and 4-7 softmax of A and B, 8 MMA issue, 9 units and copies of keys, 10 and 11 of queries and values.
// Every wait is bounded, by a limit that each unit renews.  After one has run out all waits return at once, no further
// MMA or copy is issued, and the kernel records DEV_ERR_TIMEOUT.
#include <algorithm>

#include "prefill.cuh"

namespace coli {

namespace {

constexpr int kKeys = 5, kValues = 4;    // ring slots: key blocks of 64 dims, value halves of 64 keys
constexpr uint32_t kOut = 32 * 64;       // bytes of a warp's outputs on their way: 64 of each row
constexpr float kLog2e = 1.4426950408889634f;
// f16 inputs made from f32, log2 of their powers: those of ordinary keys and values, and shifts of the factors that are kept, so that these
// and their products with scores (up to 2^37) and weights (up to 2^15) are numbers for rows of any size.
constexpr int kKeyPower = 4, kValuePower = 9, kKeyShift = 32, kValueShift = 10;
constexpr int kUp = 7;                   // log2 of what f16 weights are held times
constexpr int kMostUp = 126;             // log2 of B at the most
// A key's factors are two bf16 in a word, its scores' in the low half: powers of two, an ordinary key's this one.
constexpr uint32_t kPlainKey = (uint32_t)(127 - kKeyShift) << 7;

struct Shared {
    uint64_t q_full[2], q_empty[2], k_full[kKeys], k_empty[kKeys], v_full[kValues], v_empty[kValues], s_full[2], p_full[2][2], o_full[2],
        u_full[2], u_empty[2];
    uint64_t next_full;
    Unit unit[2];
    alignas(16) uint32_t next[4];        // the answer to the last request for a CTA's work
    uint32_t tmem;
    int abort;
};

// (x, y) = (x, y) * f + m, s += (x, y), and products: two f32 operations in one instruction.
__device__ __forceinline__ void fma2(float &x, float &y, uint32_t u, uint32_t v, float f, float m) {
    asm("{\n .reg .b64 a, b, d;\n mov.b64 a, {%2, %3};\n mov.b64 b, {%4, %4};\n mov.b64 d, {%5, %5};\n fma.rn.f32x2 a, a, b, d;\n"
        " mov.b64 {%0, %1}, a;\n}"
        : "=f"(x), "=f"(y)
        : "r"(u), "r"(v), "f"(f), "f"(m));
}
__device__ __forceinline__ void add2(float &s, float &t, float x, float y) {
    asm("{\n .reg .b64 a, b;\n mov.b64 a, {%2, %3};\n mov.b64 b, {%0, %1};\n add.rn.f32x2 b, b, a;\n mov.b64 {%0, %1}, b;\n}"
        : "+f"(s), "+f"(t)
        : "f"(x), "f"(y));
}
__device__ __forceinline__ void mul2(float &x, float &y, float u, float v) {
    asm("{\n .reg .b64 a, b;\n mov.b64 a, {%0, %1};\n mov.b64 b, {%2, %3};\n mul.rn.f32x2 a, a, b;\n mov.b64 {%0, %1}, a;\n}"
        : "+f"(x), "+f"(y)
        : "f"(u), "f"(v));
}
// 2^e, -126 <= e <= 127.
__device__ __forceinline__ float exp2i(int e) { return __uint_as_float((uint32_t)(127 + e) << 23); }
// 4 bytes from global to shared memory without a register, zeros instead where `some` is false; and the wait for all such copies of this
// thread.
__device__ __forceinline__ void copy4(uint32_t *dst, const uint32_t *src, bool some) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(smem_addr(dst)), "l"(src), "r"(some ? 4 : 0) : "memory");
}
__device__ __forceinline__ void copies_done() { asm volatile("cp.async.wait_all;" ::: "memory"); }

// A box of a 3-D tensor map, as tma_box.
__device__ __forceinline__ void tma_box3(uint32_t dst, const CUtensorMap *map, int x, int y, int z, uint64_t *bar) {
    asm volatile(
        "{\n .reg .pred q;\n elect.sync _|q, 0xffffffff;\n"
        " @q cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5}], [%2];\n}\n" ::"r"(dst),
        "l"(map), "r"(smem_addr(bar)), "r"(x), "r"(y), "r"(z)
        : "memory");
}

// Two neighbouring elements of an operand.
template <bool F16>
__device__ __forceinline__ float2 operands(uint32_t w) {
    return F16 ? __half22float2(*reinterpret_cast<const __half2 *>(&w)) : bf16x2_f32x2(w);
}
__device__ __forceinline__ bool finite(float x) { return fabsf(x) <= 3.402823466e38f; }

// Query rows whose tiles hold keys that they do not see (up to two tiles: a tile's rows have limits up to 127 apart, whose border with
// the next keys may lie anywhere): those keys' weights are 0, but 0 times an infinity or a NaN is NaN.  A
// whole warp calls this after its rows have been stored, for the rows (`mine`) with an output that is not finite: the columns where such a
// value is among the keys seen .. end - 1 are computed once more from the keys before, 32 at a time, until they are NaN.  (The
// tiles before are seen by all of a tile's rows.)  Nothing comes here unless a value or a result is not finite; a warp of 32 such rows of
// 8192 keys then takes 53 ms, which its unit's limit of waits (2.5 s) leaves room for.
template <int D, bool F16>
__device__ __noinline__ void repair(const GqaPrefillArgs &a, bool mine, int orow, int token, int q_head, int head, int krow, int seen, int end,
                                    float f, float m, float inv) {
    constexpr int kCols = D / 32;            // columns of a lane
    const int lane = threadIdx.x & 31;
    const uint16_t *k = reinterpret_cast<const uint16_t *>(a.k) + krow * a.k_stride + head * D;
    const uint16_t *v = reinterpret_cast<const uint16_t *>(a.v) + krow * a.v_stride + head * D + lane * kCols;
    const uint32_t *factors = F16 ? a.kv_power + ((long long)head * a.Tk + krow) : nullptr;
    auto value = [&](int j, float (&x)[kCols]) {
        const float by = F16 ? bf16x2_f32x2(factors[j]).y : 1.f;   // times 2^kValueShift
#pragma unroll
        for (int c = 0; c < kCols; c += 2) {
            const float2 two = operands<F16>(*reinterpret_cast<const uint32_t *>(v + j * a.v_stride + c));
            x[c] = F16 ? two.x * by * exp2i(kValueShift) : two.x, x[c + 1] = F16 ? two.y * by * exp2i(kValueShift) : two.y;
        }
    };
    for (uint32_t left = __ballot_sync(0xffffffffu, mine); left; left &= left - 1) {
        const int src = __ffs(left) - 1;
        const int n = __shfl_sync(0xffffffffu, seen, src), stop = __shfl_sync(0xffffffffu, end, src), to = __shfl_sync(0xffffffffu, orow, src);
        const float f1 = __shfl_sync(0xffffffffu, f, src), m1 = __shfl_sync(0xffffffffu, m, src), inv1 = __shfl_sync(0xffffffffu, inv, src);
        const uint16_t *q = reinterpret_cast<const uint16_t *>(a.q) + __shfl_sync(0xffffffffu, token, src) * a.q_stride +
                            __shfl_sync(0xffffffffu, q_head, src) * D;
        bool bad[kCols], some = false;
        float x[kCols], sum[kCols];
#pragma unroll
        for (int c = 0; c < kCols; c++) bad[c] = false, sum[c] = 0.f;
        for (int j = n; j < stop; j++) {
            value(j, x);
#pragma unroll
            for (int c = 0; c < kCols; c++) bad[c] = bad[c] || !finite(x[c]);
        }
#pragma unroll
        for (int c = 0; c < kCols; c++) some = some || bad[c];
        if (!__any_sync(0xffffffffu, some)) continue;
        for (int j0 = 0; j0 < n; j0 += 32) {
            float p = 0.f;
            if (j0 + lane < n) {
                const uint16_t *kj = k + (j0 + lane) * a.k_stride;
                float s = 0.f;
#pragma unroll 4
                for (int i = 0; i < D; i += 8) {
                    const uint4 u = *reinterpret_cast<const uint4 *>(q + i), w = *reinterpret_cast<const uint4 *>(kj + i);
                    const uint32_t us[4] = {u.x, u.y, u.z, u.w}, ws[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                    for (int e = 0; e < 4; e++) {
                        const float2 y = operands<F16>(us[e]), z = operands<F16>(ws[e]);
                        s = fmaf(y.y, z.y, fmaf(y.x, z.x, s));
                    }
                }
                if (a.scale < 0.f) s = -s;
                if constexpr (F16) s *= bf16x2_f32x2(factors[j0 + lane]).x;
                p = ex2(fmaf(s, f1, -m1)) * inv1;
            }
            bool open = false;               // some column is not NaN yet
            for (int j = 0; j < 32; j += 8) {
                float ahead[8][kCols];
#pragma unroll
                for (int e = 0; e < 8; e++) {
#pragma unroll
                    for (int c = 0; c < kCols; c++) ahead[e][c] = 0.f;   // past the row's keys: p is 0, too
                    if (j0 + j + e < n) value(j0 + j + e, ahead[e]);
                }
#pragma unroll
                for (int e = 0; e < 8; e++) {
                    const float pj = __shfl_sync(0xffffffffu, p, j + e);
#pragma unroll
                    for (int c = 0; c < kCols; c++) sum[c] = fmaf(pj, ahead[e][c], sum[c]);
                }
            }
#pragma unroll
            for (int c = 0; c < kCols; c++) open = open || (bad[c] && sum[c] == sum[c]);
            if (!__any_sync(0xffffffffu, open)) break;
        }
#pragma unroll
        for (int c = 0; c < kCols; c++)
            if (bad[c]) {
                const float y = sum[c];
                const long long at = (long long)to * D + lane * kCols + c;
                if (a.out_bf16) reinterpret_cast<__nv_bfloat16 *>(a.out)[at] = __float2bfloat16_rn(y);
                else reinterpret_cast<float *>(a.out)[at] = y;
            }
    }
}

template <int D, bool F16>
__global__ void __launch_bounds__(384, 1)
    gqa_prefill_kernel(const __grid_constant__ CUtensorMap q_map, const __grid_constant__ CUtensorMap k_map,
                       const __grid_constant__ CUtensorMap v_map, const GqaPrefillArgs a, long long wait_ns) {
    extern __shared__ uint8_t raw[];
    __shared__ Shared s;
    const uint32_t base = (smem_addr(raw) + 1023u) & ~1023u;
    uint8_t *sm = raw + (base - smem_addr(raw));
    const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
    constexpr int nb = D / 64;                           // blocks of a query or key tile
    constexpr uint32_t kHalf = nb * (kBlk / 2);          // 64 value rows
    constexpr uint32_t k_off = 2 * nb * kBlk, v_off = k_off + kKeys * kBlk, o_off = v_off + kValues * kHalf;
    pdl_wait();
    if (warp == 0) tmem_alloc(&s.tmem, 512);
    if (tid == 0) {
        for (int i = 0; i < 2; i++) {
            mbar_init(&s.q_full[i], 1);
            mbar_init(&s.q_empty[i], 1);
            mbar_init(&s.s_full[i], 1);
            mbar_init(&s.p_full[i][0], 4);
            mbar_init(&s.p_full[i][1], 4);
            mbar_init(&s.o_full[i], 1);
            mbar_init(&s.u_full[i], 1);
            mbar_init(&s.u_empty[i], 11);
        }
        for (int i = 0; i < kKeys; i++) {
            mbar_init(&s.k_full[i], 1);
            mbar_init(&s.k_empty[i], 1);
        }
        for (int i = 0; i < kValues; i++) {
            mbar_init(&s.v_full[i], 1);
            mbar_init(&s.v_empty[i], 1);
        }
        mbar_init(&s.next_full, 1);
        s.abort = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    tc_before_sync();
    __syncthreads();
    tc_after_sync();
    const uint32_t tmem = __shfl_sync(0xffffffffu, s.tmem, 0);
    volatile int *abort = &s.abort;
    bool ok = true;                      // this thread's waits have all ended well
    uint64_t deadline = deadline_after(wait_ns, 0);
    auto wait = [&](uint64_t *bar, uint32_t parity) {
        if (!ok) return;
        if (!warp_wait_now(bar, parity, deadline, abort, lane)) {
            ok = false;
            *abort = 1;
            atomicCAS(a.err, 0, (int)DEV_ERR_TIMEOUT);
        }
    };
    // Unit r of this CTA as the key warp has found it; the warp that has read it says so.
    auto take = [&](int r) {
        wait(&s.u_full[r & 1], (r >> 1) & 1);
        Unit u = s.unit[r & 1];
        if (!ok) u.n = -1;
        u = uniform(u);
        deadline = deadline_after(wait_ns, max(u.n, 0));
        __syncwarp();
        if (lane == 0) mbar_arrive(&s.u_empty[r & 1]);
        return u;
    };

    if (warp < 8) {
        // ---------------------------------------------------------- softmax and output
        const int x = warp >> 2, t = tid & 127;
        const uint32_t lanes = tmem + ((uint32_t)(32 * (warp & 3)) << 16), S = lanes + x * 128, O = lanes + 256 + x * D;
        // a negative scale turns the scores' sign; a factor of zero must still send masked scores (-inf) to -inf
        const bool negative = a.scale < 0.f;
        const float scale2 = fabsf(a.scale) * kLog2e;
        // f16 inputs: the factors of a tile's keys, [parity of the tile][key], in the warp's place for outputs
        uint8_t *stage = sm + o_off + warp * kOut;
        uint32_t(*power)[kRows] = reinterpret_cast<uint32_t(*)[kRows]>(stage);
        static_assert(sizeof(uint32_t[2][kRows]) <= kOut, "two tiles' factors fit");
        const int tok = t / a.group, g = t - tok * a.group;  // this thread's row: token of the tile, head of the group
        int tiles = 0, s_tiles = 0, outs = 0;            // key tiles, this tile's score tiles and outputs so far
        for (int r = 0;; r++) {
            const Unit u = take(r);
            if (u.n < 0) break;
            const int first = u.q0 + x * a.tokens, row = first + tok, nk = u.nk, nt = x ? u.nt[1] : u.nt[0];
            const int limit = min(row + nk - u.nq + 1, nk);     // keys this row sees
            const int all = min(first + nk - u.nq + 1, nk);     // keys every row of the tile sees
            const long long orow = tok < a.tokens && row < u.nq ? (long long)(u.qrow + row) * a.heads + u.head * a.group + g : -1;
            const float f = fmaxf(F16 ? scale2 * (orow >= 0 ? a.q_power[orow] : 0.f) * exp2i(-kKeyPower) : scale2, 1e-37f);
            auto fetch = [&](int j) {                    // whole warp
                const uint32_t *at = a.kv_power + ((long long)u.head * a.Tk + u.krow);
#pragma unroll
                for (int i = 0; i < kRows; i += 32) {
                    const int key = j * kRows + i + lane;
                    copy4(&power[j & 1][i + lane], at + (key < nk ? key : 0), key < nk);
                }
            };
            if (F16 && nt > 0) fetch(0);
            float m = kNone;
            float share = 0.f;                           // U
            int up = 0;                                  // log2 B
            float l4[4] = {0.f, 0.f, 0.f, 0.f};
            for (int j = 0; j < nt; j++) {
                bool keys_plain = true, plain = true;    // ordinary keys; and every value's factor is 1 / B
                if constexpr (F16) {
                    copies_done();
                    __syncwarp();                        // every lane's have come, and the last tile's factors are read
                    if (j == 0) up = 127 - (int)(power[0][0] >> 23);   // the first key, which all rows that see any see
                    const int up0 = __shfl_sync(0xffffffffu, up, 0);
                    plain = up == up0;
#pragma unroll
                    for (int i = 0; i < kRows; i += 32) {
                        const uint32_t w = power[j & 1][i + lane];
                        const bool none = j * kRows + i + lane >= nk;
                        keys_plain = keys_plain && (none || (w & 0xFFFFu) == kPlainKey);
                        plain = plain && (none || w == ((uint32_t)(127 - up0) << 23 | kPlainKey));
                    }
                    keys_plain = __all_sync(0xffffffffu, keys_plain);
                    plain = __all_sync(0xffffffffu, plain);
                    if (j + 1 < nt) fetch(j + 1);
                }
                const float ft = F16 && !keys_plain ? f * exp2i(kKeyShift) : f;
                wait(&s.s_full[x], s_tiles++ & 1);
                tc_after_sync();
                const int k0 = j * kRows;
                const bool full = k0 + kRows <= all;
                const int seen = limit - k0;                 // this row's keys in the tile
                // the row's scores, all at once: every wait for TMEM costs more than the arithmetic on a quarter of them
                uint32_t v[kRows];
#pragma unroll
                for (int c0 = 0; c0 < kRows; c0 += 32) tmem_ld(S + c0, *reinterpret_cast<uint32_t(*)[32]>(v + c0));
                tmem_ld_wait();
                if (negative)
#pragma unroll
                    for (int c = 0; c < kRows; c++) v[c] ^= 0x80000000u;
                if (F16 && !keys_plain)
#pragma unroll
                    for (int c = 0; c < kRows; c += 4) {
                        const uint4 w = *reinterpret_cast<const uint4 *>(&power[j & 1][c]);
                        const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                        for (int k = 0; k < 4; k += 2) {
                            float y = __uint_as_float(v[c + k]), z = __uint_as_float(v[c + k + 1]);
                            mul2(y, z, bf16x2_f32x2(ws[k]).x, bf16x2_f32x2(ws[k + 1]).x);
                            v[c + k] = __float_as_uint(y), v[c + k + 1] = __float_as_uint(z);
                        }
                    }
                // Rows of a warp see ever more keys: blocks of 32 keys before `least` are seen by all, from `most` on by none.
                const int least = full ? kRows : __shfl_sync(0xffffffffu, seen, 0), most = full ? kRows : __shfl_sync(0xffffffffu, seen, 31);
                if (!full)
#pragma unroll
                    for (int c0 = 0; c0 < kRows; c0 += 32)
                        if (c0 + 32 > least)
#pragma unroll
                            for (int c = c0; c < c0 + 32; c++)
                                if (c >= seen) v[c] = 0xFF800000u;
                float t4[4];
#pragma unroll
                for (int k = 0; k < 4; k++) t4[k] = max3(__uint_as_float(v[k]), __uint_as_float(v[4 + k]), __uint_as_float(v[8 + k]));
#pragma unroll
                for (int c = 12; c + 8 <= kRows; c += 8)
#pragma unroll
                    for (int k = 0; k < 4; k++) t4[k] = max3(t4[k], __uint_as_float(v[c + k]), __uint_as_float(v[c + 4 + k]));
#pragma unroll
                for (int k = 0; k < 4; k++) t4[k] = fmaxf(t4[k], __uint_as_float(v[kRows - 4 + k]));
                const float now = fmaxf(fmaxf(t4[0], t4[1]), fmaxf(t4[2], t4[3])) * ft;
                const bool move = now > m + kGrow;
                auto rescale = [&](float r) {            // O times r; whole warp
#pragma unroll 1
                    for (int c0 = 0; c0 < D; c0 += 8) {
                        uint32_t o[8];
                        tmem_ld(O + c0, o);
                        tmem_ld_wait();
#pragma unroll
                        for (int c = 0; c < 8; c++) o[c] = __float_as_uint(__uint_as_float(o[c]) * r);
                        tmem_st(O + c0, o);
                    }
                };
                float r = 1.f;
                if (__any_sync(0xffffffffu, move)) {
                    r = move ? ex2(m - now) : 1.f;
                    if (F16 && r < 0x1p-116f) r = 0.f;   // what it leaves of U can be held times B again
                    if (move) m = now;
#pragma unroll
                    for (int k = 0; k < 4; k++) l4[k] *= r;
                    if (j > 0) rescale(r);
                }
                if (k0 + kRows > nk) {
                    // value rows of other sequences may hold anything, and 0 * NaN is NaN
                    const int half = 2 * (tiles + j) + (t >> 6), slot = half % kValues;
                    wait(&s.v_full[slot], half / kValues & 1);
                    if (k0 + t >= nk)
#pragma unroll
                        for (int k = 0; k < nb; k++)
#pragma unroll
                            for (int c = 0; c < 8; c++)
                                *reinterpret_cast<uint4 *>(sm + v_off + slot * kHalf + k * (kBlk / 2) + (t & 63) * 128 + 16 * c) = make_uint4(0u, 0u, 0u, 0u);
                    fence_async_smem();
                }
                const float m0 = (F16 ? (float)kUp : 0.f) - m;
                if constexpr (F16) share *= r;
                if (F16 && plain) {
                    share = fmaxf(share, ex2(now + m0) * exp2i(-up));
                } else if constexpr (F16) {
                    // weights, times their keys' factors, times B
                    float u4[2] = {0.f, 0.f};
#pragma unroll
                    for (int c0 = 0; c0 < kRows; c0 += 32)
                        if (c0 < most)
#pragma unroll
                            for (int c = c0; c < c0 + 32; c += 4) {
                                const uint4 w = *reinterpret_cast<const uint4 *>(&power[j & 1][c]);
                                const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
                                float e[4];
                                fma2(e[0], e[1], v[c], v[c + 1], ft, m0);
                                fma2(e[2], e[3], v[c + 2], v[c + 3], ft, m0);
#pragma unroll
                                for (int k = 0; k < 4; k++) e[k] = ex2(e[k]);
                                add2(l4[0], l4[1], e[0], e[1]);
                                add2(l4[2], l4[3], e[2], e[3]);
#pragma unroll
                                for (int k = 0; k < 4; k += 2) {
                                    mul2(e[k], e[k + 1], bf16x2_f32x2(ws[k]).y, bf16x2_f32x2(ws[k + 1]).y);
                                    u4[k / 2] = max3(u4[k / 2], e[k], e[k + 1]);
                                    v[c + k] = __float_as_uint(e[k]), v[c + k + 1] = __float_as_uint(e[k + 1]);
                                }
                            }
                    share = max3(share, u4[0], u4[1]);
                    const float held = share * exp2i(up);
                    // to about 2^7, which for values of one size is 1 / their factor (2^7 less an ulp, too); an exponent field of 0
                    // gives more than kMostUp, the largest one (2^15 times 2^111) -119
                    const int next = share > 0.f && (held > 32768.f || held < 100.f) ? min(kMostUp, kUp + 127 - (int)(__float_as_uint(share * 1.5f) >> 23)) : up;
                    if (__any_sync(0xffffffffu, next != up) && j > 0) rescale(exp2i(max(-126, min(next - up, 126))));   // past that O is 0, or next to it
                    up = next;
                    const float by = exp2i(up);
#pragma unroll
                    for (int c = 0; c < kRows; c += 2) {
                        float y = __uint_as_float(v[c]), z = __uint_as_float(v[c + 1]);
                        mul2(y, z, by, by);
                        v[c] = __float_as_uint(y), v[c + 1] = __float_as_uint(z);
                    }
                }
#pragma unroll
                for (int h = 0; h < 2; h++) {
#pragma unroll
                    for (int c0 = 64 * h; c0 < 64 * h + 64; c0 += 32) {
                        uint32_t p[16];
                        if (c0 >= most) {
#pragma unroll
                            for (int c = 0; c < 16; c++) p[c] = 0;
                            tmem_st(S + c0 / 2, p);
                            continue;
                        }
#pragma unroll
                        for (int c = 0; c < 32; c += 2) {
                            float x, y;
                            if (F16 && !plain) {
                                x = __uint_as_float(v[c0 + c]), y = __uint_as_float(v[c0 + c + 1]);
                            } else {
                                fma2(x, y, v[c0 + c], v[c0 + c + 1], f, m0);
                                x = ex2(x), y = ex2(y);
                                add2(l4[c & 2], l4[(c & 2) + 1], x, y);
                            }
                            p[c / 2] = F16 ? pack_f16(x, y) : pack_bf16(x, y);
                        }
                        tmem_st(S + c0 / 2, p);              // over scores that have been read
                    }
                    tmem_st_wait();
                    tc_before_sync();
                    __syncwarp();
                    if (lane == 0 && ok) mbar_arrive(&s.p_full[x][h]);
                }
            }
            tiles += u.n;
            const float l = (l4[0] + l4[1]) + (l4[2] + l4[3]);
            // no weight at all: a row without keys, or one whose scores are all -infinity, which is NaN
            const float none = limit > 0 ? __uint_as_float(0x7FC00000u) : 0.f, inv = l != 0.f ? 1.f / l : none;
            if (nt > 0) {
                wait(&s.o_full[x], outs++ & 1);
                tc_after_sync();
            }
            // Rows go out through shared memory, 64 bytes of each at a time: 4 threads then write a row's piece together, where a thread's
            // own 16 bytes of 32 different rows cost 2.5 us a unit.
            if constexpr (F16) __syncwarp();             // the last tile's factors are read
            int dst[4];                                  // the output rows of this thread's pieces
#pragma unroll
            for (int i = 0; i < 4; i++) dst[i] = __shfl_sync(0xffffffffu, (int)orow, 8 * i + (lane >> 2));
            auto send = [&](const uint32_t (&w)[16], int byte) {   // 64 bytes of this thread's row
                const int x = lane >> 1 & 3;             // pieces of 16 bytes in an order of the row's own: no bank twice
#pragma unroll
                for (int c = 0; c < 4; c++)
                    *reinterpret_cast<uint4 *>(stage + lane * 64 + ((c ^ x) << 4)) = make_uint4(w[4 * c], w[4 * c + 1], w[4 * c + 2], w[4 * c + 3]);
                __syncwarp();
#pragma unroll
                for (int i = 0; i < 4; i++) {
                    const int row = 8 * i + (lane >> 2), piece = lane & 3;
                    const uint4 y = *reinterpret_cast<const uint4 *>(stage + row * 64 + ((piece ^ (row >> 1 & 3)) << 4));
                    if (dst[i] >= 0)
                        *reinterpret_cast<uint4 *>(reinterpret_cast<char *>(a.out) + (long long)dst[i] * (D * (a.out_bf16 ? 2 : 4)) + byte + 16 * piece) = y;
                }
                __syncwarp();
            };
            const uint32_t some = limit > 0 ? 0xFFFFFFFFu : 0u;   // a row without keys beside ones that have some: 0 times their values may be NaN
            const float out_inv = F16 ? inv * exp2i(kValueShift) : inv, down = exp2i(-up);   // what P and the values are held times, taken back
            float odd = 0.f;                             // NaN once an output is not finite
#pragma unroll 1
            for (int c0 = 0; c0 < D; c0 += 32) {
                uint32_t o[32];
                if (nt > 0) {
                    tmem_ld(O + c0, o);
                    tmem_ld_wait();
                } else {
#pragma unroll
                    for (int c = 0; c < 32; c++) o[c] = 0u;
                }
#pragma unroll
                for (int c = 0; c < 32; c++) o[c] = __float_as_uint(F16 ? __uint_as_float(o[c]) * out_inv * down : __uint_as_float(o[c]) * inv) & some;
#pragma unroll
                for (int c = 0; c < 32; c++) odd = fmaf(__uint_as_float(o[c]), 0.f, odd);
                uint32_t w[16];
                if (a.out_bf16) {
#pragma unroll
                    for (int c = 0; c < 16; c++) w[c] = pack_bf16(__uint_as_float(o[2 * c]), __uint_as_float(o[2 * c + 1]));
                    send(w, 2 * c0);
                } else {
#pragma unroll
                    for (int k = 0; k < 2; k++) {
#pragma unroll
                        for (int c = 0; c < 16; c++) w[c] = o[16 * k + c];
                        send(w, 4 * c0 + 64 * k);
                    }
                }
            }
            const int end = min(nt * kRows, nk);
            const bool again = odd != odd && orow >= 0 && limit > 0 && limit < end;
            if (__any_sync(0xffffffffu, again))
                repair<D, F16>(a, again, (int)orow, u.qrow + row, u.head * a.group + g, u.head, u.krow, limit, end, F16 ? f * exp2i(kKeyShift) : f, F16 ? m - kUp : m, inv);
            if (orow >= 0 && a.lse) a.lse[orow] = l != 0.f ? (m - (F16 ? kUp : 0) + log2f(l)) * 0.6931471805599453f : none - INFINITY;
            tc_before_sync();
        }
    } else if (warp == 8) {
        // ---------------------------------------------------------- MMA issue
        constexpr uint32_t id_s = f16_idesc(!F16, false, false, kRows, kRows), id_o = f16_idesc(!F16, false, true, kRows, D);
        const uint64_t dq = sw128_desc(base, 16, 1024), dk = sw128_desc(base + k_off, 16, 1024), dv = sw128_desc(base + v_off, kBlk / 2, 1024);
        // scores of query tile x with the keys at c; fresh: nobody has waited for them yet, last: nobody uses them after
        auto scores = [&](int x, Ring c, bool fresh, bool last) {
            const uint64_t qa = dq + ((x * nb * kBlk) >> 4);
#pragma unroll
            for (int b = 0; b < nb; b++) {
                if (fresh) {
                    wait(&s.k_full[c.slot], c.par);
                    tc_after_sync();
                }
                if (!ok) return;
                const uint64_t ka = dk + ((c.slot * kBlk) >> 4);
#pragma unroll
                for (int k = 0; k < 4; k++) mma_ss(tmem + x * 128, qa + ((b * kBlk) >> 4) + 2 * k, ka + 2 * k, id_s, b || k);
                if (last) tc_commit(&s.k_empty[c.slot]);
                c.step(1, kKeys);
            }
            tc_commit(&s.s_full[x]);
        };
        // the products of query tile x with the values at c, in halves of 64 keys
        auto output = [&](int x, int tile, bool more, Ring c, bool fresh, bool last) {
#pragma unroll
            for (int h = 0; h < 2; h++) {
                wait(&s.p_full[x][h], tile & 1);
                if (fresh) wait(&s.v_full[c.slot], c.par);
                tc_after_sync();
                if (!ok) return;
                const uint64_t va = dv + ((c.slot * kHalf) >> 4);
#pragma unroll
                for (int k = 0; k < 4; k++) mma_ts(tmem + 256 + x * D, tmem + x * 128 + 8 * (4 * h + k), va + ((k * 2048) >> 4), id_o, more || h || k);
                if (last) tc_commit(&s.v_empty[c.slot]);
                c.step(1, kValues);
            }
        };
        Ring kr{0, 0}, vr{0, 0};                         // this unit's next keys and values
        int st[2] = {0, 0}, qs[2] = {0, 0};              // score tiles and query tiles before this unit
        for (int r = 0;; r++) {
            const Unit u = take(r);
            if (u.n < 0) break;
            if (u.n == 0) continue;
#pragma unroll
            for (int x = 0; x < 2; x++)
                if (u.nt[x] > 0) {
                    wait(&s.q_full[x], qs[x]++ & 1);
                    tc_after_sync();
                    scores(x, kr, x == 0 || u.nt[0] == 0, x == 1 || u.nt[1] == 0);
                    if (ok && u.nt[x] == 1) tc_commit(&s.q_empty[x]);
                }
            kr.step(nb, kKeys);
            for (int j = 0; j < u.n; j++) {
#pragma unroll
                for (int x = 0; x < 2; x++) {
                    if (j >= u.nt[x]) continue;
                    output(x, st[x] + j, j > 0, vr, x == 0 || j >= u.nt[0], x == 1 || j >= u.nt[1]);
                    if (j + 1 < u.nt[x]) {
                        scores(x, kr, x == 0 || j + 1 >= u.nt[0], x == 1 || j + 1 >= u.nt[1]);
                        if (ok && j + 2 == u.nt[x]) tc_commit(&s.q_empty[x]);
                    } else if (ok) {
                        tc_commit(&s.o_full[x]);
                    }
                }
                vr.step(2, kValues);
                if (j + 1 < u.n) kr.step(nb, kKeys);
            }
            st[0] += u.nt[0];
            st[1] += u.nt[1];
        }
    } else if (warp == 9) {
        // ---------------------------------------------------------- units and bulk copies of keys
        int most, blocks = 0, i = blockIdx.x, asked = 0;
        Ring c{0, 0};
        const int pairs = all_pairs(a, lane, blockIdx.x == 0, most), units = pairs * a.H;
        Place at = no_place(most);
        for (int r = 0;; r++) {
            Unit u;
            u.n = -1;
            u.nt[0] = u.nt[1] = u.head = u.q0 = u.nq = u.nk = u.qrow = u.krow = 0;
            if (i >= 0 && i < units) u = uniform(unit_of(a, i, pairs, at, lane));
            if (i < 0 || u.n >= 0) {
                if (r > 1) wait(&s.u_empty[r & 1], ((r >> 1) - 1) & 1);
                if (!ok) break;
                if (lane == 0) {
                    s.unit[r & 1] = u;
                    mbar_arrive(&s.u_full[r & 1]);
                }
                if (i < 0) break;
            } else {
                r--;                     // more CTAs than units: nothing to do for this one
            }
            deadline = deadline_after(wait_ns, max(u.n, 0));
            // Which work comes next is asked for late: at the start every CTA would be given its second unit, the longest one to
            // the CTA that has the longest already (1x2432, 2 units an SM: 53 us, this way 43).
            const int last = max(u.n - 1, 0);
            for (int j = 0; j <= last; j++) {
                if (j == last) {
                    if (lane == 0) {
                        mbar_expect_tx(&s.next_full, 16);
                        ask_next(s);
                    }
                    __syncwarp();
                }
                if (j >= u.n) break;
                for (int b = 0; b < nb; b++) {
                    if (blocks++ >= kKeys) wait(&s.k_empty[c.slot], c.par ^ 1);
                    if (!ok) break;
                    expect_bytes(&s.k_full[c.slot], kBlk);
                    tma_box(base + k_off + c.slot * kBlk, &k_map, u.head * D + 64 * b, u.krow + j * kRows, &s.k_full[c.slot]);
                    c.step(1, kKeys);
                }
            }
            wait(&s.next_full, asked++ & 1);
            if (!ok) break;
            i = read_next(s);
            __syncwarp();                // all lanes have read before the next request
        }
    } else {
        // ---------------------------------------------------------- bulk copies of a query tile and of half the values
        const int h = warp - 10;
        int tiles = 0, qs = 0;
        Ring c{h, 0};
        for (int r = 0;; r++) {
            const Unit u = take(r);
            if (u.n < 0) break;
            if ((h ? u.nt[1] : u.nt[0]) > 0) {
                if (qs > 0) wait(&s.q_empty[h], (qs - 1) & 1);
                qs++;
                if (ok) expect_bytes(&s.q_full[h], nb * a.tokens * a.group * 128);
                for (int b = 0; b < nb && ok; b++)
                    tma_box3(base + (h * nb + b) * kBlk, &q_map, 64 * b, u.head * a.group, u.qrow + u.q0 + h * a.tokens, &s.q_full[h]);
            }
            for (int j = 0; j < u.n; j++) {
                if (2 * tiles++ + h >= kValues) wait(&s.v_empty[c.slot], c.par ^ 1);
                if (!ok) break;
                expect_bytes(&s.v_full[c.slot], kHalf);
                for (int b = 0; b < nb; b++)
                    tma_box(base + v_off + c.slot * kHalf + b * (kBlk / 2), &v_map, u.head * D + 64 * b, u.krow + j * kRows + 64 * h, &s.v_full[c.slot]);
                c.step(2, kValues);
            }
        }
    }
    pdl_trigger();
    tc_before_sync();
    __syncthreads();
    if (warp == 0) {
        if (*abort) settle();
        tc_after_sync();
        tmem_free(tmem, 512);
    }
}

// Boxes of 64 dims x a group's heads x a tile's tokens of q.
cudaError_t query_map(const GqaPrefillArgs &a, CUtensorMap *out) {
    const PFN_cuTensorMapEncodeTiled_v12000 fn = encode_tiled();
    if (!fn) return cudaErrorNotSupported;
    const cuuint64_t dims[3] = {(cuuint64_t)a.dim, (cuuint64_t)a.heads, (cuuint64_t)a.Tq};
    const cuuint64_t strides[2] = {(cuuint64_t)a.dim * 2, (cuuint64_t)a.q_stride * 2};
    const cuuint32_t box[3] = {64, (cuuint32_t)a.group, (cuuint32_t)a.tokens}, estr[3] = {1, 1, 1};
    return fn(out, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(a.q), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
              CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS
               ? cudaSuccess
               : cudaErrorInvalidValue;
}

// f32 -> f16: each row of q, k and v times a power of two of its own, whose factor goes to q_power (by rows) or, by heads and tokens,
// to kv_power.  Rows of q, then of k, then of v; one thread per 8 elements.
template <int D>
__global__ void __launch_bounds__(256) gqa_round_kernel(const GqaPrefillArgs a, __half *q16, __half *k16, __half *v16, float *q_power,
                                                        __nv_bfloat16 *kv_power) {
    constexpr int kUnits = D / 8;
    auto finite = [](float x) {
        const uint32_t b = __float_as_uint(x) & 0x7FFFFFFFu;
        return b < 0x7F800000u ? b : 0u;
    };
    const long long n_q = (long long)a.Tq * a.heads, n_k = (long long)a.Tk * a.H, rows = n_q + 2 * n_k;
    const int u = threadIdx.x % kUnits;
    // Factors are numbers, at 2^-126 the smallest: rows that would need a smaller one get a power that is less.
    const int most_q = min(126, 118 + max(-230, min(8, ilogbf(a.scale * kLog2e)))), most_k = 126 + kKeyPower - kKeyShift, most_v = 126 - kValueShift;
    pdl_wait();
    for (long long r0 = blockIdx.x * (256LL / kUnits); r0 < rows; r0 += gridDim.x * (256LL / kUnits)) {   // the CTA stays together
        const long long r = r0 + threadIdx.x / kUnits;
        const bool query = r < n_q, value = r >= n_q + n_k;
        const uint32_t i = (uint32_t)(query ? r : value ? r - n_q - n_k : r - n_q), heads = query ? a.heads : a.H, t = i / heads, h = i - t * heads;   // rows of each < 2^31
        float4 x = make_float4(0.f, 0.f, 0.f, 0.f), y = x;
        if (r < rows) {
            const float *p = (const float *)(query ? a.q : value ? a.v : a.k) + t * (query ? a.q_stride : value ? a.v_stride : a.k_stride) + h * D + 8 * u;
            x = *reinterpret_cast<const float4 *>(p);
            y = *reinterpret_cast<const float4 *>(p + 4);
        }
        uint32_t m = max(max(max(finite(x.x), finite(x.y)), max(finite(x.z), finite(x.w))), max(max(finite(y.x), finite(y.y)), max(finite(y.z), finite(y.w))));
#pragma unroll
        for (int o = 1; o < kUnits; o <<= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
        if (r >= rows) continue;
        const int size = m ? (int)(m >> 23) - 127 : 0;   // below 2^-126 any small number will do
        int e = min(14 - size, query ? most_q : most_k);
        if (!query && !value && size >= -5 && size <= 10) e = kKeyPower;
        if (value) e = min(kValuePower - 10 * ((size + 204) / 10 - 20), most_v);
        const float by = query && a.scale == 0.f ? 0.f : exp2i(e);
        if (u == 0) {
            if (query) q_power[i] = exp2i(-e);
            else kv_power[2 * (h * (long long)a.Tk + t) + value] = __float2bfloat16_rn(exp2i(value ? -kValueShift - e : kKeyPower - kKeyShift - e));
        }
        reinterpret_cast<uint4 *>(query ? q16 : value ? v16 : k16)[i * (long long)kUnits + u] =
            make_uint4(pack_f16(x.x * by, x.y * by), pack_f16(x.z * by, x.w * by), pack_f16(y.x * by, y.y * by), pack_f16(y.z * by, y.w * by));
    }
    pdl_trigger();
}

// What a call with f32 inputs keeps in scratch.
struct Rounded {
    size_t q, k, v, q_power, kv_power, end;
};
Rounded rounded(const GqaPrefillArgs &a) {
    Rounded z;
    z.q = 0;
    z.k = z.q + round256((size_t)a.Tq * a.heads * a.dim * 2);
    z.v = z.k + round256((size_t)a.Tk * a.H * a.dim * 2);
    z.q_power = z.v + round256((size_t)a.Tk * a.H * a.dim * 2);
    z.kv_power = z.q_power + round256((size_t)a.Tq * a.heads * sizeof(float));
    z.end = z.kv_power + round256((size_t)a.Tk * a.H * sizeof(uint32_t));
    return z;
}

template <int D>
cudaError_t round_inputs(GqaPrefillArgs &a, const DevInfo &d, cudaStream_t st, int *n_launch) {
    const Rounded z = rounded(a);
    char *at = (char *)d.scratch;
    const long long rows = (long long)a.Tq * a.heads + 2LL * a.Tk * a.H, ctas = (rows * (D / 8) + 255) / 256;
    if (cudaError_t e = launch_pdl(gqa_round_kernel<D>, dim3((unsigned)std::min(ctas, 16LL * d.n_sm)), dim3(256), 0, st, a, (__half *)(at + z.q),
                                   (__half *)(at + z.k), (__half *)(at + z.v), (float *)(at + z.q_power), (__nv_bfloat16 *)(at + z.kv_power)))
        return e;
    ++*n_launch;
    a.q = at + z.q;
    a.k = at + z.k;
    a.v = at + z.v;
    a.q_stride = a.heads * a.dim;
    a.k_stride = a.v_stride = a.H * a.dim;
    a.q_power = (const float *)(at + z.q_power);
    a.kv_power = (const uint32_t *)(at + z.kv_power);
    return cudaSuccess;
}

template <int D, bool F16>
cudaError_t run(const GqaPrefillArgs &a, const DevInfo &d, cudaStream_t st) {
    CUtensorMap q, k, v;
    if (cudaError_t e = query_map(a, &q)) return e;
    k = v = q;                                // no keys: never read
    if (a.Tk > 0) {
        if (cudaError_t e = matrix_map(a.k, (long long)a.H * D, a.Tk, a.k_stride, kRows, &k)) return e;
        if (cudaError_t e = matrix_map(a.v, (long long)a.H * D, a.Tk, a.v_stride, kRows / 2, &v)) return e;
    }
    // at most; every unit that is not empty has a row of its own
    const long long units = std::min((long long)a.Tq, ((long long)a.Tq + 2 * a.tokens - 1) / (2 * a.tokens) + a.n_seq - 1) * a.H;
    constexpr size_t smem = (2 * (D / 64) + kKeys) * kBlk + kValues * (D / 64) * (kBlk / 2) + 8 * kOut + 1024;
    static std::atomic<uint64_t> done{0};
    if (cudaError_t e = allow_smem(gqa_prefill_kernel<D, F16>, smem, d.device, done)) return e;
    return launch_pdl(gqa_prefill_kernel<D, F16>, dim3((unsigned)units), dim3(384), smem, st, q, k, v, a, d.wait_ns);
}

template <int D>
cudaError_t launch(GqaPrefillArgs a, const DevInfo &d, cudaStream_t st, int *n_launch) {
    *n_launch = 1;
    if (!a.in_f32) return run<D, false>(a, d, st);
    if (cudaError_t e = round_inputs<D>(a, d, st, n_launch)) return e;
    return run<D, true>(a, d, st);
}

}  // namespace

size_t gqa_prefill_scratch(const GqaPrefillArgs &a) { return a.in_f32 ? rounded(a).end : 0; }

cudaError_t launch_gqa_prefill(const GqaPrefillArgs &a, const DevInfo &d, cudaStream_t st, int *n_launch) {
    return a.dim == 64 ? launch<64>(a, d, st, n_launch) : launch<128>(a, d, st, n_launch);
}

}  // namespace coli

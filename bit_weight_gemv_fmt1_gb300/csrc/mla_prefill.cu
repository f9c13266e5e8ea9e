// mla_prefill.cu -- causal attention of packed sequences in the expanded form,
// on the 5th-generation tensor cores.
//
// A unit of work is one head and 256 query rows of one sequence, two tiles A and
// B of 128, and a walk over the keys in tiles of 128.  The grid has a CTA per unit, longest first; a CTA that nears its
// unit's end takes over one that has not started (cluster launch control), so that the next queries, keys and
// scores come while the last output is written.  Only the key warp looks units up; it hands them on through a ring of
// two, and every warp spreads them from lane 0: MMA and copy operands that the compiler cannot prove uniform cost 300 of
// 2900 cycles a tile.  Times of 8192 tokens x 32 heads / 4 x 2048 x 32 / 3 x 4000 with 4000 cached x 8, us: a CTA per
// unit in the order of heads 515 / 124 / 236; units of a fixed share 485 / 120 / 235; this 474 / 96 / 233.  Taking heads in groups
// whose keys fit L2: 494 / 105 / 238; keys and values asked into L2 four tiles ahead: slower by 2 %.
//   S = Q K^T   M = 128 queries, N = 128 keys, K = nope + rope (K-major operands in shared memory)
//   O += P V    M = 128 queries, N = v, K = 128 keys (P in TMEM, V as stored: N-major)
// The two tiles alternate: while the softmax of one runs, the tensor cores work
// on the other.  One thread holds one query row; P overwrites S in TMEM.
//
// Softmax: x = log2(e) * scale * score, e = 2^(x - m), l += e, P = bf16(e).  m is
// the row's running maximum, moved (and O and l rescaled) only when a tile's
// maximum passes it by 8: weights up to 2^8 lose nothing in bf16.  m, l and O are
// f32; rounding P to bf16 is within 2^-8 of each weight, as the values' own.
//
// Bound: shared memory, close to the tensor cores.  A round (128 keys, nope + rope = 192, v = 128) is 24 score MMAs that read 8 KB,
// 16 output MMAs that read 4 KB and 82 KB of copies coming in, 342 KB or 2670 cycles at 128 bytes each; the tensor cores
// alone need 2340.  Measured: 3300, in which the MMA warp issues without a pause (scores 86 cycles each, 59 alone) and
// either softmax (1300) has 2000 to spare.  Q from TMEM would spare a third of the reads, but S and O fill TMEM.
// Shared memory holds Q (96 KB), a ring of 5 key blocks of 128 keys x 64 dims (80 KB) and a
// ring of 3 value halves of 64 keys (48 KB), each freed and asked for by itself after its last use.  In a round
// the values lie idle for 770 cycles and the keys for 500, less than a copy takes (1000 to 1500): what the rings hold
// beyond a tile covers that.  Two whole key tiles and one value tile, of the same size: 474 / 96 / 233 us against
// 452 / 96 / 231 (8 x 1000 x 16 heads: 40 against 41, the price of more barriers); all blocks of a key tile waited for at once: 471.
// (These compare versions of their day on the same inputs again and again.)  8192 tokens x 32 heads now: 435 to 465 us that
// way, 474 us with new inputs each call, 1.45 PFLOP/s, 0.75 of the measured bf16 rate.
//
// Keys past a causal row's limit are masked by selection; value rows past the
// sequence's end belong to its neighbours and are zeroed in shared memory.
// Warps: 0-3 and 4-7 softmax of A and B, 8 MMA issue, 9 units and copies of keys, 10 and 11 of queries and values.
// Every wait is bounded, by a limit that each unit renews: a CTA that takes over units lives as
// long as the call.  After one has run out all waits return at once, no further MMA or copy is
// issued, and the kernel records DEV_ERR_TIMEOUT.
#include <cudaTypedefs.h>

#include <algorithm>

#include "mla_units.cuh"
#include "tcgen05.cuh"

namespace coli {

namespace {

constexpr uint32_t kBlk = kRows * 128;   // 128 rows x 64 bf16, 128-byte swizzle
constexpr float kGrow = 8.f;             // log2 of the weight that moves the reference
constexpr float kNone = -3e38f;          // reference of a row that has seen no key

__device__ __forceinline__ float max3(float a, float b, float c) {
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}

struct Shared {
    uint64_t q_full[2], q_empty[2], k_full[5], k_empty[5], v_full[3], v_empty[3], s_full[2], p_full[2], o_full[2], u_full[2], u_empty[2];
    uint64_t next_full;
    Unit unit[2];
    alignas(16) uint32_t next[4];        // the answer to the last request for a CTA's work
    uint32_t tmem;
    int abort;
};


// A place in a ring of n buffers and the parity of its use.
struct Ring {
    int slot, par;
    __device__ __forceinline__ void step(int by, int n) {
        slot += by;
        if (slot >= n) {
            slot -= n;
            par ^= 1;
        }
    }
};

// The same values, all from lane 0: the compiler then keeps them, and the operands of MMAs and copies that derive from
// them, in uniform registers.
__device__ __forceinline__ Unit uniform(Unit u) {
    for (int *p : {&u.head, &u.q0, &u.nq, &u.nk, &u.qrow, &u.krow, &u.nt[0], &u.nt[1], &u.n}) *p = __shfl_sync(0xffffffffu, *p, 0);
    return u;
}

// Asks for the work of a CTA that has not started yet, in its stead; the answer (16 bytes) comes to `next`.
__device__ __forceinline__ void ask_next(Shared &s) {
    asm volatile("clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];" ::"r"(smem_addr(s.next)),
                 "r"(smem_addr(&s.next_full))
                 : "memory");
}
// That CTA's index; -1: all have started, and no further request may be made.
__device__ __forceinline__ int read_next(Shared &s) {
    int i;
    asm volatile(
        "{\n .reg .b128 r;\n .reg .pred p;\n mov.s32 %0, -1;\n ld.shared.b128 r, [%1];\n"
        " clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, r;\n"
        " @p clusterlaunchcontrol.query_cancel.get_first_ctaid::x.b32.b128 %0, r;\n"
        " fence.proxy.async.shared::cta;\n}\n"
        : "=&r"(i)
        : "r"(smem_addr(s.next))
        : "memory");
    return i;
}

template <int V>
__global__ void __launch_bounds__(384, 1)
    mla_prefill_kernel(const __grid_constant__ CUtensorMap q_map, const __grid_constant__ CUtensorMap kv_map,
                       const __grid_constant__ CUtensorMap kr_map, const __grid_constant__ CUtensorMap v_map, const MlaPrefillArgs a, long long wait_ns) {
    extern __shared__ uint8_t raw[];
    __shared__ Shared s;
    const uint32_t base = (smem_addr(raw) + 1023u) & ~1023u;
    uint8_t *sm = raw + (base - smem_addr(raw));
    const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
    const int nn = a.nope / 64, nb = nn + 1;             // blocks of a query or key tile: no-position part, rotary part
    const int nk_ring = 2 * nb - 1;                      // key blocks of 64 dims
    constexpr uint32_t kHalf = V / 64 * (kBlk / 2);      // 64 value rows
    const uint32_t k_off = 2 * nb * kBlk, v_off = k_off + nk_ring * kBlk;
    pdl_wait();
    pdl_trigger();
    if (warp == 0) tmem_alloc(&s.tmem, 512);
    if (tid == 0) {
        for (int i = 0; i < 2; i++) {
            mbar_init(&s.q_full[i], 1);
            mbar_init(&s.q_empty[i], 1);
            mbar_init(&s.s_full[i], 1);
            mbar_init(&s.p_full[i], 4);
            mbar_init(&s.o_full[i], 1);
            mbar_init(&s.u_full[i], 1);
            mbar_init(&s.u_empty[i], 11);
        }
        for (int i = 0; i < 5; i++) {
            mbar_init(&s.k_full[i], 1);
            mbar_init(&s.k_empty[i], 1);
        }
        for (int i = 0; i < 3; i++) {
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
    // Unit r of this CTA as the key warp has found it; the warp that has read it says so.  It comes when the keys of the unit
    // before have been asked for: a warp with no tile in that one waits for all of its time.
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
        const uint32_t lanes = tmem + ((uint32_t)(32 * (warp & 3)) << 16), S = lanes + x * 128, O = lanes + 256 + x * V;
        // a negative scale turns the scores' sign; a zero one must still send masked scores (-inf) to -inf
        const bool negative = a.scale < 0.f;
        const float f = a.scale == 0.f ? 1e-37f : fabsf(a.scale) * 1.4426950408889634f;
        int k3 = 0, s_tiles = 0, outs = 0;               // key tiles so far mod 3, this tile's score tiles and outputs so far
        for (int r = 0;; r++) {
            const Unit u = take(r);
            if (u.n < 0) break;
            const int row = u.q0 + x * kRows + t, nk = u.nk, nt = x ? u.nt[1] : u.nt[0];
            const int limit = min(row + nk - u.nq + 1, nk);  // keys this row sees
            const int all = min(row - t + nk - u.nq + 1, nk);   // keys every row of the tile sees
            const long long orow = row < u.nq ? (long long)(u.qrow + row) * a.H + u.head : -1;
            float m = kNone;
            float l4[4] = {0.f, 0.f, 0.f, 0.f};
            for (int j = 0; j < nt; j++, k3 = k3 == 2 ? 0 : k3 + 1) {
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
                if (!full)
#pragma unroll
                    for (int c = 0; c < kRows; c++)
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
                const float now = fmaxf(fmaxf(t4[0], t4[1]), fmaxf(t4[2], t4[3])) * f;
                const bool move = now > m + kGrow;
                if (__any_sync(0xffffffffu, move)) {
                    const float r = move ? ex2(m - now) : 1.f;
                    if (move) m = now;
#pragma unroll
                    for (int k = 0; k < 4; k++) l4[k] *= r;
                    if (j > 0) {
#pragma unroll 1
                        for (int c0 = 0; c0 < V; c0 += 8) {
                            uint32_t o[8];
                            tmem_ld(O + c0, o);
                            tmem_ld_wait();
#pragma unroll
                            for (int c = 0; c < 8; c++) o[c] = __float_as_uint(__uint_as_float(o[c]) * r);
                            tmem_st(O + c0, o);
                        }
                    }
                }
                const float m0 = -m;
#pragma unroll
                for (int c0 = 0; c0 < kRows; c0 += 32) {
                    uint32_t p[16];
#pragma unroll
                    for (int c = 0; c < 32; c += 2) {
                        const float x = ex2(fmaf(__uint_as_float(v[c0 + c]), f, m0)), y = ex2(fmaf(__uint_as_float(v[c0 + c + 1]), f, m0));
                        l4[c & 3] += x;
                        l4[(c + 1) & 3] += y;
                        p[c / 2] = pack_bf16(x, y);
                    }
                    tmem_st(S + c0 / 2, p);                  // over scores that have been read
                }
                if (k0 + kRows > nk) {
                    // value rows of other sequences may hold anything, and 0 * NaN is NaN
                    const int half = 2 * k3 + (t >> 6), slot = half < 3 ? half : half - 3;
                    wait(&s.v_full[slot], half >= 3);
                    if (k0 + t >= nk)
#pragma unroll
                        for (int k = 0; k < V / 64; k++)
#pragma unroll
                            for (int c = 0; c < 8; c++)
                                *reinterpret_cast<uint4 *>(sm + v_off + slot * kHalf + k * (kBlk / 2) + (t & 63) * 128 + 16 * c) = make_uint4(0u, 0u, 0u, 0u);
                    fence_async_smem();
                }
                tmem_st_wait();
                tc_before_sync();
                __syncwarp();
                if (lane == 0 && ok) mbar_arrive(&s.p_full[x]);
            }
            k3 = (k3 + u.n - nt) % 3;
            const float l = (l4[0] + l4[1]) + (l4[2] + l4[3]);
            const float inv = l != 0.f ? 1.f / l : 0.f;
            if (nt > 0) {
                wait(&s.o_full[x], outs++ & 1);
                tc_after_sync();
            }
#pragma unroll 1
            for (int c0 = 0; c0 < V; c0 += 32) {
                uint32_t o[32];
                if (nt > 0) {
                    tmem_ld(O + c0, o);
                    tmem_ld_wait();
                } else {
#pragma unroll
                    for (int c = 0; c < 32; c++) o[c] = 0u;
                }
                if (orow < 0) continue;
#pragma unroll
                for (int c = 0; c < 32; c++) o[c] = __float_as_uint(__uint_as_float(o[c]) * inv);
                if (a.out_bf16) {
                    uint4 *d = reinterpret_cast<uint4 *>(reinterpret_cast<__nv_bfloat16 *>(a.out) + orow * V + c0);
#pragma unroll
                    for (int c = 0; c < 32; c += 8) {
                        uint32_t w[4];
#pragma unroll
                        for (int k = 0; k < 4; k++) w[k] = pack_bf16(__uint_as_float(o[c + 2 * k]), __uint_as_float(o[c + 2 * k + 1]));
                        d[c / 8] = make_uint4(w[0], w[1], w[2], w[3]);
                    }
                } else {
                    uint4 *d = reinterpret_cast<uint4 *>(reinterpret_cast<float *>(a.out) + orow * V + c0);
#pragma unroll
                    for (int c = 0; c < 32; c += 4) d[c / 4] = make_uint4(o[c], o[c + 1], o[c + 2], o[c + 3]);
                }
            }
            if (orow >= 0 && a.lse) a.lse[orow] = l != 0.f ? (m + log2f(l)) * 0.6931471805599453f : -INFINITY;
            tc_before_sync();
        }
    } else if (warp == 8) {
        // ---------------------------------------------------------- MMA issue
        constexpr uint32_t id_s = f16_idesc(1, false, false, kRows, kRows), id_o = f16_idesc(1, false, true, kRows, V);
        const uint64_t dq = sw128_desc(base, 16, 1024), dk = sw128_desc(base + k_off, 16, 1024), dv = sw128_desc(base + v_off, kBlk / 2, 1024);
        // scores of query tile x with the keys at c; fresh: nobody has waited for them yet, last: nobody uses them after
        auto scores = [&](int x, Ring c, bool fresh, bool last) {
            const uint64_t qa = dq + ((x * nb * kBlk) >> 4);
            for (int b = 0; b < nn; b++) {
                if (fresh) {
                    wait(&s.k_full[c.slot], c.par);
                    tc_after_sync();
                }
                if (!ok) return;
                const uint64_t ka = dk + ((c.slot * kBlk) >> 4);
#pragma unroll
                for (int k = 0; k < 4; k++) mma_ss(tmem + x * 128, qa + ((b * kBlk) >> 4) + 2 * k, ka + 2 * k, id_s, b || k);
                if (last) tc_commit(&s.k_empty[c.slot]);
                c.step(1, nk_ring);
            }
            if (fresh) {
                wait(&s.k_full[c.slot], c.par);
                tc_after_sync();
            }
            if (!ok) return;
            const uint64_t ka = dk + ((c.slot * kBlk) >> 4);
#pragma unroll
            for (int k = 0; k < 4; k++)
                if (16 * k < a.rope) mma_ss(tmem + x * 128, qa + ((nn * kBlk) >> 4) + 2 * k, ka + 2 * k, id_s, true);
            if (last) tc_commit(&s.k_empty[c.slot]);
            tc_commit(&s.s_full[x]);
        };
        // the products of query tile x with the values at c, in halves of 64 keys
        auto output = [&](int x, bool more, Ring c, bool fresh, bool last) {
#pragma unroll
            for (int h = 0; h < 2; h++) {
                if (fresh) {
                    wait(&s.v_full[c.slot], c.par);
                    tc_after_sync();
                }
                if (!ok) return;
                const uint64_t va = dv + ((c.slot * kHalf) >> 4);
#pragma unroll
                for (int k = 0; k < 4; k++) mma_ts(tmem + 256 + x * V, tmem + x * 128 + 8 * (4 * h + k), va + ((k * 2048) >> 4), id_o, more || h || k);
                if (last) tc_commit(&s.v_empty[c.slot]);
                c.step(1, 3);
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
            kr.step(nb, nk_ring);
            for (int j = 0; j < u.n; j++) {
#pragma unroll
                for (int x = 0; x < 2; x++) {
                    if (j >= u.nt[x]) continue;
                    wait(&s.p_full[x], (st[x] + j) & 1);
                    tc_after_sync();
                    output(x, j > 0, vr, x == 0 || j >= u.nt[0], x == 1 || j >= u.nt[1]);
                    if (j + 1 < u.nt[x]) {
                        scores(x, kr, x == 0 || j + 1 >= u.nt[0], x == 1 || j + 1 >= u.nt[1]);
                        if (ok && j + 2 == u.nt[x]) tc_commit(&s.q_empty[x]);
                    } else if (ok) {
                        tc_commit(&s.o_full[x]);
                    }
                }
                vr.step(2, 3);
                if (j + 1 < u.n) kr.step(nb, nk_ring);
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
            if (lane == 0) {
                mbar_expect_tx(&s.next_full, 16);
                ask_next(s);
            }
            __syncwarp();
            deadline = deadline_after(wait_ns, max(u.n, 0));
            const int hk = u.head * (a.nope + V);
            for (int j = 0; j < u.n; j++)
                for (int b = 0; b < nb; b++) {
                    if (blocks++ >= nk_ring) wait(&s.k_empty[c.slot], c.par ^ 1);
                    if (!ok) break;
                    expect_bytes(&s.k_full[c.slot], kBlk);
                    tma_box(base + k_off + c.slot * kBlk, b < nn ? &kv_map : &kr_map, b < nn ? hk + 64 * b : 0, u.krow + j * kRows, &s.k_full[c.slot]);
                    c.step(1, nk_ring);
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
            const int hk = u.head * (a.nope + V), hq = u.head * (a.nope + a.rope);
            if ((h ? u.nt[1] : u.nt[0]) > 0) {
                if (qs > 0) wait(&s.q_empty[h], (qs - 1) & 1);
                qs++;
                if (ok) expect_bytes(&s.q_full[h], nb * kBlk);
                for (int b = 0; b < nb && ok; b++) tma_box(base + (h * nb + b) * kBlk, &q_map, hq + 64 * b, u.qrow + u.q0 + h * kRows, &s.q_full[h]);
            }
            for (int j = 0; j < u.n; j++) {
                if (2 * tiles++ + h >= 3) wait(&s.v_empty[c.slot], c.par ^ 1);
                if (!ok) break;
                expect_bytes(&s.v_full[c.slot], kHalf);
                for (int b = 0; b < V / 64; b++)
                    tma_box(base + v_off + c.slot * kHalf + b * (kBlk / 2), &v_map, hk + a.nope + 64 * b, u.krow + j * kRows + 64 * h, &s.v_full[c.slot]);
                c.step(2, 3);
            }
        }
    }
    tc_before_sync();
    __syncthreads();
    if (warp == 0) {
        if (*abort) settle();
        tc_after_sync();
        tmem_free(tmem, 512);
    }
}

// f32 -> bf16, rows of `cols` (a multiple of 8) at `stride` to packed ones.
__global__ void __launch_bounds__(256) mla_round_kernel(const float *src, long long stride, long long rows, int cols, __nv_bfloat16 *dst) {
    pdl_wait();
    pdl_trigger();
    const int units = cols / 8;
    const long long n = rows * units;
    for (long long i = blockIdx.x * 256LL + threadIdx.x; i < n; i += gridDim.x * 256LL) {
        const long long r = i / units;
        const int u = (int)(i - r * units);
        const float4 x = *reinterpret_cast<const float4 *>(src + r * stride + 8 * u), y = *reinterpret_cast<const float4 *>(src + r * stride + 8 * u + 4);
        reinterpret_cast<uint4 *>(dst)[i] = make_uint4(pack_bf16(x.x, x.y), pack_bf16(x.z, x.w), pack_bf16(y.x, y.y), pack_bf16(y.z, y.w));
    }
}

cudaError_t matrix_map(const void *p, long long cols, long long rows, long long stride, int box_rows, CUtensorMap *out) {
    static PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
        void *f = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) != cudaSuccess ||
            q != cudaDriverEntryPointSuccess)
            f = nullptr;
        return (PFN_cuTensorMapEncodeTiled_v12000)f;
    }();
    if (!fn) return cudaErrorNotSupported;
    const cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows}, strides[1] = {(cuuint64_t)stride * 2};
    const cuuint32_t box[2] = {64, (cuuint32_t)box_rows}, estr[2] = {1, 1};
    return fn(out, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void *>(p), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
              CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS
               ? cudaSuccess
               : cudaErrorInvalidValue;
}

template <int V>
cudaError_t run(const MlaPrefillArgs &a, const DevInfo &d, cudaStream_t st) {
    CUtensorMap q, kv, kr, vm;
    if (cudaError_t e = matrix_map(a.q, (long long)a.H * (a.nope + a.rope), a.Tq, a.q_stride, kRows, &q)) return e;
    kv = kr = vm = q;                         // no keys: never read
    if (a.Tk > 0) {
        if (cudaError_t e = matrix_map(a.kv, (long long)a.H * (a.nope + V), a.Tk, a.kv_stride, kRows, &kv)) return e;
        if (cudaError_t e = matrix_map(a.kv, (long long)a.H * (a.nope + V), a.Tk, a.kv_stride, kRows / 2, &vm)) return e;
        if (cudaError_t e = matrix_map(a.k_rope, a.rope, a.Tk, a.kr_stride, kRows, &kr)) return e;
    }
    const int nb = a.nope / 64 + 1;
    // at most; every unit that is not empty has a row of its own
    const long long units = std::min((long long)a.Tq, (long long)(a.Tq + 2 * kRows - 1) / (2 * kRows) + a.n_seq - 1) * a.H;
    auto bytes = [](int nb) { return (size_t)(4 * nb - 1) * kBlk + 3 * (V / 64) * (kBlk / 2) + 1024; };
    const size_t smem = bytes(nb);
    auto kern = mla_prefill_kernel<V>;
    static std::atomic<uint64_t> done{0};
    if (cudaError_t e = allow_smem(kern, bytes(3), d.device, done)) return e;   // nope = 128

    return launch_pdl(kern, dim3((unsigned)units), dim3(384), smem, st, q, kv, kr, vm, a, d.wait_ns);
}

size_t round256(size_t n) { return (n + 255) / 256 * 256; }

}  // namespace

size_t mla_prefill_scratch(const MlaPrefillArgs &a) {
    if (!a.in_f32) return 0;
    return round256((size_t)a.Tq * a.H * (a.nope + a.rope) * 2) + round256((size_t)a.Tk * a.H * (a.nope + a.v) * 2) +
           round256((size_t)a.Tk * a.rope * 2);
}

cudaError_t launch_mla_prefill(const MlaPrefillArgs &a0, const DevInfo &d, cudaStream_t st, int *n_launch) {
    MlaPrefillArgs a = a0;
    *n_launch = 1;
    if (a.in_f32) {
        const int cols[3] = {a.H * (a.nope + a.rope), a.H * (a.nope + a.v), a.rope};
        const long long rows[3] = {a.Tq, a.Tk, a.Tk}, strides[3] = {a.q_stride, a.kv_stride, a.kr_stride};
        const void *src[3] = {a.q, a.kv, a.k_rope};
        __nv_bfloat16 *dst[3];
        char *at = (char *)d.scratch;
        for (int i = 0; i < 3; i++) {
            dst[i] = (__nv_bfloat16 *)at;
            at += round256((size_t)rows[i] * cols[i] * 2);
            const long long want = (rows[i] * (cols[i] / 8) + 255) / 256;
            if (want == 0) continue;
            if (cudaError_t e = launch_pdl(mla_round_kernel, dim3((unsigned)(want < 32LL * d.n_sm ? want : 32LL * d.n_sm)), dim3(256), 0, st,
                                           (const float *)src[i], strides[i], rows[i], cols[i], dst[i]))
                return e;
            ++*n_launch;
        }
        a.q = dst[0];
        a.kv = dst[1];
        a.k_rope = dst[2];
        a.q_stride = cols[0];
        a.kv_stride = cols[1];
        a.kr_stride = cols[2];
    }
    return a.v == 64 ? run<64>(a, d, st) : run<128>(a, d, st);
}

}  // namespace coli

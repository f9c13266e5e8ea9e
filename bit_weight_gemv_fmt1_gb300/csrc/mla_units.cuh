// mla_units.cuh -- the units of work of the expanded attention (mla_prefill.cu) and the search for one by its number.
#pragma once

#include "mla.cuh"

namespace coli {

constexpr int kRows = 128;               // rows of a query or key tile

// One unit of work: a head's pair of query tiles.
struct Unit {
    int head, q0, nq, nk, qrow, krow;    // first query of the pair in its sequence, the sequence's sizes and first rows
    int nt[2], n;                        // key tiles that each query tile sees, the larger of them; n < 0: no more units
};

// Sequence b's offsets (all 0 where they are bad) and its number of pairs.
__device__ __forceinline__ int pairs_of(const MlaPrefillArgs &a, int b, bool report, int4 &c) {
    c = make_int4(0, 0, 0, 0);
    if (b >= a.n_seq) return 0;
    const int4 d = make_int4(a.cu_q[b], a.cu_q[b + 1], a.cu_k[b], a.cu_k[b + 1]);
    const bool good = d.x >= 0 && d.y >= d.x && d.y <= a.Tq && d.z >= 0 && d.w >= d.z && d.w <= a.Tk;
    if (report && !good) mla_bad_index(a.err);
    if (good) c = d;
    return (c.y - c.x + 2 * kRows - 1) / (2 * kRows);
}
// How many of a sequence's n pairs see v key tiles or more: the last pair sees all nk keys, each one before it 256
// fewer rows' worth.
__device__ __forceinline__ int pairs_with(int n, int4 c, int v) {
    if (v <= 0) return n;
    const int spare = c.w - c.z - ((v - 1) * kRows + 1);   // rows that may lie behind the pair's last
    if (spare < 0) return 0;
    const int need = max(1, (c.y - c.x - spare + 2 * kRows - 1) / (2 * kRows));
    return min(n, max(0, n - need + 1));
}
// Whole warp: the pairs of all sequences, and the most key tiles that one sees.
__device__ __forceinline__ int all_pairs(const MlaPrefillArgs &a, int lane, bool report, int &most) {
    int total = 0;
    most = 0;
    for (int b = lane; b < a.n_seq; b += 32) {
        int4 c;
        total += pairs_of(a, b, report, c);
        most = max(most, (c.w - c.z + kRows - 1) / kRows);
    }
    most = __reduce_max_sync(0xffffffffu, most);
    return __reduce_add_sync(0xffffffffu, total);
}
// How far a CTA has come in the order of units: the pairs that see v tiles have the numbers below..upto - 1, and those
// of sequences before b0 end at run.  A CTA's units rise as a rule, so most of them are found from here in one look at 32
// sequences; nothing promises that they do, and a lower one is searched from the start (512 sequences of up to 200 rows x 16
// heads: 333 us, with a search from the start each time 853; 8192 x 32 heads, which needs none of it, 459 against 452, or 472
// with the count unrolled at five places: it is one loop for its size).
struct Place {
    int v, below, upto, b0, run, most;
};
// Before the first unit.
__device__ __forceinline__ Place no_place(int most) { return Place{most + 1, 0, 0, 0, 0, most}; }
// Whole warp: unit i, in the order of key tiles, most first, all heads of a pair together.
__device__ __forceinline__ Unit unit_of(const MlaPrefillArgs &a, int i, int pairs, Place &at, int lane) {
    Unit u;
    const int p = i / a.H;
    u.head = i - p * a.H;
    if (p < at.below) at = no_place(at.most);
    if (p < at.run) {
        at.b0 = 0;
        at.run = at.below;
    }
    if (p >= at.upto) {
        // count(lo) > p >= count(hi), the pairs that see so many tiles or more; first the next number of tiles, then halves
        int lo = 0, hi = at.v, above = pairs, below = at.upto, v = hi - 1;
        while (hi - lo > 1) {
            int t = 0;
#pragma unroll 2
            for (int b = lane; b < a.n_seq; b += 32) {
                int4 c;
                const int n = pairs_of(a, b, false, c);
                t += pairs_with(n, c, v);
            }
            t = __reduce_add_sync(0xffffffffu, t);
            if (t > p) {
                lo = v;
                above = t;
            } else {
                hi = v;
                below = t;
            }
            v = (lo + hi) / 2;
        }
        at.v = lo;
        at.below = below;
        at.upto = above;
        at.b0 = 0;
        at.run = below;
    }
    const int v = at.v;
    int run = at.run;
    u.q0 = u.nq = u.nk = u.qrow = u.krow = 0;
    for (int b0 = at.b0; b0 < a.n_seq; b0 += 32) {
        int4 c;
        const int n = pairs_of(a, b0 + lane, false, c);
        const int above = pairs_with(n, c, v + 1), here = pairs_with(n, c, v) - above;
        int incl = here;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int w = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += w;
        }
        const int before = run + incl - here;
        const uint32_t hit = __ballot_sync(0xffffffffu, before <= p && p < before + here);
        if (hit) {
            at.b0 = b0;
            at.run = run;
            const int src = __ffs(hit) - 1;
            u.q0 = __shfl_sync(0xffffffffu, (n - 1 - above - (p - before)) * 2 * kRows, src);
            u.qrow = __shfl_sync(0xffffffffu, c.x, src);
            u.nq = __shfl_sync(0xffffffffu, c.y, src) - u.qrow;
            u.krow = __shfl_sync(0xffffffffu, c.z, src);
            u.nk = __shfl_sync(0xffffffffu, c.w, src) - u.krow;
            break;
        }
        run += __shfl_sync(0xffffffffu, incl, 31);
    }
#pragma unroll
    for (int x = 0; x < 2; x++) {
        // the last live row's limit
        const int rows = min(kRows, u.nq - u.q0 - x * kRows);
        const int limit = rows > 0 ? u.q0 + x * kRows + rows + u.nk - u.nq : 0;
        u.nt[x] = limit > 0 ? (min(limit, u.nk) + kRows - 1) / kRows : 0;
    }
    u.n = max(u.nt[0], u.nt[1]);
    return u;
}

}  // namespace coli

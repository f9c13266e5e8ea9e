// mla_attend.cuh -- what the two kernels of the absorbed attention share: how
// the work is cut, the walk over a CTA's tiles, token slots and query rows.
#pragma once

#include "mla.cuh"
#include "tcgen05.cuh"

namespace coli {

constexpr int kTile = 128;               // tokens per tile
constexpr int kSoft = 256;               // softmax threads
constexpr int kStraddle = 3;              // tiles that a piece's second sequence costs
constexpr float kNone = -3e38f;          // reference of a column that has none yet

struct AttendPlan {
    int cols;              // query rows (columns) of a CTA
    int n_rows;            // query rows of a sequence: n_q * H
    int nrb;               // blocks of `cols` rows
    int n_groups, n_slots; // pieces of the line of tiles; CTAs of a group
    float *part;           // [n_groups * nrb * 2][cols][L] partial O, then [..][cols][2] m, l
    float *part_ml;
    int2 *pieces;          // [n_seq] first group and number of groups of each sequence
    int pbox;              // tokens per copy box
    long long wait_ns;     // bound of the waits (deadline_after)
};

// The piece of a CTA's group: tiles [u0, u1), beginning in sequence b0 with p0 tiles before it.
struct Piece {
    int u0, u1, b0, p0;
};

__device__ __forceinline__ int seq_len(const MlaAttendArgs &a, int b) {
    const int n = a.lens[b];
    return n < 0 || n > a.pages_stride * a.c.page ? 0 : n;
}
__device__ __forceinline__ int tiles_of(int len) { return len > 0 ? (len + kTile - 1) / kTile : 1; }

// The tiles of a CTA's piece, for each of its row blocks, in order.
struct Walk {
    const MlaAttendArgs &a;
    const AttendPlan &g;
    const Piece s;
    int rb, u, b, p, T, len;
    __device__ Walk(const MlaAttendArgs &a_, const AttendPlan &g_, const Piece &s_, int slot) : a(a_), g(g_), s(s_), rb(slot) { start(); }
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
    __device__ int rest() const { return min(s.u1, p + T) - u; }               // tiles left of this part
    __device__ void skip(int n) { u += n; }                                    // within this part
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

__device__ __forceinline__ void store_out(const MlaAttendArgs &a, long long e, float v) {
    if (a.out_bf16) reinterpret_cast<__nv_bfloat16 *>(a.out)[e] = __float2bfloat16_rn(v);
    else reinterpret_cast<float *>(a.out)[e] = v;
}

__device__ __forceinline__ bool finite_bits(uint32_t v) { return (v & 0x7F800000u) != 0x7F800000u; }

// Address of unit u (8 elements) of query row `row`: latent units first, then rope ones.
template <bool QB>
__device__ __forceinline__ const uint4 *query_unit(const MlaAttendArgs &a, long long row, int u) {
    const int nu = a.c.L / 8;
    const long long e = u < nu ? row * a.c.L + 8 * u : row * a.c.R + 8 * (u - nu);
    return reinterpret_cast<const uint4 *>(reinterpret_cast<const uint8_t *>(u < nu ? a.q_latent : a.q_rope) + e * (QB ? 2 : 4));
}

// Warp 0: this group's piece of the line of all sequences' tiles, and (block 0) the table of the sequences' groups.
// Where that leaves no piece more than kStraddle tiles longer than an even cut, each sequence gets one group and its
// share of the others, so that no piece straddles two sequences; otherwise the line is cut evenly.  A second start and
// end cost a CTA about as much as kStraddle tiles (4 x 9000 tokens, 16 heads x 3 queries, bf16: 31.5 us cut evenly, 28.4
// by sequences; 24 sequences of 3000 to 12000 tokens on 38 groups: 180 us by sequences, 98 cut evenly).
__device__ __forceinline__ void find_piece(const MlaAttendArgs &a, const AttendPlan &g, int group, int lane, Piece &out) {
    auto tiles = [&](int b, bool check) {
        if (b >= a.n_seq) return 0;
        const int n = a.lens[b];
        const bool good = n >= 0 && n <= a.pages_stride * a.c.page;
        if (check && !good) mla_bad_index(a.err);
        return tiles_of(good ? n : 0);
    };
    auto scan = [&](int v) {              // inclusive prefix sum over the warp
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int w = __shfl_up_sync(0xffffffffu, v, o);
            if (lane >= o) v += w;
        }
        return v;
    };
    const int mine = tiles(lane, true);   // the first 32 sequences' lengths are read once
    int total = mine;
    for (int b = lane + 32; b < a.n_seq; b += 32) total += tiles(b, true);
    total = __reduce_add_sync(0xffffffffu, total);
    const int chunk = (total + g.n_groups - 1) / g.n_groups, spare = g.n_groups - a.n_seq;
    auto groups_of = [&](int T) { return min(T, 1 + (int)((long long)spare * T / total)); };
    bool shares = spare >= 0;
    if (shares) {
        int longest = 0;
        for (int b = lane; b < a.n_seq; b += 32) {
            const int T = b < 32 ? mine : tiles(b, false), n = groups_of(T);
            longest = max(longest, (T + n - 1) / n);
        }
        shares = __reduce_max_sync(0xffffffffu, longest) <= chunk + kStraddle;
    }
    int u0 = shares ? 0 : min(total, group * chunk), u1 = shares ? 0 : min(total, u0 + chunk);
    if (lane == 0) {
        out.u0 = u0;
        out.u1 = u1;
    }
    __syncwarp();
    int run_t = 0, run_g = 0;
    for (int b0 = 0; b0 < a.n_seq; b0 += 32) {
        const int b = b0 + lane, T = b0 ? tiles(b, false) : mine;
        const int n = shares && b < a.n_seq ? groups_of(T) : 0;
        const int incl_t = scan(T), incl_g = shares ? scan(n) : 0;
        const int p = run_t + incl_t - T, g0 = shares ? run_g + incl_g - n : p / chunk;
        if (b < a.n_seq) {
            if (shares ? g0 <= group && group < g0 + n : p <= u0 && u0 < p + T) {
                out.b0 = b;
                out.p0 = p;
                if (shares) {
                    const int k = group - g0;
                    out.u0 = p + (int)((long long)T * k / n);
                    out.u1 = p + (int)((long long)T * (k + 1) / n);
                }
            }
            if (g.pieces && blockIdx.x == 0) g.pieces[b] = make_int2(g0, shares ? n : (p + T - 1) / chunk - g0 + 1);
        }
        run_t += __shfl_sync(0xffffffffu, incl_t, 31);
        run_g += __shfl_sync(0xffffffffu, incl_g, 31);
    }
}

// Reduces each of a thread's NC columns over the warp's lanes by halving: 31 exchanges for 32 columns instead of 160.
// Lane i returns column i / (32 / NC).
template <int NC, class Op>
__device__ __forceinline__ float reduce_columns(float (&v)[NC], int lane, Op op) {
    int o = 16;
#pragma unroll
    for (int w = NC / 2; w >= 1; w /= 2, o /= 2) {
        const bool up = lane & o;
#pragma unroll
        for (int i = 0; i < w; i++) {
            const float keep = up ? v[i + w] : v[i], send = up ? v[i] : v[i + w];
            v[i] = op(keep, __shfl_xor_sync(0xffffffffu, send, o));
        }
    }
    for (; o >= 1; o /= 2) v[0] = op(v[0], __shfl_xor_sync(0xffffffffu, v[0], o));
    return v[0];
}

// A copy warp's lanes: the slot of this lane's box of pbox tokens in the current
// tile, looked up two tiles ahead, whose rows are then asked into L2 (each of the
// group's CTAs asks for a share).  A tile's buffers come free only about 1000
// cycles before they are needed again, less than HBM's latency under load.
struct BoxAhead {
    Walk w;                // two tiles ahead of the current one
    int lane, nbox, pbox, share;
    bool fetch;
    int slot[3];
    struct Asked {
        int id, off;
        bool live;
    };
    __device__ BoxAhead(const MlaAttendArgs &a, const AttendPlan &g, const Piece &s, int slot_, int lane_, bool fetch_)
        : w(a, g, s, slot_), lane(lane_), nbox(kTile / g.pbox), pbox(g.pbox), share(slot_), fetch(fetch_) {
        // one round trip for the first three tiles' page ids
        const Asked a0 = ask(), a1 = ask(), a2 = ask();
        slot[0] = answer(a0);
        slot[1] = answer(a1);
        slot[2] = answer(a2);
    }
    __device__ Asked ask() {
        Asked q{-1, 0, false};
        if (!w.valid()) return q;
        const int t = w.tile() * kTile + lane * pbox;
        if (lane < nbox && t < w.len) {
            const int pi = t / w.a.c.page;
            q.off = t - pi * w.a.c.page;
            q.id = w.a.pages[(long long)w.b * w.a.pages_stride + pi];
            q.live = true;
        }
        w.next();
        return q;
    }
    __device__ int answer(const Asked &q) {
        if (!q.live) return -1;
        if (q.id < 0 || q.id >= w.a.c.n_pages) {
            mla_bad_index(w.a.err);
            return -1;
        }
        const int sl = q.id * w.a.c.page + q.off;
        if (fetch) {
            // this CTA's share of the box's rows
            const int per = (pbox + w.g.n_slots - 1) / w.g.n_slots, r0 = min(pbox, share * per), r1 = min(pbox, r0 + per);
            if (r1 > r0) bulk_prefetch(mla_row(w.a.c, sl + r0), (r1 - r0) * w.a.c.row_bytes);
        }
        return sl;
    }
    __device__ void next() {
        slot[0] = slot[1];
        slot[1] = slot[2];
        slot[2] = answer(ask());
    }
};

// The E4M3 kernel (mla_attend_e4m3.cu).
cudaError_t launch_mla_attend_e4m3(const MlaAttendArgs &a, const AttendPlan &g, int device, cudaStream_t st);
// Tensor map of the cache's rows: boxes of `inner` elements x `pbox` rows, with that swizzle.
cudaError_t mla_row_map(const MlaCache &c, int inner, int pbox, CUtensorMapSwizzle swizzle, CUtensorMap *out);

}  // namespace coli

// gqa_evict.cu -- which cached tokens stay by their accumulated attention weight,
// and their way to the sequence's new pages.
//
// Selection, one CTA per sequence and head: the weights become integers of the
// same order (a NaN last), up to three passes of a radix selection (12, 10 and 10 bits,
// counts in shared memory; none after one whose last bin stays whole) give the smallest one that stays and how many equal to it
// do; one more pass writes the tokens that stay in their order.  The move is a
// kernel of its own, so that few sequences use every SM.
//
// 12 sequences up to 16000 to 4001 tokens, 8 heads: selection 18 us (96 CTAs: barriers and latency of a few passes over 16 keys a
// thread), move 22 us: of a scattered row's 64 + 64 bytes of codes, 16 of scales and 4 of weight each piece costs DRAM an access of its
// own, 97 MB for 58 MB.  One sequence of 4096 to 1024: 12 us on the device with the read back (13 with always three passes).
#include <algorithm>

#include "gqa.cuh"

namespace coli {

namespace {

constexpr int kSelect = 1024, kBins = 4096, kRoom = 48000;   // kRoom keys of 4 bytes in shared memory

// Integers ordered as the weights; +0 and -0 alike, every NaN the largest.
__device__ __forceinline__ uint32_t ordered(float w) {
    if (w != w) return 0xFFFFFFFFu;
    const uint32_t b = __float_as_uint(w + 0.f);
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}

// A sequence's length; 0 (and a record) where it is out of range.
__device__ __forceinline__ int length_of(const GqaEvictArgs &a, int b, bool report) {
    const int n = a.lens[b];
    if (n >= 0 && n <= a.longest) return n;
    if (report) mla_bad_index(a.err);
    return 0;
}

// Inclusive sums over the CTA's threads of x and y; x_all and y_all get the totals.
__device__ __forceinline__ void scan(int &x, int &y, int &x_all, int &y_all, int2 *sums) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(0xffffffffu, x, o), v = __shfl_up_sync(0xffffffffu, y, o);
        if (lane >= o) x += u, y += v;
    }
    if (lane == 31) sums[warp] = make_int2(x, y);
    __syncthreads();
    int2 s = sums[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(0xffffffffu, s.x, o), v = __shfl_up_sync(0xffffffffu, s.y, o);
        if (lane >= o) s.x += u, s.y += v;
    }
    x_all = __shfl_sync(0xffffffffu, s.x, 31);
    y_all = __shfl_sync(0xffffffffu, s.y, 31);
    const int u = __shfl_sync(0xffffffffu, s.x, max(warp - 1, 0)), v = __shfl_sync(0xffffffffu, s.y, max(warp - 1, 0));
    if (warp) x += u, y += v;
    __syncthreads();                                     // sums is free again
}

__global__ void __launch_bounds__(kSelect) gqa_select_kernel(const GqaEvictArgs a, int room) {
    extern __shared__ __align__(16) uint32_t keys[];     // the first `room` candidates'; more are read again each time
    __shared__ __align__(16) int count[kBins];
    __shared__ int2 sums[kSelect / 32];
    __shared__ int s_bin, s_left, s_in;
    const int b = blockIdx.x / a.c.n_kv, h = blockIdx.x - b * a.c.n_kv, tid = threadIdx.x;
    pdl_wait();
    const int n = length_of(a, b, tid == 0 && h == 0);
    const int stay = min(n, a.keep);
    int32_t *kept = a.kept + (long long)blockIdx.x * a.keep;
    if (tid == 0 && h == 0) a.new_lens[b] = stay;
    for (int i = stay + tid; i < a.keep; i += kSelect) kept[i] = -1;
    if (n <= a.keep) {
        for (int i = tid; i < n; i += kSelect) kept[i] = i;
        return;
    }
    const int old = n - a.recent, want = a.keep - a.recent;   // the candidates, and how many of them stay
    for (int i = tid; i < a.recent; i += kSelect) kept[want + i] = old + i;
    if (want == 0) return;
    const int32_t *pages = a.pages + b * a.pages_stride;
    auto read_key = [&](int t) {
        const int p = t / a.c.page, id = pages[p];
        if (id < 0 || id >= a.c.n_pages) {
            mla_bad_index(a.err);
            return ordered(0.f);
        }
        return ordered(a.c.w[gqa_row(a.c, id, h) + t - p * a.c.page]);
    };
    auto key = [&](int t) { return t < room ? keys[t] : read_key(t); };
    for (int i = tid; i < kBins; i += kSelect) count[i] = 0;
    __syncthreads();
    // 4 tokens at a time, which share a page and 16 bytes of weights
#pragma unroll 4
    for (int t = 4 * tid; t < old; t += 4 * kSelect) {
        const int p = t / a.c.page, id = pages[p];
        float4 w = make_float4(0.f, 0.f, 0.f, 0.f);
        if (id < 0 || id >= a.c.n_pages) mla_bad_index(a.err);
        else w = *reinterpret_cast<const float4 *>(a.c.w + gqa_row(a.c, id, h) + t - p * a.c.page);
        const uint32_t k[4] = {ordered(w.x), ordered(w.y), ordered(w.z), ordered(w.w)};
        if (t < room) *reinterpret_cast<uint4 *>(keys + t) = make_uint4(k[0], k[1], k[2], k[3]);
#pragma unroll
        for (int i = 0; i < 4; i++)
            if (t + i < old) atomicAdd(&count[k[i] >> 20], 1);
    }
    uint32_t prefix = 0;
    int left = want;                                     // of the keys that begin with the prefix, how many stay
    for (int pass = 0; pass < 3; pass++) {
        const int shift = pass == 0 ? 20 : pass == 1 ? 10 : 0, bits = pass == 0 ? 12 : 10;
        if (pass > 0) {
            const int known = shift + bits;
            for (int t = tid; t < old; t += kSelect) {
                const uint32_t k = key(t);
                if ((k >> known) == (prefix >> known)) atomicAdd(&count[(k >> shift) & ((1 << bits) - 1)], 1);
            }
        }
        __syncthreads();
        // counts from the top: thread i has the bins 4095 - 4i .. 4092 - 4i
        int4 *bins = reinterpret_cast<int4 *>(&count[kBins - 4 - 4 * tid]);
        const int4 c = *bins;
        *bins = make_int4(0, 0, 0, 0);                   // for the next pass
        int incl = c.x + c.y + c.z + c.w, none = 0, all, all2;
        scan(incl, none, all, all2, sums);
        int before = incl - c.x - c.y - c.z - c.w;
        const int each[4] = {c.w, c.z, c.y, c.x};
#pragma unroll
        for (int i = 0; i < 4; i++) {
            if (before < left && left <= before + each[i]) {
                s_bin = kBins - 1 - 4 * tid - i;
                s_left = left - before;
                s_in = each[i];
            }
            before += each[i];
        }
        __syncthreads();
        prefix |= (uint32_t)s_bin << shift;
        left = s_left;
        if (left == s_in) break;                         // all of the bin stay: those above the prefix and those equal to it
    }
    // In order: every key above the last one that stays, and the first `left` equal ones.  A thread has as many neighbours as the
    // next one, an odd number: its lane's words lie in banks of their own.
    const int each = ((old + kSelect - 1) / kSelect) | 1, t0 = min((long long)tid * each, (long long)old), t1 = min(t0 + each, old);
    int over = 0, same = 0, all, all2;
    for (int t = t0; t < t1; t++) {
        const uint32_t k = key(t);
        over += k > prefix;
        same += k == prefix;
    }
    const int over_here = over, same_here = same;
    scan(over, same, all, all2, sums);
    int equal = same - same_here, at = over - over_here + min(equal, left);
    for (int t = t0; t < t1; t++) {
        const uint32_t k = key(t);
        if (k > prefix || (k == prefix && equal++ < left)) kept[at++] = t;
    }
    pdl_trigger();
}

// A warp has 32 rows that stay: each lane finds one's old and new place and moves its scales and weight, then the lanes move all their
// codes, 16 bytes each, keys first.
template <int D>
__global__ void __launch_bounds__(256, 6) gqa_move_kernel(const GqaEvictArgs a) {
    constexpr int kHalf = D / 32;        // 16-byte pieces of a row's key, and of its value
    const int lane = threadIdx.x & 31, per = (a.keep + 31) / 32;
    const long long w = blockIdx.x * 8LL + (threadIdx.x >> 5);
    const int pair = (int)(w / per), i = (int)(w - (long long)pair * per) * 32 + lane;
    pdl_wait();
    if (pair >= a.n_seq * a.c.n_kv) return;
    const int b = pair / a.c.n_kv, h = pair - b * a.c.n_kv;
    const int t = i < a.keep ? a.kept[(long long)pair * a.keep + i] : -1;
    int s = -1, d = -1;
    if (t >= 0) {
        const int sp = t / a.c.page, dp = i / a.c.page;
        const int from = a.pages[b * a.pages_stride + sp], to = a.dst[b * a.dst_stride + dp];
        if (from < 0 || from >= a.c.n_pages || to < 0 || to >= a.c.n_pages) {
            mla_bad_index(a.err);
        } else {
            s = (int)gqa_row(a.c, from, h) + (t - sp * a.c.page);   // rows < 2^31, a row plus a token need not be
            d = (int)gqa_row(a.c, to, h) + (i - dp * a.c.page);
        }
    }
    // keys, then values: half the registers of both at once, and more warps
#pragma unroll 1
    for (int value = 0; value < 2; value++) {
        uint4 *codes = reinterpret_cast<uint4 *>(value ? a.c.v : a.c.k);
        uint4 x[kHalf];
#pragma unroll
        for (int k = 0; k < kHalf; k++) {
            const int piece = k * 32 + lane, row = __shfl_sync(0xffffffffu, s, piece / kHalf);
            if (row >= 0) x[k] = codes[(long long)row * kHalf + piece % kHalf];
        }
        if (s >= 0) {
            void *sc = value ? a.c.vs : a.c.ks;
            const int ng = D / a.c.gs;
            if (ng == 4) reinterpret_cast<uint2 *>(sc)[d] = reinterpret_cast<const uint2 *>(sc)[s];
            else if (ng == 2) reinterpret_cast<uint32_t *>(sc)[d] = reinterpret_cast<const uint32_t *>(sc)[s];
            else reinterpret_cast<uint16_t *>(sc)[d] = reinterpret_cast<const uint16_t *>(sc)[s];
            if (value) a.c.w[d] = a.c.w[s];
        }
#pragma unroll
        for (int k = 0; k < kHalf; k++) {
            const int piece = k * 32 + lane, row = __shfl_sync(0xffffffffu, d, piece / kHalf);
            if (row >= 0) codes[(long long)row * kHalf + piece % kHalf] = x[k];
        }
    }
    pdl_trigger();
}

}  // namespace

cudaError_t launch_gqa_evict(const GqaEvictArgs &a, const DevInfo &d, cudaStream_t st, int *n_launch) {
    const long long pairs = (long long)a.n_seq * a.c.n_kv;
    const int room = (int)std::min(a.pages_stride * a.c.page, (long long)kRoom);
    static std::atomic<uint64_t> done{0};
    if (cudaError_t e = allow_smem(gqa_select_kernel, kRoom * sizeof(uint32_t), d.device, done)) return e;
    *n_launch = 2;
    if (cudaError_t e = launch_pdl(gqa_select_kernel, dim3((unsigned)pairs), dim3(kSelect), room * sizeof(uint32_t), st, a, room)) return e;
    const dim3 grid((unsigned)((pairs * ((a.keep + 31) / 32) + 7) / 8));
    return a.c.dim == 64 ? launch_pdl(gqa_move_kernel<64>, grid, dim3(256), 0, st, a) : launch_pdl(gqa_move_kernel<128>, grid, dim3(256), 0, st, a);
}

}  // namespace coli

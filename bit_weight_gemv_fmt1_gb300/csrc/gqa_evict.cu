// gqa_evict.cu -- which cached tokens stay by their accumulated attention weight,
// and their way to the sequence's new pages.
//
// Selection, one CTA per sequence and head: the weights become integers of the
// same order (a NaN last), three passes of a radix selection (11, 11 and 10 bits,
// counts in shared memory) give the smallest one that stays and how many equal to it
// do; one more pass writes the tokens that stay in their order.  The move is a
// kernel of its own, so that few sequences use every SM.
#include "gqa.cuh"

namespace coli {

namespace {

constexpr int kSelect = 1024, kBins = 2048;

// Integers ordered as the weights; +0 and -0 alike, every NaN the largest.
__device__ __forceinline__ uint32_t ordered(float w) {
    if (w != w) return 0xFFFFFFFFu;
    const uint32_t b = __float_as_uint(w + 0.f);
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}

// A sequence's length; 0 (and a record) where it is out of range.
__device__ __forceinline__ int length_of(const GqaEvictArgs &a, int b, bool report) {
    const int n = a.lens[b];
    if (n >= 0 && n <= a.pages_stride * a.c.page) return n;
    if (report) mla_bad_index(a.err);
    return 0;
}

__global__ void __launch_bounds__(kSelect) gqa_select_kernel(const GqaEvictArgs a) {
    __shared__ int count[kBins];
    __shared__ int sums[kSelect / 32], above[kSelect / 32];
    __shared__ int s_bin, s_left;
    const int b = blockIdx.x / a.c.n_kv, h = blockIdx.x - b * a.c.n_kv, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    pdl_wait();
    pdl_trigger();
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
    auto key = [&](int t) {
        const int p = t / a.c.page, id = pages[p];
        if (id < 0 || id >= a.c.n_pages) {
            mla_bad_index(a.err);
            return ordered(0.f);
        }
        return ordered(a.c.w[gqa_row(a.c, id, h) + t - p * a.c.page]);
    };
    uint32_t prefix = 0;
    int left = want;                                     // of the keys that begin with the prefix, how many stay
    for (int pass = 0; pass < 3; pass++) {
        const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0, bits = pass == 2 ? 10 : 11, known = shift + bits;
        for (int i = tid; i < kBins; i += kSelect) count[i] = 0;
        __syncthreads();
        for (int t = tid; t < old; t += kSelect) {
            const uint32_t k = key(t);
            if (pass == 0 || (k >> known) == (prefix >> known)) atomicAdd(&count[(k >> shift) & ((1 << bits) - 1)], 1);
        }
        __syncthreads();
        // counts from the top: thread i has the bins 2047 - 2i and 2046 - 2i
        const int c0 = count[kBins - 1 - 2 * tid], c1 = count[kBins - 2 - 2 * tid];
        int incl = c0 + c1;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += v;
        }
        if (lane == 31) sums[warp] = incl;
        __syncthreads();
        if (warp == 0) {
            int v = sums[lane];
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int w = __shfl_up_sync(0xffffffffu, v, o);
                if (lane >= o) v += w;
            }
            sums[lane] = v;
        }
        __syncthreads();
        const int before = incl - c0 - c1 + (warp ? sums[warp - 1] : 0);
        if (before < left && left <= before + c0) {
            s_bin = kBins - 1 - 2 * tid;
            s_left = left - before;
        } else if (before + c0 < left && left <= before + c0 + c1) {
            s_bin = kBins - 2 - 2 * tid;
            s_left = left - before - c0;
        }
        __syncthreads();
        prefix |= (uint32_t)s_bin << shift;
        left = s_left;
    }
    // in order: every key above the last one that stays, and the first `left` equal ones
    int done = 0, equal = 0;                             // written so far, equal ones met so far
    for (int t0 = 0; t0 < old; t0 += kSelect) {
        const int t = t0 + tid;
        const uint32_t k = t < old ? key(t) : 0;
        const bool over = t < old && k > prefix, same = t < old && k == prefix;
        const uint32_t mo = __ballot_sync(0xffffffffu, over), ms = __ballot_sync(0xffffffffu, same);
        __syncthreads();
        if (lane == 0) {
            above[warp] = __popc(mo);
            sums[warp] = __popc(ms);
        }
        __syncthreads();
        int o0 = 0, e0 = 0, o_all = 0, e_all = 0;
        for (int w = 0; w < kSelect / 32; w++) {
            if (w == warp) o0 = o_all, e0 = e_all;
            o_all += above[w];
            e_all += sums[w];
        }
        const uint32_t lower = (1u << lane) - 1;
        const int my_over = o0 + __popc(mo & lower), my_equal = e0 + __popc(ms & lower);
        const int room = max(0, left - equal);           // equal ones that still stay
        if (over || (same && my_equal < room)) kept[done + my_over + min(my_equal, room)] = t;
        done += o_all + min(e_all, room);
        equal += e_all;
    }
}

// dim / 16 neighbouring threads per row that stays: 16 bytes of the key's codes or of the value's each, the first of either half the
// scales too, the second one the weight.
__global__ void __launch_bounds__(256) gqa_move_kernel(const GqaEvictArgs a) {
    const int half = a.c.dim / 32, tpr = 2 * half, rows = 256 / tpr;
    const int blocks = (a.keep + rows - 1) / rows, pair = blockIdx.x / blocks;
    const int i = (blockIdx.x - pair * blocks) * rows + threadIdx.x / tpr, c = threadIdx.x & (tpr - 1);
    const int b = pair / a.c.n_kv, h = pair - b * a.c.n_kv;
    pdl_wait();
    pdl_trigger();
    if (i >= a.keep) return;
    const int t = a.kept[(long long)pair * a.keep + i];
    if (t < 0) return;
    const int sp = t / a.c.page, dp = i / a.c.page;
    const int from = a.pages[b * a.pages_stride + sp], to = a.dst[b * a.dst_stride + dp];
    if (from < 0 || from >= a.c.n_pages || to < 0 || to >= a.c.n_pages) {
        mla_bad_index(a.err);
        return;
    }
    const long long s = gqa_row(a.c, from, h) + t - sp * a.c.page, d = gqa_row(a.c, to, h) + i - dp * a.c.page;
    const bool value = c >= half;
    uint8_t *codes = value ? a.c.v : a.c.k;
    const int u = value ? c - half : c, ng = a.c.dim / a.c.gs;
    const uint4 x = reinterpret_cast<const uint4 *>(codes)[s * half + u];
    if (u == 0) {
        __nv_bfloat16 *sc = value ? a.c.vs : a.c.ks;
        if (ng == 4) reinterpret_cast<uint2 *>(sc)[d] = reinterpret_cast<const uint2 *>(sc)[s];
        else if (ng == 2) reinterpret_cast<uint32_t *>(sc)[d] = reinterpret_cast<const uint32_t *>(sc)[s];
        else sc[d] = sc[s];
    }
    if (c == 1) a.c.w[d] = a.c.w[s];
    reinterpret_cast<uint4 *>(codes)[d * half + u] = x;
}

}  // namespace

cudaError_t launch_gqa_evict(const GqaEvictArgs &a, cudaStream_t st, int *n_launch) {
    const unsigned pairs = (unsigned)a.n_seq * a.c.n_kv;
    *n_launch = 2;
    if (cudaError_t e = launch_pdl(gqa_select_kernel, dim3(pairs), dim3(kSelect), 0, st, a)) return e;
    const int rows = 256 / (a.c.dim / 16);
    return launch_pdl(gqa_move_kernel, dim3((a.keep + rows - 1) / rows * pairs), dim3(256), 0, st, a);
}

}  // namespace coli

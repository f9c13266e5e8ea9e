// gqa_api.cu -- the grouped-head attention entry points of include/coli.h:
// argument checks and launches.  Nothing is launched unless every check passed.
#include <algorithm>

#include "api_checks.cuh"
#include "gqa.cuh"

using namespace coli;

namespace {

constexpr long long kIntMax = (1LL << 31) - 1;
constexpr long long kLongest = 1LL << 30;    // tokens of a sequence: the kernels' places, some tiles past its end too, fit an int

int longest(int64_t pages_stride, const GqaCache &c) { return (int)std::min((long long)pages_stride * c.page, kLongest); }

int check_cache(const coli_gqa_cache *c, GqaCache *out) {
    if (!c) return bad(COLI_EINVAL, "cache is NULL");
    if (c->n_kv < 1 || c->n_kv > 1024) return bad(COLI_EINVAL, "n_kv must be in 1..1024 (got %d)", c->n_kv);
    if (c->dim != 64 && c->dim != 128) return bad(COLI_EINVAL, "dim must be 64 or 128 (got %d)", c->dim);
    if ((c->gs != 32 && c->gs != 64 && c->gs != 128) || c->gs > c->dim)
        return bad(COLI_EINVAL, "gs must be 32, 64 or 128, at most dim (got %d)", c->gs);
    if (c->page_size < 16 || c->page_size > 65536 || c->page_size % 16)
        return bad(COLI_EINVAL, "page_size must be a multiple of 16 in 16..65536 (got %d)", c->page_size);
    if (c->n_pages < 1 || c->n_pages > kIntMax / c->page_size / c->n_kv)
        return bad(COLI_EINVAL, "n_pages must be >= 1 and n_pages * n_kv * page_size <= 2^31 - 1 (got %lld)", (long long)c->n_pages);
    if (int rc = need(c->k, 16, "cache k")) return rc;
    if (int rc = need(c->v, 16, "cache v")) return rc;
    if (int rc = need(c->k_scales, 16, "cache k_scales")) return rc;
    if (int rc = need(c->v_scales, 16, "cache v_scales")) return rc;
    if (c->weights)
        if (int rc = need(c->weights, 16, "cache weights")) return rc;
    *out = GqaCache{c->k, c->v, (__nv_bfloat16 *)c->k_scales, (__nv_bfloat16 *)c->v_scales, c->weights, c->n_kv, c->dim, c->gs,
                    c->page_size, (int)c->n_pages};
    return COLI_OK;
}

int check_stride(long long stride, int T, int heads, int dim, const char *name) {
    if (T > 1 && (stride < (long long)heads * dim || stride % 8))
        return bad(COLI_EINVAL, "%s must be a multiple of 8 that holds a token's heads (got %lld)", name, stride);
    return COLI_OK;
}

bool overlap(const void *a, int64_t bytes_a, const void *b, int64_t bytes_b) {
    const char *x = (const char *)a, *y = (const char *)b;
    return x < y + bytes_b && y < x + bytes_a;
}

int append(const coli_gqa_cache *cache, int dtype, const void *k, int64_t k_stride, const void *v, int64_t v_stride, int T,
           const int64_t *slots, void *stream) {
    clear_last_error();
    GqaAppendArgs a{};
    if (int rc = check_cache(cache, &a.c)) return rc;
    if (int rc = float_type(dtype, "dtype")) return rc;
    if (T < 0) return bad(COLI_EINVAL, "T must be >= 0 (got %d)", T);
    if ((int64_t)T * a.c.n_kv > kIntMax / 2) return bad(COLI_EINVAL, "T * n_kv is too large (got %d, %d)", T, a.c.n_kv);
    if (int rc = check_stride(k_stride, T, a.c.n_kv, a.c.dim, "k_stride")) return rc;
    if (int rc = check_stride(v_stride, T, a.c.n_kv, a.c.dim, "v_stride")) return rc;
    if (T) {
        if (int rc = need(k, 16, "k")) return rc;
        if (int rc = need(v, 16, "v")) return rc;
        if (int rc = need(slots, 8, "slots")) return rc;
    }
    if (int rc = injected_gate()) return rc;
    if (!T) return COLI_OK;
    DevInfo d;
    if (int rc = device_info(&d)) return rc;
    a.k = k;
    a.v = v;
    a.k_stride = k_stride;
    a.v_stride = v_stride;
    a.T = T;
    a.slots = slots;
    a.err = d.err;
    return launched(launch_gqa_append(a, dtype == COLI_BF16, d.n_sm, (cudaStream_t)stream), "coli_gqa_append", 1);
}

int read(const coli_gqa_cache *cache, const int32_t *pages, int64_t pages_stride, int n_seq, const int32_t *cu, int T, int dtype,
         void *k, int64_t k_stride, void *v, int64_t v_stride, void *stream) {
    clear_last_error();
    GqaReadArgs a{};
    if (int rc = check_cache(cache, &a.c)) return rc;
    if (int rc = float_type(dtype, "dtype")) return rc;
    if (T < 0 || n_seq < 0) return bad(COLI_EINVAL, "T and n_seq must be >= 0 (got %d, %d)", T, n_seq);
    if ((int64_t)T * a.c.n_kv > kIntMax / 2) return bad(COLI_EINVAL, "T * n_kv is too large (got %d, %d)", T, a.c.n_kv);
    if (pages_stride < 1 || pages_stride > kIntMax)
        return bad(COLI_EINVAL, "pages_stride must be in 1..2^31-1 (got %lld)", (long long)pages_stride);
    if (int rc = check_stride(k_stride, T, a.c.n_kv, a.c.dim, "k_stride")) return rc;
    if (int rc = check_stride(v_stride, T, a.c.n_kv, a.c.dim, "v_stride")) return rc;
    if (T && n_seq) {
        if (int rc = need(pages, 4, "pages")) return rc;
        if (int rc = need(cu, 4, "cu")) return rc;
        if (int rc = need(k, 16, "k")) return rc;
        if (int rc = need(v, 16, "v")) return rc;
    }
    if (int rc = injected_gate()) return rc;
    if (!T || !n_seq) return COLI_OK;
    DevInfo d;
    if (int rc = device_info(&d)) return rc;
    a.pages = pages;
    a.pages_stride = pages_stride;
    a.n_seq = n_seq;
    a.cu = cu;
    a.T = T;
    a.k = k;
    a.v = v;
    a.k_stride = k_stride;
    a.v_stride = v_stride;
    a.err = d.err;
    return launched(launch_gqa_read(a, dtype == COLI_BF16, (cudaStream_t)stream), "coli_gqa_read", 1);
}

int attend(const coli_gqa_cache *cache, int dtype_q, const void *q, int n_seq, int n_q, int H, const int32_t *pages,
           int64_t pages_stride, const int32_t *lens, float scale, int weigh, int dtype_out, void *out, float *lse, void *stream) {
    clear_last_error();
    GqaAttendArgs a{};
    if (int rc = check_cache(cache, &a.c)) return rc;
    if (int rc = float_type(dtype_q, "dtype_q")) return rc;
    if (int rc = float_type(dtype_out, "dtype_out")) return rc;
    if (n_seq < 0 || n_q < 1 || H < 1 || H > 1024 || (int64_t)n_q * H > 65536)
        return bad(COLI_EINVAL, "need n_seq >= 0, n_q >= 1, 1 <= n_heads <= 1024, n_q * n_heads <= 65536 (got %d, %d, %d)", n_seq, n_q, H);
    if (H % a.c.n_kv) return bad(COLI_EINVAL, "n_heads must be a multiple of n_kv (got %d, %d)", H, a.c.n_kv);
    if ((int64_t)n_seq * n_q * H > kIntMax) return bad(COLI_EINVAL, "n_seq * n_q * n_heads is too large");
    if (pages_stride < 1 || pages_stride > kIntMax)
        return bad(COLI_EINVAL, "pages_stride must be in 1..2^31-1 (got %lld)", (long long)pages_stride);
    if (n_seq && pages_stride * a.c.page / 32 + 1 > kIntMax / n_seq)   // tiles of 32 tokens; a product would pass 2^63
        return bad(COLI_EINVAL, "n_seq * pages_stride * page_size is too large");
    if (!(scale == scale)) return bad(COLI_EINVAL, "scale must not be NaN");
    if (weigh && !a.c.w) return bad(COLI_EINVAL, "weigh needs a cache with weights");
    if (n_seq) {
        if (int rc = need(q, 16, "q")) return rc;
        if (int rc = need(pages, 4, "pages")) return rc;
        if (int rc = need(lens, 4, "lens")) return rc;
        if (int rc = need(out, 16, "out")) return rc;
        if (lse)
            if (int rc = need(lse, 4, "lse")) return rc;
        // A segment's queries are read before its outputs are written, but not before other segments', and again for the weights.
        const int64_t rows = (int64_t)n_seq * n_q * H, bytes_q = rows * a.c.dim * (dtype_q == COLI_BF16 ? 2 : 4);
        if (overlap(out, rows * a.c.dim * (dtype_out == COLI_BF16 ? 2 : 4), q, bytes_q) && (weigh || out != q || dtype_out != dtype_q))
            return bad(COLI_EINVAL, "out may be q itself, of its type and without weigh, and must not overlap it otherwise");
        if (lse && overlap(lse, rows * 4, q, bytes_q)) return bad(COLI_EINVAL, "lse must not overlap q");
    }
    if (int rc = injected_gate()) return rc;
    if (!n_seq) return COLI_OK;
    a.q = q;
    a.q_bf16 = dtype_q == COLI_BF16;
    a.out_bf16 = dtype_out == COLI_BF16;
    a.weigh = weigh != 0;
    a.n_seq = n_seq;
    a.n_q = n_q;
    a.H = H;
    a.pages = pages;
    a.pages_stride = pages_stride;
    a.lens = lens;
    a.longest = longest(pages_stride, a.c);
    a.scale = scale;
    a.out = out;
    a.lse = lse;
    DevInfo d;
    if (int rc = device_info(&d)) return rc;
    if (const size_t bytes = gqa_attend_scratch(a, d.n_sm))
        if (int rc = device_scratch(&d, (cudaStream_t)stream, bytes)) return rc;
    a.err = d.err;
    int n = 0;
    const cudaError_t e = launch_gqa_attend(a, d, (cudaStream_t)stream, &n);
    return launched(e, "coli_gqa_attend", n);
}

int evict(const coli_gqa_cache *cache, const int32_t *pages, int64_t pages_stride, int n_seq, const int32_t *lens, int keep, int recent,
          const int32_t *dst, int64_t dst_stride, int32_t *kept, int32_t *new_lens, void *stream) {
    clear_last_error();
    GqaEvictArgs a{};
    if (int rc = check_cache(cache, &a.c)) return rc;
    if (!a.c.w) return bad(COLI_EINVAL, "an eviction needs a cache with weights");
    if (n_seq < 0) return bad(COLI_EINVAL, "n_seq must be >= 0 (got %d)", n_seq);
    if (keep < 1 || keep > kLongest || recent < 0 || recent > keep)
        return bad(COLI_EINVAL, "need 1 <= keep <= 2^30 and 0 <= recent <= keep (got %d, %d)", keep, recent);
    if (pages_stride < 1 || pages_stride > kIntMax || dst_stride < 1 || dst_stride > kIntMax)
        return bad(COLI_EINVAL, "pages_stride and dst_stride must be in 1..2^31-1 (got %lld, %lld)", (long long)pages_stride, (long long)dst_stride);
    if (dst_stride * a.c.page < keep) return bad(COLI_EINVAL, "dst_stride pages must hold keep tokens (got %lld, %d)", (long long)dst_stride, keep);
    if ((int64_t)n_seq * a.c.n_kv > kIntMax || ((int64_t)keep + 31) / 32 > kIntMax / ((int64_t)n_seq * a.c.n_kv + 1))
        return bad(COLI_EINVAL, "n_seq * n_kv * keep is too large");
    if (n_seq) {
        if (int rc = need(pages, 4, "pages")) return rc;
        if (int rc = need(lens, 4, "lens")) return rc;
        if (int rc = need(dst, 4, "dst")) return rc;
        if (int rc = need(kept, 4, "kept")) return rc;
        if (int rc = need(new_lens, 4, "new_lens")) return rc;
        if (new_lens == lens) return bad(COLI_EINVAL, "new_lens must not be lens");
    }
    if (int rc = injected_gate()) return rc;
    if (!n_seq) return COLI_OK;
    DevInfo d;
    if (int rc = device_info(&d)) return rc;
    a.pages = pages;
    a.pages_stride = pages_stride;
    a.n_seq = n_seq;
    a.lens = lens;
    a.longest = longest(pages_stride, a.c);
    a.keep = keep;
    a.recent = recent;
    a.dst = dst;
    a.dst_stride = dst_stride;
    a.kept = kept;
    a.new_lens = new_lens;
    a.err = d.err;
    int n = 0;
    const cudaError_t e = launch_gqa_evict(a, d, (cudaStream_t)stream, &n);
    return launched(e, "coli_gqa_evict", n);
}

int prefill(int dtype, const void *q, int64_t q_stride, const void *k, int64_t k_stride, const void *v, int64_t v_stride, int Tq, int Tk,
            int n_seq, const int32_t *cu_q, const int32_t *cu_k, int heads, int n_kv, int dim, float scale, int dtype_out, void *out,
            float *lse, void *stream) {
    clear_last_error();
    if (int rc = float_type(dtype, "dtype")) return rc;
    if (int rc = float_type(dtype_out, "dtype_out")) return rc;
    if (dim != 64 && dim != 128) return bad(COLI_EINVAL, "dim must be 64 or 128 (got %d)", dim);
    if (heads < 1 || heads > 1024 || n_kv < 1 || heads % n_kv || heads / n_kv > 128)
        return bad(COLI_EINVAL, "need 1 <= n_heads <= 1024, a multiple of n_kv and at most 128 times it (got %d, %d)", heads, n_kv);
    if (Tq < 0 || Tk < 0 || n_seq < 0) return bad(COLI_EINVAL, "need Tq, Tk, n_seq >= 0 (got %d, %d, %d)", Tq, Tk, n_seq);
    const int group = heads / n_kv, tokens = 128 / group;
    if ((int64_t)Tq * heads > kIntMax || (int64_t)Tk * n_kv > kIntMax || ((int64_t)Tq / (2 * tokens) + 1 + n_seq) * n_kv > kIntMax)
        return bad(COLI_EINVAL, "Tq * n_heads, Tk * n_kv or n_seq * n_kv is too large");
    if (int rc = check_stride(q_stride, Tq, heads, dim, "q_stride")) return rc;
    if (int rc = check_stride(k_stride, Tk, n_kv, dim, "k_stride")) return rc;
    if (int rc = check_stride(v_stride, Tk, n_kv, dim, "v_stride")) return rc;
    if (!(scale == scale)) return bad(COLI_EINVAL, "scale must not be NaN");
    if (Tq && n_seq) {
        if (int rc = need(q, 16, "q")) return rc;
        if (Tk) {
            if (int rc = need(k, 16, "k")) return rc;
            if (int rc = need(v, 16, "v")) return rc;
        }
        if (int rc = need(cu_q, 4, "cu_q")) return rc;
        if (int rc = need(cu_k, 4, "cu_k")) return rc;
        if (int rc = need(out, 16, "out")) return rc;
        if (lse)
            if (int rc = need(lse, 4, "lse")) return rc;
    }
    if (int rc = injected_gate()) return rc;
    if (!Tq || !n_seq) return COLI_OK;
    GqaPrefillArgs a{};
    a.q = q;
    a.k = k;
    a.v = v;
    // the stride of a single token means nothing
    a.q_stride = Tq > 1 ? q_stride : (int64_t)heads * dim;
    a.k_stride = Tk > 1 ? k_stride : (int64_t)n_kv * dim;
    a.v_stride = Tk > 1 ? v_stride : (int64_t)n_kv * dim;
    a.in_f32 = dtype == COLI_F32;
    a.out_bf16 = dtype_out == COLI_BF16;
    a.Tq = Tq;
    a.Tk = Tk;
    a.n_seq = n_seq;
    a.cu_q = cu_q;
    a.cu_k = cu_k;
    a.heads = heads;
    a.H = n_kv;
    a.group = group;
    a.tokens = tokens;
    a.dim = dim;
    a.scale = scale;
    a.out = out;
    a.lse = lse;
    DevInfo d;
    if (int rc = device_info(&d)) return rc;
    if (const size_t bytes = gqa_prefill_scratch(a))
        if (int rc = device_scratch(&d, (cudaStream_t)stream, bytes)) return rc;
    a.err = d.err;
    int n = 0;
    const cudaError_t e = launch_gqa_prefill(a, d, (cudaStream_t)stream, &n);
    return launched(e, "coli_gqa_prefill", n);
}

}  // namespace

extern "C" {

int coli_gqa_prefill(int dtype, const void *q, int64_t q_stride, const void *k, int64_t k_stride, const void *v, int64_t v_stride,
                     int Tq, int Tk, int n_seq, const int32_t *cu_q, const int32_t *cu_k, int n_heads, int n_kv, int dim, float scale,
                     int dtype_out, void *out, float *lse, void *stream) {
    return guarded([&] {
        return prefill(dtype, q, q_stride, k, k_stride, v, v_stride, Tq, Tk, n_seq, cu_q, cu_k, n_heads, n_kv, dim, scale, dtype_out,
                       out, lse, stream);
    });
}

int coli_gqa_append(const coli_gqa_cache *cache, int dtype, const void *k, int64_t k_stride, const void *v, int64_t v_stride, int T,
                    const int64_t *slots, void *stream) {
    return guarded([&] { return append(cache, dtype, k, k_stride, v, v_stride, T, slots, stream); });
}

int coli_gqa_read(const coli_gqa_cache *cache, const int32_t *pages, int64_t pages_stride, int n_seq, const int32_t *cu, int T,
                  int dtype, void *k, int64_t k_stride, void *v, int64_t v_stride, void *stream) {
    return guarded([&] { return read(cache, pages, pages_stride, n_seq, cu, T, dtype, k, k_stride, v, v_stride, stream); });
}

int coli_gqa_attend(const coli_gqa_cache *cache, int dtype_q, const void *q, int n_seq, int n_q, int n_heads, const int32_t *pages,
                    int64_t pages_stride, const int32_t *lens, float scale, int weigh, int dtype_out, void *out, float *lse,
                    void *stream) {
    return guarded(
        [&] { return attend(cache, dtype_q, q, n_seq, n_q, n_heads, pages, pages_stride, lens, scale, weigh, dtype_out, out, lse, stream); });
}

int coli_gqa_evict(const coli_gqa_cache *cache, const int32_t *pages, int64_t pages_stride, int n_seq, const int32_t *lens, int keep,
                   int recent, const int32_t *dst, int64_t dst_stride, int32_t *kept, int32_t *new_lens, void *stream) {
    return guarded(
        [&] { return evict(cache, pages, pages_stride, n_seq, lens, keep, recent, dst, dst_stride, kept, new_lens, stream); });
}

}  // extern "C"

// mla_api.cu -- the latent-attention entry points of include/coli.h: argument
// checks and launches.  Nothing is launched unless every check passed.
#include "api_checks.cuh"
#include "mla.cuh"

using namespace coli;

namespace {

int check_cache(const coli_mla_cache *c, MlaCache *out) {
    if (!c) return bad(COLI_EINVAL, "cache is NULL");
    if (c->dtype != COLI_BF16 && c->dtype != COLI_E4M3)
        return bad(COLI_EFMT, "the cache's dtype must be COLI_BF16 or COLI_E4M3 (got %d)", c->dtype);
    if (c->latent < 128 || c->latent > 512 || c->latent % 128)
        return bad(COLI_EINVAL, "latent must be 128, 256, 384 or 512 (got %d)", c->latent);
    if (c->rope < 16 || c->rope > 64 || c->rope % 16)
        return bad(COLI_EINVAL, "rope must be a multiple of 16 in 16..64 (got %d)", c->rope);
    if (c->page_size < 16 || c->page_size > 65536 || c->page_size % 16)
        return bad(COLI_EINVAL, "page_size must be a multiple of 16 in 16..65536 (got %d)", c->page_size);
    if (c->n_pages < 1 || c->n_pages > ((1LL << 31) - 1) / c->page_size)
        return bad(COLI_EINVAL, "n_pages must be >= 1 and n_pages * page_size <= 2^31 - 1 (got %lld)", (long long)c->n_pages);
    if (int rc = need(c->rows, 16, "cache rows")) return rc;
    out->e4m3 = c->dtype == COLI_E4M3;
    if (out->e4m3)
        if (int rc = need(c->scales, 16, "cache scales")) return rc;
    out->rows = (uint8_t *)c->rows;
    out->scales = out->e4m3 ? c->scales : nullptr;
    out->L = c->latent;
    out->R = c->rope;
    out->page = c->page_size;
    out->n_pages = (int)c->n_pages;
    out->row_bytes = (c->latent + c->rope) * (out->e4m3 ? 1 : 2);
    return COLI_OK;
}

int check_rot(const int32_t *pos, const float *rot, int n_pos) {
    if (int rc = need(pos, 4, "pos")) return rc;
    if (int rc = need(rot, 16, "rot")) return rc;
    if (n_pos < 1) return bad(COLI_EINVAL, "n_pos must be >= 1 (got %d)", n_pos);
    return COLI_OK;
}

int query(const float *q, int64_t q_stride, int T, int H, int nope, int rope, const int32_t *pos, const float *rot, int n_pos,
          int interleaved, int dn, void *out_nope, int64_t ld_nope, int dr, void *out_rope, int64_t ld_rope, void *stream) {
    clear_last_error();
    if (T < 0 || H < 1) return bad(COLI_EINVAL, "need T >= 0 and n_heads >= 1 (got %d, %d)", T, H);
    if (nope < 0 || nope % 8 || nope > 65536) return bad(COLI_EINVAL, "nope must be a multiple of 8 >= 0 (got %d)", nope);
    if (rope < 16 || rope > 256 || rope % 16) return bad(COLI_EINVAL, "rope must be a multiple of 16 in 16..256 (got %d)", rope);
    if (nope)
        if (int rc = float_type(dn, "dtype_nope")) return rc;
    if (int rc = float_type(dr, "dtype_rope")) return rc;
    if (T > 1 && (q_stride < (int64_t)H * (nope + rope) || q_stride % 8))
        return bad(COLI_EINVAL, "q_stride must be a multiple of 8 that holds a token's heads (got %lld)", (long long)q_stride);
    if ((nope && (ld_nope < nope || ld_nope % 8)) || ld_rope < rope || ld_rope % 8)
        return bad(COLI_EINVAL, "ld_nope and ld_rope must be multiples of 8 that hold a row (got %lld, %lld)", (long long)ld_nope, (long long)ld_rope);
    if (T) {
        if (int rc = need(q, 16, "q")) return rc;
        if (int rc = check_rot(pos, rot, n_pos)) return rc;
        if (nope)
            if (int rc = need(out_nope, 16, "out_nope")) return rc;
        if (int rc = need(out_rope, 16, "out_rope")) return rc;
    }
    if (int rc = injected_gate()) return rc;
    if (!T) return COLI_OK;
    DevInfo d;
    if (int rc = device_info(&d)) return rc;
    const MlaQueryArgs a{q, q_stride, T, H, nope, rope, pos, rot, n_pos, interleaved, out_nope, out_rope, ld_nope, ld_rope, d.err};
    return launched(launch_mla_query(a, dn == COLI_BF16, dr == COLI_BF16, d.n_sm, (cudaStream_t)stream), "coli_mla_query", 1);
}

int append(const coli_mla_cache *cache, const float *kv, int64_t kv_stride, int T, const float *norm, float eps, const int32_t *pos,
           const float *rot, int n_pos, int interleaved, const int64_t *slots, void *stream) {
    clear_last_error();
    MlaAppendArgs a{};
    if (int rc = check_cache(cache, &a.c)) return rc;
    if (T < 0) return bad(COLI_EINVAL, "T must be >= 0 (got %d)", T);
    if (T > 1 && (kv_stride < a.c.L + a.c.R || kv_stride % 4))
        return bad(COLI_EINVAL, "kv_stride must be a multiple of 4 that holds a token (got %lld)", (long long)kv_stride);
    if (norm && !(eps > 0.f)) return bad(COLI_EINVAL, "eps must be > 0");
    if (T) {
        if (int rc = need(kv, 16, "kv")) return rc;
        if (norm)
            if (int rc = need(norm, 16, "norm")) return rc;
        if (int rc = check_rot(pos, rot, n_pos)) return rc;
        if (int rc = need(slots, 8, "slots")) return rc;
    }
    if (int rc = injected_gate()) return rc;
    if (!T) return COLI_OK;
    DevInfo d;
    if (int rc = device_info(&d)) return rc;
    a.kv = kv;
    a.kv_stride = kv_stride;
    a.T = T;
    a.norm = norm;
    a.eps = eps;
    a.pos = pos;
    a.rot = rot;
    a.n_pos = n_pos;
    a.interleaved = interleaved;
    a.slots = slots;
    a.err = d.err;
    return launched(launch_mla_append(a, (cudaStream_t)stream), "coli_mla_append", 1);
}

int read(const coli_mla_cache *cache, const int32_t *pages, int64_t pages_stride, int n_seq, const int32_t *cu, int T, int dtype,
         void *out, int64_t out_stride, void *stream) {
    clear_last_error();
    MlaReadArgs a{};
    if (int rc = check_cache(cache, &a.c)) return rc;
    if (int rc = float_type(dtype, "dtype")) return rc;
    if (T < 0 || n_seq < 0) return bad(COLI_EINVAL, "T and n_seq must be >= 0 (got %d, %d)", T, n_seq);
    if (pages_stride < 1) return bad(COLI_EINVAL, "pages_stride must be >= 1 (got %lld)", (long long)pages_stride);
    if (out_stride < a.c.L + a.c.R || out_stride % 8)
        return bad(COLI_EINVAL, "out_stride must be a multiple of 8 that holds a row (got %lld)", (long long)out_stride);
    if (T && n_seq) {
        if (int rc = need(pages, 4, "pages")) return rc;
        if (int rc = need(cu, 4, "cu")) return rc;
        if (int rc = need(out, 16, "out")) return rc;
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
    a.out = out;
    a.out_stride = out_stride;
    a.err = d.err;
    return launched(launch_mla_read(a, dtype == COLI_BF16, (cudaStream_t)stream), "coli_mla_read", 1);
}

int attend(const coli_mla_cache *cache, int dtype_q, const void *q_latent, const void *q_rope, int n_seq, int n_q, int H,
           const int32_t *pages, int64_t pages_stride, const int32_t *lens, float scale, int dtype_out, void *out, float *lse,
           void *stream) {
    clear_last_error();
    MlaAttendArgs a{};
    if (int rc = check_cache(cache, &a.c)) return rc;
    if (int rc = float_type(dtype_q, "dtype_q")) return rc;
    if (int rc = float_type(dtype_out, "dtype_out")) return rc;
    if (n_seq < 0 || n_q < 1 || H < 1 || H > 1024 || (int64_t)n_q * H > 65536)
        return bad(COLI_EINVAL, "need n_seq >= 0, n_q >= 1, 1 <= n_heads <= 1024, n_q * n_heads <= 65536 (got %d, %d, %d)", n_seq, n_q, H);
    if ((int64_t)n_seq * n_q * H > (1LL << 31) - 1) return bad(COLI_EINVAL, "n_seq * n_q * n_heads is too large");
    if (pages_stride < 1 || pages_stride > (1LL << 31) - 1)
        return bad(COLI_EINVAL, "pages_stride must be in 1..2^31-1 (got %lld)", (long long)pages_stride);
    if (n_seq && pages_stride * a.c.page / 128 + 1 > ((1LL << 31) - 1) / n_seq)   // a product would pass 2^63
        return bad(COLI_EINVAL, "n_seq * pages_stride * page_size is too large");
    if (!(scale == scale)) return bad(COLI_EINVAL, "scale must not be NaN");
    if (n_seq) {
        if (int rc = need(q_latent, 16, "q_latent")) return rc;
        if (int rc = need(q_rope, 16, "q_rope")) return rc;
        if (int rc = need(pages, 4, "pages")) return rc;
        if (int rc = need(lens, 4, "lens")) return rc;
        if (int rc = need(out, 16, "out")) return rc;
        if (lse)
            if (int rc = need(lse, 4, "lse")) return rc;
    }
    if (int rc = injected_gate()) return rc;
    if (!n_seq) return COLI_OK;
    a.q_latent = q_latent;
    a.q_rope = q_rope;
    a.q_bf16 = dtype_q == COLI_BF16;
    a.out_bf16 = dtype_out == COLI_BF16;
    a.n_seq = n_seq;
    a.n_q = n_q;
    a.H = H;
    a.pages = pages;
    a.pages_stride = pages_stride;
    a.lens = lens;
    a.scale = scale;
    a.out = out;
    a.lse = lse;
    DevInfo d;
    if (int rc = device_info(&d)) return rc;
    if (const size_t bytes = mla_attend_scratch(a, d.n_sm))
        if (int rc = device_scratch(&d, (cudaStream_t)stream, bytes)) return rc;
    a.err = d.err;
    int n = 0;
    const cudaError_t e = launch_mla_attend(a, d, (cudaStream_t)stream, &n);
    return launched(e, "coli_mla_attend", n);
}

int prefill(int dtype, const void *q, int64_t q_stride, const void *kv, int64_t kv_stride, const void *k_rope, int64_t kr_stride,
            int Tq, int Tk, int n_seq, const int32_t *cu_q, const int32_t *cu_k, int H, int nope, int rope, int v, float scale,
            int dtype_out, void *out, float *lse, void *stream) {
    clear_last_error();
    if (int rc = float_type(dtype, "dtype")) return rc;
    if (int rc = float_type(dtype_out, "dtype_out")) return rc;
    if ((nope != 64 && nope != 128) || (v != 64 && v != 128))
        return bad(COLI_EINVAL, "nope and v must be 64 or 128 (got %d, %d)", nope, v);
    if (rope < 16 || rope > 64 || rope % 16) return bad(COLI_EINVAL, "rope must be a multiple of 16 in 16..64 (got %d)", rope);
    if (Tq < 0 || Tk < 0 || n_seq < 0 || H < 1 || H > 1024)
        return bad(COLI_EINVAL, "need Tq, Tk, n_seq >= 0 and 1 <= n_heads <= 1024 (got %d, %d, %d, %d)", Tq, Tk, n_seq, H);
    if ((int64_t)Tq * H > (1LL << 31) - 1 || ((int64_t)Tq / 256 + 1 + n_seq) * H > (1LL << 31) - 1)
        return bad(COLI_EINVAL, "Tq * n_heads or n_seq * n_heads is too large");
    if (q_stride < (int64_t)H * (nope + rope) || kv_stride < (int64_t)H * (nope + v) || kr_stride < rope || q_stride % 8 ||
        kv_stride % 8 || kr_stride % 8)
        return bad(COLI_EINVAL, "strides must be multiples of 8 that hold a token (got %lld, %lld, %lld)", (long long)q_stride,
                   (long long)kv_stride, (long long)kr_stride);
    if (!(scale == scale)) return bad(COLI_EINVAL, "scale must not be NaN");
    if (Tq && n_seq) {
        if (int rc = need(q, 16, "q")) return rc;
        if (Tk) {
            if (int rc = need(kv, 16, "kv")) return rc;
            if (int rc = need(k_rope, 16, "k_rope")) return rc;
        }
        if (int rc = need(cu_q, 4, "cu_q")) return rc;
        if (int rc = need(cu_k, 4, "cu_k")) return rc;
        if (int rc = need(out, 16, "out")) return rc;
        if (lse)
            if (int rc = need(lse, 4, "lse")) return rc;
    }
    if (int rc = injected_gate()) return rc;
    if (!Tq || !n_seq) return COLI_OK;
    MlaPrefillArgs a{};
    a.q = q;
    a.kv = kv;
    a.k_rope = k_rope;
    a.q_stride = q_stride;
    a.kv_stride = kv_stride;
    a.kr_stride = kr_stride;
    a.in_f32 = dtype == COLI_F32;
    a.out_bf16 = dtype_out == COLI_BF16;
    a.Tq = Tq;
    a.Tk = Tk;
    a.n_seq = n_seq;
    a.cu_q = cu_q;
    a.cu_k = cu_k;
    a.H = H;
    a.nope = nope;
    a.rope = rope;
    a.v = v;
    a.scale = scale;
    a.out = out;
    a.lse = lse;
    DevInfo d;
    if (int rc = device_info(&d)) return rc;
    if (const size_t bytes = mla_prefill_scratch(a))
        if (int rc = device_scratch(&d, (cudaStream_t)stream, bytes)) return rc;
    a.err = d.err;
    int n = 0;
    const cudaError_t e = launch_mla_prefill(a, d, (cudaStream_t)stream, &n);
    return launched(e, "coli_mla_prefill", n);
}

}  // namespace

extern "C" {

int coli_mla_query(const float *q, int64_t q_stride, int T, int n_heads, int nope, int rope, const int32_t *pos, const float *rot,
                   int n_pos, int interleaved, int dtype_nope, void *out_nope, int64_t ld_nope, int dtype_rope, void *out_rope,
                   int64_t ld_rope, void *stream) {
    return guarded([&] {
        return query(q, q_stride, T, n_heads, nope, rope, pos, rot, n_pos, interleaved, dtype_nope, out_nope, ld_nope, dtype_rope,
                     out_rope, ld_rope, stream);
    });
}

int coli_mla_append(const coli_mla_cache *cache, const float *kv, int64_t kv_stride, int T, const float *norm, float eps,
                    const int32_t *pos, const float *rot, int n_pos, int interleaved, const int64_t *slots, void *stream) {
    return guarded([&] { return append(cache, kv, kv_stride, T, norm, eps, pos, rot, n_pos, interleaved, slots, stream); });
}

int coli_mla_read(const coli_mla_cache *cache, const int32_t *pages, int64_t pages_stride, int n_seq, const int32_t *cu, int T,
                  int dtype, void *out, int64_t out_stride, void *stream) {
    return guarded([&] { return read(cache, pages, pages_stride, n_seq, cu, T, dtype, out, out_stride, stream); });
}

int coli_mla_attend(const coli_mla_cache *cache, int dtype_q, const void *q_latent, const void *q_rope, int n_seq, int n_q,
                    int n_heads, const int32_t *pages, int64_t pages_stride, const int32_t *lens, float scale, int dtype_out,
                    void *out, float *lse, void *stream) {
    return guarded([&] {
        return attend(cache, dtype_q, q_latent, q_rope, n_seq, n_q, n_heads, pages, pages_stride, lens, scale, dtype_out, out, lse,
                      stream);
    });
}

int coli_mla_prefill(int dtype, const void *q, int64_t q_stride, const void *kv, int64_t kv_stride, const void *k_rope,
                     int64_t kr_stride, int Tq, int Tk, int n_seq, const int32_t *cu_q, const int32_t *cu_k, int n_heads, int nope,
                     int rope, int v, float scale, int dtype_out, void *out, float *lse, void *stream) {
    return guarded([&] {
        return prefill(dtype, q, q_stride, kv, kv_stride, k_rope, kr_stride, Tq, Tk, n_seq, cu_q, cu_k, n_heads, nope, rope, v,
                       scale, dtype_out, out, lse, stream);
    });
}

}  // extern "C"

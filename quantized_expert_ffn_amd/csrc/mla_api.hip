// C-ABI entry points of latent attention (include/coli_mla.h): argument
// checks, workspace carve-up and kernel launches.
#include <hip/hip_runtime.h>

#include <cmath>
#include <cstdarg>
#include <cstdio>

#include "coli_mla.h"
#include "kernels.h"
#include "mla.h"

using namespace coli;

namespace {

// The status word has the workspace's first 256 bytes to itself.
constexpr size_t WS_HEAD = 256;

int fail(int code, const char *fmt, ...) {
    char buf[512];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(buf, sizeof buf, fmt, ap);
    va_end(ap);
    return api_fail(code, buf);
}

int launched(hipError_t e, const char *who) {
    return e == hipSuccess ? COLI_OK : fail(COLI_EHIP, "%s launch: %s", who, hipGetErrorString(e));
}

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

int check_mla_dims(const coli_mla_dims *d) {
    if (!d) return fail(COLI_EINVAL, "dims is NULL");
    if (d->n_heads < 1 || d->n_heads > 256) return fail(COLI_EINVAL, "n_heads=%d: must be in 1..256", d->n_heads);
    if (d->rank != 256 && d->rank != 512) return fail(COLI_EINVAL, "rank=%d: must be 256 or 512", d->rank);
    if (!(d->nope == 128 && d->v_dim == 128) && !(d->nope == 192 && d->v_dim == 256))
        return fail(COLI_EINVAL, "nope=%d, v_dim=%d: must be (128, 128) or (192, 256)", d->nope, d->v_dim);
    if (d->page_size < 1 || d->page_size > 65536)
        return fail(COLI_EINVAL, "page_size=%d: must be in 1..65536", d->page_size);
    if (d->dtype != COLI_BF16 && d->dtype != COLI_FP16)
        return fail(COLI_EINVAL, "dtype=%d: must be COLI_BF16 (0) or COLI_FP16 (1)", d->dtype);
    if (d->kv_format != COLI_KV_PLAIN && d->kv_format != COLI_KV_E4M3)
        return fail(COLI_EINVAL, "kv_format=%d: must be COLI_KV_PLAIN (0) or COLI_KV_E4M3 (1)", d->kv_format);
    if (d->rope_style != COLI_ROPE_PAIRS && d->rope_style != COLI_ROPE_HALVES)
        return fail(COLI_EINVAL, "rope_style=%d: must be COLI_ROPE_PAIRS (0) or COLI_ROPE_HALVES (1)", d->rope_style);
    if (!(d->norm_eps >= 0.0f) || !std::isfinite(d->norm_eps))
        return fail(COLI_EINVAL, "norm_eps=%g: must be finite and not negative", (double)d->norm_eps);
    if (!(d->softmax_scale > 0.0f) || !std::isfinite(d->softmax_scale))
        return fail(COLI_EINVAL, "softmax_scale=%g: must be finite and positive", (double)d->softmax_scale);
    return COLI_OK;
}

int check_ws(const void *ws, size_t have, size_t need, const char *who) {
    if (!ws) return fail(COLI_EINVAL, "%s: workspace is NULL", who);
    if (!aligned16(ws)) return fail(COLI_EINVAL, "%s: the workspace must be 16-byte aligned", who);
    if (have < need) return fail(COLI_EWORKSPACE, "%s: workspace %zu bytes < %zu needed", who, have, need);
    return COLI_OK;
}

int check_cache(const coli_mla_dims *d, const void *pages, const float *kv_scale, int32_t n_pages, const char *who) {
    if (!pages || !aligned16(pages)) return fail(COLI_EINVAL, "%s: pages must be a 16-byte aligned pointer", who);
    if (n_pages < 1) return fail(COLI_EINVAL, "%s: n_pages=%d: must be positive", who, n_pages);
    if ((d->kv_format == COLI_KV_E4M3) != (kv_scale != nullptr))
        return fail(COLI_EINVAL, "%s: kv_scale goes with COLI_KV_E4M3, and only with it", who);
    return COLI_OK;
}

bool bad_stride(int64_t s) { return s < 0 || s % 8 != 0; }

MlaCache cache(const coli_mla_dims *d, const void *pages, const float *kv_scale, int32_t n_pages,
               const int32_t *table, int32_t width) {
    MlaCache c;
    c.pages = static_cast<const uint8_t *>(pages);
    c.scale = kv_scale;
    c.table = table;
    c.n_pages = n_pages;
    c.page = d->page_size;
    c.width = width;
    return c;
}

}  // namespace

extern "C" {

size_t coli_mla_row_bytes(const coli_mla_dims *d) {
    if (check_mla_dims(d) != COLI_OK) return 0;
    return d->kv_format == COLI_KV_E4M3 ? (size_t)d->rank + 2 * MLA_ROPE : 2 * ((size_t)d->rank + MLA_ROPE);
}

size_t coli_mla_workspace_bytes(const coli_mla_dims *d, int32_t batch, int32_t n_q, int32_t max_kv) {
    if (check_mla_dims(d) != COLI_OK) return 0;
    if (batch < 0 || batch > COLI_MLA_MAX_BATCH || n_q < 1 || max_kv < 0 || max_kv > COLI_MLA_MAX_LENGTH ||
        (int64_t)n_q * d->n_heads > COLI_MLA_MAX_ROWS || (int64_t)batch * max_kv > COLI_MLA_MAX_TOKENS) {
        fail(COLI_EINVAL, "batch=%d, n_q=%d, max_kv=%d: batch in 0..%d, n_q >= 1 with n_q * n_heads <= %d, "
                          "max_kv in 0..%d with batch * max_kv <= %lld", batch, n_q, max_kv, COLI_MLA_MAX_BATCH,
             COLI_MLA_MAX_ROWS, COLI_MLA_MAX_LENGTH, COLI_MLA_MAX_TOKENS);
        return 0;
    }
    return WS_HEAD + (batch ? mla_decode_part_bytes(*d, batch, n_q, max_kv) : 0);
}

int coli_mla_append(const coli_mla_dims *d, int32_t n_tokens, const void *kv_a, const void *norm_w,
                    const int32_t *positions, const int64_t *slots, const double *inv_freq, const void *q_pe,
                    int64_t q_token_stride, int64_t q_head_stride, void *q_pe_out, int64_t out_token_stride,
                    int64_t out_head_stride, void *pages, float *kv_scale, int32_t n_pages, void *ws,
                    size_t ws_bytes, void *stream) {
    int rc = check_mla_dims(d);
    if (rc) return rc;
    if (n_tokens < 0) return fail(COLI_EINVAL, "n_tokens=%d < 0", n_tokens);
    if (n_tokens == 0) return COLI_OK;
    if (!kv_a || !positions || !slots || !inv_freq) return fail(COLI_EINVAL, "coli_mla_append: NULL pointer argument");
    if ((q_pe == nullptr) != (q_pe_out == nullptr))
        return fail(COLI_EINVAL, "coli_mla_append: q_pe and q_pe_out go together");
    if (!aligned16(kv_a) || !aligned16(norm_w) || !aligned16(q_pe) || !aligned16(q_pe_out))
        return fail(COLI_EINVAL, "coli_mla_append: kv_a, norm_w, q_pe and q_pe_out must be 16-byte aligned");
    if (bad_stride(q_token_stride) || bad_stride(q_head_stride) || bad_stride(out_token_stride) ||
        bad_stride(out_head_stride))
        return fail(COLI_EINVAL, "coli_mla_append: strides must be non-negative multiples of 8");
    if ((rc = check_cache(d, pages, kv_scale, n_pages, "coli_mla_append"))) return rc;
    if ((rc = check_ws(ws, ws_bytes, WS_HEAD, "coli_mla_append"))) return rc;
    if ((rc = api_check_device())) return rc;
    MlaAppendArgs a{};
    a.kv_a = kv_a;
    a.norm_w = norm_w;
    a.q_pe = q_pe;
    a.q_out = q_pe_out;
    a.positions = positions;
    a.slots = slots;
    a.inv_freq = inv_freq;
    a.pages = static_cast<uint8_t *>(pages);
    a.kv_scale = kv_scale;
    a.status = static_cast<uint32_t *>(ws);
    a.q_ts = q_token_stride;
    a.q_hs = q_head_stride;
    a.o_ts = out_token_stride;
    a.o_hs = out_head_stride;
    a.n_slots = (int64_t)n_pages * d->page_size;
    a.tokens = n_tokens;
    a.heads = q_pe ? d->n_heads : 0;
    a.eps = d->norm_eps;
    return launched(launch_mla_append(a, *d, static_cast<hipStream_t>(stream)), "append");
}

int coli_mla_project(int32_t dtype, int32_t n_tokens, int32_t n_heads, int32_t n_in, int32_t n_out, const void *x,
                     int64_t x_token_stride, int64_t x_head_stride, const void *w, void *out, void *stream) {
    if (dtype != COLI_BF16 && dtype != COLI_FP16)
        return fail(COLI_EINVAL, "dtype=%d: must be COLI_BF16 (0) or COLI_FP16 (1)", dtype);
    if (n_tokens < 0) return fail(COLI_EINVAL, "n_tokens=%d < 0", n_tokens);
    if (n_heads < 1 || n_heads > 256) return fail(COLI_EINVAL, "n_heads=%d: must be in 1..256", n_heads);
    if (n_in < 64 || n_in > 1024 || n_in % 64)
        return fail(COLI_EINVAL, "n_in=%d: must be a multiple of 64 in 64..1024", n_in);
    if (n_out < 64 || n_out > 4096 || n_out % 64)
        return fail(COLI_EINVAL, "n_out=%d: must be a multiple of 64 in 64..4096", n_out);
    if ((int64_t)n_heads * n_tokens >= (int64_t)1 << 30)
        return fail(COLI_EINVAL, "n_tokens=%d: too many for %d heads", n_tokens, n_heads);
    if (n_tokens == 0) return COLI_OK;
    if (!x || !w || !out) return fail(COLI_EINVAL, "coli_mla_project: NULL pointer argument");
    if (!aligned16(x) || !aligned16(w) || !aligned16(out))
        return fail(COLI_EINVAL, "coli_mla_project: x, w and out must be 16-byte aligned");
    if (bad_stride(x_token_stride) || bad_stride(x_head_stride))
        return fail(COLI_EINVAL, "coli_mla_project: strides must be non-negative multiples of 8");
    const int rc = api_check_device();
    if (rc) return rc;
    MlaProjectArgs a{x, w, out, x_token_stride, x_head_stride, n_tokens, n_heads, n_in, n_out};
    return launched(launch_mla_project(a, dtype, static_cast<hipStream_t>(stream)), "project");
}

int coli_mla_decode(const coli_mla_dims *d, int32_t batch, int32_t n_q, const void *q_lat, const void *q_pe,
                    const void *pages, const float *kv_scale, int32_t n_pages, const int32_t *table,
                    int32_t table_width, const int32_t *kv_lens, int32_t max_kv, void *out, float *lse, void *ws,
                    size_t ws_bytes, void *stream) {
    int rc = check_mla_dims(d);
    if (rc) return rc;
    if (batch < 0 || batch > COLI_MLA_MAX_BATCH)
        return fail(COLI_EINVAL, "batch=%d: must be in 0..%d", batch, COLI_MLA_MAX_BATCH);
    if (n_q < 1 || (int64_t)n_q * d->n_heads > COLI_MLA_MAX_ROWS)
        return fail(COLI_EINVAL, "n_q=%d: must be positive, with n_q * n_heads at most %d", n_q, COLI_MLA_MAX_ROWS);
    if (max_kv < 0 || max_kv > COLI_MLA_MAX_LENGTH || (int64_t)batch * max_kv > COLI_MLA_MAX_TOKENS)
        return fail(COLI_EINVAL, "max_kv=%d: must be in 0..%d, with batch * max_kv at most %lld", max_kv,
                    COLI_MLA_MAX_LENGTH, COLI_MLA_MAX_TOKENS);
    if (batch == 0) return COLI_OK;
    if (!q_lat || !q_pe || !table || !kv_lens || !out)
        return fail(COLI_EINVAL, "coli_mla_decode: NULL pointer argument");
    if (!aligned16(q_lat) || !aligned16(q_pe) || !aligned16(out))
        return fail(COLI_EINVAL, "coli_mla_decode: q_lat, q_pe and out must be 16-byte aligned");
    if (table_width < 1 || (int64_t)table_width * d->page_size < max_kv)
        return fail(COLI_EINVAL, "coli_mla_decode: table_width=%d pages do not hold max_kv=%d tokens", table_width,
                    max_kv);
    if ((rc = check_cache(d, pages, kv_scale, n_pages, "coli_mla_decode"))) return rc;
    const size_t need = WS_HEAD + mla_decode_part_bytes(*d, batch, n_q, max_kv);
    if ((rc = check_ws(ws, ws_bytes, need, "coli_mla_decode"))) return rc;
    if ((rc = api_check_device())) return rc;
    MlaDecodeArgs a{};
    a.c = cache(d, pages, kv_scale, n_pages, table, table_width);
    a.q_lat = q_lat;
    a.q_pe = q_pe;
    a.kv_lens = kv_lens;
    a.out = out;
    a.lse = lse;
    a.status = static_cast<uint32_t *>(ws);
    a.part = reinterpret_cast<float *>(static_cast<uint8_t *>(ws) + WS_HEAD);
    a.batch = batch;
    a.n_q = n_q;
    a.heads = d->n_heads;
    a.max_kv = max_kv;
    a.scale = d->softmax_scale;
    return launched(launch_mla_decode(a, *d, static_cast<hipStream_t>(stream)), "decode");
}

int coli_mla_expand(const coli_mla_dims *d, int32_t batch, int32_t n_rows, const void *pages,
                    const float *kv_scale, int32_t n_pages, const int32_t *table, int32_t table_width,
                    const int32_t *cu_k, const void *w, void *kv, void *k_pe, void *ws, size_t ws_bytes,
                    void *stream) {
    int rc = check_mla_dims(d);
    if (rc) return rc;
    if (batch < 0 || batch > COLI_MLA_MAX_BATCH)
        return fail(COLI_EINVAL, "batch=%d: must be in 0..%d", batch, COLI_MLA_MAX_BATCH);
    if (n_rows < 0 || n_rows > COLI_MLA_MAX_LENGTH)
        return fail(COLI_EINVAL, "n_rows=%d: must be in 0..%d", n_rows, COLI_MLA_MAX_LENGTH);
    if (batch == 0 || n_rows == 0) return COLI_OK;
    if (!table || !cu_k || !w || !kv || !k_pe) return fail(COLI_EINVAL, "coli_mla_expand: NULL pointer argument");
    if (!aligned16(w) || !aligned16(kv) || !aligned16(k_pe))
        return fail(COLI_EINVAL, "coli_mla_expand: w, kv and k_pe must be 16-byte aligned");
    if (table_width < 1) return fail(COLI_EINVAL, "coli_mla_expand: table_width=%d: must be positive", table_width);
    if ((rc = check_cache(d, pages, kv_scale, n_pages, "coli_mla_expand"))) return rc;
    if ((rc = check_ws(ws, ws_bytes, WS_HEAD, "coli_mla_expand"))) return rc;
    if ((rc = api_check_device())) return rc;
    MlaExpandArgs a{};
    a.c = cache(d, pages, kv_scale, n_pages, table, table_width);
    a.cu_k = cu_k;
    a.w = w;
    a.kv = kv;
    a.k_pe = k_pe;
    a.status = static_cast<uint32_t *>(ws);
    a.batch = batch;
    a.rows = n_rows;
    a.n_out = d->n_heads * (d->nope + d->v_dim);
    return launched(launch_mla_expand(a, *d, static_cast<hipStream_t>(stream)), "expand");
}

int coli_mla_prefill(const coli_mla_dims *d, int32_t batch, int32_t n_q_rows, int32_t n_k_rows, const void *q,
                     int64_t q_token_stride, int64_t q_head_stride, const void *k_nope, int64_t k_token_stride,
                     int64_t k_head_stride, const void *k_pe, const void *v, int64_t v_token_stride,
                     int64_t v_head_stride, const int32_t *cu_q, const int32_t *cu_k, int32_t max_q, int32_t causal,
                     void *out, float *lse, void *ws, size_t ws_bytes, void *stream) {
    int rc = check_mla_dims(d);
    if (rc) return rc;
    if (batch < 0 || batch > COLI_MLA_MAX_BATCH)
        return fail(COLI_EINVAL, "batch=%d: must be in 0..%d", batch, COLI_MLA_MAX_BATCH);
    if (n_q_rows < 0 || n_k_rows < 0 || max_q < 0)
        return fail(COLI_EINVAL, "n_q_rows=%d, n_k_rows=%d, max_q=%d: must not be negative", n_q_rows, n_k_rows, max_q);
    if (n_q_rows > COLI_MLA_MAX_LENGTH || n_k_rows > COLI_MLA_MAX_LENGTH)
        return fail(COLI_EINVAL, "n_q_rows=%d, n_k_rows=%d: must be at most %d", n_q_rows, n_k_rows, COLI_MLA_MAX_LENGTH);
    if (causal != 0 && causal != 1) return fail(COLI_EINVAL, "causal=%d: must be 0 or 1", causal);
    if (batch == 0 || n_q_rows == 0 || max_q == 0) return COLI_OK;
    if (!q || !cu_q || !cu_k || !out || (n_k_rows > 0 && (!k_nope || !k_pe || !v)))
        return fail(COLI_EINVAL, "coli_mla_prefill: NULL pointer argument");
    if (!aligned16(q) || !aligned16(k_nope) || !aligned16(k_pe) || !aligned16(v) || !aligned16(out))
        return fail(COLI_EINVAL, "coli_mla_prefill: q, k_nope, k_pe, v and out must be 16-byte aligned");
    if (bad_stride(q_token_stride) || bad_stride(q_head_stride) || bad_stride(k_token_stride) ||
        bad_stride(k_head_stride) || bad_stride(v_token_stride) || bad_stride(v_head_stride))
        return fail(COLI_EINVAL, "coli_mla_prefill: strides must be non-negative multiples of 8");
    if (k_token_stride > COLI_MLA_MAX_STRIDE || v_token_stride > COLI_MLA_MAX_STRIDE)
        return fail(COLI_EINVAL, "coli_mla_prefill: token strides of k_nope and v must be at most %d", COLI_MLA_MAX_STRIDE);
    if ((int64_t)batch * d->n_heads * (((int64_t)max_q + 127) / 128) >= (int64_t)1 << 28)
        return fail(COLI_EINVAL, "coli_mla_prefill: batch=%d, max_q=%d: too many blocks of queries", batch, max_q);
    if ((rc = check_ws(ws, ws_bytes, WS_HEAD, "coli_mla_prefill"))) return rc;
    if ((rc = api_check_device())) return rc;
    MlaPrefillArgs a{};
    a.q = q;
    a.k_nope = k_nope;
    a.k_pe = k_pe;
    a.v = v;
    a.cu_q = cu_q;
    a.cu_k = cu_k;
    a.out = out;
    a.lse = lse;
    a.status = static_cast<uint32_t *>(ws);
    a.q_ts = q_token_stride;
    a.q_hs = q_head_stride;
    a.k_ts = k_token_stride;
    a.k_hs = k_head_stride;
    a.v_ts = v_token_stride;
    a.v_hs = v_head_stride;
    a.batch = batch;
    a.heads = d->n_heads;
    a.n_q_rows = n_q_rows;
    a.n_k_rows = n_k_rows;
    a.max_q = max_q < n_q_rows ? max_q : n_q_rows;   // no sequence has more
    a.causal = causal;
    a.scale = d->softmax_scale;
    return launched(launch_mla_prefill(a, *d, static_cast<hipStream_t>(stream)), "prefill");
}

}  // extern "C"

// C-ABI entry points of the 8-bit products (include/coli_w8.h): argument
// checks and kernel launches.
#include <hip/hip_runtime.h>

#include <cstdarg>
#include <cstdio>

#include "kernels.h"
#include "w8.h"

using namespace coli;

namespace {

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

bool aligned(const void *p, uintptr_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

uintptr_t size_of(int32_t dtype) { return dtype == COLI_F32 ? 4 : 2; }

int check_sizes(int32_t dtype, int32_t n_tokens, int32_t k) {
    if (dtype != COLI_BF16 && dtype != COLI_FP16 && dtype != COLI_F32)
        return fail(COLI_EINVAL, "dtype=%d: must be COLI_BF16 (0), COLI_FP16 (1) or COLI_F32 (2)", dtype);
    if (n_tokens < 0 || n_tokens > COLI_W8_MAX_ROWS)
        return fail(COLI_EINVAL, "n_tokens=%d: must be in 0..%d", n_tokens, COLI_W8_MAX_ROWS);
    if (k < 16 || k > COLI_W8_MAX_K || k % 16)
        return fail(COLI_EINVAL, "k=%d: must be a multiple of 16 in 16..%d", k, COLI_W8_MAX_K);
    return COLI_OK;
}

// Strides whose rows lie apart and whose offsets stay in 64 bits.
bool bad_stride(int64_t stride, int64_t least) { return stride < least || stride > (int64_t)1 << 36; }

}  // namespace

extern "C" {

int coli_w8_quantize(int32_t dtype, int32_t n_tokens, int32_t k, const void *x, int64_t token_stride, int8_t *codes,
                     float *scale, void *stream) {
    int rc = check_sizes(dtype, n_tokens, k);
    if (rc) return rc;
    if (n_tokens == 0) return COLI_OK;
    if (!x || !codes || !scale) return fail(COLI_EINVAL, "coli_w8_quantize: NULL pointer argument");
    if (!aligned(x, 16) || !aligned(codes, 16) || !aligned(scale, 4))
        return fail(COLI_EINVAL, "coli_w8_quantize: x and codes must be 16-byte aligned, scale 4-byte");
    const int64_t bytes = size_of(dtype);
    if ((token_stride < 0 || token_stride > (int64_t)1 << 36) || token_stride * bytes % 16)
        return fail(COLI_EINVAL, "coli_w8_quantize: token_stride=%lld: rows must be 16-byte aligned, in 0..2^36",
                    (long long)token_stride);
    if ((rc = api_check_device())) return rc;
    W8QuantizeArgs a{x, codes, scale, token_stride * bytes, n_tokens, k};
    return launched(launch_w8_quantize(a, dtype, static_cast<hipStream_t>(stream)), "quantize");
}

int coli_w8_linear(int32_t dtype, int32_t n_tokens, int32_t k, int32_t n_out, const int8_t *codes, int64_t code_stride,
                   const float *scale, const int8_t *w, const float *w_scale, const float *bias, void *out,
                   int64_t out_stride, void *stream) {
    int rc = check_sizes(dtype, n_tokens, k);
    if (rc) return rc;
    if (n_out < 1 || n_out > COLI_W8_MAX_ROWS)
        return fail(COLI_EINVAL, "n_out=%d: must be in 1..%d", n_out, COLI_W8_MAX_ROWS);
    if (n_tokens == 0) return COLI_OK;
    if (!codes || !scale || !w || !w_scale || !out) return fail(COLI_EINVAL, "coli_w8_linear: NULL pointer argument");
    if (!aligned(codes, 16) || !aligned(w, 16) || !aligned(scale, 4) || !aligned(w_scale, 4) || !aligned(bias, 4) ||
        !aligned(out, size_of(dtype)))
        return fail(COLI_EINVAL, "coli_w8_linear: codes and w must be 16-byte aligned, the others to their elements");
    if (code_stride < 0 || code_stride > (int64_t)1 << 36 || code_stride % 16)
        return fail(COLI_EINVAL, "coli_w8_linear: code_stride=%lld: must be a multiple of 16 in 0..2^36",
                    (long long)code_stride);
    if (bad_stride(out_stride, n_out))
        return fail(COLI_EINVAL, "coli_w8_linear: out_stride=%lld: must be in n_out=%d..2^36", (long long)out_stride, n_out);
    if ((rc = api_check_device())) return rc;
    W8LinearArgs a{codes, w, scale, w_scale, bias, out, code_stride, out_stride, n_tokens, k, n_out};
    return launched(launch_w8_linear(a, dtype, static_cast<hipStream_t>(stream)), "linear");
}

}  // extern "C"

// Private interface between the latent-attention entry points and their
// kernels: arguments (passed by value) and launchers.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "coli_mla.h"

namespace coli {

constexpr int MLA_ROPE = COLI_MLA_ROPE;

// A paged cache as the kernels see it.
struct MlaCache {
    const uint8_t *pages;     // [n_pages * page_size] rows
    const float *scale;       // [n_pages * page_size], E4M3 only
    const int32_t *table;     // [batch, width]
    int32_t n_pages, page, width;
};

struct MlaAppendArgs {
    const void *kv_a, *norm_w, *q_pe;
    void *q_out;
    const int32_t *positions;
    const int64_t *slots;
    const double *inv_freq;
    uint8_t *pages;
    float *kv_scale;
    uint32_t *status;
    int64_t q_ts, q_hs, o_ts, o_hs, n_slots;
    int32_t tokens, heads;
    float eps;
};
hipError_t launch_mla_append(const MlaAppendArgs &a, const coli_mla_dims &d, hipStream_t st);

struct MlaProjectArgs {
    const void *x, *w;
    void *out;
    int64_t x_ts, x_hs;
    int32_t tokens, heads, n_in, n_out;
};
hipError_t launch_mla_project(const MlaProjectArgs &a, int dtype, hipStream_t st);

struct MlaExpandArgs {
    MlaCache c;
    const int32_t *cu_k;
    const void *w;
    void *kv, *k_pe;
    uint32_t *status;
    int32_t batch, rows, n_out;   // n_out = n_heads * (nope + v_dim)
};
hipError_t launch_mla_expand(const MlaExpandArgs &a, const coli_mla_dims &d, hipStream_t st);

struct MlaDecodeArgs {
    MlaCache c;
    const void *q_lat, *q_pe;
    const int32_t *kv_lens;
    void *out;
    float *lse;
    uint32_t *status;
    float *part;                  // partial results (workspace)
    int32_t batch, n_q, heads, max_kv;
    float scale;
};
hipError_t launch_mla_decode(const MlaDecodeArgs &a, const coli_mla_dims &d, hipStream_t st);
// Bytes of partial results a decode call needs behind the status page.
size_t mla_decode_part_bytes(const coli_mla_dims &d, int batch, int n_q, int max_kv);

struct MlaPrefillArgs {
    const void *q, *k_nope, *k_pe, *v;
    const int32_t *cu_q, *cu_k;
    void *out;
    float *lse;
    uint32_t *status;
    int64_t q_ts, q_hs, k_ts, k_hs, v_ts, v_hs;
    int32_t batch, heads, n_q_rows, n_k_rows, max_q, causal;
    float scale;
};
hipError_t launch_mla_prefill(const MlaPrefillArgs &a, const coli_mla_dims &d, hipStream_t st);

// Calls f with the element type of `dtype` (a value of it, for its type).
template <class F>
hipError_t mla_with_type(int dtype, F f) {
    return dtype == COLI_BF16 ? f(__bf16()) : f(_Float16());
}

}  // namespace coli

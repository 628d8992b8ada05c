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
    float *full;                  // and those of whole sequences, where only partial results are wanted
    const int32_t *prefix_table;  // pages of tokens that come before every sequence's own (launch_mla_decode_prefix)
    int32_t batch, n_q, heads, max_kv, prefix;
    float scale;
};
hipError_t launch_mla_decode(const MlaDecodeArgs &a, const coli_mla_dims &d, hipStream_t st);
// The same where sequences begin with a.prefix > 0 tokens that they share, which each reads for itself.
hipError_t launch_mla_decode_prefix(const MlaDecodeArgs &a, const coli_mla_dims &d, hipStream_t st);
// Bytes of partial results a decode call needs behind the status page.
size_t mla_decode_part_bytes(const coli_mla_dims &d, int batch, int n_q, int max_kv);

// Partial results of a decode call, without the join: a sequence whose plan
// entry (two int32 at part, first and last workgroup) names one workgroup has
// its result in slot sequence * blocks + block of `full`; others in slots
// 2 (block * groups + g) + (g == first) of part + first floats.  A slot holds
// `rows` rows, [32 rows][column tile][4][64 lanes] of four floats, then their
// (maximum, sum) pairs.
struct MlaParts {
    int rows, blocks, groups, slot, first;
};
MlaParts mla_decode_parts(const coli_mla_dims &d, int batch, int n_q, int max_kv);
hipError_t launch_mla_decode_parts(const MlaDecodeArgs &a, const coli_mla_dims &d, hipStream_t st);

// Attention behind a prefix that all sequences share: its partial results, and
// the join with those of the sequences' own tokens.
struct MlaSharedArgs {
    MlaCache c;                   // the prefix's pages
    const void *q_lat, *q_pe;
    const int32_t *kv_lens, *own_table;   // the sequences' own tokens, and their pages
    void *out;
    float *lse;
    uint32_t *status;
    int64_t *plan;                // how the work is shared out
    float *part;                  // partial results over the prefix
    const float *own, *full;      // of the sequences' own tokens (MlaParts), or null
    int32_t own_width, batch, n_q, heads, prefix, max_kv, shares;
    int32_t whole;                // blocks of rows are of one sequence, and take its own tokens too
    MlaParts p;
    float scale;
};
// Whether a call's sequences read the prefix each for itself: where that is faster (path 0), never (1), wherever lengths fit (2).
bool mla_prefix_by_sequence(const coli_mla_dims &d, int batch, int n_q, int prefix, int max_kv, int path);
// The sizes of a call and where its workspace's part is.
MlaSharedArgs mla_shared_args(const coli_mla_dims &d, void *part, int batch, int n_q, int prefix, int max_kv);
hipError_t launch_mla_shared(const MlaSharedArgs &a, const coli_mla_dims &d, hipStream_t st);
hipError_t launch_mla_shared_join(const MlaSharedArgs &a, const coli_mla_dims &d, hipStream_t st);
// Bytes of the prefix's partial results.
size_t mla_shared_part_bytes(const coli_mla_dims &d, int batch, int n_q, int prefix, int max_kv);

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

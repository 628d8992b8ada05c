// Device building blocks of the latent-attention kernels.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "device_common.h"
#include "mla.h"

namespace coli {

// Eight values of a 16-bit type: one 16-byte access.
template <class T>
using x8 = T __attribute__((ext_vector_type(8)));
template <class T>
using x4 = T __attribute__((ext_vector_type(4)));
template <class T>
using x2 = T __attribute__((ext_vector_type(2)));
typedef float f32x2 __attribute__((ext_vector_type(2)));

// Row of a cache that holds token t of sequence b; a page id outside the
// cache raises the status and reads as page 0.
__device__ __forceinline__ int64_t mla_slot(const MlaCache &c, int b, int t, uint32_t *status) {
    const int pi = t / c.page;
    int pid = c.table[(int64_t)b * c.width + pi];
    if ((uint32_t)pid >= (uint32_t)c.n_pages) {
        raise_status(status, ST_BADPAGE);
        pid = 0;
    }
    return (int64_t)pid * c.page + (t - pi * c.page);
}

// Length of sequence b inside what the call was told to cover.
__device__ __forceinline__ int mla_len(const int32_t *lens, int b, int max_kv, uint32_t *status) {
    const int n = lens[b];
    if (n < 0 || n > max_kv) {
        raise_status(status, ST_BADPAGE);
        return n < 0 ? 0 : max_kv;
    }
    return n;
}

__device__ __forceinline__ float wave_sum(float v) {
    for (int o = 32; o; o >>= 1) v += __shfl_xor(v, o);
    return v;
}

}  // namespace coli

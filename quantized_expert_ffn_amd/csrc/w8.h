// Private interface between the 8-bit product entry points and their kernels:
// arguments (passed by value) and launchers.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "coli_w8.h"

namespace coli {

struct W8QuantizeArgs {
    const void *x;
    int8_t *codes;
    float *scale;
    int64_t stride;   // bytes
    int tokens, k;
};
hipError_t launch_w8_quantize(const W8QuantizeArgs &a, int dtype, hipStream_t st);

struct W8LinearArgs {
    const int8_t *x, *w;
    const float *x_scale, *w_scale, *bias;
    void *out;
    int64_t x_stride, o_stride;
    int tokens, k, n_out;
};
hipError_t launch_w8_linear(const W8LinearArgs &a, int dtype, hipStream_t st);

// Calls f with a value of the element type of `dtype`.
template <class F>
hipError_t w8_with_type(int dtype, F f) {
    return dtype == COLI_BF16 ? f(__bf16()) : dtype == COLI_FP16 ? f(_Float16()) : f(float());
}

}  // namespace coli

// Products of 8-bit codes with scales for each token and output channel
// (coli_w8_linear): out[t, o] = s_t s_o sum_k q_tk w_ok + bias_o.
//
// v_mfma_i32_32x32x32_i8 with the channels as its rows and the tokens as its
// columns: a wavefront takes 32 of each, its operands straight from memory.
#include "kernels.h"
#include "mfma.h"
#include "w8.h"

namespace coli {
namespace {

template <class T>
__global__ __launch_bounds__(256) void k_w8_linear(W8LinearArgs a) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, n = lane & 31, hf = lane >> 5;
    const int across = (a.n_out + 127) / 128;
    const int o0 = (blockIdx.x % across * 4 + wave) * 32, t0 = blockIdx.x / across * 32;
    if (o0 >= a.n_out) return;
    const int8_t *w = a.w + (int64_t)min(o0 + n, a.n_out - 1) * a.k;
    const int8_t *x = a.x + (int64_t)min(t0 + n, a.tokens - 1) * a.x_stride;
    i32x16 acc = {0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0};
    for (int k = 0; k < a.k; k += 32) {
        i32x4 av = {0, 0, 0, 0}, bv = {0, 0, 0, 0};
        if (k + 16 * hf < a.k) {
            av = *reinterpret_cast<const i32x4 *>(w + k + 16 * hf);
            bv = *reinterpret_cast<const i32x4 *>(x + k + 16 * hf);
        }
        acc = __builtin_amdgcn_mfma_i32_32x32x32_i8(av, bv, acc, 0, 0, 0);
    }
    const int t = t0 + n;
    if (t >= a.tokens) return;
    const float s = a.x_scale[t];
    T *out = static_cast<T *>(a.out) + (int64_t)t * a.o_stride;
#pragma unroll
    for (int r = 0; r < 16; ++r) {
        const int o = o0 + 8 * (r / 4) + 4 * hf + r % 4;
        if (o < a.n_out) {
            float v = (float)acc[r] * s * a.w_scale[o];
            if (a.bias) v += a.bias[o];
            out[o] = (T)v;
        }
    }
}

}  // namespace

hipError_t launch_w8_linear(const W8LinearArgs &a, int dtype, hipStream_t st) {
    return w8_with_type(dtype, [&](auto t) {
        const int64_t grid = (int64_t)((a.n_out + 127) / 128) * ((a.tokens + 31) / 32);
        if (grid > INT32_MAX) return hipErrorInvalidConfiguration;
        hipLaunchKernelGGL(k_w8_linear<decltype(t)>, dim3((uint32_t)grid), dim3(256), 0, st, a);
        return hipGetLastError();
    });
}

}  // namespace coli

// A token's activations as 8-bit codes and one scale (coli_w8_quantize).
#include "device_common.h"
#include "kernels.h"
#include "w8.h"

namespace coli {
namespace {

// Sixteen values of T in binary32.
template <class T>
__device__ __forceinline__ void load16(const void *p, float (&v)[16]) {
    typedef T vec __attribute__((ext_vector_type(16 / sizeof(T))));
    constexpr int N = 16 / sizeof(T);
#pragma unroll
    for (int i = 0; i < 16 / N; ++i) {
        const vec x = static_cast<const vec *>(p)[i];
#pragma unroll
        for (int j = 0; j < N; ++j) v[N * i + j] = (float)x[j];
    }
}

// The code of x by the scale s > 0, inv = 1 / s: the integer next to x / s,
// ties to even.  x * inv is off by less than 2^-16 of a step, so its integer r
// is one of the quotient's two neighbours, and x - r s, which fma forms
// exactly (a multiple of half a unit of s, at most s), says which.
__device__ __forceinline__ int code(float x, float s, float inv) {
    const float r = __builtin_rintf(x * inv), t = 2.0f * __builtin_fmaf(-r, s, x);
    int c = (int)r;
    const bool odd = c & 1;
    if (t > s || (t == s && odd)) ++c;
    if (t < -s || (t == -s && odd)) --c;
    return min(max(c, -127), 127);
}

template <class T>
__global__ __launch_bounds__(256) void k_w8_quantize(W8QuantizeArgs a) {
    __shared__ uint32_t part[4];
    const int tid = threadIdx.x, chunks = a.k / 16;
    const uint8_t *row = static_cast<const uint8_t *>(a.x) + blockIdx.x * a.stride;
    // the largest magnitude, as bits: above every number stand the infinities, then NaN
    uint32_t top = 0;
    for (int c = tid; c < chunks; c += 256) {
        float v[16];
        load16<T>(row + (int64_t)c * 16 * sizeof(T), v);
#pragma unroll
        for (int i = 0; i < 16; ++i) top = max(top, __float_as_uint(v[i]) & 0x7fffffffu);
    }
    for (int o = 32; o; o >>= 1) top = max(top, (uint32_t)__shfl_xor((int)top, o));
    if ((tid & 63) == 0) part[tid >> 6] = top;
    __syncthreads();
    top = max(max(part[0], part[1]), max(part[2], part[3]));
    const bool bad = top >= 0x7f800000u;
    const float s = bad ? __uint_as_float(0x7fc00000u) : __uint_as_float(top) / 127.0f;
    if (tid == 0) a.scale[blockIdx.x] = s;
    // Scales whose reciprocal binary32 does not hold: both sides 2^64 larger, which is exact.
    const float lift = s < 0x1p-60f ? 0x1p64f : 1.0f, sl = s * lift, inv = 1.0f / sl;
    int8_t *out = a.codes + (int64_t)blockIdx.x * a.k;
    for (int c = tid; c < chunks; c += 256) {
        float v[16];
        load16<T>(row + (int64_t)c * 16 * sizeof(T), v);
        u32x4 w = {0, 0, 0, 0};
        if (s > 0.0f) {
#pragma unroll
            for (int i = 0; i < 16; ++i) w[i / 4] |= (uint32_t)(code(v[i] * lift, sl, inv) & 0xff) << (8 * (i % 4));
        }
        *reinterpret_cast<u32x4 *>(out + 16 * c) = w;
    }
}

}  // namespace

hipError_t launch_w8_quantize(const W8QuantizeArgs &a, int dtype, hipStream_t st) {
    return w8_with_type(dtype, [&](auto t) {
        hipLaunchKernelGGL(k_w8_quantize<decltype(t)>, dim3(a.tokens), dim3(256), 0, st, a);
        return hipGetLastError();
    });
}

}  // namespace coli

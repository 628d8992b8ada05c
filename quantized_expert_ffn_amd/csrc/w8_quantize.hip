// A token's activations as 8-bit codes and one scale (coli_w8_quantize).
#include "device_common.h"
#include "kernels.h"
#include "w8.h"

namespace coli {
namespace {

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

// A workgroup has a token, whose values stay in registers between the pass for
// their largest and the one for their codes: read once, 16 bytes a lane, all
// lanes in a row.  What bounds it is memory: 8191 x 6144 in binary32, 252 MB,
// takes 45.4 us, 5.55 TB/s; with the values read again for their codes, and a
// lane's codes apart from its neighbours', 61.9.  One token takes a launch and
// one round trip to memory, 3.8 us.
template <class T, int UNITS>
__global__ __launch_bounds__(1024) void k_w8_quantize(W8QuantizeArgs a) {
    constexpr int N = 16 / sizeof(T);
    typedef T vec __attribute__((ext_vector_type(N)));
    __shared__ uint32_t part[16];
    const int tid = threadIdx.x, threads = blockDim.x, units = a.k / N;
    const vec *row = reinterpret_cast<const vec *>(static_cast<const uint8_t *>(a.x) + blockIdx.x * a.stride);
    vec v[UNITS];
#pragma unroll
    for (int i = 0; i < UNITS; ++i) v[i] = row[min(tid + i * threads, units - 1)];   // behind the end: the last again
    // the largest magnitude, as bits: above every number stand the infinities, then NaN
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < UNITS; ++i)
#pragma unroll
        for (int j = 0; j < N; ++j) top = max(top, __float_as_uint((float)v[i][j]) & 0x7fffffffu);
    for (int o = 32; o; o >>= 1) top = max(top, (uint32_t)__shfl_xor((int)top, o));
    if (threads > 64) {
        if ((tid & 63) == 0) part[tid >> 6] = top;
        __syncthreads();
        for (int w = 0; w < threads >> 6; ++w) top = max(top, part[w]);
    }
    const bool bad = top >= 0x7f800000u;
    const float s = bad ? __uint_as_float(0x7fc00000u) : __uint_as_float(top) / 127.0f;
    if (tid == 0) a.scale[blockIdx.x] = s;
    // Scales whose reciprocal binary32 does not hold: both sides 2^64 larger, which is exact.
    const float lift = s < 0x1p-60f ? 0x1p64f : 1.0f, sl = s * lift, inv = 1.0f / sl;
    uint32_t *out = reinterpret_cast<uint32_t *>(a.codes + (int64_t)blockIdx.x * a.k);
#pragma unroll
    for (int i = 0; i < UNITS; ++i) {
        const int u = tid + i * threads;
        if (u >= units) continue;
        uint32_t w[N / 4] = {};
        if (s > 0.0f) {
#pragma unroll
            for (int j = 0; j < N; ++j) w[j / 4] |= (uint32_t)(code((float)v[i][j] * lift, sl, inv) & 0xff) << (8 * (j % 4));
        }
#pragma unroll
        for (int j = 0; j < N / 4; ++j) out[u * (N / 4) + j] = w[j];
    }
}

template <class T, int UNITS>
hipError_t quantize(W8QuantizeArgs a, int units, hipStream_t st) {
    const int threads = (((units + UNITS - 1) / UNITS + 63) & ~63);
    const int most = 1 << 21;   // tokens of a launch, whose threads are to be fewer than 2^32
    for (int left = a.tokens; left > 0; left -= most) {
        hipLaunchKernelGGL((k_w8_quantize<T, UNITS>), dim3(min(left, most)), dim3(threads), 0, st, a);
        a.x = static_cast<const uint8_t *>(a.x) + most * a.stride;
        a.codes += (int64_t)most * a.k;
        a.scale += most;
    }
    return hipGetLastError();
}

}  // namespace

// Four units of 16 bytes a thread, up to 1024 threads; 16 for longer rows.
hipError_t launch_w8_quantize(const W8QuantizeArgs &a, int dtype, hipStream_t st) {
    return w8_with_type(dtype, [&](auto t) {
        using T = decltype(t);
        const int units = a.k / (16 / (int)sizeof(T));
        return units <= 4096 ? quantize<T, 4>(a, units, st) : quantize<T, 16>(a, units, st);
    });
}

}  // namespace coli

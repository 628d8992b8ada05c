// Products with the latent projections: project (per head) and expand (all
// heads, rows gathered from the paged cache).
#include "mla_common.h"

namespace coli {
namespace {

template <class T>
__global__ __launch_bounds__(256) void k_mla_project(MlaProjectArgs a) {
    const int o = blockIdx.x * 256 + threadIdx.x, h = blockIdx.y;
    if (o >= a.n_out) return;
    const T *w = static_cast<const T *>(a.w) + ((int64_t)h * a.n_out + o) * a.n_in;
    for (int t = blockIdx.z; t < a.tokens; t += gridDim.z) {
        const T *x = static_cast<const T *>(a.x) + t * a.x_ts + h * a.x_hs;
        float s = 0.0f;
        for (int k = 0; k < a.n_in; k += 8) {
            const x8<T> u = *reinterpret_cast<const x8<T> *>(x + k), v = *reinterpret_cast<const x8<T> *>(w + k);
#pragma unroll
            for (int i = 0; i < 8; ++i) s = __builtin_fmaf((float)u[i], (float)v[i], s);
        }
        static_cast<T *>(a.out)[((int64_t)t * a.heads + h) * a.n_out + o] = (T)s;
    }
}

template <class T, bool FP8>
__global__ __launch_bounds__(256) void k_mla_expand(MlaExpandArgs a, int rank) {
    __shared__ float c[512];
    const int r = blockIdx.y, tid = threadIdx.x;
    int b = 0;
    while (b < a.batch && a.cu_k[b + 1] <= r) ++b;
    if (b == a.batch) return;
    const int t = r - a.cu_k[b];
    if (t < 0 || t >= a.c.width * a.c.page) {
        raise_status(a.status, ST_BADPAGE);
        return;
    }
    const int64_t slot = mla_slot(a.c, b, t, a.status);
    const int row = FP8 ? rank + 2 * MLA_ROPE : 2 * (rank + MLA_ROPE);
    const uint8_t *src = a.c.pages + slot * row;
    for (int i = tid; i < rank; i += 256)
        c[i] = FP8 ? fp8_to_f32(src[i]) : (float)reinterpret_cast<const T *>(src)[i];
    const float scale = FP8 ? a.c.scale[slot] : 1.0f;
    if (blockIdx.x == 0 && tid < MLA_ROPE)
        static_cast<T *>(a.k_pe)[(int64_t)r * MLA_ROPE + tid] =
            reinterpret_cast<const T *>(src + (FP8 ? rank : 2 * rank))[tid];
    __syncthreads();
    const int o = blockIdx.x * 256 + tid;
    if (o >= a.n_out) return;
    const T *w = static_cast<const T *>(a.w) + (int64_t)o * rank;
    float s = 0.0f;
    for (int k = 0; k < rank; k += 8) {
        const x8<T> v = *reinterpret_cast<const x8<T> *>(w + k);
#pragma unroll
        for (int i = 0; i < 8; ++i) s = __builtin_fmaf(c[k + i], (float)v[i], s);
    }
    static_cast<T *>(a.kv)[(int64_t)r * a.n_out + o] = (T)(s * scale);
}

}  // namespace

hipError_t launch_mla_project(const MlaProjectArgs &a, int dtype, hipStream_t st) {
    const dim3 grid((a.n_out + 255) / 256, a.heads, a.tokens < 256 ? a.tokens : 256);
    return mla_with_type(dtype, [&](auto t) {
        hipLaunchKernelGGL((k_mla_project<decltype(t)>), grid, dim3(256), 0, st, a);
        return hipGetLastError();
    });
}

hipError_t launch_mla_expand(const MlaExpandArgs &a, const coli_mla_dims &d, hipStream_t st) {
    const dim3 grid((a.n_out + 255) / 256, a.rows);
    return mla_with_type(d.dtype, [&](auto t) {
        using T = decltype(t);
        if (d.kv_format == COLI_KV_E4M3)
            hipLaunchKernelGGL((k_mla_expand<T, true>), grid, dim3(256), 0, st, a, d.rank);
        else
            hipLaunchKernelGGL((k_mla_expand<T, false>), grid, dim3(256), 0, st, a, d.rank);
        return hipGetLastError();
    });
}

}  // namespace coli

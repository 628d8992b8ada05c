// Attention of prompts over expanded keys and values.  One pass over the
// keys with the running maximum and sum of the softmax; a wavefront takes
// one (query, head).
#include "mla_common.h"

namespace coli {
namespace {

template <class T, int NOPE, int V>
__global__ __launch_bounds__(256) void k_mla_prefill(MlaPrefillArgs a) {
    constexpr int KP = NOPE / 64, VP = V / 64;
    const int lane = threadIdx.x & 63, i = blockIdx.x * 4 + (threadIdx.x >> 6), h = blockIdx.y, b = blockIdx.z;
    const int q0 = a.cu_q[b], n = a.cu_q[b + 1] - q0, k0 = a.cu_k[b], m_keys = a.cu_k[b + 1] - k0;
    if (q0 < 0 || n < 0 || q0 + n > a.n_q_rows || n > a.max_q || k0 < 0 || m_keys < 0 || k0 + m_keys > a.n_k_rows) {
        if (threadIdx.x == 0) raise_status(a.status, ST_BADPAGE);
        return;
    }
    if (i >= n) return;
    const int seen = a.causal ? min(m_keys, i + m_keys - n + 1) : m_keys;
    const T *q = static_cast<const T *>(a.q) + (q0 + i) * a.q_ts + h * a.q_hs;
    float qn[KP], o[VP];
    for (int x = 0; x < KP; ++x) qn[x] = (float)q[64 * x + lane];
    for (int x = 0; x < VP; ++x) o[x] = 0.0f;
    const float qp = (float)q[NOPE + lane];
    float m = -__builtin_inff(), l = 0.0f;
    for (int t = 0; t < seen; ++t) {
        const T *k = static_cast<const T *>(a.k_nope) + (k0 + t) * a.k_ts + h * a.k_hs;
        const T *v = static_cast<const T *>(a.v) + (k0 + t) * a.v_ts + h * a.v_hs;
        float s = qp * (float)static_cast<const T *>(a.k_pe)[(int64_t)(k0 + t) * MLA_ROPE + lane];
        for (int x = 0; x < KP; ++x) s = __builtin_fmaf(qn[x], (float)k[64 * x + lane], s);
        s = wave_sum(s) * a.scale;
        const float top = fmaxf(m, s), f = expf(m - top), p = expf(s - top);
        l = l * f + p;
        for (int x = 0; x < VP; ++x) o[x] = o[x] * f + p * (float)v[64 * x + lane];
        m = top;
    }
    const int64_t row = (int64_t)(q0 + i) * a.heads + h;
    for (int x = 0; x < VP; ++x) static_cast<T *>(a.out)[row * V + 64 * x + lane] = (T)(seen > 0 ? o[x] / l : 0.0f);
    if (a.lse && lane == 0) a.lse[row] = seen > 0 ? m + logf(l) : -__builtin_inff();
}

}  // namespace

hipError_t launch_mla_prefill(const MlaPrefillArgs &a, const coli_mla_dims &d, hipStream_t st) {
    const dim3 grid((a.max_q + 3) / 4, a.heads, a.batch);
    return mla_with_type(d.dtype, [&](auto t) {
        using T = decltype(t);
        if (d.nope == 128)
            hipLaunchKernelGGL((k_mla_prefill<T, 128, 128>), grid, dim3(256), 0, st, a);
        else
            hipLaunchKernelGGL((k_mla_prefill<T, 192, 256>), grid, dim3(256), 0, st, a);
        return hipGetLastError();
    });
}

}  // namespace coli

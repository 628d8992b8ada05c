// Absorbed attention of a few new tokens a sequence over the paged latents.
// One pass over the tokens with the running maximum and sum of the softmax:
// a workgroup takes one (query, head), its wavefronts every fourth token, and
// their four results are joined at the end.
#include "mla_common.h"

namespace coli {
namespace {

template <class T, int RANK, bool FP8>
__global__ __launch_bounds__(256) void k_mla_decode(MlaDecodeArgs a) {
    __shared__ float so[4][RANK];
    __shared__ float sm[4], sl[4];
    constexpr int PER = RANK / 64, ROW = FP8 ? RANK + 2 * MLA_ROPE : 2 * (RANK + MLA_ROPE);
    const int64_t row = (int64_t)blockIdx.x * a.heads + blockIdx.y;
    const int b = blockIdx.x / a.n_q, j = blockIdx.x % a.n_q, lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int seen = mla_len(a.kv_lens, b, a.max_kv, a.status) - a.n_q + 1 + j;
    float q[PER], o[PER];
    for (int i = 0; i < PER; ++i) {
        q[i] = (float)static_cast<const T *>(a.q_lat)[row * RANK + PER * lane + i];
        o[i] = 0.0f;
    }
    const float qp = (float)static_cast<const T *>(a.q_pe)[row * MLA_ROPE + lane];
    float m = -__builtin_inff(), l = 0.0f;
    for (int t = wave; t < seen; t += 4) {
        const int64_t slot = mla_slot(a.c, b, t, a.status);
        const uint8_t *src = a.c.pages + slot * ROW;
        float c[PER];
        for (int i = 0; i < PER; ++i)
            c[i] = FP8 ? fp8_to_f32(src[PER * lane + i]) * a.c.scale[slot]
                       : (float)reinterpret_cast<const T *>(src)[PER * lane + i];
        float s = qp * (float)reinterpret_cast<const T *>(src + (FP8 ? RANK : 2 * RANK))[lane];
        for (int i = 0; i < PER; ++i) s = __builtin_fmaf(q[i], c[i], s);
        s = wave_sum(s) * a.scale;
        const float top = fmaxf(m, s), f = expf(m - top), p = expf(s - top);
        l = l * f + p;
        for (int i = 0; i < PER; ++i) o[i] = o[i] * f + p * c[i];
        m = top;
    }
    for (int i = 0; i < PER; ++i) so[wave][PER * lane + i] = o[i];
    if (lane == 0) {
        sm[wave] = m;
        sl[wave] = l;
    }
    __syncthreads();
    const float top = fmaxf(fmaxf(sm[0], sm[1]), fmaxf(sm[2], sm[3]));
    float f[4], total = 0.0f;
    for (int w = 0; w < 4; ++w) {
        f[w] = sm[w] == -__builtin_inff() ? 0.0f : expf(sm[w] - top);
        total += f[w] * sl[w];
    }
    for (int i = threadIdx.x; i < RANK; i += 256) {
        float v = 0.0f;
        for (int w = 0; w < 4; ++w) v += f[w] * so[w][i];
        static_cast<T *>(a.out)[row * RANK + i] = (T)(seen > 0 ? v / total : 0.0f);
    }
    if (a.lse && threadIdx.x == 0) a.lse[row] = seen > 0 ? top + logf(total) : -__builtin_inff();
}

}  // namespace

size_t mla_decode_part_bytes(const coli_mla_dims &, int, int, int) { return 0; }

hipError_t launch_mla_decode(const MlaDecodeArgs &a, const coli_mla_dims &d, hipStream_t st) {
    const dim3 grid(a.batch * a.n_q, a.heads);
    return mla_with_type(d.dtype, [&](auto t) {
        using T = decltype(t);
        const bool fp8 = d.kv_format == COLI_KV_E4M3;
        if (d.rank == 512 && fp8) hipLaunchKernelGGL((k_mla_decode<T, 512, true>), grid, dim3(256), 0, st, a);
        if (d.rank == 512 && !fp8) hipLaunchKernelGGL((k_mla_decode<T, 512, false>), grid, dim3(256), 0, st, a);
        if (d.rank == 256 && fp8) hipLaunchKernelGGL((k_mla_decode<T, 256, true>), grid, dim3(256), 0, st, a);
        if (d.rank == 256 && !fp8) hipLaunchKernelGGL((k_mla_decode<T, 256, false>), grid, dim3(256), 0, st, a);
        return hipGetLastError();
    });
}

}  // namespace coli

// Append: RMS norm of the latent, rotation of the shared key and of the
// queries, and the write into the paged cache.
//
//   c = a / sqrt(mean(a^2) + eps) * g,  r_i = (x_i + j y_i) e^{j position f_i}
//
// One workgroup a token.  The first wavefront takes the latent (rank / 64
// values a lane) and the key while the second forms the token's 32 angles,
// reduced to a turn in 64 bits: a position of 1e5 times a frequency near one
// has no fraction left in binary32.  All wavefronts then rotate the queries,
// sixteen values (eight pairs) a thread.
//
// What bounds it: bytes, of which the queries' are the most: 8191 tokens, 64
// heads, E4M3 latents: 26 us and 149 MB, 5.7 TB/s, from a warm cache, 36 us
// from a cold one; one token: 2.7 us.
#include "mla_common.h"

namespace coli {
namespace {

constexpr int APPEND_THREADS = 256;

// Sixteen values of a head, pairs i0 .. i0 + 7: contiguous for PAIRS, two
// runs of eight, 32 apart, for HALVES.
template <class T, bool HALVES>
__device__ __forceinline__ void rotate16(const T *src, T *dst, const float2 *cs, int u) {
    const int lo = HALVES ? 8 * u : 16 * u, hi = HALVES ? 32 + 8 * u : 16 * u + 8;
    const x8<T> a = *reinterpret_cast<const x8<T> *>(src + lo);
    const x8<T> b = *reinterpret_cast<const x8<T> *>(src + hi);
    x8<T> p, q;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float2 e = cs[8 * u + i];
        if (HALVES) {
            const float x = (float)a[i], y = (float)b[i];
            p[i] = (T)__builtin_fmaf(x, e.x, -(y * e.y));
            q[i] = (T)__builtin_fmaf(y, e.x, x * e.y);
        } else {
            const float x = i < 4 ? (float)a[2 * i] : (float)b[2 * i - 8];
            const float y = i < 4 ? (float)a[2 * i + 1] : (float)b[2 * i - 7];
            const T s = (T)__builtin_fmaf(x, e.x, -(y * e.y)), t = (T)__builtin_fmaf(y, e.x, x * e.y);
            if (i < 4) {
                p[2 * i] = s;
                p[2 * i + 1] = t;
            } else {
                q[2 * i - 8] = s;
                q[2 * i - 7] = t;
            }
        }
    }
    *reinterpret_cast<x8<T> *>(dst + lo) = p;
    *reinterpret_cast<x8<T> *>(dst + hi) = q;
}

template <class T, int RANK, bool FP8, bool HALVES>
__global__ __launch_bounds__(APPEND_THREADS) void k_mla_append(MlaAppendArgs a) {
    __shared__ float2 cs[MLA_ROPE / 2];
    const int t = blockIdx.x, tid = threadIdx.x, lane = tid & 63;
    constexpr int PER = RANK / 64;           // latent values a lane
    constexpr int ROW = FP8 ? RANK + 2 * MLA_ROPE : 2 * (RANK + MLA_ROPE);
    if (tid >= 64 && tid < 64 + MLA_ROPE / 2) {
        const int i = tid - 64;
        double turns = (double)a.positions[t] * a.inv_freq[i] * 0.15915494309189533577;   // 1 / (2 pi)
        turns -= rint(turns);
        float s, c;
        sincosf((float)(turns * 6.283185307179586477), &s, &c);
        cs[i] = make_float2(c, s);
    }
    const int64_t slot = a.slots[t];
    const bool store = slot >= 0 && slot < a.n_slots;
    const T *x = static_cast<const T *>(a.kv_a) + (int64_t)t * (RANK + MLA_ROPE);
    uint8_t *row = a.pages + (store ? slot : 0) * (int64_t)ROW;
    if (tid < 64) {
        if (slot >= a.n_slots && lane == 0) raise_status(a.status, ST_BADPAGE);
        typedef T vec __attribute__((ext_vector_type(PER)));
        const vec raw = *reinterpret_cast<const vec *>(x + PER * lane);
        float v[PER];
#pragma unroll
        for (int i = 0; i < PER; ++i) v[i] = (float)raw[i];
        if (a.norm_w) {
            float ss = 0.0f;
#pragma unroll
            for (int i = 0; i < PER; ++i) ss = __builtin_fmaf(v[i], v[i], ss);
            const float r = 1.0f / sqrtf(wave_sum(ss) * (1.0f / RANK) + a.eps);
            const vec g = *reinterpret_cast<const vec *>(static_cast<const T *>(a.norm_w) + PER * lane);
#pragma unroll
            for (int i = 0; i < PER; ++i) v[i] = v[i] * r * (float)g[i];
        }
        if (FP8) {
            // the largest magnitude as an integer: a NaN's bits lie above infinity's, so it comes through
            uint32_t top = 0;
#pragma unroll
            for (int i = 0; i < PER; ++i) top = max(top, __float_as_uint(v[i]) & 0x7fffffffu);
            for (int o = 32; o; o >>= 1) top = max(top, (uint32_t)__shfl_xor((int)top, o));
            const float s = __uint_as_float(top) / 448.0f;
            uint32_t code[PER / 4];
#pragma unroll
            for (int i = 0; i < PER; i += 4) {
                float q[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    q[j] = s > 0.0f ? v[i + j] / s : 0.0f;
                    // a scale below the normal numbers is so coarse that quotients pass the largest code (NaN stays)
                    if (fabsf(q[j]) > 448.0f) q[j] = copysignf(448.0f, q[j]);
                }
                int w = __builtin_amdgcn_cvt_pk_fp8_f32(q[0], q[1], 0, false);
                code[i / 4] = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(q[2], q[3], w, true);
            }
            if (store) {
#pragma unroll
                for (int i = 0; i < PER / 4; ++i) reinterpret_cast<uint32_t *>(row)[lane * (PER / 4) + i] = code[i];
                if (lane == 0) a.kv_scale[slot] = s;
            }
        } else if (store) {
            vec o;
#pragma unroll
            for (int i = 0; i < PER; ++i) o[i] = (T)v[i];
            *reinterpret_cast<vec *>(row + 2 * PER * lane) = o;
        }
    }
    __syncthreads();
    if (store && tid < 4)
        rotate16<T, HALVES>(x + RANK, reinterpret_cast<T *>(row + (FP8 ? RANK : 2 * RANK)), cs, tid);
    for (int u = tid; u < 4 * a.heads; u += APPEND_THREADS) {
        const int h = u >> 2;
        rotate16<T, HALVES>(static_cast<const T *>(a.q_pe) + t * a.q_ts + h * a.q_hs,
                            static_cast<T *>(a.q_out) + t * a.o_ts + h * a.o_hs, cs, u & 3);
    }
}

template <class T, int RANK, bool FP8>
hipError_t launch(const MlaAppendArgs &a, bool halves, hipStream_t st) {
    if (halves)
        hipLaunchKernelGGL((k_mla_append<T, RANK, FP8, true>), dim3(a.tokens), dim3(APPEND_THREADS), 0, st, a);
    else
        hipLaunchKernelGGL((k_mla_append<T, RANK, FP8, false>), dim3(a.tokens), dim3(APPEND_THREADS), 0, st, a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_mla_append(const MlaAppendArgs &a, const coli_mla_dims &d, hipStream_t st) {
    const bool fp8 = d.kv_format == COLI_KV_E4M3, halves = d.rope_style == COLI_ROPE_HALVES;
    return mla_with_type(d.dtype, [&](auto t) {
        using T = decltype(t);
        if (d.rank == 512) return fp8 ? launch<T, 512, true>(a, halves, st) : launch<T, 512, false>(a, halves, st);
        return fp8 ? launch<T, 256, true>(a, halves, st) : launch<T, 256, false>(a, halves, st);
    });
}

}  // namespace coli

// Routing from logits (coli_moe_select): scores, groups, top-k, weights.
//
// Scores and choices are formed in binary64, so that experts are ranked by
// what their choices are; a wavefront takes a token, a lane every 64th expert.
#include "device_common.h"
#include "kernels.h"

namespace coli {
namespace {

__device__ __forceinline__ double wave_sum64(double v) {
    for (int o = 32; o; o >>= 1) v += __shfl_xor(v, o);
    return v;
}
__device__ __forceinline__ double wave_max64(double v) {
    for (int o = 32; o; o >>= 1) v = fmax(v, __shfl_xor(v, o));
    return v;
}

template <class T>
__global__ __launch_bounds__(64) void k_select(SelectArgs a) {
    extern __shared__ double lds[];
    double *score = lds, *choice = lds + a.experts, *best = lds + 2 * a.experts;
    const int lane = threadIdx.x, size = a.experts / a.groups;
    const T *row = static_cast<const T *>(a.logits) + blockIdx.x * a.stride;
    bool bad = false;
    double top = -__builtin_inf();
    for (int e = lane; e < a.experts; e += 64) {
        float l = (float)row[e];
        if (!finite_f32(l)) {
            bad = true;
            l = 0.0f;
        }
        score[e] = l;
        top = fmax(top, (double)l);
    }
    double scale = 1.0;
    if (a.softmax) {
        top = wave_max64(top);
        double sum = 0.0;
        for (int e = lane; e < a.experts; e += 64) sum += exp(score[e] - top);
        scale = 1.0 / wave_sum64(sum);
    }
    for (int e = lane; e < a.experts; e += 64) {
        const double l = score[e], s = a.softmax ? exp(l - top) * scale : 1.0 / (1.0 + exp(-l));
        float b = a.bias ? a.bias[e] : 0.0f;
        if (!finite_f32(b)) {
            bad = true;
            b = 0.0f;
        }
        score[e] = s;
        choice[e] = s + b;
    }
    __syncthreads();
    uint64_t open = ~0ull;
    if (a.topk_group < a.groups) {
        if (lane < a.groups) {
            double first = -__builtin_inf(), second = -__builtin_inf();
            for (int e = lane * size; e < (lane + 1) * size; ++e) {
                const double c = choice[e];
                second = fmax(second, fmin(first, c));
                first = fmax(first, c);
            }
            best[lane] = a.top2 && size > 1 ? first + second : first;
        }
        __syncthreads();
        int before = 0;
        if (lane < a.groups)
            for (int g = 0; g < a.groups; ++g) before += best[g] > best[lane] || (best[g] == best[lane] && g < lane);
        open = __ballot(lane < a.groups && before < a.topk_group);
    }
    double mine = 0.0, sum = 0.0;
    int mine_e = 0;
    for (int k = 0; k < a.top_k; ++k) {
        double c = -__builtin_inf();
        int at = a.experts;
        for (int e = lane; e < a.experts; e += 64)
            if ((open >> (e / size) & 1) && choice[e] > c) {
                c = choice[e];
                at = e;
            }
        for (int o = 32; o; o >>= 1) {
            const double oc = __shfl_xor(c, o);
            const int oa = __shfl_xor(at, o);
            if (oc > c || (oc == c && oa < at)) {
                c = oc;
                at = oa;
            }
        }
        const double s = score[at];
        sum += s;
        if (lane == k) {
            mine = s;
            mine_e = at;
        }
        __syncthreads();
        if (lane == 0) choice[at] = -__builtin_inf();
        __syncthreads();
    }
    if (lane < a.top_k) {
        const float w = (float)((a.norm ? mine / sum : mine) * a.rsf);
        bad |= !finite_f32(w);
        const int64_t o = (int64_t)blockIdx.x * a.top_k + lane;
        a.idx[o] = mine_e;
        a.w[o] = w;
    }
    if (__ballot(bad) && lane == 0) raise_status(a.status, ST_NONFINITE);
}

}  // namespace

hipError_t launch_select(const SelectArgs &a, int dtype, hipStream_t st) {
    const size_t smem = (2 * a.experts + 64) * sizeof(double);
    auto go = [&](auto t) {
        hipLaunchKernelGGL(k_select<decltype(t)>, dim3(a.tokens), dim3(64), smem, st, a);
        return hipGetLastError();
    };
    return dtype == COLI_BF16 ? go(__bf16()) : dtype == COLI_FP16 ? go(_Float16()) : go(float());
}

}  // namespace coli

// Routing from logits (coli_moe_select): scores, groups, top-k, weights.
//
// Experts are to be chosen as in 64 bits, yet a sigmoid in binary64 for each of
// them would cost more than all else.  Choices are formed in binary32 first,
// with a bound on their error; experts that could be among the best K by it,
// hardly more than K, are ranked by choices in binary64.  Without a bias the
// order is the logits', which binary32 holds.  Where the bound leaves groups
// undecided, or too many experts (equal ones), the token is done over in
// binary64 by a whole wavefront.
//
// What bounds it: instructions.  A token has LANES lanes, each PER experts in a
// row: sixteen lanes where tokens are many, so that what goes across lanes is
// shared by four of them, a whole wavefront where they are few or the experts
// too many.
#include <type_traits>

#include "device_common.h"
#include "kernels.h"
#include "mla_mfma.h"

namespace coli {
namespace {

// A value of another lane of the same row of sixteen, N lanes on.
template <int N>
__device__ __forceinline__ float ror(float v) {
    return __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(v), 0x120 + N, 0xf, 0xf, true));
}
template <int N>
__device__ __forceinline__ double ror(double v) {
    const uint64_t b = __double_as_longlong(v);
    const uint32_t lo = __builtin_amdgcn_mov_dpp((int)(uint32_t)b, 0x120 + N, 0xf, 0xf, true);
    const uint32_t hi = __builtin_amdgcn_mov_dpp((int)(b >> 32), 0x120 + N, 0xf, 0xf, true);
    return __longlong_as_double((uint64_t)hi << 32 | lo);
}
// Reductions over a token's lanes, for all of them.
template <int LANES, class V, class F>
__device__ __forceinline__ V all_lanes(V v, F f) {
    v = f(v, ror<8>(v));
    v = f(v, ror<4>(v));
    v = f(v, ror<2>(v));
    v = f(v, ror<1>(v));
    if constexpr (LANES == 64) {
        v = f(v, __shfl_xor(v, 16));
        v = f(v, __shfl_xor(v, 32));
    }
    return v;
}
struct Max {
    template <class V>
    __device__ __forceinline__ V operator()(V a, V b) const { return a > b ? a : b; }
};
struct Min {
    template <class V>
    __device__ __forceinline__ V operator()(V a, V b) const { return a < b ? a : b; }
};
struct Add {
    template <class V>
    __device__ __forceinline__ V operator()(V a, V b) const { return a + b; }
};

// A wavefront's accesses to its own LDS before this, of whatever type, come
// before those after it.
__device__ __forceinline__ void wave_sync() {
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    __builtin_amdgcn_wave_barrier();
}

constexpr float LOG2E = 1.44269504088896340736f;

// The place of an expert's value in LDS, in words: runs of sixteen, four apart.
__device__ __forceinline__ int place(int e) { return e + (e >> 4) * 4; }
__host__ __device__ constexpr int row_words(int experts) { return (experts + 15) / 16 * 20; }
// Bytes of a wavefront's room in LDS: two rows of values a token, the second
// of which also holds one token's choices in binary64 and 64 groups' scores;
// then a candidate a lane, in 8 + 4 bytes.
__host__ __device__ constexpr size_t select_room(int lanes, int experts) {
    const size_t rows = (size_t)(64 / lanes) * row_words(experts) * 4, slow = 8 * ((size_t)experts + 64);
    return (rows + (rows > slow ? rows : slow) + 15) / 16 * 16 + 64 * 12;
}

// An expert's score in binary64.
__device__ __forceinline__ double score64(const SelectArgs &a, float l, float top, double inv_sum) {
    return a.softmax ? exp((double)l - top) * inv_sum : 1.0 / (1.0 + exp(-(double)l));
}

__device__ __forceinline__ float bias_of(const SelectArgs &a, int e) {
    const float b = a.bias ? a.bias[e] : 0.0f;
    return finite_f32(b) ? b : 0.0f;
}

// One token by a whole wavefront, all in binary64: `logit` its logits, `choice`
// room for as many choices and, behind them, 64 group scores.  Lane k gets the k-th
// expert.  What a choice is without a bias is left to the logits.
__device__ __forceinline__ int select_slow(const SelectArgs &a, const float *logit, double *choice, float top, double inv_sum) {
    const int lane = threadIdx.x & 63, size = a.experts / a.groups;
    double *best = choice + a.experts;
    wave_sync();
    for (int e = lane; e < a.experts; e += 64) choice[e] = score64(a, logit[place(e)], top, inv_sum) + bias_of(a, e);
    wave_sync();
    uint64_t open = ~0ull;
    if (a.topk_group < a.groups) {
        double group = 0.0;
        if (lane < a.groups) {
            double first = -__builtin_inf(), second = -__builtin_inf();
            for (int e = lane * size; e < (lane + 1) * size; ++e) {
                const double c = a.top2 || a.bias ? choice[e] : (double)logit[place(e)];
                second = fmax(second, fmin(first, c));
                first = fmax(first, c);
            }
            best[lane] = group = a.top2 && size > 1 ? first + second : first;
        }
        wave_sync();
        int before = 0;
        for (int g = 0; g < a.groups; ++g) before += best[g] > group || (best[g] == group && g < lane);
        open = __ballot(lane < a.groups && before < a.topk_group);
    }
    int chosen = 0;
    uint32_t mine = 0;   // bit i: this lane's expert lane + 64 i is taken
    for (int k = 0; k < a.top_k; ++k) {
        double c = -__builtin_inf();
        int at = a.experts;
        for (int i = 0, e = lane; e < a.experts; ++i, e += 64)
            if ((open >> (e / size) & 1) && !(mine >> i & 1)) {
                const double v = a.bias ? choice[e] : (double)logit[place(e)];
                if (v > c) {
                    c = v;
                    at = e;
                }
            }
        for (int o = 32; o; o >>= 1) {
            const double oc = __shfl_xor(c, o);
            const int oa = __shfl_xor(at, o);
            if (oc > c || (oc == c && oa < at)) {
                c = oc;
                at = oa;
            }
        }
        if ((at & 63) == lane) mine |= 1u << (at >> 6);
        if (lane == k) chosen = at;
    }
    return chosen;
}

template <class T, int LANES, int PER>
__global__ __launch_bounds__(256) void k_select(SelectArgs a, int vector) {
    constexpr int TOK = 64 / LANES, SUB = PER / 4;   // tokens a wavefront; experts a maximum stands for
    extern __shared__ double lds[];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, tok = lane / LANES, sub = lane % LANES;
    const int words = row_words(a.experts), size = a.experts / a.groups;
    // a wavefront's room: logits [TOK], approximate choices [TOK] (or one token's in binary64 and its groups'), candidates
    const size_t room = select_room(LANES, a.experts);
    char *mem = reinterpret_cast<char *>(lds) + wave * room;
    float *logit = reinterpret_cast<float *>(mem) + tok * words;
    char *second_row = mem + (size_t)TOK * words * 4;
    float *near = reinterpret_cast<float *>(second_row) + tok * words;
    double *cand_key = reinterpret_cast<double *>(mem + room - 64 * 12) + tok * LANES;
    int *cand = reinterpret_cast<int *>(mem + room - 64 * 4) + tok * LANES;

    const int64_t token = ((int64_t)blockIdx.x * (blockDim.x >> 6) + wave) * TOK + tok;
    if (token - tok >= a.tokens) return;
    const bool real = token < a.tokens;
    const T *row = static_cast<const T *>(a.logits) + (real ? token : a.tokens - 1) * a.stride;
    const int e0 = sub * PER;
    constexpr float NEG = -__builtin_inff();
    float key[PER];
    bool bad = false;
    if (vector) {   // whole runs, 16-byte aligned
        constexpr int N = sizeof(T) == 4 ? 4 : PER < 8 ? 4 : 8;
        typedef T vec __attribute__((ext_vector_type(N)));
#pragma unroll
        for (int i = 0; i < PER; i += N) {
            vec v;
            if (e0 + i < a.experts) v = *reinterpret_cast<const vec *>(row + e0 + i);
#pragma unroll
            for (int j = 0; j < N; ++j) key[i + j] = e0 + i < a.experts ? (float)v[j] : NEG;
        }
    } else {
#pragma unroll
        for (int i = 0; i < PER; ++i) key[i] = e0 + i < a.experts ? (float)row[e0 + i] : NEG;
    }
    float top = NEG;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        if (e0 + i < a.experts && !finite_f32(key[i])) {
            bad = true;
            key[i] = 0.0f;
        }
        top = fmaxf(top, key[i]);
    }
    if (e0 < a.experts) {
#pragma unroll
        for (int i = 0; i < PER; i += 4) *reinterpret_cast<f32x4 *>(logit + place(e0 + i)) = f32x4{key[i], key[i + 1], key[i + 2], key[i + 3]};
    }
    top = all_lanes<LANES>(top, Max());
    // ---- the softmax's sum, where something needs it: in renormalised weights without a bias it cancels
    double inv_sum = 1.0;
    if (a.softmax && (a.bias || !a.norm || (a.top2 && a.topk_group < a.groups))) {
        double sum = 0.0;
#pragma unroll
        for (int i = 0; i < PER; ++i)
            if (e0 + i < a.experts) sum += exp((double)key[i] - top);
        inv_sum = 1.0 / all_lanes<LANES>(sum, Add());
    }
    // ---- approximate choices, off by at most eps: a sigmoid by 2^-21 (0.2 of the exponential's relative error, sum and
    // quotient by a step each, the sum with the bias by half of one), a softmax by 2^-20 of the largest (the exponent by two
    // steps and a half of itself, d 2^-d < 1, the exponential and its product by a step each), and half a step of the bias
    const bool groups = a.topk_group < a.groups, approximate = a.bias || (groups && a.top2);
    float eps = 0.0f;
    if (approximate) {
        const float inv = (float)inv_sum;
        float most = 0.0f;
        float c[PER];
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int e = e0 + i;
            float b = 0.0f;
            if (a.bias && e < a.experts) {
                b = a.bias[e];
                if (!finite_f32(b)) {
                    bad = true;
                    b = 0.0f;
                }
            }
            most = fmaxf(most, fabsf(b));
            const float x = a.softmax ? __builtin_amdgcn_exp2f((key[i] - top) * LOG2E) * inv
                                      : __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-LOG2E * key[i]));
            c[i] = e < a.experts ? x + b : NEG;
        }
        eps = 0x1p-20f * (a.softmax ? inv : 0.5f) + 0x1p-22f * all_lanes<LANES>(most, Max());
        if (groups && e0 < a.experts) {
#pragma unroll
            for (int i = 0; i < PER; i += 4) *reinterpret_cast<f32x4 *>(near + place(e0 + i)) = f32x4{c[i], c[i + 1], c[i + 2], c[i + 3]};
        }
        if (a.bias) {
#pragma unroll
            for (int i = 0; i < PER; ++i) key[i] = c[i];
        }
    }
    wave_sync();
    // ---- groups: a lane each (there are at most LANES)
    bool slow = false;
    if (groups) {
        const float *from = approximate ? near : logit;
        float first = NEG, second = NEG;
        if (sub < a.groups)
            for (int e = sub * size; e < (sub + 1) * size; ++e) {
                const float v = from[place(e)];
                second = fmaxf(second, fminf(first, v));
                first = fmaxf(first, v);
            }
        const float mine = a.top2 && size > 1 ? first + second : first;
        int before = 0;
        for (int g = 0; g < a.groups; ++g) {
            const float other = __shfl(mine, lane - sub + g);
            before += other > mine || (other == mine && g < sub);
        }
        const bool in = sub < a.groups && before < a.topk_group;
        const uint64_t open = __ballot(in) >> (lane - sub);
        if (approximate) {
            const float least = all_lanes<LANES>(in ? mine : -NEG, Min()), next = all_lanes<LANES>(sub < a.groups && !in ? mine : NEG, Max());
            // sums of two are off by 2 eps and their own rounding
            slow = !(least - next > 4.0f * eps + 0x1p-22f * (fabsf(least) + fabsf(next)));
        }
        int g = e0 / size, rest = e0 - g * size;
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            if (!(open >> g & 1)) key[i] = NEG;
            if (++rest == size) {
                rest = 0;
                ++g;
            }
        }
    }
    // ---- a bound from below on the K-th best: the K-th of the maxima of SUB experts each
    float most[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        most[q] = key[SUB * q];
#pragma unroll
        for (int i = 1; i < SUB; ++i) most[q] = fmaxf(most[q], key[SUB * q + i]);
    }
    float bound = NEG;
    for (int k = 0; k < a.top_k; ++k) {
        const float mine = fmaxf(fmaxf(most[0], most[1]), fmaxf(most[2], most[3]));
        bound = all_lanes<LANES>(mine, Max());
        uint64_t has = __ballot(mine == bound);
        if (LANES < 64) has = has >> (lane - sub) & ((1ull << (LANES & 63)) - 1);
        if (sub == (int)__builtin_ctzll(has)) {   // of equal ones, one lane's at a time
            bool done = false;
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const bool it = !done && most[q] == bound;
                if (it) most[q] = NEG;
                done |= it;
            }
        }
    }
    // ---- candidates, in the order of their experts
    bound = a.bias ? bound - 2.0f * eps - 0x1p-22f * fabsf(bound) : bound;
    uint32_t mask = 0;
#pragma unroll
    for (int i = 0; i < PER; ++i)
        if (key[i] >= bound && key[i] > NEG) mask |= 1u << i;
    int count = __popc(mask), upto = count;
    upto = dpp_add<0x111, 0xf>(upto);
    upto = dpp_add<0x112, 0xf>(upto);
    upto = dpp_add<0x114, 0xf>(upto);
    upto = dpp_add<0x118, 0xf>(upto);
    if constexpr (LANES == 64) {
        upto = dpp_add<0x142, 0xa>(upto);
        upto = dpp_add<0x143, 0xc>(upto);
    }
    const int total = __shfl(upto, lane - sub + LANES - 1);
    slow |= total > LANES;
    for (int at = upto - count; mask && at < LANES; ++at) {
        const int i = __builtin_ctz(mask);
        mask &= mask - 1;
        cand[at] = e0 + i;
    }
    wave_sync();
    // ---- their scores, and their order by choices in binary64 (without a bias, by logits)
    int mine = sub < min(total, LANES) ? cand[sub] : -1;
    double score = 0.0, choice = -__builtin_inf();
    if (mine >= 0) {
        const float l = logit[place(mine)];
        score = score64(a, l, top, inv_sum);
        choice = a.bias ? score + bias_of(a, mine) : (double)l;
        cand_key[sub] = choice;
    }
    wave_sync();
    int rank = 0;
    const int longest = LANES == 64 ? total : (int)all_lanes<64>((float)total, Max());
    for (int i = 0; i < min(longest, LANES); ++i) {
        const double other = cand_key[i];
        rank += i < total && (other > choice || (other == choice && i < sub));
    }
    bool chosen = mine >= 0 && rank < a.top_k;
    // ---- tokens to be done over, one after the other
    uint64_t again = __ballot(slow && real && sub == 0);
    while (again) {
        const int at = __builtin_ctzll(again), its = at / LANES;
        again &= again - 1;
        const float its_top = __shfl(top, at);
        const double its_inv = __shfl(inv_sum, at);
        const int e = select_slow(a, reinterpret_cast<const float *>(mem) + its * words, reinterpret_cast<double *>(second_row), its_top, its_inv);
        // lane k's expert to the token's lane k; with sixteen lanes, K is at most that
        const int from = __shfl(e, sub);
        if (tok == its) {
            chosen = sub < a.top_k;
            mine = from;
            rank = sub;
            score = chosen ? score64(a, logit[place(mine)], top, inv_sum) : 0.0;
        }
    }
    const double sum = all_lanes<LANES>(chosen ? score : 0.0, Add());
    if (chosen && real) {
        const float w = (float)((a.norm ? score / sum : score) * a.rsf);
        bad |= !finite_f32(w);
        a.idx[token * a.top_k + rank] = mine;
        a.w[token * a.top_k + rank] = w;
    }
    if (__ballot(bad && real) && lane == 0) raise_status(a.status, ST_NONFINITE);
}

template <class T, int LANES, int PER>
hipError_t launch_shape(const SelectArgs &a, hipStream_t st) {
    constexpr int TOK = 64 / LANES;
    const size_t room = select_room(LANES, a.experts);
    int waves = a.tokens > 256 * TOK ? 4 : 1;
    const int64_t groups = (a.tokens + TOK - 1) / TOK;
    constexpr int N = sizeof(T) == 4 ? 4 : PER < 8 ? 4 : 8;
    const bool vector = a.experts % N == 0 && a.stride % N == 0 && reinterpret_cast<uintptr_t>(a.logits) % (N * sizeof(T)) == 0;
    const hipError_t e = ensure_dyn_smem(reinterpret_cast<const void *>(&k_select<T, LANES, PER>), room * waves);
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL((k_select<T, LANES, PER>), dim3((uint32_t)((groups + waves - 1) / waves)), dim3(64 * waves), room * waves, st, a,
                       (int)vector);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_select(const SelectArgs &a, int dtype, hipStream_t st) {
    auto go = [&](auto t) {
        using T = decltype(t);
        if (a.tokens >= 2048 && a.experts <= 256 && a.top_k <= 10 && a.groups <= 16)
            return a.experts <= 64 ? launch_shape<T, 16, 4>(a, st) : launch_shape<T, 16, 16>(a, st);
        return a.experts <= 256 ? launch_shape<T, 64, 4>(a, st) : launch_shape<T, 64, 16>(a, st);
    };
    return dtype == COLI_BF16 ? go(__bf16()) : dtype == COLI_FP16 ? go(_Float16()) : go(float());
}

}  // namespace coli

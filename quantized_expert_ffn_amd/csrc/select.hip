// Routing from logits (coli_moe_select): scores, groups, top-k, weights.
//
// Experts are to be chosen as in 64 bits, yet a sigmoid in binary64 for each of
// them would cost more than all else.  Choices are formed in binary32 first,
// with a bound on their error; experts that could be among the best K by it,
// hardly more than K, are ranked by choices in binary64.  Without a bias scores
// rise with the logits, which binary32 holds, and the bound is on what binary64
// rounds away (least_equal).  Where the bound leaves groups undecided, or too many
// experts (equal ones), the token is done over in binary64 by a whole wavefront.
//
// What bounds it: a launch where tokens are few (one token, 256 experts in 8
// groups: 5.9 us, of which 3.8 are a launch's), then instructions (16384 tokens
// of 256 experts, sigmoid with a bias, 4 of 8 groups: 12.0 to 12.7 us, 1.4 TB/s
// of logits, 16.8 MB).  A token has LANES lanes, each PER experts in a row:
// sixteen lanes where tokens are many, so that what goes across lanes is shared by
// four of them, a whole wavefront where they are few or the experts too many.
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
// This lane's value and that of the lane 16, or 32, away, in some order.
__device__ __forceinline__ void swap16(float v, float &a, float &b) {
    const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    a = __uint_as_float(r[0]), b = __uint_as_float(r[1]);
}
__device__ __forceinline__ void swap32(float v, float &a, float &b) {
    const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    a = __uint_as_float(r[0]), b = __uint_as_float(r[1]);
}
template <bool FAR>
__device__ __forceinline__ void swap64(double v, double &a, double &b) {
    const uint64_t u = __double_as_longlong(v);
    const uint32_t l = (uint32_t)u, h = (uint32_t)(u >> 32);
    const auto lo = FAR ? __builtin_amdgcn_permlane32_swap(l, l, false, false) : __builtin_amdgcn_permlane16_swap(l, l, false, false);
    const auto hi = FAR ? __builtin_amdgcn_permlane32_swap(h, h, false, false) : __builtin_amdgcn_permlane16_swap(h, h, false, false);
    a = __longlong_as_double((uint64_t)hi[0] << 32 | lo[0]), b = __longlong_as_double((uint64_t)hi[1] << 32 | lo[1]);
}
__device__ __forceinline__ void swap16(double v, double &a, double &b) { swap64<false>(v, a, b); }
__device__ __forceinline__ void swap32(double v, double &a, double &b) { swap64<true>(v, a, b); }
// Reductions over a token's lanes, for all of them.
template <int LANES, class V, class F>
__device__ __forceinline__ V all_lanes(V v, F f) {
    v = f(v, ror<8>(v));
    v = f(v, ror<4>(v));
    v = f(v, ror<2>(v));
    v = f(v, ror<1>(v));
    if constexpr (LANES == 64) {
        V x, y;
        swap16(v, x, y);
        v = f(x, y);
        swap32(v, x, y);
        v = f(x, y);
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
// Bytes of a wavefront's room in LDS: its tokens' logits; their approximate
// choices, where groups are read from there, and in the same place one token's
// choices in binary64 and 64 groups' scores; a candidate a lane, in 8 + 4 bytes.
__host__ __device__ constexpr size_t select_room(int lanes, int experts, bool near) {
    const size_t rows = (size_t)(64 / lanes) * row_words(experts) * 4, slow = 8 * ((size_t)experts + 64);
    return (rows + (near && rows > slow ? rows : slow) + 15) / 16 * 16 + 64 * 12;
}
// Lanes of a group, if it is whole ones and a power of two of them; else 0.
__host__ __device__ constexpr int group_span(int size, int per) {
    const int span = size % per ? 0 : size / per;
    return span & (span - 1) ? 0 : span;
}

// An expert's score in binary64.
__device__ __forceinline__ double score64(const SelectArgs &a, float l, float top, double inv_sum) {
    return a.softmax ? exp((double)l - top) * inv_sum : 1.0 / (1.0 + exp(-(double)l));
}

// A logit below which no score in binary64 comes up to that of l; next to l itself
// except far out.  Computed scores of two logits differ as the exact ones do if
// those are 2^-50 apart: of one where l >= 0 (exponential, sum and quotient are
// off by 2^-51 in all), of themselves below.  A sigmoid rises by 1 / (2 (1 + e^l))
// or more up to l, and below 0 by half of itself; an exponential by itself, and
// its argument, d below the largest, is off by 2^-53 d.  Scores near the
// least number binary64 holds keep too few bits: nothing is below.  2^-48 leaves
// room for the roundings here.
__device__ __forceinline__ float least_equal(const SelectArgs &a, float l, float top) {
    const float d = top - l;
    if (a.softmax ? d > 690.0f : l < -700.0f) return -__builtin_inff();
    return l - 0x1p-48f * (1.0f + (a.softmax ? d : __builtin_amdgcn_exp2f(l * LOG2E)));
}

__device__ __forceinline__ float bias_of(const SelectArgs &a, int e) {
    const float b = a.bias ? a.bias[e] : 0.0f;
    return finite_f32(b) ? b : 0.0f;
}

// One token by a whole wavefront, all in binary64: `logit` its logits, `choice`
// room for as many choices and, behind them, 64 group scores.  Lane k gets the k-th
// expert.
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
                const double c = choice[e];
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
                const double v = choice[e];
                if (v > c) {
                    c = v;
                    at = e;
                }
            }
        at = (int)all_lanes<64>(c == all_lanes<64>(c, Max()) ? (float)at : 1024.0f, Min());
        if ((at & 63) == lane) mine |= 1u << (at >> 6);
        if (lane == k) chosen = at;
    }
    return chosen;
}

template <class T, int LANES, int PER>
__global__ __launch_bounds__(64) void k_select(SelectArgs a, int vector) {
    constexpr int TOK = 64 / LANES, SUB = PER / 4;   // tokens a wavefront; experts a maximum stands for
    extern __shared__ double lds[];
    const int lane = threadIdx.x, tok = lane / LANES, sub = lane % LANES;
    const int words = row_words(a.experts), size = a.experts / a.groups;
    // in LDS: logits [TOK], approximate choices [TOK] (or one token's in binary64 and its groups'), candidates
    const bool groups = a.topk_group < a.groups;
    const int span = group_span(size, PER);
    const size_t room = select_room(LANES, a.experts, groups && !span);
    char *mem = reinterpret_cast<char *>(lds);
    float *logit = reinterpret_cast<float *>(mem) + tok * words;
    char *second_row = mem + (size_t)TOK * words * 4;
    float *near = reinterpret_cast<float *>(second_row) + tok * words;
    double *cand_key = reinterpret_cast<double *>(mem + room - 64 * 12) + tok * LANES;
    int *cand = reinterpret_cast<int *>(mem + room - 64 * 4) + tok * LANES;

    const int64_t token = (int64_t)blockIdx.x * TOK + tok;
    const bool real = token < a.tokens;
    const T *row = static_cast<const T *>(a.logits) + (real ? token : a.tokens - 1) * a.stride;
    const int e0 = sub * PER;
    constexpr float NEG = -__builtin_inff();
    float key[PER];
    bool bad = false;
    // No load of these waits for another: places behind the last expert read the last, or the first again.
    if (vector) {   // whole runs, 16-byte aligned
        constexpr int N = sizeof(T) == 4 ? 4 : PER < 8 ? 4 : 8;
        typedef T vec __attribute__((ext_vector_type(N)));
        vec v[PER / N];
#pragma unroll
        for (int i = 0; i < PER / N; ++i) v[i] = *reinterpret_cast<const vec *>(row + (e0 + N * i < a.experts ? e0 + N * i : 0));
#pragma unroll
        for (int i = 0; i < PER; ++i) key[i] = (float)v[i / N][i % N];
    } else {
        T v[PER];
#pragma unroll
        for (int i = 0; i < PER; ++i) v[i] = row[min(e0 + i, a.experts - 1)];
#pragma unroll
        for (int i = 0; i < PER; ++i) key[i] = (float)v[i];
    }
    float b[PER];
    float most_bias = 0.0f;
    if (a.bias) {
        if (vector) {
            f32x4 v[PER / 4];
#pragma unroll
            for (int i = 0; i < PER / 4; ++i) v[i] = *reinterpret_cast<const f32x4 *>(a.bias + (e0 + 4 * i < a.experts ? e0 + 4 * i : 0));
#pragma unroll
            for (int i = 0; i < PER; ++i) b[i] = v[i / 4][i % 4];
        } else {
#pragma unroll
            for (int i = 0; i < PER; ++i) b[i] = a.bias[min(e0 + i, a.experts - 1)];
        }
        float odd = 0.0f;
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            odd = __builtin_fmaf(b[i], 0.0f, odd);   // NaN from what is not finite
            most_bias = fmaxf(most_bias, fabsf(b[i]));
        }
        if (odd != 0.0f) {
            bad = true;
            most_bias = 0.0f;
#pragma unroll
            for (int i = 0; i < PER; ++i) {
                b[i] = finite_f32(b[i]) ? b[i] : 0.0f;
                most_bias = fmaxf(most_bias, fabsf(b[i]));
            }
        }
    }
    float top = NEG, odd = 0.0f;
    const int left = a.experts - e0;   // where not all are there, those of a lane are or are not, or some are
    const bool some = left > 0;
#pragma unroll
    for (int i = 0; i < PER; ++i) odd = __builtin_fmaf(key[i], 0.0f, odd);
    if (odd != 0.0f) {
        bad = true;
#pragma unroll
        for (int i = 0; i < PER; ++i) key[i] = finite_f32(key[i]) ? key[i] : 0.0f;
    }
    if (a.experts % PER) {
#pragma unroll
        for (int i = 0; i < PER; ++i) key[i] = i < left ? key[i] : NEG;
    } else if (a.experts < LANES * PER) {
#pragma unroll
        for (int i = 0; i < PER; ++i) key[i] = some ? key[i] : NEG;
    }
#pragma unroll
    for (int i = 0; i < PER; ++i) top = fmaxf(top, key[i]);
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
        for (int i = 0; i < PER; ++i) sum += exp((double)key[i] - top);   // none behind the last expert: exp(-inf)
        inv_sum = 1.0 / all_lanes<LANES>(sum, Add());
    }
    // ---- approximate choices, off by at most eps: a sigmoid by 2^-21 (0.2 of the exponential's relative error, sum and
    // quotient by a step each, the sum with the bias by half of one), a softmax by 2^-20 of the largest (the exponent by two
    // steps and a half of itself, d 2^-d < 1, the exponential and its product by a step each), and half a step of the bias
    const bool approximate = a.bias || (groups && a.top2);
    float eps = 0.0f, seen[PER];   // seen: what groups go by
#pragma unroll
    for (int i = 0; i < PER; ++i) seen[i] = key[i];
    if (approximate) {
        const float inv = (float)inv_sum;
        float c[PER];
        if (a.softmax) {
#pragma unroll
            for (int i = 0; i < PER; ++i) c[i] = __builtin_amdgcn_exp2f((key[i] - top) * LOG2E) * inv;
        } else {
#pragma unroll
            for (int i = 0; i < PER; ++i) c[i] = __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-LOG2E * key[i]));
        }
        if (a.bias) {
#pragma unroll
            for (int i = 0; i < PER; ++i) c[i] += b[i];
        }
        if (a.experts < LANES * PER) {
#pragma unroll
            for (int i = 0; i < PER; ++i) c[i] = key[i] == NEG ? NEG : c[i];
        }
        eps = 0x1p-20f * (a.softmax ? inv : 0.5f) + 0x1p-22f * all_lanes<LANES>(most_bias, Max());
        if (groups && !span && e0 < a.experts) {
#pragma unroll
            for (int i = 0; i < PER; i += 4) *reinterpret_cast<f32x4 *>(near + place(e0 + i)) = f32x4{c[i], c[i + 1], c[i + 2], c[i + 3]};
        }
#pragma unroll
        for (int i = 0; i < PER; ++i) seen[i] = c[i];
        if (a.bias) {
#pragma unroll
            for (int i = 0; i < PER; ++i) key[i] = c[i];
        }
    }
    wave_sync();
    // ---- groups: a lane each (there are at most LANES)
    bool slow = false;
    if (groups) {
        float first = NEG, second = NEG;
        if (span) {
#pragma unroll
            for (int i = 0; i < PER; ++i) {
                second = fmaxf(second, fminf(first, seen[i]));
                first = fmaxf(first, seen[i]);
            }
            for (int o = 1; o < span; o += o) {
                const float f = __shfl_xor(first, o), t = __shfl_xor(second, o);
                second = fmaxf(fmaxf(second, t), fminf(first, f));
                first = fmaxf(first, f);
            }
        } else {
            const float *from = approximate ? near : logit;
            if (sub < a.groups)
                for (int e = sub * size, end = e + size; e < end; e += 8) {   // the last of them again, if eight do not divide
                    float v[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i) v[i] = from[place(min(e + i, end - 1))];
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const float w = e + i < end ? v[i] : NEG;
                        second = fmaxf(second, fminf(first, w));
                        first = fmaxf(first, w);
                    }
                }
        }
        // its number, and the lane that has another's
        const int shift = span ? __builtin_ctz(span) : 0, self = sub >> shift;
        const bool two = a.top2 && size > 1, there = self < a.groups;
        const float mine = two ? first + second : first;
        bool in;
        auto stand = [&](auto v) {
            int before = 0;
            for (int g = 0; g < a.groups; ++g) {
                const auto other = __shfl(v, lane - sub + (g << shift));
                before += other > v || (other == v && g < self);
            }
            in = there && before < a.topk_group;
        };
        stand(mine);
        if (approximate) {
            const float least = all_lanes<LANES>(in ? mine : -NEG, Min()), next = all_lanes<LANES>(there && !in ? mine : NEG, Max());
            // sums of two are off by 2 eps and their own rounding
            slow = !(least - next > 4.0f * eps + 0x1p-22f * (fabsf(least) + fabsf(next)));
        } else {   // logits: equal ones are, others where binary64 tells the scores apart
            const float least = all_lanes<LANES>(in ? mine : -NEG, Min()), d = top - least;
            // elsewhere binary32's steps, 2^-24 of a logit, are the wider ones
            if (__ballot(fabsf(least) < 0x1p-20f * (a.softmax ? 1.0f + d : 1.0f) || (a.softmax ? d > 690.0f : top > 14.0f || least < -700.0f))) {
                const float below = all_lanes<LANES>(there && mine < least ? mine : NEG, Max());
                const float above = all_lanes<LANES>(there && mine > least ? mine : -NEG, Min());
                slow = below >= least_equal(a, least, top) || least_equal(a, above, top) <= least;
            }
        }
        if (span && __ballot(slow)) {   // scores in binary64, of the experts that could be a group's best
            const float from = two ? second : first;
            const float least_seen = approximate ? from - 2.0f * eps - 0x1p-22f * fabsf(from) : least_equal(a, from, top);
            uint32_t open = 0;
#pragma unroll
            for (int i = 0; i < PER; ++i) open |= seen[i] >= least_seen && seen[i] > NEG ? 1u << i : 0;
            double f = -__builtin_inf(), t = f;
            while (open) {
                const int e = e0 + __builtin_ctz(open);
                open &= open - 1;
                const double v = score64(a, logit[place(e)], top, inv_sum) + bias_of(a, e);
                t = fmax(t, fmin(f, v));
                f = fmax(f, v);
            }
            for (int o = 1; o < span; o += o) {
                const double of = __shfl_xor(f, o), ot = __shfl_xor(t, o);
                t = fmax(fmax(t, ot), fmin(f, of));
                f = fmax(f, of);
            }
            stand(two ? f + t : f);
            slow = false;
        }
        if (span) {
#pragma unroll
            for (int i = 0; i < PER; ++i) key[i] = in ? key[i] : NEG;
        } else {
            const uint64_t open = __ballot(in) >> (lane - sub);
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
    }
    // ---- a bound from below on the K-th best: the K-th of the maxima of SUB experts each
    float most[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        most[q] = key[SUB * q];
#pragma unroll
        for (int i = 1; i < SUB; ++i) most[q] = fmaxf(most[q], key[SUB * q + i]);
    }
    const uint64_t lower = ((1ull << sub) - 1) << (lane - sub);   // the token's lanes before this one
    float bound = NEG;
    for (int k = 0; k < a.top_k; ++k) {
        const float mine = fmaxf(fmaxf(most[0], most[1]), fmaxf(most[2], most[3]));
        bound = all_lanes<LANES>(mine, Max());
        const uint64_t has = __ballot(mine == bound);
        if (mine == bound && !(has & lower)) {   // of equal ones, one lane's at a time
#pragma unroll
            for (int q = 0; q < 4; ++q) most[q] = most[q] == bound ? NEG : most[q];
        }
    }
    // ---- candidates, in the order of their experts
    bound = a.bias ? bound - 2.0f * eps - 0x1p-22f * fabsf(bound) : least_equal(a, bound, top);
    bound = fmaxf(bound, -0x1.fffffep+127f);   // closed ones are below every number
    uint32_t mask = 0;
#pragma unroll
    for (int i = 0; i < PER; ++i) mask |= key[i] >= bound ? 1u << i : 0;
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
    // ---- their scores, and their order by choices in binary64
    int mine = sub < min(total, LANES) ? cand[sub] : -1;
    double score = 0.0, choice = -__builtin_inf();
    if (mine >= 0) {
        const float l = logit[place(mine)];
        score = score64(a, l, top, inv_sum);
        choice = a.bias ? score + bias_of(a, mine) : score;
        cand_key[sub] = choice;
    }
    wave_sync();
    int rank = 0;
    const int longest = LANES == 64 ? total : (int)all_lanes<64>((float)total, Max());
    for (int i = 0; i < min(longest, LANES); i += 4) {
        double other[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) other[j] = cand_key[i + j];   // LANES are a multiple
#pragma unroll
        for (int j = 0; j < 4; ++j) rank += i + j < total && (other[j] > choice || (other[j] == choice && i + j < sub));
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
    const size_t room = select_room(LANES, a.experts, a.topk_group < a.groups && !group_span(a.experts / a.groups, PER));
    constexpr int N = sizeof(T) == 4 ? 4 : PER < 8 ? 4 : 8;
    const bool vector = a.experts % N == 0 && a.stride % N == 0 && reinterpret_cast<uintptr_t>(a.logits) % (N * sizeof(T)) == 0 &&
                        reinterpret_cast<uintptr_t>(a.bias) % 16 == 0;
    const hipError_t e = ensure_dyn_smem(reinterpret_cast<const void *>(&k_select<T, LANES, PER>), room);
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL((k_select<T, LANES, PER>), dim3((uint32_t)(((int64_t)a.tokens + TOK - 1) / TOK)), dim3(64), room, st, a, (int)vector);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_select(const SelectArgs &a, int dtype, hipStream_t st) {
    auto go = [&](auto t) {
        using T = decltype(t);
        // Sixteen lanes against a wavefront a token, us: 256 experts in 8 groups of which 4 are kept, K = 8, 1024 tokens 6.8 and
        // 6.5, 2048 7.3, 7.3, 4096 7.4, 9.5, 16384 11.6, 25.4; 64 experts 4.3, 4.4; 4.4, 4.8; 4.5, 6.2; 6.2, 15.6.  Candidates
        // need a lane each, hence few of K, and groups too.  The bound is a maximum of four experts each: with few in the kept
        // groups it lets more than sixteen candidates in, and tokens are done over (K = 8, 32 experts kept: 2048 tokens 42.4,
        // 7.6, 16384 59.5, 25.5; 64 kept: 7.5, 7.3; 20.7, 25.3; K = 6, 20 kept: 33.9, 8.0; 55.4, 30.0).
        const int open = a.experts / a.groups * a.topk_group;
        const bool fit = a.experts <= 64 || open <= 16 || open >= 8 * a.top_k;
        if (a.tokens >= 2048 && a.experts <= 256 && a.top_k <= 10 && a.groups <= 16 && fit)
            return a.experts <= 64 ? launch_shape<T, 16, 4>(a, st) : launch_shape<T, 16, 16>(a, st);
        return a.experts <= 256 ? launch_shape<T, 64, 4>(a, st) : launch_shape<T, 64, 16>(a, st);
    };
    return dtype == COLI_BF16 ? go(__bf16()) : dtype == COLI_FP16 ? go(_Float16()) : go(float());
}

}  // namespace coli

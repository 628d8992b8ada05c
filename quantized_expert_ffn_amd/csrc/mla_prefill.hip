// Attention of prompts over expanded keys and values:
//
//   s_ij = scale (<q_i, k_j> + <p_i, r_j>),  out_i = sum_j e^{s_ij} v_j / sum_j e^{s_ij}
//
// over the keys j that query i sees, in one pass with the running maximum and
// sum of the softmax.
//
// What bounds it: no one part.  8192 tokens, 64 heads, widths 192 + 64 and 256,
// bf16, causal: 1.94 ms, 1.14 PFLOP/s, 0.81 of what a large library product of
// the same type reaches on the card (two runs of the same code: 1.94 and 1.97;
// single kernels under a profiler 2.0 to 2.17); counters: matrix cores 62% busy,
// LDS 31%, hardly a bank conflict, wavefronts waiting 30% of their time.  A
// build of 1.94 ms took 1.72 without the loads after the first tiles and 1.85
// without the exponentials.  Short calls are bound by the chain of a tile:
// ragged prompts of up to 513 queries over 1500 keys, 32 heads, widths 128 + 64
// and 128, fp16: 36 us, 24 tiles in a row for the longest.
#include "kernels.h"
#include "mla_mfma.h"

namespace coli {
namespace {

constexpr float LOG2E = 1.44269504088896340736f, LN2 = 0.69314718055994530942f;
// The running maximum moves only when a score exceeds it by this many powers
// of two: weights then reach 2^8 (binary16, lifted by 2^7: 2^15), which both
// types hold, and most tiles spare the pass over the accumulators.
constexpr float MAX_LAG = 8.0f;

// NW wavefronts share tiles of KT keys and values: NW / KG groups of 32
// queries, each of KG wavefronts that take 32 keys of a tile each.  Eight
// wavefronts of 256 registers are two a SIMD, so that one's softmax runs under
// the other's products (four on tiles of 32 keys took 1.97 and 2.38 ms in two
// builds in which eight on 64 took 1.94).
template <class T_, int NOPE_, int V_, int NW_, int KT_, int KG_>
struct Pre {
    using T = T_;
    static constexpr int NOPE = NOPE_, V = V_, NW = NW_, KT = KT_, KG = KG_;
    static constexpr int ROWS = 32 * NW / KG;
    static constexpr int KS = (NOPE + MLA_ROPE) / 16;   // matrix steps of a score
    static constexpr int KB = (NOPE + MLA_ROPE) / 64;   // blocks of eight 16-byte chunks in a key,
    static constexpr int VB = V / 64;                   // and in a value
    static constexpr int CT = V / 32;
    static constexpr int KTILE = KT * 128 * KB, TILE = KTILE + KT * 128 * VB;
    static constexpr int L_ML = NW * (CT / 2) * 4096;   // to join the keys' halves: accumulators, then pairs [NW][32]
    static_assert(KG == 1 || KT == 64, "two halves of 32 keys");
    static constexpr int JOIN = KG == 2 ? L_ML + NW * 32 * 8 : 0;
    static constexpr int STAGES = 3 * TILE <= 160 * 1024 ? 3 : 2;   // tiles in LDS: loads run one or two ahead
    static constexpr int L_ODD = STAGES * TILE > JOIN ? STAGES * TILE : JOIN;   // int: a wavefront set a value aside
    static constexpr int LDS = L_ODD + 16;
    static_assert(LDS <= 160 * 1024, "the LDS of a CU");
    static constexpr int LOADS = KB + VB;                            // of a wavefront, for a tile
};

// As in the decode kernel: LDS holds a tile as [8 tokens][8 chunks] blocks of
// 1 KiB, chunk c of token t at position c ^ swz(t) of its 128 bytes.
__device__ __forceinline__ int pre_swz(int t) { return 4 * ((t >> 1) & 1) + 2 * ((t >> 2) & 1) + ((t >> 3) & 1); }

template <class D>
__global__ __launch_bounds__(64 * D::NW, 2) void k_mla_prefill(MlaPrefillArgs a, int blocks) {
    using T = typename D::T;
    constexpr int V = D::V, CT = D::CT, KS = D::KS, THREADS = 64 * D::NW;
    constexpr float NEG = -__builtin_inff();
    const int tid = threadIdx.x, lane = tid & 63, wave = uniform(tid >> 6), n = lane & 31, hf = lane >> 5;

    // Workgroups go to the eight XCDs in turn; the blocks of one head of one sequence stay on one XCD, whose L2 then holds
    // its keys, the longest first.
    const int pair = (blockIdx.x & 7) + 8 * ((blockIdx.x >> 3) / blocks), blk = blocks - 1 - (blockIdx.x >> 3) % blocks;
    if (pair >= a.batch * a.heads) return;
    const int h = pair % a.heads;
    int b = pair / a.heads;
    if (a.batch > 1 && a.batch <= 64) {
        // the sequences with the most keys first: a long one begun last would leave the other CUs idle
        const int keys = lane < a.batch ? a.cu_k[lane + 1] - a.cu_k[lane] : -1;
        int rank = 0;
        for (int i = 0; i < a.batch; ++i) {
            const int other = __builtin_amdgcn_readlane(keys, i);
            rank += other > keys || (other == keys && i < lane);
        }
        b = __builtin_ctzll(__ballot(lane < a.batch && rank == b));
    }

    const int q0 = uniform(a.cu_q[b]), nq = uniform(a.cu_q[b + 1]) - q0;
    const int k0 = uniform(a.cu_k[b]), nk = uniform(a.cu_k[b + 1]) - k0;
    if (q0 < 0 || nq < 0 || nq > a.n_q_rows - q0 || nq > a.max_q || k0 < 0 || nk < 0 || nk > a.n_k_rows - k0) {
        if (tid == 0) raise_status(a.status, ST_BADPAGE);
        return;
    }
    const int group = wave % (D::NW / D::KG), half = wave / (D::NW / D::KG);   // the keys' half with KG = 2
    const int row0 = blk * D::ROWS, wrow = row0 + 32 * group, row = wrow + n;
    if (row0 >= nq) return;
    const int shift = a.causal ? nk - nq + 1 : nk;            // query i sees shift + i (or all nk) keys
    auto sees = [&](int i) { return min(nk, max(0, a.causal ? shift + i : nk)); };
    const int last = min(row0 + D::ROWS, nq) - 1;
    const int tiles = (sees(last) + D::KT - 1) / D::KT;
    const int block_seen = sees(row0);                        // keys every query of the block sees,
    const int wave_seen = sees(min(wrow, nq - 1));            // every query of the wavefront,
    const int wave_any = wrow < nq ? sees(min(wrow + 31, nq - 1)) : 0;   // any of them
    const int seen = sees(min(row, nq - 1));

    // ---- lane addresses inside a tile
    uint32_t ka[4], va[4];
    {
        const int f = pre_swz(n);
#pragma unroll
        for (int v = 0; v < 4; ++v) ka[v] = (n >> 3) * D::KB * 1024 + (n & 7) * 128 + (((2 * v + hf) ^ f) << 4);
        const int x = lane & 15, cb = (lane >> 4) & 1, t8 = 4 * hf + (x >> 2);
#pragma unroll
        for (int v = 0; v < 4; ++v) {   // va[2 e + (ct & 1)], e the token group of a step
            const int e = v >> 1, fv = pre_swz(8 * e + t8);
            va[v] = D::KTILE + e * D::VB * 1024 + t8 * 128 + (((4 * (v & 1) + 2 * cb + ((x & 3) >> 1)) ^ fv) << 4) + 8 * (x & 1);
        }
    }

    // ---- loads: a wavefront takes chunk lane % 8 of tokens 8 wave + lane / 8 of a tile, keys and values apart
    static_assert(D::KT == 8 * D::NW, "one group of eight tokens a wavefront");
    const char *kn = reinterpret_cast<const char *>(static_cast<const T *>(a.k_nope) + k0 * a.k_ts + h * a.k_hs);
    const char *kp = reinterpret_cast<const char *>(static_cast<const T *>(a.k_pe) + (int64_t)k0 * MLA_ROPE);
    const char *vv = reinterpret_cast<const char *>(static_cast<const T *>(a.v) + k0 * a.v_ts + h * a.v_hs);
    const int my_token = 8 * wave + (lane >> 3);
    const uint32_t my_chunk = ((lane & 7) ^ pre_swz(my_token)) << 4;
    const uint32_t k_step = 2 * (uint32_t)a.k_ts, v_step = 2 * (uint32_t)a.v_ts;
    uint32_t k_off = my_token * k_step + my_chunk, p_off = my_token * (2 * MLA_ROPE) + my_chunk, v_off = my_token * v_step + my_chunk;
    // Tiles come in order, so the last, where tokens behind the end are the last token again, can change the offsets.
    auto clamp = [&](int tile) {
        const int end = nk - tile * D::KT;
        if (end < D::KT) {
            const int t = min(my_token, end - 1);
            k_off = t * k_step + my_chunk;
            p_off = t * (2 * MLA_ROPE) + my_chunk;
            v_off = t * v_step + my_chunk;
        }
    };
    auto issue_k = [&](int tile) {
        clamp(tile);
        const uint32_t d = tile % D::STAGES * D::TILE + wave * D::KB * 1024;
        const char *n0 = kn + (int64_t)tile * D::KT * (2 * a.k_ts), *p0 = kp + (int64_t)tile * (D::KT * 2 * MLA_ROPE);
        load_to_lds_from<0>(n0, k_off, d, 0);
        load_to_lds_from<128>(n0, k_off, d, 1024);
        if (D::KB == 4) load_to_lds_from<256>(n0, k_off, d, 2048);
        load_to_lds_from<0>(p0, p_off, d, (D::KB - 1) * 1024);
    };
    auto issue_v = [&](int tile) {
        const uint32_t d = tile % D::STAGES * D::TILE + D::KTILE + wave * D::VB * 1024;
        const char *v0 = vv + (int64_t)tile * D::KT * (2 * a.v_ts);
        load_to_lds_from<0>(v0, v_off, d, 0);
        load_to_lds_from<128>(v0, v_off, d, 1024);
        if (D::VB == 4) {
            load_to_lds_from<256>(v0, v_off, d, 2048);
            load_to_lds_from<384>(v0, v_off, d, 3 * 1024);
        }
    };
    auto issue = [&](int tile) {
        issue_k(tile);
        issue_v(tile);
    };
    // Cleared before the first tile's barrier, set after it.  A word of the kernel's own: a barrier that carries a value
    // would take one of the device library's, at the byte where the dynamic allocation is addressed from.
    if (tid == 0) lds_write<int>(D::L_ODD, 0);
    if (tiles > 0) issue(0);
    if (D::STAGES == 3 && tiles > 1) issue(1);

    x8<T> qf[KS];
    {
        const T *q = static_cast<const T *>(a.q) + (q0 + min(row, nq - 1)) * a.q_ts + h * a.q_hs + 8 * hf;
#pragma unroll
        for (int s = 0; s < KS; ++s) qf[s] = *reinterpret_cast<const x8<T> *>(q + 16 * s);
#pragma unroll
        for (int s = 0; s < KS; ++s) arrived(qf[s]);
    }
    f32x16 o[CT];
#pragma unroll
    for (int c = 0; c < CT; ++c)
#pragma unroll
        for (int r = 0; r < 16; ++r) o[c][r] = 0.0f;
    constexpr float LIFT = WEIGHT_LIFT<T>, LAG = LIFT + MAX_LAG;
    float m = NEG, l = 0.0f;   // m: the running maximum less LIFT
    const float scale = a.scale * LOG2E;
    bool odd = false;   // a value that is not finite was set aside

    for (int tile = 0; tile < tiles; ++tile) {
        const int t0 = tile * D::KT;
        const uint32_t base = tile % D::STAGES * D::TILE;
        if (D::STAGES == 3 && tile + 1 < tiles)
            wait_vm<D::LOADS>();
        else
            wait_vm<0>();
        barrier_lds();   // the tile is there, and every wavefront is done with the one before
        // With two stages the values' loads follow the first scores: a burst of all of them would hold up the products.
        const int coming = tile + D::STAGES - 1;
        bool v_due = coming < tiles;
        if (v_due) {
            issue_k(coming);
            if (D::STAGES == 3) {
                issue_v(coming);
                v_due = false;
            }
        }
        if (t0 + D::KT > block_seen) {
            // A tile that some queries see only in part: values that are not finite would reach those that do not see
            // them as 0 * NaN.  They are set aside, and added at the end where they are seen.  Places behind the last
            // key hold its value again, for nobody.
            const int from = block_seen > t0 ? block_seen - t0 : 0;
            for (int i = tid; i < (D::KT - from) * D::VB * 8; i += THREADS) {
                const int t = from + i / (D::VB * 8), c = i % (D::VB * 8);
                const uint32_t w = base + D::KTILE + ((t >> 3) * D::VB + (c >> 3)) * 1024 + (t & 7) * 128 + ((c & 7) << 4);
                x8<T> v = lds_read<x8<T>>(w);
                bool bad = false;
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    if (!finite_f32((float)v[k])) {
                        v[k] = (T)0.0f;
                        bad = true;
                    }
                if (bad) lds_write(w, v);
                odd |= bad && t0 + t < nk;
            }
            barrier_lds();
        }
#pragma unroll
        for (int k = 0; k < D::KT / 32 / D::KG; ++k) {
            const int kh = D::KG == 2 ? half : k, tw = t0 + 32 * kh;
            if (tw >= wave_any) break;
            const uint32_t kb = base + kh * 4 * D::KB * 1024, vb = base + kh * 4 * D::VB * 1024;
            f32x16 s;
#pragma unroll
            for (int r = 0; r < 16; ++r) s[r] = 0.0f;
            x8<T> ahead[2][2];   // operands two reads ahead of their products
            auto fetch = [&](int i) { return lds_read<x8<T>>(kb + ka[i & 3], (i >> 2) * 1024); };
            ahead[0][0] = fetch(0);
            ahead[0][1] = fetch(1);
#pragma unroll
            for (int c = 0; c < KS; c += 2) {
                __builtin_amdgcn_sched_barrier(0);
                if (c + 2 < KS) {
                    ahead[(c / 2 + 1) & 1][0] = fetch(c + 2);
                    ahead[(c / 2 + 1) & 1][1] = fetch(c + 3);
                }
                s = mfma32<T>(ahead[(c / 2) & 1][0], qf[c], s);
                s = mfma32<T>(ahead[(c / 2) & 1][1], qf[c + 1], s);
            }
            __builtin_amdgcn_sched_barrier(0);
            if (tw + 32 > wave_seen) {
                int rem = seen - tw - 4 * hf;
                arrived(rem);   // a branch, not selects that every tile would pay for
#pragma unroll
                for (int r = 0; r < 16; ++r)
                    if (8 * (r >> 2) + (r & 3) >= rem) s[r] = NEG;
            }
            float top = s[0];
#pragma unroll
            for (int r = 1; r < 16; ++r) top = fmaxf(top, s[r]);
            top = half_max(top) * scale;
            if (__ballot(top > m + LAG)) {
                const float to = top > m + LAG ? top - LIFT : m;
                const float f = m == to ? 1.0f : __builtin_amdgcn_exp2f(m - to);
                l *= f;
                m = to;
#pragma unroll
                for (int c = 0; c < CT; ++c)
#pragma unroll
                    for (int r = 0; r < 16; ++r) o[c][r] *= f;
            }
            const float ref = m == NEG ? 0.0f : m;
            float sum = 0.0f;
            x8<T> p[2];
#pragma unroll
            for (int r = 0; r < 16; ++r) {
                const float w = __builtin_amdgcn_exp2f(__builtin_fmaf(s[r], scale, -ref));
                sum += w;
                p[r >> 3][r & 7] = (T)w;
            }
            l += sum;
            if (v_due) {
                issue_v(coming);
                v_due = false;
            }
            u32x4 av[2][2];   // a column tile's two matrix steps
            auto fetch_v = [&](int c, int k) {
                const int imm = 2 * k * D::VB * 1024 + (c >> 1) * 1024;
                const u32x2 v0 = lds_read_tr16(vb + va[c & 1], imm), v1 = lds_read_tr16(vb + va[2 + (c & 1)], imm);
                return u32x4{v0[0], v0[1], v1[0], v1[1]};
            };
            av[0][0] = fetch_v(0, 0);
            av[0][1] = fetch_v(0, 1);
#pragma unroll
            for (int c = 0; c < CT; ++c) {
                __builtin_amdgcn_sched_barrier(0);
                if (c + 1 < CT) {
                    av[(c + 1) & 1][0] = fetch_v(c + 1, 0);
                    av[(c + 1) & 1][1] = fetch_v(c + 1, 1);
                }
                o[c] = mfma32<T>(__builtin_bit_cast(x8<T>, av[c & 1][0]), p[0], o[c]);
                o[c] = mfma32<T>(__builtin_bit_cast(x8<T>, av[c & 1][1]), p[1], o[c]);
            }
            __builtin_amdgcn_sched_barrier(0);
        }
        if (v_due) issue_v(coming);
    }

    l = half_sum(l);
    int c0 = 0;
    if (D::KG == 2) {
        // each wavefront hands half of its columns to the one with the other keys, and both add first half to second
        barrier_lds();
        if (hf == 0) lds_write(D::L_ML + 8 * (32 * wave + n), f32x2{m, l});
#pragma unroll
        for (int c = 0; c < CT / 2; ++c)
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                f32x4 v;
#pragma unroll
                for (int i = 0; i < 4; ++i) v[i] = half ? o[c][4 * q + i] : o[CT / 2 + c][4 * q + i];
                lds_write((wave * (CT / 2) + c) * 4096 + 16 * lane, v, q * 1024);
            }
        barrier_lds();
        const int other = wave ^ (D::NW / 2);
        const f32x2 ml = lds_read<f32x2>(D::L_ML + 8 * (32 * other + n));
        const float to = fmaxf(m, ml[0]);
        const float fa = m == to ? 1.0f : __builtin_amdgcn_exp2f(m - to);
        const float fb = ml[0] == to ? 1.0f : __builtin_amdgcn_exp2f(ml[0] - to);
        l = half ? ml[1] * fb + l * fa : l * fa + ml[1] * fb;
        m = to;
#pragma unroll
        for (int c = 0; c < CT / 2; ++c)
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const f32x4 v = lds_read<f32x4>((other * (CT / 2) + c) * 4096 + 16 * lane, q * 1024);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float own = half ? o[CT / 2 + c][4 * q + i] : o[c][4 * q + i];
                    o[c][4 * q + i] = own * fa + v[i] * fb;
                }
            }
        c0 = half * (CT / 2);
    }
    if (row < nq) {
        const int64_t r = (int64_t)(q0 + row) * a.heads + h;
        const float f = l == 0.0f ? 0.0f : 1.0f / l;
        T *dst = static_cast<T *>(a.out) + r * V + 32 * c0 + 4 * hf;
#pragma unroll
        for (int c = 0; c < CT / D::KG; ++c)
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                x4<T> v;
#pragma unroll
                for (int i = 0; i < 4; ++i) v[i] = (T)(o[c][4 * q + i] * f);
                *reinterpret_cast<x4<T> *>(dst + 32 * c + 8 * q) = v;
            }
        if (a.lse && hf == 0 && half == 0) a.lse[r] = l == 0.0f ? NEG : (m + __builtin_amdgcn_logf(l)) * LN2;
    }
    if (__ballot(odd) && lane == 0) lds_write<int>(D::L_ODD, 1);
    barrier_lds();
    if (lds_read<int>(D::L_ODD)) {
        wait_vm<0>();   // the results are there for the others to add to
        barrier_lds();
        // the values set aside: their column of every query that sees them
        for (int c = tid; c < V; c += THREADS)
            for (int t = block_seen; t < sees(last); ++t) {
                const float x = (float)reinterpret_cast<const T *>(vv)[t * a.v_ts + c];
                if (finite_f32(x)) continue;
                for (int i = row0; i <= last; ++i)
                    if (t < sees(i)) {
                        T *dst = static_cast<T *>(a.out) + ((int64_t)(q0 + i) * a.heads + h) * V + c;
                        *dst = (T)((float)*dst + x);
                    }
            }
    }
}

template <class D>
hipError_t launch(const MlaPrefillArgs &a, hipStream_t st) {
    const int blocks = (a.max_q + D::ROWS - 1) / D::ROWS;
    const hipError_t e = ensure_dyn_smem(reinterpret_cast<const void *>(&k_mla_prefill<D>), D::LDS);
    if (e != hipSuccess) return e;
    // A launch has less than 2^32 threads: as many sequences as that leaves (one whose blocks alone passed it would have
    // more results than the card has memory).
    const int64_t groups = ((int64_t)1 << 32) / (64 * D::NW) / ((int64_t)blocks * 8) - 1;   // of eight sequences' heads
    const int64_t most = groups * 8 / a.heads;
    const int each = (int)(most < 1 ? 1 : most < a.batch ? most : a.batch);
    for (int b = 0; b < a.batch; b += each) {
        MlaPrefillArgs part = a;
        part.cu_q += b;
        part.cu_k += b;
        part.batch = a.batch - b < each ? a.batch - b : each;
        hipLaunchKernelGGL(k_mla_prefill<D>, dim3((uint32_t)blocks * 8 * ((a.heads * part.batch + 7) / 8)), dim3(64 * D::NW),
                           D::LDS, st, part, blocks);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

template <class T, int NOPE, int V>
hipError_t by_size(const MlaPrefillArgs &a, hipStream_t st) {
    // Workgroups of 256 queries if they fill the 256 CUs, else of 128 whose keys two wavefronts share: 512 tokens, 64
    // heads, widths 192 + 64 and 256: 41 against 33 us; 1024 tokens: 66 against 83 us; 8192: 1.94 against 2.16 ms.
    const int64_t by_max = (int64_t)a.batch * ((a.max_q + 255) / 256), by_rows = (a.n_q_rows + 255) / 256 + a.batch - 1;
    if (a.heads * (by_max < by_rows ? by_max : by_rows) < 256) return launch<Pre<T, NOPE, V, 8, 64, 2>>(a, st);
    return launch<Pre<T, NOPE, V, 8, 64, 1>>(a, st);
}

}  // namespace

hipError_t launch_mla_prefill(const MlaPrefillArgs &a, const coli_mla_dims &d, hipStream_t st) {
    return mla_with_type(d.dtype, [&](auto t) {
        using T = decltype(t);
        return d.nope == 128 ? by_size<T, 128, 128>(a, st) : by_size<T, 192, 256>(a, st);
    });
}

}  // namespace coli

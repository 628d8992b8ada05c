// Absorbed attention of a batch's new tokens over a prefix that all its
// sequences share, and the join with what they see of their own tokens.
//
// The query rows of all sequences are one product with the prefix's latents:
// s = scale (<q, c> + <p, k>), out = sum e^s c / sum e^s over tiles of 32
// tokens.  A workgroup takes 128 rows, a wavefront 32 of them with all columns,
// so that weights stay in the registers they are formed in: 256 accumulators
// and 144 registers of queries beside them.
#include "kernels.h"
#include "mla_mfma.h"

namespace coli {
namespace {

constexpr int SHD_TILE = 32, SHD_ROWS = 128;
constexpr float LOG2E = 1.44269504088896340736f, LN2 = 0.69314718055994530942f;
// The running maximum moves only when a score exceeds it by this many powers of two.
constexpr float MAX_LAG = 8.0f;

template <class T_, int RANK_, bool FP8_>
struct Shd {
    using T = T_;
    static constexpr int RANK = RANK_;
    static constexpr bool FP8 = FP8_;
    static constexpr int ROW = FP8 ? RANK + 2 * MLA_ROPE : 2 * (RANK + MLA_ROPE);   // bytes of a cached token
    static constexpr int CB = (RANK + MLA_ROPE) / 64;   // 128-byte lines of a token in LDS, where codes are widened
    static constexpr int KS = (RANK + MLA_ROPE) / 16;   // matrix steps of a score
    static constexpr int CT = RANK / 32;                // 32-column tiles of the output
    static constexpr int RING = 4;
    static constexpr int TILE = SHD_TILE * CB * 128;
    static constexpr int L_ID = RING * TILE;                    // int32 [RING][4 wavefronts][64]: page ids of tiles to come
    static constexpr int L_SCALE = L_ID + RING * 1024;          // float [RING][32]: E4M3 scales
    static constexpr int L_EXP = L_SCALE + RING * 4 * SHD_TILE; // float [RING][32]: their exponents
    static constexpr int LDS = L_EXP + RING * 4 * SHD_TILE;
    static constexpr int SLOT = SHD_ROWS * RANK + 2 * SHD_ROWS;
    static_assert(LDS <= 160 * 1024, "the LDS of a CU");
};

// Work is shared out evenly in units of one tile of one block of rows.
struct Units {
    int64_t units;
    int tiles, shares;
    __host__ __device__ int64_t first(int g) const { return units * g / shares; }
    // the workgroup that has a unit
    __host__ __device__ int owner(int64_t unit) const { return (int)(((unit + 1) * shares - 1) / units); }
};
Units shd_units(int64_t rows, int prefix) {
    Units u;
    u.tiles = (prefix + SHD_TILE - 1) / SHD_TILE;
    u.units = (rows + SHD_ROWS - 1) / SHD_ROWS * u.tiles;
    u.shares = (int)(u.units < 256 ? u.units : 256);
    return u;
}

__device__ __forceinline__ int shd_swz(int t) { return 4 * ((t >> 1) & 1) + 2 * ((t >> 2) & 1) + ((t >> 3) & 1); }

// The tokens of the prefix that a query row sees: all, unless its sequence has
// fewer tokens of its own than new ones.
__device__ __forceinline__ int shd_seen(const MlaSharedArgs &a, int64_t row) {
    const int per = a.n_q * a.heads, b = (int)(row / per), j = (int)(row - (int64_t)b * per) / a.heads;
    const int len = mla_len(a.kv_lens, b, a.max_kv, a.status);
    return max(0, a.prefix + min(0, len - a.n_q + 1 + j));
}

template <class D>
__global__ __launch_bounds__(256, 1) void k_mla_shared(MlaSharedArgs a, Units u) {
    using T = typename D::T;
    constexpr int RANK = D::RANK, CT = D::CT, KS = D::KS;
    constexpr bool FP8 = D::FP8;
    constexpr float NEG = -__builtin_inff();
    constexpr float LIFT = WEIGHT_LIFT<T>, LAG = LIFT + MAX_LAG;
    const int tid = threadIdx.x, lane = tid & 63, wave = uniform(tid >> 6);
    const int n = lane & 31, hf = lane >> 5, g = blockIdx.x;
    const int64_t rows = (int64_t)a.batch * a.n_q * a.heads;
    int64_t unit = u.first(g);
    const int64_t end = u.first(g + 1);
    const float scale = a.scale * LOG2E;
    const uint32_t page_inv = 0xffffffffu / (uint32_t)a.c.page;
    bool bad_page = false;

    // ---- lane addresses inside a tile
    uint32_t ka[4], va[4];
    {
        const int f = shd_swz(n), x = lane & 15, cb = (lane >> 4) & 1;
#pragma unroll
        for (int v = 0; v < 4; ++v) {
            ka[v] = (n >> 3) * D::CB * 1024 + (n & 7) * 128 + (((2 * v + hf) ^ f) << 4);
            const int e = v >> 1, t8 = 4 * hf + (x >> 2), fv = shd_swz(8 * e + t8);
            va[v] = e * D::CB * 1024 + t8 * 128 + (((4 * (v & 1) + 2 * cb + ((x & 3) >> 1)) ^ fv) << 4) + 8 * (x & 1);
        }
    }
    const int lt = 8 * wave + (lane >> 3), lf = shd_swz(lt);   // the token whose chunks this thread loads

    while (unit < end) {
        const int blk = (int)(unit / u.tiles), lo = (int)(unit - (int64_t)blk * u.tiles);
        const int hi = (int)min((int64_t)u.tiles, lo + end - unit);
        unit += hi - lo;
        const int64_t row = (int64_t)blk * SHD_ROWS + 32 * wave + n, wave_row = (int64_t)blk * SHD_ROWS + 32 * wave;
        const bool works = wave_row < rows;
        const int64_t at_row = row < rows ? row : rows - 1;
        x8<T> qf[KS];
#pragma unroll
        for (int s = 0; s < KS; ++s)
            qf[s] = *reinterpret_cast<const x8<T> *>(s < RANK / 16
                                                         ? static_cast<const T *>(a.q_lat) + at_row * RANK + 16 * s + 8 * hf
                                                         : static_cast<const T *>(a.q_pe) + at_row * MLA_ROPE + 16 * (s - RANK / 16) + 8 * hf);
        const int seen = shd_seen(a, at_row);
        int wave_seen = seen;
        for (int o = 16; o; o >>= 1) wave_seen = min(wave_seen, __shfl_xor(wave_seen, o));
        wave_seen = uniform(wave_seen);
        int block_seen = a.prefix;   // the least of the block's rows
        for (int64_t r = (int64_t)blk * SHD_ROWS + lane; r < min((int64_t)(blk + 1) * SHD_ROWS, rows); r += 64)
            block_seen = min(block_seen, shd_seen(a, r));
        for (int o = 32; o; o >>= 1) block_seen = min(block_seen, __shfl_xor(block_seen, o));
        block_seen = uniform(block_seen);

        f32x16 o[CT];
#pragma unroll
        for (int c = 0; c < CT; ++c)
#pragma unroll
            for (int r = 0; r < 16; ++r) o[c][r] = 0.0f;
        float m = NEG, l = 0.0f, mv = NEG;

        for (int tile = lo; tile < hi; ++tile) {
            const int t0 = tile * SHD_TILE;
            __syncthreads();   // the tile before is done with
            {
                const int t = min(t0 + lt, a.prefix - 1), pi = div_by(t, a.c.page, page_inv);
                int id = a.c.table[pi];
                if ((uint32_t)id >= (uint32_t)a.c.n_pages) {
                    bad_page = true;
                    id = 0;
                }
                const int64_t slot = (int64_t)id * a.c.page + (t - pi * a.c.page);
                const uint8_t *src = a.c.pages + slot * D::ROW;
                const uint32_t dst = wave * D::CB * 1024 + (lane >> 3) * 128;
                if (FP8) {
#pragma unroll
                    for (int i = 0; i < RANK / 128; ++i) {
                        const int c = (lane & 7) + 8 * i;   // of sixteen codes: chunks 2 c and 2 c + 1
                        const u32x4 w = *reinterpret_cast<const u32x4 *>(src + 16 * c);
                        const uint32_t line = dst + (c >> 2) * 1024;
                        lds_write(line + (((2 * c & 7) ^ lf) << 4), widen8<T>(u32x2{w[0], w[1]}));
                        lds_write(line + (((2 * c + 1 & 7) ^ lf) << 4), widen8<T>(u32x2{w[2], w[3]}));
                    }
                    const x8<T> v = *reinterpret_cast<const x8<T> *>(src + RANK + 16 * (lane & 7));
                    lds_write(dst + (D::CB - 1) * 1024 + (((lane & 7) ^ lf) << 4), v);
                    if ((lane & 7) == 0) {
                        const float sc = a.c.scale[slot];
                        lds_write<float>(D::L_SCALE + 4 * lt, sc);
                        lds_write<float>(D::L_EXP + 4 * lt, sc == 0.0f ? NEG : (float)__builtin_amdgcn_frexp_expf(sc));
                    }
                } else {
#pragma unroll
                    for (int c = 0; c < D::CB; ++c) {
                        const x8<T> v = *reinterpret_cast<const x8<T> *>(src + 128 * c + 16 * (lane & 7));
                        lds_write(dst + c * 1024 + (((lane & 7) ^ lf) << 4), v);
                    }
                }
            }
            __syncthreads();
            f32x16 s;
            float sc[16];
#pragma unroll
            for (int r = 0; r < 16; ++r) s[r] = 0.0f;
#pragma unroll
            for (int k = 0; k < RANK / 16; ++k) s = mfma32<T>(lds_read<x8<T>>(ka[k & 3], (k >> 2) * 1024), qf[k], s);
            if (FP8) {
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const f32x4 v = lds_read<f32x4>(D::L_SCALE + 16 * hf, 32 * q);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        s[4 * q + i] *= v[i];
                        sc[4 * q + i] = __builtin_amdgcn_frexp_mantf(v[i]);
                    }
                }
            }
#pragma unroll
            for (int k = RANK / 16; k < KS; ++k) s = mfma32<T>(lds_read<x8<T>>(ka[k & 3], (k >> 2) * 1024), qf[k], s);
            if (t0 + SHD_TILE > wave_seen) {
                const int rem = seen - t0 - 4 * hf;
#pragma unroll
                for (int r = 0; r < 16; ++r)
                    if (8 * (r >> 2) + (r & 3) >= rem) {
                        s[r] = NEG;
                        sc[r] = 0.0f;
                    }
            }
            // ---- softmax
            float top = s[0], sv[16];
#pragma unroll
            for (int r = 1; r < 16; ++r) top = fmaxf(top, s[r]);
            top = half_max(top) * scale;
            float topv = NEG;
            if (FP8) {
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const f32x4 e = lds_read<f32x4>(D::L_EXP + 16 * hf, 32 * q);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        sv[4 * q + i] = __builtin_fmaf(s[4 * q + i], scale, e[i]);
                        topv = fmaxf(topv, sv[4 * q + i]);
                    }
                }
                topv = half_max(topv);
            }
            if (__ballot(top > m + LAG || (FP8 && topv > mv + LAG))) {
                const float to = top > m + LAG ? top - LIFT : m;
                float f = m == to ? 1.0f : __builtin_amdgcn_exp2f(m - to);
                l *= f;
                m = to;
                if (FP8) {
                    const float tov = topv > mv + LAG ? rintf(topv) - LIFT : mv;
                    f = mv == tov ? 1.0f : __builtin_amdgcn_exp2f(mv - tov);
                    mv = tov;
                }
#pragma unroll
                for (int c = 0; c < CT; ++c)
#pragma unroll
                    for (int r = 0; r < 16; ++r) o[c][r] *= f;
            }
            const float ref = m == NEG ? 0.0f : m, refv = mv == NEG ? 0.0f : mv;
            x8<T> p[2];
#pragma unroll
            for (int r = 0; r < 16; ++r) {
                float w = __builtin_amdgcn_exp2f(__builtin_fmaf(s[r], scale, -ref));
                l += w;
                if (FP8) w = sc[r] * __builtin_amdgcn_exp2f(sv[r] - refv);
                p[r >> 3][r & 7] = (T)w;
            }
            // A tile that some rows see only in part: values that are not finite would reach rows that do not see them.
            if (block_seen < a.prefix && t0 + SHD_TILE > block_seen) {
                __syncthreads();
                const int from = block_seen > t0 ? block_seen - t0 : 0;
                constexpr int CH = (D::CB - 1) * 8;
                for (int i = tid; i < (SHD_TILE - from) * CH; i += 256) {
                    const int t = from + i / CH, c = i % CH;
                    const uint32_t w = ((t >> 3) * D::CB + (c >> 3)) * 1024 + (t & 7) * 128 + ((c & 7) << 4);
                    x8<T> v = lds_read<x8<T>>(w);
#pragma unroll
                    for (int k = 0; k < 8; ++k)
                        if (!finite_f32((float)v[k])) v[k] = (T)0.0f;
                    lds_write(w, v);
                }
                __syncthreads();
            }
#pragma unroll
            for (int c = 0; c < CT; ++c)
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const int imm = 2 * k * D::CB * 1024 + (c >> 1) * 1024;
                    const u32x2 v0 = lds_read_tr16(va[c & 1], imm), v1 = lds_read_tr16(va[2 + (c & 1)], imm);
                    o[c] = mfma32<T>(__builtin_bit_cast(x8<T>, u32x4{v0[0], v0[1], v1[0], v1[1]}), p[k], o[c]);
                }
        }

        // ---- the segment's result, divided by its sum
        l = half_sum(l);
        if (works) {
            const float half_off = FP8 && l != 0.0f ? __builtin_amdgcn_exp2f(0.5f * (mv - m)) : 1.0f;
            const float f = l == 0.0f ? 0.0f : half_off / l;
            float *dst = a.part + (int64_t)(g + blk) * D::SLOT, *at = dst + wave * CT * 1024 + 4 * lane;
#pragma unroll
            for (int c = 0; c < CT; ++c)
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    f32x4 v;
#pragma unroll
                    for (int i = 0; i < 4; ++i) v[i] = FP8 ? o[c][4 * q + i] * f * half_off : o[c][4 * q + i] * f;
                    *reinterpret_cast<f32x4 *>(at + (c * 4 + q) * 256) = v;
                }
            if (hf == 0) *reinterpret_cast<float2 *>(dst + SHD_ROWS * RANK + 2 * (32 * wave + n)) = make_float2(m, l);
        }
    }
    if (bad_page) raise_status(a.status, ST_BADPAGE);
}

// Joins the partial results of 32 rows by 8 columns: out = sum 2^{m_i - M} l_i
// o_i / sum 2^{m_i - M} l_i, those over the prefix in order, then those of the
// rows' sequences.  A workgroup's W wavefronts take every W-th each.
template <class T, int RANK, int W>
__global__ __launch_bounds__(64 * W) void k_mla_shared_join(MlaSharedArgs a, Units u) {
    constexpr int SLOT = SHD_ROWS * RANK + 2 * SHD_ROWS;
    constexpr float NEG = -__builtin_inff();
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, n = lane & 31, cq = blockIdx.x % (RANK / 8);
    const int64_t rows = (int64_t)a.batch * a.n_q * a.heads, row = (int64_t)(blockIdx.x / (RANK / 8)) * 32 + n;
    const int64_t at_row = row < rows ? row : rows - 1;
    __shared__ f32x4 so[W][64];
    __shared__ float sm[W][64], sl[W][64];
    float m = NEG, l = 0.0f;
    f32x4 o = {0.0f, 0.0f, 0.0f, 0.0f};
    auto add = [&](const float *at, const float *ml) {
        const float2 x = *reinterpret_cast<const float2 *>(ml);
        const f32x4 v = *reinterpret_cast<const f32x4 *>(at);
        const float to = fmaxf(m, x.x), old = m == to ? 1.0f : __builtin_amdgcn_exp2f(m - to);
        const float f = x.y * (x.x == to ? 1.0f : __builtin_amdgcn_exp2f(x.x - to));
        m = to;
        l = __builtin_fmaf(l, old, f);
#pragma unroll
        for (int i = 0; i < 4; ++i) o[i] = __builtin_fmaf(v[i], f, o[i] * old);
    };
    {
        const int64_t blk = row / SHD_ROWS, unit = blk * u.tiles;
        const int r = (int)(row - blk * SHD_ROWS), g0 = u.owner(unit), g1 = u.owner(unit + u.tiles - 1);
        for (int g = g0 + wave; g <= g1; g += W) {
            const float *slot = a.part + (g + blk) * SLOT;
            add(slot + (r / 32 * (RANK / 8) + cq) * 256 + 4 * lane, slot + SHD_ROWS * RANK + 2 * r);
        }
    }
    if (a.own) {
        const int per = a.n_q * a.heads, b = (int)(at_row / per), w = (int)(at_row - (int64_t)b * per);
        const int block = w / a.p.rows, r = w - block * a.p.rows;
        const int32_t *plan = reinterpret_cast<const int32_t *>(a.own) + 2 * b;
        const int g0 = plan[0], g1 = plan[1];
        const int at = (r / 32 * (RANK / 8) + cq) * 256 + 4 * (r % 32 + 32 * (lane >> 5)), ml = a.p.rows * RANK + 2 * r;
        for (int g = g0 + wave; g <= g1; g += W) {
            const float *slot = g0 == g1 ? a.full + ((int64_t)b * a.p.blocks + block) * a.p.slot
                                         : a.own + a.p.first + (2 * ((int64_t)block * a.p.groups + g) + (g == g0 ? 1 : 0)) * a.p.slot;
            add(slot + at, slot + ml);
        }
    }
    if (W > 1) {
        so[wave][lane] = o;
        sm[wave][lane] = m;
        sl[wave][lane] = l;
        __syncthreads();
        if (wave) return;
#pragma unroll
        for (int w = 1; w < W; ++w) m = fmaxf(m, sm[w][lane]);
        o = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        l = 0.0f;
#pragma unroll
        for (int w = 0; w < W; ++w) {
            const float f = sm[w][lane] == m ? 1.0f : __builtin_amdgcn_exp2f(sm[w][lane] - m);
            const f32x4 v = so[w][lane];
            l = __builtin_fmaf(sl[w][lane], f, l);
#pragma unroll
            for (int i = 0; i < 4; ++i) o[i] = __builtin_fmaf(v[i], f, o[i]);
        }
    }
    if (row >= rows) return;
    const float f = l == 0.0f ? 0.0f : 1.0f / l;
    x4<T> v;
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = (T)(o[i] * f);
    *reinterpret_cast<x4<T> *>(static_cast<T *>(a.out) + row * RANK + 8 * cq + 4 * (lane >> 5)) = v;
    if (a.lse && cq == 0 && lane < 32) a.lse[row] = l == 0.0f ? NEG : (m + __builtin_amdgcn_logf(l)) * LN2;
}

// Calls f with the type, rank and format of the dims as types.
template <class F>
hipError_t with_shape(const coli_mla_dims &d, F f) {
    return mla_with_type(d.dtype, [&](auto t) {
        using T = decltype(t);
        if (d.kv_format == COLI_KV_E4M3) return d.rank == 512 ? f(Shd<T, 512, true>()) : f(Shd<T, 256, true>());
        return d.rank == 512 ? f(Shd<T, 512, false>()) : f(Shd<T, 256, false>());
    });
}

}  // namespace

size_t mla_shared_part_bytes(const coli_mla_dims &d, int64_t rows, int prefix) {
    // slots are counted by workgroup + block of rows: a bound that grows with each argument
    const Units u = shd_units(rows, prefix);
    return 4 * (size_t)(SHD_ROWS * d.rank + 2 * SHD_ROWS) * (size_t)(u.shares + (rows + SHD_ROWS - 1) / SHD_ROWS);
}

hipError_t launch_mla_shared(const MlaSharedArgs &a, const coli_mla_dims &d, hipStream_t st) {
    const Units u = shd_units((int64_t)a.batch * a.n_q * a.heads, a.prefix);
    return with_shape(d, [&](auto shape) {
        using D = decltype(shape);
        const hipError_t e = ensure_dyn_smem(reinterpret_cast<const void *>(&k_mla_shared<D>), D::LDS);
        if (e != hipSuccess) return e;
        hipLaunchKernelGGL(k_mla_shared<D>, dim3(u.shares), dim3(256), D::LDS, st, a, u);
        return hipGetLastError();
    });
}

hipError_t launch_mla_shared_join(const MlaSharedArgs &a, const coli_mla_dims &d, hipStream_t st) {
    const int64_t rows = (int64_t)a.batch * a.n_q * a.heads;
    const Units u = shd_units(rows, a.prefix);
    return with_shape(d, [&](auto shape) {
        using D = decltype(shape);
        const dim3 grid((uint32_t)((rows + 31) / 32 * (D::RANK / 8)));
        hipLaunchKernelGGL((k_mla_shared_join<typename D::T, D::RANK, 4>), grid, dim3(256), 0, st, a, u);
        return hipGetLastError();
    });
}

}  // namespace coli

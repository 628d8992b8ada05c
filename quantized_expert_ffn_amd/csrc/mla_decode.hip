// Absorbed attention of a few new tokens a sequence over the paged latents:
//
//   s_rt = scale (<q_r, c_t> + <p_r, k_t>),  out_r = sum_t e^{s_rt} c_t / sum_t e^{s_rt}
//
// for the n_q * n_heads query rows r of a sequence.  Every row reads the same
// latents, so a sequence is one product [rows x (rank + 64)] x [tokens] and
// one [tokens] x [rank], of the same cached tile: read from memory once, used
// twice from LDS.
#include "kernels.h"
#include "mla_mfma.h"

namespace coli {
namespace {

constexpr int DEC_TILE = 64;     // tokens a tile
constexpr float LOG2E = 1.44269504088896340736f, LN2 = 0.69314718055994530942f;
// The running maximum moves only when a score exceeds it by this many powers
// of two: weights then reach 2^8, which every type here holds, and most tiles
// spare the pass over the accumulators.
constexpr float MAX_LAG = 8.0f;

// Four wavefronts: RG groups of 32 rows, each of CG = 4 / RG wavefronts that
// share the output's columns.  Wavefronts 0 and 1 of a group score half of a
// tile's tokens each and hand their weights to the others through LDS.
template <class T_, int RANK_, bool FP8_, int RG_>
struct Dec {
    using T = T_;
    static constexpr int RANK = RANK_, RG = RG_, CG = 4 / RG_;
    static constexpr bool FP8 = FP8_;
    static constexpr int ROWS = 32 * RG;
    static constexpr int ROW = FP8 ? RANK + 2 * MLA_ROPE : 2 * (RANK + MLA_ROPE);   // bytes of a cached token
    static constexpr int CB = ROW / 128;              // blocks of eight 16-byte chunks in it
    static constexpr int PE = CB - 1;                 // the last holds the rotated key
    static constexpr int KS = (RANK + MLA_ROPE) / 16; // matrix steps of a score
    static constexpr int CT = RANK / 32 / CG;         // 32-column tiles of a wavefront's output
    static constexpr int TILE = DEC_TILE * ROW;
    static constexpr int L_OFF = 2 * TILE;                    // int64 [2][64]: row offsets of tiles to come
    static constexpr int L_SCALE = L_OFF + 2 * 8 * DEC_TILE;  // float [2][64]: E4M3 scales
    static constexpr int L_TOP = L_SCALE + 2 * 4 * DEC_TILE;  // float [RG][2][32]: maxima, at the end sums
    static constexpr int L_UNIT = L_TOP + RG * 2 * 32 * 4;    // float [2]: largest scale of a tile
    static constexpr int L_P = L_UNIT + 16;                   // weights: [RG][2][2][64 lanes] of 16 bytes
    static constexpr int LDS = L_P + RG * 2 * 2048;
    static constexpr int SLOT = ROWS * RANK + 2 * ROWS;       // floats of a partial result
};

// A sequence's tiles; one without tokens keeps an empty tile, whose owner
// writes its zeros.
__device__ __forceinline__ int dec_tiles(int len) { return len > 0 ? (len + DEC_TILE - 1) / DEC_TILE : 1; }

__device__ __forceinline__ int wave_scan(int v, int lane) {
    for (int o = 1; o < 64; o <<= 1) {
        const int u = __shfl_up(v, o);
        if (lane >= o) v += u;
    }
    return v;
}

// Tiles are shared out evenly: workgroup g of `groups` has tiles
// first(g) .. first(g + 1) - 1 of the batch's tiles in order.
__device__ __forceinline__ int64_t dec_first(int64_t tiles, int groups, int g) { return tiles * g / groups; }
__device__ __forceinline__ int dec_owner(int64_t tiles, int groups, int64_t tile) {
    return (int)(((tile + 1) * groups - 1) / tiles);
}

// Swizzle of a token's 16-byte chunks: LDS holds a tile as [8 tokens][8
// chunks] blocks of 1 KiB, which is what a wavefront's load writes, chunk c of
// token t at position (c ^ swz(t)) of its 128 bytes.  Sixteen tokens' same
// chunk, and four tokens' neighbouring ones, then lie in sixteen different
// groups of banks.
__device__ __forceinline__ int dec_swz(int t) { return (t & 6) | ((t >> 3) & 1); }

template <class D>
__global__ __launch_bounds__(256, 1) void k_mla_decode(MlaDecodeArgs a, int groups) {
    using T = typename D::T;
    constexpr int RANK = D::RANK, CT = D::CT, KS = D::KS;
    constexpr float NEG = -__builtin_inff();
    const int tid = threadIdx.x, lane = tid & 63, wave = uniform(tid >> 6);
    const int n = lane & 31, hf = lane >> 5;
    const int rg = wave / D::CG, cg = wave % D::CG, th = cg & 1;
    const int g = blockIdx.x, rows = a.n_q * a.heads;
    const int block_row = blockIdx.y * D::ROWS, wave_row = block_row + 32 * rg;
    const bool has_rows = wave_row < rows;

    // ---- this workgroup's tiles
    int64_t tiles = 0;
    for (int b = 0; b < a.batch; b += 64) {
        const int len = b + lane < a.batch ? mla_len(a.kv_lens, b + lane, a.max_kv, a.status) : 0;
        tiles += uniform(__shfl(wave_scan(b + lane < a.batch ? dec_tiles(len) : 0, lane), 63));
    }
    const int shares = groups < tiles ? groups : (int)tiles;   // none of them empty
    if (g >= shares) return;
    int64_t at = dec_first(tiles, shares, g);
    const int64_t stop = dec_first(tiles, shares, g + 1);
    int seq = 0;
    int64_t seq_first = 0;
    {
        int64_t base = 0;
        bool found = false;
        for (int b = 0; b < a.batch; b += 64) {
            const int mine = b + lane < a.batch ? dec_tiles(mla_len(a.kv_lens, b + lane, a.max_kv, a.status)) : 0;
            const int incl = wave_scan(mine, lane);
            const int64_t f = base + incl - mine;
            if (g == 0 && blockIdx.y == 0 && wave == 0 && b + lane < a.batch) {   // for the join
                int32_t *plan = reinterpret_cast<int32_t *>(a.part) + 2 * (b + lane);
                plan[0] = dec_owner(tiles, shares, f);
                plan[1] = dec_owner(tiles, shares, f + mine - 1);
            }
            const uint64_t hit = __ballot(base + incl > at);
            if (!found && hit) {
                const int l = __builtin_ctzll(hit);
                seq = b + l;
                seq_first = base + __shfl(incl - mine, l);
                found = true;
            }
            base += __shfl(incl, 63);
        }
    }
    seq = uniform(seq);
    int left = uniform((int)(stop - at));
    at = uniform64(at - seq_first);  // from here on in tiles of the sequence

    // ---- lane addresses inside a tile
    uint32_t ka[4], va[4];
    {
        const int t = 32 * th + n, f = dec_swz(t);
#pragma unroll
        for (int v = 0; v < 4; ++v)
            ka[v] = (t >> 3) * D::CB * 1024 + (t & 7) * 128 + (((2 * v + hf) ^ f) << 4);
        const int x = lane & 15, cb = (lane >> 4) & 1;
#pragma unroll
        for (int v = 0; v < 4; ++v) {
            if (D::FP8) {   // va[ct & 3], matrix step s at + 2 s groups of tokens
                const int jr = x >> 1, t8 = 4 * hf + (jr & 3);
                const int fv = dec_swz(8 * (jr >> 2) + t8);
                va[v] = (jr >> 2) * D::CB * 1024 + t8 * 128 + (((2 * v + cb) ^ fv) << 4) + 8 * (x & 1);
            } else {        // va[2 e + (ct & 1)], e the token group of a step
                const int e = v >> 1, t8 = 4 * hf + (x >> 2);
                const int fv = dec_swz(8 * e + t8);
                va[v] = e * D::CB * 1024 + t8 * 128 +
                        (((4 * (v & 1) + 2 * cb + ((x & 3) >> 1)) ^ fv) << 4) + 8 * (x & 1);
            }
        }
    }
    // what this thread loads: chunk (lane % 8) of tokens 16 wave + lane / 8 and + 8
    const int lt0 = 16 * wave + (lane >> 3), lt1 = lt0 + 8;
    const uint8_t *src0 = a.c.pages + (((lane & 7) ^ dec_swz(lt0)) << 4);
    const uint8_t *src1 = a.c.pages + (((lane & 7) ^ dec_swz(lt1)) << 4);

    while (left > 0) {
        const int len = uniform(mla_len(a.kv_lens, seq, a.max_kv, a.status));
        const int n_tiles = dec_tiles(len);
        const int lo = (int)at, hi = (int)(left < n_tiles - at ? at + left : n_tiles);
        const int first_j = block_row / a.heads;
        const int block_seen = len - a.n_q + 1 + first_j;          // tokens every row here sees
        const int wave_seen = len - a.n_q + 1 + wave_row / a.heads;
        const int row = wave_row + n;
        const int seen = row < rows ? len - a.n_q + 1 + row / a.heads : len;

        // The tiles' loads run one tile ahead, their row offsets two, their page ids three.
        auto token = [&](int tile) { return min(tile * DEC_TILE + tid, len - 1); };   // behind the end: the last again
        auto page_of = [&](int tile) -> int {
            return tid < DEC_TILE && tile < hi && len > 0 ? a.c.table[(int64_t)seq * a.c.width + token(tile) / a.c.page] : 0;
        };
        auto slot_of = [&](int tile, int pid) -> int64_t {
            if ((uint32_t)pid >= (uint32_t)a.c.n_pages) {
                raise_status(a.status, ST_BADPAGE);
                pid = 0;
            }
            return (int64_t)pid * a.c.page + (len > 0 ? token(tile) % a.c.page : 0);
        };
        // Offsets (and scales) of a tile, from its page id; the scales are put down a tile later.
        float sc_next = 0.0f;
        auto put_offsets = [&](int tile, int pid) {
            const int64_t slot = slot_of(tile, pid);
            lds_write<int64_t>(D::L_OFF + 8 * (((tile - lo) & 1) * DEC_TILE + tid), slot * D::ROW);
            if (D::FP8) sc_next = a.c.scale[slot];
        };
        auto put_scales = [&](int tile) {
            const int buf = (tile - lo) & 1;
            lds_write<float>(D::L_SCALE + 4 * (buf * DEC_TILE + tid), sc_next);
            float top = finite_f32(sc_next) ? fabsf(sc_next) : 0.0f;
            for (int x = 32; x; x >>= 1) top = fmaxf(top, __shfl_xor(top, x));
            if (tid == 0) lds_write<float>(D::L_UNIT + 4 * buf, top);
        };
        auto issue = [&](int tile) {
            const int buf = (tile - lo) & 1;
            const uint8_t *p0 = src0 + lds_read<int64_t>(D::L_OFF + 8 * (buf * DEC_TILE + lt0));
            const uint8_t *p1 = src1 + lds_read<int64_t>(D::L_OFF + 8 * (buf * DEC_TILE + lt1));
            const uint32_t d = buf * D::TILE + 2 * wave * D::CB * 1024;
#pragma unroll
            for (int c = 0; c < D::CB; ++c) {
                load_to_lds(p0 + 128 * c, d + 1024 * c);
                load_to_lds(p1 + 128 * c, d + (D::CB + c) * 1024);
            }
        };

        int pid = page_of(lo), pid2 = page_of(lo + 1);
        __syncthreads();   // LDS of the segment before is free
        if (wave == 0) {
            put_offsets(lo, pid);
            if (D::FP8) put_scales(lo);
            if (lo + 1 < hi) put_offsets(lo + 1, pid2);
        }
        __syncthreads();
        issue(lo);
        pid = page_of(lo + 2);
        x8<T> qf[KS];
        {
            const int64_t r = (int64_t)seq * rows + (row < rows ? row : 0);
            const T *ql = static_cast<const T *>(a.q_lat) + r * RANK, *qp = static_cast<const T *>(a.q_pe) + r * MLA_ROPE;
#pragma unroll
            for (int s = 0; s < KS; ++s) {
                const int k = s < RANK / 16 ? (D::FP8 ? 32 * (s >> 1) + 16 * hf + 8 * (s & 1) : 16 * s + 8 * hf)
                                            : 16 * (s - RANK / 16) + 8 * hf;
                qf[s] = *reinterpret_cast<const x8<T> *>((s < RANK / 16 ? ql : qp) + k);
            }
#pragma unroll
            for (int s = 0; s < KS; ++s) arrived(qf[s]);
        }
        f32x16 o[CT];
#pragma unroll
        for (int c = 0; c < CT; ++c)
#pragma unroll
            for (int r = 0; r < 16; ++r) o[c][r] = 0.0f;
        float m = NEG, l = 0.0f, unit = 0.0f;   // unit: E4M3 accumulators are in units of it
        const bool works = has_rows && len > 0, scores = works && cg < 2;
        const uint32_t top_at = D::L_TOP + 4 * (64 * rg + n), p_at = D::L_P + 4096 * rg + 16 * lane;

        for (int tile = lo; tile < hi; ++tile) {
            const int buf = (tile - lo) & 1;
            const uint32_t base = buf * D::TILE;
            const int t0 = tile * DEC_TILE, tw = t0 + 32 * th;
            wait_vm<0>();
            arrived(pid);
            arrived(sc_next);
            barrier_lds();   // the tile is there, and every wavefront is done with the one before
            if (tile + 1 < hi) issue(tile + 1);

            f32x16 s;
            float sc[16];
            if (scores) {
#pragma unroll
                for (int r = 0; r < 16; ++r) s[r] = 0.0f;
                // operands four reads ahead of their products; no more, or the compiler hoists reads until it spills
                u32x4 ahead[2][4];
                auto fetch = [&](int i) {
                    const uint32_t w = D::FP8 && i >= RANK / 32 ? base + ka[i & 3] + D::PE * 1024 : base + ka[i & 3] + (i >> 2) * 1024;
                    return lds_read<u32x4>(w);
                };
                constexpr int READS = D::CB * 4;
#pragma unroll
                for (int i = 0; i < 4; ++i) ahead[0][i] = fetch(i);
                if (D::FP8) {
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const f32x4 v = lds_read<f32x4>(D::L_SCALE + 4 * (buf * DEC_TILE + 32 * th + 8 * q + 4 * hf));
#pragma unroll
                        for (int i = 0; i < 4; ++i) sc[4 * q + i] = v[i];
                    }
                }
#pragma unroll
                for (int c = 0; c < READS; c += 4) {
                    __builtin_amdgcn_sched_barrier(0);
                    if (c + 4 < READS) {
#pragma unroll
                        for (int i = 0; i < 4; ++i) ahead[(c / 4 + 1) & 1][i] = fetch(c + 4 + i);
                    }
                    if (D::FP8 && c == RANK / 32) {
#pragma unroll
                        for (int r = 0; r < 16; ++r) s[r] *= sc[r];
                    }
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const u32x4 w = ahead[(c / 4) & 1][i];
                        const int k = c + i;
                        if (D::FP8 && k < RANK / 32) {
                            s = mfma32<T>(widen8<T>(u32x2{w[0], w[1]}), qf[2 * k], s);
                            s = mfma32<T>(widen8<T>(u32x2{w[2], w[3]}), qf[2 * k + 1], s);
                        } else {
                            s = mfma32<T>(__builtin_bit_cast(x8<T>, w), qf[D::FP8 ? k + RANK / 32 : k], s);
                        }
                    }
                }
                __builtin_amdgcn_sched_barrier(0);
                const float scale = a.scale * LOG2E;
                if (tw + 32 > wave_seen) {
#pragma unroll
                    for (int r = 0; r < 16; ++r)
                        s[r] = tw + 8 * (r >> 2) + 4 * hf + (r & 3) < seen ? s[r] * scale : NEG;
                } else {
#pragma unroll
                    for (int r = 0; r < 16; ++r) s[r] *= scale;
                }
                float top = s[0];
#pragma unroll
                for (int r = 1; r < 16; ++r) top = fmaxf(top, s[r]);
                lds_write<float>(top_at + 128 * th, half_max(top));
            }
            if (wave == 0 && tile + 1 < hi) {
                if (D::FP8) put_scales(tile + 1);
                if (tile + 2 < hi) {
                    put_offsets(tile + 2, pid);
                    pid = page_of(tile + 3);
                }
            }
            barrier_lds();
            if (works) {
                const float top = fmaxf(lds_read<float>(top_at), lds_read<float>(top_at + 128));
                float grown = unit;
                // the largest scale so far: weights times scales stay in the type's range
                if (D::FP8) grown = fmaxf(unit, lds_read<float>(D::L_UNIT + 4 * buf));
                if (__ballot(top > m + MAX_LAG || grown > unit)) {
                    const float to = top > m + MAX_LAG ? top : m;
                    float f = m == to ? 1.0f : __builtin_amdgcn_exp2f(m - to);
                    l *= f;
                    m = to;
                    if (D::FP8 && grown > unit) {
                        f *= unit / grown;
                        unit = grown;
                    }
#pragma unroll
                    for (int c = 0; c < CT; ++c)
#pragma unroll
                        for (int r = 0; r < 16; ++r) o[c][r] *= f;
                }
                if (scores) {
                    const float ref = m == NEG ? 0.0f : m;
                    const float inv = D::FP8 ? (unit > 0.0f ? 1.0f / unit : 0.0f) : 1.0f;
                    float sum = 0.0f;
                    x8<T> p[2];
#pragma unroll
                    for (int r = 0; r < 16; ++r) {
                        float w = __builtin_amdgcn_exp2f(s[r] - ref);
                        sum += w;
                        if (D::FP8) w = s[r] == NEG ? 0.0f : w * (sc[r] * inv);
                        p[r >> 3][r & 7] = (T)w;
                    }
                    l += sum;
                    lds_write(p_at + 2048 * th, p[0]);
                    lds_write(p_at + 2048 * th + 1024, p[1]);
                }
            }
            // A tile that some rows see only in part, though its tokens exist: values that are not finite would reach
            // rows that do not see them as 0 * NaN; a row that does see them has them in its scores already.
            if (block_seen < len && t0 + DEC_TILE > block_seen) {
                const int from = block_seen > t0 ? block_seen - t0 : 0;
                constexpr int CH = (D::CB - 1) * 8;
                for (int i = tid; i < (DEC_TILE - from) * CH; i += 256) {
                    const int t = from + i / CH, c = i % CH;
                    const uint32_t w = base + ((t >> 3) * D::CB + (c >> 3)) * 1024 + (t & 7) * 128 + ((c & 7) << 4);
                    if (D::FP8) {
                        u32x4 v = lds_read<u32x4>(w);
#pragma unroll
                        for (int k = 0; k < 4; ++k)
#pragma unroll
                            for (int y = 0; y < 32; y += 8)
                                if (((v[k] >> y) & 0x7f) == 0x7f) v[k] &= ~(0xffu << y);
                        lds_write(w, v);
                    } else {
                        x8<T> v = lds_read<x8<T>>(w);
#pragma unroll
                        for (int k = 0; k < 8; ++k)
                            if (!finite_f32((float)v[k])) v[k] = (T)0.0f;
                        lds_write(w, v);
                    }
                }
            }
            barrier_lds();
            if (works) {
                x8<T> p[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) p[k] = lds_read<x8<T>>(p_at + 1024 * k);
                u32x4 ahead[2][4];   // a column tile's four matrix steps (E4M3: two words each)
                auto fetch = [&](int c, int k) {
                    const int col = cg * CT + c;
                    u32x4 v = {0, 0, 0, 0};
                    if (D::FP8) {
                        // CT is 2 or a multiple of 4: where it is 2, the column tile's low bits are not c's
                        const uint32_t lo_bits = CT % 4 ? va[0] ^ ((col & 3) << 5) : va[c & 3];
                        const u32x2 w = lds_read_tr8(base + lo_bits + 2 * k * D::CB * 1024 + (col >> 2) * 1024);
                        v[0] = w[0];
                        v[1] = w[1];
                        return v;
                    }
                    const uint32_t w = base + 2 * k * D::CB * 1024 + (col >> 1) * 1024;
                    const u32x2 v0 = __builtin_bit_cast(u32x2, lds_read_tr16<T>(w + va[c & 1]));
                    const u32x2 v1 = __builtin_bit_cast(u32x2, lds_read_tr16<T>(w + va[2 + (c & 1)]));
                    return u32x4{v0[0], v0[1], v1[0], v1[1]};
                };
#pragma unroll
                for (int k = 0; k < 4; ++k) ahead[0][k] = fetch(0, k);
#pragma unroll
                for (int c = 0; c < CT; ++c) {
                    __builtin_amdgcn_sched_barrier(0);
                    if (c + 1 < CT) {
#pragma unroll
                        for (int k = 0; k < 4; ++k) ahead[(c + 1) & 1][k] = fetch(c + 1, k);
                    }
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const u32x4 w = ahead[c & 1][k];
                        const x8<T> v = D::FP8 ? widen8<T>(u32x2{w[0], w[1]}) : __builtin_bit_cast(x8<T>, w);
                        o[c] = mfma32<T>(v, p[k], o[c]);
                    }
                }
                __builtin_amdgcn_sched_barrier(0);
            }
        }

        // ---- the segment's result: the sums of both halves of the tokens, then out or a partial result
        barrier_lds();
        if (scores) {
            l = half_sum(l);
            lds_write<float>(top_at + 128 * th, l);
        }
        barrier_lds();
        l = works ? lds_read<float>(top_at) + lds_read<float>(top_at + 128) : 0.0f;
        if (D::FP8) {
#pragma unroll
            for (int c = 0; c < CT; ++c)
#pragma unroll
                for (int r = 0; r < 16; ++r) o[c][r] *= unit;
        }
        if (lo == 0 && hi == n_tiles) {
            if (row < rows) {
                const int64_t r = (int64_t)seq * rows + row;
                const float f = l == 0.0f ? 0.0f : 1.0f / l;
                T *dst = static_cast<T *>(a.out) + r * RANK + cg * CT * 32 + 4 * hf;
#pragma unroll
                for (int c = 0; c < CT; ++c)
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        x4<T> v;
#pragma unroll
                        for (int i = 0; i < 4; ++i) v[i] = (T)(o[c][4 * q + i] * f);
                        *reinterpret_cast<x4<T> *>(dst + 32 * c + 8 * q) = v;
                    }
                if (a.lse && hf == 0 && cg == 0) a.lse[r] = l == 0.0f ? NEG : (m + __builtin_amdgcn_logf(l)) * LN2;
            }
        } else if (has_rows) {
            // slot 0: the segment begins inside its sequence, slot 1: with it
            const int64_t slot = ((int64_t)blockIdx.y * groups + g) * 2 + (lo == 0 ? 1 : 0);
            float *dst = a.part + 2 * ((a.batch + 7) & ~7) + slot * D::SLOT;
#pragma unroll
            for (int c = 0; c < CT; ++c)
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    f32x4 v;
#pragma unroll
                    for (int i = 0; i < 4; ++i) v[i] = o[c][4 * q + i];
                    *reinterpret_cast<f32x4 *>(dst + ((rg * (RANK / 32) + cg * CT + c) * 4 + q) * 256 + 4 * lane) = v;
                }
            if (hf == 0 && cg == 0)
                *reinterpret_cast<float2 *>(dst + D::ROWS * RANK + 2 * (32 * rg + n)) = make_float2(m, l);
        }
        left -= hi - lo;
        at = 0;
        ++seq;
    }
}

// Joins the partial results of a sequence: out = sum_g 2^{m_g - M} o_g / sum_g
// 2^{m_g - M} l_g, over the workgroups in order.  One workgroup takes 32 rows
// by 8 columns (of each lane half), its wavefronts every fourth partial.
template <class T, int RANK, int ROWS>
__global__ __launch_bounds__(256) void k_mla_join(MlaDecodeArgs a, int groups) {
    constexpr int SLOT = ROWS * RANK + 2 * ROWS;
    constexpr float NEG = -__builtin_inff();
    const int b = blockIdx.z, lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int32_t *plan = reinterpret_cast<const int32_t *>(a.part) + 2 * b;
    const int g0 = plan[0], g1 = plan[1];
    if (g0 == g1) return;
    __shared__ f32x4 so[4][64];
    __shared__ float sm[4][64], sl[4][64];
    const int rgs = blockIdx.y, rb = rgs / (ROWS / 32), rg = rgs % (ROWS / 32), cq = blockIdx.x, n = lane & 31;
    const float *part = a.part + 2 * ((a.batch + 7) & ~7) + (int64_t)rb * groups * 2 * SLOT;
    f32x4 o = {0.0f, 0.0f, 0.0f, 0.0f};
    float m = NEG, l = 0.0f;
#pragma unroll 4
    for (int g = g0 + wave; g <= g1; g += 4) {
        const float *p = part + (int64_t)(2 * g + (g == g0 ? 1 : 0)) * SLOT;
        const float2 ml = *reinterpret_cast<const float2 *>(p + ROWS * RANK + 2 * (32 * rg + n));
        const f32x4 v = *reinterpret_cast<const f32x4 *>(p + (rg * (RANK / 32) * 4 + cq) * 256 + 4 * lane);
        const float to = fmaxf(m, ml.x);
        const float fa = m == to ? 1.0f : __builtin_amdgcn_exp2f(m - to);
        const float fb = ml.x == to ? 1.0f : __builtin_amdgcn_exp2f(ml.x - to);
        l = l * fa + ml.y * fb;
#pragma unroll
        for (int i = 0; i < 4; ++i) o[i] = o[i] * fa + v[i] * fb;
        m = to;
    }
    so[wave][lane] = o;
    sm[wave][lane] = m;
    sl[wave][lane] = l;
    __syncthreads();
    if (wave) return;
#pragma unroll
    for (int w = 1; w < 4; ++w) {
        const float mb = sm[w][lane], lb = sl[w][lane];
        const f32x4 v = so[w][lane];
        const float to = fmaxf(m, mb);
        const float fa = m == to ? 1.0f : __builtin_amdgcn_exp2f(m - to);
        const float fb = mb == to ? 1.0f : __builtin_amdgcn_exp2f(mb - to);
        l = l * fa + lb * fb;
#pragma unroll
        for (int i = 0; i < 4; ++i) o[i] = o[i] * fa + v[i] * fb;
        m = to;
    }
    const int rows = a.n_q * a.heads, row = 32 * rgs + n;
    if (row >= rows) return;
    const int64_t r = (int64_t)b * rows + row;
    const float f = l == 0.0f ? 0.0f : 1.0f / l;
    x4<T> v;
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = (T)(o[i] * f);
    *reinterpret_cast<x4<T> *>(static_cast<T *>(a.out) + r * RANK + 8 * cq + 4 * (lane >> 5)) = v;
    if (a.lse && cq == 0 && lane < 32) a.lse[r] = l == 0.0f ? NEG : (m + __builtin_amdgcn_logf(l)) * LN2;
}

// Rows of a workgroup, and how many workgroups share the batch's tiles: as
// many as fill the 256 CUs once (a workgroup's LDS and registers take one).
int dec_rows(int rows) { return rows <= 32 ? 32 : 64; }
int dec_groups(int batch, int rows, int max_kv) {
    const int per = dec_rows(rows), blocks = (rows + per - 1) / per;
    const int64_t tiles = (int64_t)batch * (max_kv > 0 ? (max_kv + DEC_TILE - 1) / DEC_TILE : 1);
    int64_t groups = blocks < 256 ? 256 / blocks : 1;
    if (groups > tiles) groups = tiles;
    return (int)groups;
}

template <class D>
hipError_t launch(const MlaDecodeArgs &a, hipStream_t st) {
    const int rows = a.n_q * a.heads, groups = dec_groups(a.batch, rows, a.max_kv);
    const int blocks = (rows + D::ROWS - 1) / D::ROWS;
    const hipError_t e = ensure_dyn_smem(reinterpret_cast<const void *>(&k_mla_decode<D>), D::LDS);
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(k_mla_decode<D>, dim3(groups, blocks), dim3(256), D::LDS, st, a, groups);
    if (groups > 1)
        hipLaunchKernelGGL((k_mla_join<typename D::T, D::RANK, D::ROWS>),
                           dim3(D::RANK / 8, (rows + 31) / 32, a.batch), dim3(256), 0, st, a, groups);
    return hipGetLastError();
}

template <class T, int RANK, bool FP8>
hipError_t by_rows(const MlaDecodeArgs &a, hipStream_t st) {
    return dec_rows(a.n_q * a.heads) == 32 ? launch<Dec<T, RANK, FP8, 1>>(a, st)
                                           : launch<Dec<T, RANK, FP8, 2>>(a, st);
}

}  // namespace

// A bound that grows with each argument, so that a workspace serves every
// smaller call: blocks * groups partial results, twice.
size_t mla_decode_part_bytes(const coli_mla_dims &d, int batch, int n_q, int max_kv) {
    const int rows = n_q * d.n_heads, per = dec_rows(rows), blocks = (rows + per - 1) / per;
    const int64_t tiles = (int64_t)batch * (max_kv > 0 ? (max_kv + DEC_TILE - 1) / DEC_TILE : 1);
    int64_t slots = blocks > 256 ? blocks : 256;
    if (slots > blocks * tiles) slots = blocks * tiles;
    return 8 * (((size_t)batch + 7) & ~(size_t)7) + 4 * 2 * ((size_t)per * d.rank + 2 * per) * (size_t)slots;
}

hipError_t launch_mla_decode(const MlaDecodeArgs &a, const coli_mla_dims &d, hipStream_t st) {
    return mla_with_type(d.dtype, [&](auto t) {
        using T = decltype(t);
        const bool fp8 = d.kv_format == COLI_KV_E4M3;
        if (d.rank == 512) return fp8 ? by_rows<T, 512, true>(a, st) : by_rows<T, 512, false>(a, st);
        return fp8 ? by_rows<T, 256, true>(a, st) : by_rows<T, 256, false>(a, st);
    });
}

}  // namespace coli

// Products with the latent projections, out[t, o] = sum_k w[o, k] x[t, k]:
// project (a product a head) and expand (all heads at once, the rows x
// gathered out of the paged cache).
//
// Both keep their reduction dimension contiguous in both operands, so one
// tiled product serves them: a workgroup takes tiles of TM output features by
// its TN tokens, w as the A operand, so that a lane's results are four
// consecutive features of one token.  Steps of 64 along k, a line of 128 bytes
// of every row, form one stream over a workgroup's tiles, through a ring of
// LDS stages loaded straight from memory; results pass through the stage that
// was used last, to leave in whole lines.
//
// What bounds it: expand of 8192 rows, 64 heads, rank 512, 192 + 256 features,
// bf16: 236 us, 1.0 PFLOP/s and 470 MB written.  A build of 239 us took 174
// without its loads and 167 with one product in eight: with two stages a step
// waits for all of them, and they have been out for one step.  LDS serves them
// beside 0.75 KiB of operands a product (128 x 128 a wavefront would read 0.5,
// and spills; 128 x 96 takes 300 us).  Stores that
// pass L2 by took it there from 275 us, 216 of them without any store.  Project
// is bound by its bytes: 133 tokens, 128 heads, 512 -> 128, fp16: 8.2 us, 4.7
// TB/s; one token, 64 heads, 192 -> 512, bf16: 4.1 us.
#include "kernels.h"
#include "mla_mfma.h"

namespace coli {
namespace {

// NW wavefronts in WM x NW / WM pieces of a tile; WGS workgroups fit a CU.
// STREAM: results go past the L2, which keeps the operands (8192 rows, 64
// heads, 470 MB of results: 275 us without, 240 us with).
template <class T_, bool FP8_, int TM_, int TN_, int NW_, int WM_, int STAGES_, int WGS_, bool STREAM_ = false>
struct Gemm {
    using T = T_;
    static constexpr bool FP8 = FP8_, STREAM = STREAM_;
    static constexpr int TM = TM_, TN = TN_, NW = NW_, WM = WM_, WN = NW_ / WM_, STAGES = STAGES_, WGS = WGS_;
    static constexpr int FM = TM / WM / 32, FN = TN / WN / 32;       // 32 x 32 tiles of a wavefront
    static constexpr int BROW = FP8 ? 64 : 128;                      // bytes of a token's step
    static constexpr int ASTAGE = TM * 128, STAGE = ASTAGE + TN * BROW;
    static constexpr int LA = TM / 8 / NW;                           // 1 KiB loads a wavefront and step
    static constexpr int LB_ALL = TN * BROW / 1024, LB = LB_ALL < NW ? 1 : LB_ALL / NW;
    static constexpr int OF = FM < 2 ? 1 : 2;                        // 32-feature tiles that leave together
    static constexpr int OROW = 64 * OF + 16, OUT = NW * 32 * OROW;  // bytes of a token's, of the wavefronts'
    static constexpr int LDS = STAGES * STAGE;
    static_assert(OUT <= STAGE && LDS * WGS <= 160 * 1024, "LDS");
};

// Lane's place in a 1 KiB load: eight rows of eight chunks (sixteen of four
// for codes), swizzled so that sixteen rows' same chunk lies in sixteen groups
// of banks.
__device__ __forceinline__ int swz(int r) { return 4 * ((r >> 1) & 1) + 2 * ((r >> 2) & 1) + ((r >> 3) & 1); }
__device__ __forceinline__ int swz8(int r) { return (r >> 2) & 3; }

// The products of the tiles mt .. mt_end - 1 of TM features.  w: [features]
// [64 steps]; xp: this lane's sources of its B loads at k = 0; row_of: where a
// token's features go, or null.
template <class D, class Row>
__device__ __forceinline__ void gemm_tiles(const typename D::T *w, int features, const uint8_t *const (&xp)[D::LB], int steps,
                                           int mt, int mt_end, const float (&scale)[D::FN], Row row_of) {
    using T = typename D::T;
    const int tid = threadIdx.x, lane = tid & 63, wave = uniform(tid >> 6), n = lane & 31, hf = lane >> 5;
    const int wm = wave % D::WM, wn = wave / D::WM;
    // ---- the stream of loads
    const uint8_t *wp[D::LA];
    int load_mt = mt, load_k = 0, load_slot = 0;
    auto aim = [&] {
#pragma unroll
        for (int i = 0; i < D::LA; ++i) {
            const int r = (wave * D::LA + i) * 8 + (lane >> 3), o = min(load_mt * D::TM + r, features - 1);
            wp[i] = reinterpret_cast<const uint8_t *>(w + (int64_t)o * (64 * steps)) + (((lane & 7) ^ swz(r)) << 4);
        }
    };
    auto issue = [&] {
        if (load_mt >= mt_end) return;
        const uint32_t base = load_slot * D::STAGE;
#pragma unroll
        for (int i = 0; i < D::LA; ++i) load_to_lds(wp[i] + load_k * 128, base + (wave * D::LA + i) * 1024);
#pragma unroll
        for (int i = 0; i < D::LB; ++i)   // fewer loads than wavefronts: some load the same once more
            load_to_lds(xp[i] + load_k * D::BROW, base + D::ASTAGE + (wave * D::LB + i) % D::LB_ALL * 1024);
        load_slot = load_slot == D::STAGES - 1 ? 0 : load_slot + 1;
        if (++load_k == steps) {
            load_k = 0;
            ++load_mt;
            aim();
        }
    };
    aim();
#pragma unroll
    for (int i = 0; i < D::STAGES - 1; ++i) issue();
    // Matrix step e of a stage takes k = 32 (e / 2) + 16 hf + 8 (e % 2) + 0..7 on both sides: 16 bytes of codes then hold
    // two steps.
    uint32_t aa[4], ba[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const uint32_t c = ((4 * (e >> 1) + 2 * hf + (e & 1)) ^ swz(n)) << 4, r = (n >> 3) * 1024 + (n & 7) * 128;
        aa[e] = wm * D::FM * 4096 + r + c;
        ba[e] = D::ASTAGE + wn * D::FN * 32 * D::BROW + (D::FP8 ? n * 64 + (((e & 2) + hf) ^ swz8(n)) * 16 : r + c);
    }
    int slot = 0, ready = 0;   // steps whose loads are known to have arrived
    for (; mt < mt_end; ++mt) {
        f32x16 acc[D::FM][D::FN];
#pragma unroll
        for (int i = 0; i < D::FM; ++i)
#pragma unroll
            for (int j = 0; j < D::FN; ++j)
#pragma unroll
                for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.0f;
        uint32_t base = 0;
        for (int k = 0; k < steps; ++k) {
            if (ready > 0)
                --ready;
            else if (D::STAGES > 2 && (mt + 1 < mt_end || k + 1 < steps))
                wait_vm<(D::STAGES - 2) * (D::LA + D::LB)>();
            else
                wait_vm<0>();
            barrier_lds();
            issue();
            base = slot * D::STAGE;
            slot = slot == D::STAGES - 1 ? 0 : slot + 1;
#pragma unroll
            for (int h = 0; h < 2; ++h) {   // two matrix steps at a time
                x8<T> av[2][D::FM], bv[2][D::FN];
#pragma unroll
                for (int j = 0; j < D::FN; ++j) {
                    if (D::FP8) {
                        const u32x4 c = lds_read<u32x4>(base + ba[2 * h], j * 32 * D::BROW);
                        bv[0][j] = widen8<T>(u32x2{c[0], c[1]});
                        bv[1][j] = widen8<T>(u32x2{c[2], c[3]});
                    } else {
#pragma unroll
                        for (int e = 0; e < 2; ++e) bv[e][j] = lds_read<x8<T>>(base + ba[2 * h + e], j * 32 * D::BROW);
                    }
                }
#pragma unroll
                for (int i = 0; i < D::FM; ++i)
#pragma unroll
                    for (int e = 0; e < 2; ++e) av[e][i] = lds_read<x8<T>>(base + aa[2 * h + e], i * 4096);
#pragma unroll
                for (int e = 0; e < 2; ++e)
#pragma unroll
                    for (int i = 0; i < D::FM; ++i)
#pragma unroll
                        for (int j = 0; j < D::FN; ++j) acc[i][j] = mfma32<T>(av[e][i], bv[e][j], acc[i][j]);
            }
        }
        // The loads that are out, before the stores: a later count of loads must not wait for those.
        wait_vm<0>();
        ready = D::STAGES - 1;
        barrier_lds();
        const uint32_t at = base + wave * 32 * D::OROW;
        constexpr int PER = 4 * D::OF;   // lanes a token's run of features
#pragma unroll
        for (int j = 0; j < D::FN; ++j)
#pragma unroll
            for (int i = 0; i < D::FM; i += D::OF) {
#pragma unroll
                for (int q = 0; q < 4 * D::OF; ++q) {
                    x4<T> v;
#pragma unroll
                    for (int k = 0; k < 4; ++k) v[k] = (T)(acc[i + q / 4][j][4 * (q % 4) + k] * scale[j]);
                    lds_write(at + n * D::OROW + 8 * hf, v, 16 * q);
                }
                const int o = mt * D::TM + (wm * D::FM + i) * 32 + 8 * (lane % PER);
#pragma unroll
                for (int p = 0; p < PER / 2; ++p) {
                    const int t = p * (64 / PER) + lane / PER;
                    const x8<T> v = lds_read<x8<T>>(at + t * D::OROW + 16 * (lane % PER));
                    T *dst = row_of((wn * D::FN + j) * 32 + t);
                    if (dst && o < features) {
                        if (D::STREAM)
                            __builtin_nontemporal_store(__builtin_bit_cast(u32x4, v), reinterpret_cast<u32x4 *>(dst + o));
                        else
                            *reinterpret_cast<x8<T> *>(dst + o) = v;
                    }
                }
            }
    }
}

// Work items to XCDs: workgroups go to the eight XCDs in turn; each XCD takes
// a contiguous run of items.
__device__ __forceinline__ int xcd_item(int block, int total) {
    const int share = (total + 7) / 8, rest = total - (share - 1) * 8, xcd = block & 7, nth = block >> 3;
    return xcd < rest ? xcd * share + nth : rest * share + (xcd - rest) * (share - 1) + nth;
}

template <class D>
__global__ __launch_bounds__(64 * D::NW, 2) void k_mla_project(MlaProjectArgs a, int m_tiles, int parts, int n_tiles) {
    using T = typename D::T;
    const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
    const int id = xcd_item(blockIdx.x, gridDim.x);
    const int h = id / (parts * n_tiles), part = id / n_tiles % parts, t0 = id % n_tiles * D::TN;
    const uint8_t *xp[D::LB];
#pragma unroll
    for (int i = 0; i < D::LB; ++i) {
        const int r = (wave * D::LB + i) % D::LB_ALL * 8 + (lane >> 3);
        const int64_t t = min(t0 + r, a.tokens - 1);
        xp[i] = reinterpret_cast<const uint8_t *>(static_cast<const T *>(a.x) + t * a.x_ts + h * a.x_hs) +
                (((lane & 7) ^ swz(r)) << 4);
    }
    float scale[D::FN];
#pragma unroll
    for (int j = 0; j < D::FN; ++j) scale[j] = 1.0f;
    gemm_tiles<D>(static_cast<const T *>(a.w) + (int64_t)h * a.n_out * a.n_in, a.n_out, xp, a.n_in / 64,
                  part * m_tiles / parts, (part + 1) * m_tiles / parts, scale, [&](int t) -> T * {
                      return t0 + t < a.tokens ? static_cast<T *>(a.out) + ((int64_t)(t0 + t) * a.heads + h) * a.n_out : nullptr;
                  });
}

// A workgroup keeps its tokens and goes through the feature tiles of its part,
// so the rows are looked up once.  An XCD has all parts of few token tiles: its
// L2 keeps those rows while the weights pass through it once (8192 rows, 64
// heads: 302 us with one part of all tokens an XCD, whose rows its L2 does not
// hold).
template <class D>
__global__ __launch_bounds__(64 * D::NW, 2) void k_mla_expand(MlaExpandArgs a, int rank, int m_tiles, int parts, int n_tiles) {
    using T = typename D::T;
    const int tid = threadIdx.x, lane = tid & 63, wave = uniform(tid >> 6);
    const int id = xcd_item(blockIdx.x, gridDim.x);
    const int across = 4 * parts, run = id / across, wide = min(4, n_tiles - 4 * run);
    const int part = (id - run * across) / wide, t0 = (4 * run + (id - run * across) % wide) * D::TN;
    if (blockIdx.x == 0 && wave == 0) {   // the offsets, for all: from 0, ascending, inside the rows
        bool bad = a.cu_k[0] != 0 || a.cu_k[a.batch] > a.rows;
        for (int b = lane; b < a.batch; b += 64) bad |= a.cu_k[b + 1] < a.cu_k[b];
        if (__ballot(bad) && lane == 0) raise_status(a.status, ST_BADPAGE);
    }
    const int rows = min(a.rows, a.cu_k[a.batch]);
    if (t0 >= rows) return;
    const int row_bytes = D::FP8 ? rank + 2 * MLA_ROPE : 2 * (rank + MLA_ROPE);
    // Where the tile's rows are, a thread a row, in the stage that is loaded last: int64 row offsets, then scales.
    constexpr uint32_t AT = (D::STAGES - 1) * D::STAGE, SCALES = AT + 8 * D::TN;
    {
        // the sequence of the tile's first row: how many end at or before it
        int first = 0;
        for (int b = 0; b < a.batch; b += 64)
            first += __popcll(__ballot(b + lane < a.batch && a.cu_k[min(b + lane, a.batch - 1) + 1] <= t0));
        for (int t = tid; t < D::TN; t += 64 * D::NW) {
            const int r = min(t0 + t, rows - 1);
            int b = min(first, a.batch - 1);
            while (b + 1 < a.batch && a.cu_k[b + 1] <= r) ++b;
            const int at = r - a.cu_k[b];
            int64_t slot = 0;
            if (at < 0 || at >= (int64_t)a.c.width * a.c.page)
                raise_status(a.status, ST_BADPAGE);
            else
                slot = mla_slot(a.c, b, at, a.status);
            lds_write<int64_t>(AT + 8 * t, slot * row_bytes);
            if (D::FP8) lds_write<float>(SCALES + 4 * t, a.c.scale[slot]);
        }
        __syncthreads();
    }
    const uint8_t *xp[D::LB];
#pragma unroll
    for (int i = 0; i < D::LB; ++i) {
        const int l = (wave * D::LB + i) % D::LB_ALL;
        const int r = D::FP8 ? l * 16 + (lane >> 2) : l * 8 + (lane >> 3);
        xp[i] = a.c.pages + lds_read<int64_t>(AT + 8 * r) + ((D::FP8 ? (lane & 3) ^ swz8(r) : (lane & 7) ^ swz(r)) << 4);
    }
    float scale[D::FN];
#pragma unroll
    for (int j = 0; j < D::FN; ++j)
        scale[j] = D::FP8 ? lds_read<float>(SCALES + 4 * ((wave / D::WM * D::FN + j) * 32 + (lane & 31))) : 1.0f;
    if (part == 0)   // one part also copies the keys
        for (int i = tid; i < D::TN * 8; i += 64 * D::NW)
            if (t0 + i / 8 < rows)
                *reinterpret_cast<x8<T> *>(static_cast<T *>(a.k_pe) + (int64_t)(t0 + i / 8) * MLA_ROPE + i % 8 * 8) =
                    *reinterpret_cast<const x8<T> *>(a.c.pages + lds_read<int64_t>(AT + 8 * (i / 8)) + row_bytes - 2 * MLA_ROPE +
                                                     i % 8 * 16);
    barrier_lds();   // the offsets are read: the stage is free
    gemm_tiles<D>(static_cast<const T *>(a.w), a.n_out, xp, rank / 64, part * m_tiles / parts, (part + 1) * m_tiles / parts, scale,
                  [&](int t) -> T * { return t0 + t < rows ? static_cast<T *>(a.kv) + (int64_t)(t0 + t) * a.n_out : nullptr; });
}

// Parts the feature tiles of `items` token tiles are cut into: workgroups
// enough to fill the 256 CUs once, if there are tiles enough.
template <class D>
int gemm_parts(int64_t items, int m_tiles) {
    const int64_t parts = 256 * D::WGS / items;
    return (int)(parts < 1 ? 1 : parts < m_tiles ? parts : m_tiles);
}

// How many m x n tiles cover features x tokens.
int64_t gemm_tile_count(int64_t features, int64_t tokens, int m, int n) {
    return (features + m - 1) / m * ((tokens + n - 1) / n);
}
// 128 x 32 tiles of three stages, two workgroups a CU, start soonest: they are
// taken where all run at once.
constexpr int64_t SMALL_TILES = 512;

template <class D>
hipError_t project(const MlaProjectArgs &a, hipStream_t st) {
    const int mt = (a.n_out + D::TM - 1) / D::TM, nt = (a.tokens + D::TN - 1) / D::TN;
    const int parts = gemm_parts<D>((int64_t)nt * a.heads, mt);
    const hipError_t e = ensure_dyn_smem(reinterpret_cast<const void *>(&k_mla_project<D>), D::LDS);
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(k_mla_project<D>, dim3((uint32_t)parts * nt * a.heads), dim3(64 * D::NW), D::LDS, st, a, mt, parts, nt);
    return hipGetLastError();
}

template <class D>
hipError_t expand(const MlaExpandArgs &a, int rank, hipStream_t st) {
    const int mt = (a.n_out + D::TM - 1) / D::TM, nt = (a.rows + D::TN - 1) / D::TN, parts = gemm_parts<D>(nt, mt);
    const hipError_t e = ensure_dyn_smem(reinterpret_cast<const void *>(&k_mla_expand<D>), D::LDS);
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(k_mla_expand<D>, dim3((uint32_t)parts * nt), dim3(64 * D::NW), D::LDS, st, a, rank, mt, parts, nt);
    return hipGetLastError();
}

// Which tiles, at rank 512, bf16.  128 x 32 against 256 x 128: 16 heads of 256
// features, 512 rows (512 tiles): 9.1 us against 12.8; 64 heads of 448, 64 rows
// (448): 9.4 against 13.1; 160 rows of those (1120): 21.5 against 14.7.  256 x
// 128 against 256 x 256, 64 heads of 448, where the fuller last round decides:
// 1034 rows: 44.2 against 53.3; 8192 rows: 286 against 249.
template <class T, bool FP8>
hipError_t expand_by_size(const MlaExpandArgs &a, int rank, hipStream_t st) {
    if (a.rows <= 32 || gemm_tile_count(a.n_out, a.rows, 128, 32) <= SMALL_TILES) return expand<Gemm<T, FP8, 128, 32, 4, 4, 3, 2>>(a, rank, st);
    // rounds of 256 workgroups, in tokens
    auto rounds = [&](int tn) {
        const int64_t mt = (a.n_out + 255) / 256, nt = (a.rows + tn - 1) / tn, parts = nt < 256 ? 256 / nt : 1;
        return (mt + parts - 1) / parts * ((nt * parts + 255) / 256) * tn;
    };
    if (rounds(128) < rounds(256)) return expand<Gemm<T, FP8, 256, 128, 8, 4, 3, 1, true>>(a, rank, st);
    return expand<Gemm<T, FP8, 256, 256, 8, 2, 2, 1, true>>(a, rank, st);
}

}  // namespace

// Which tiles, bf16.  128 x 32 against 128 x 128: 16 heads, 512 -> 128, 300
// tokens (160 tiles): 6.7 us against 8.5; 64 heads, 512 -> 256, 100 tokens
// (512): 8.2 against 8.7, 200 tokens (896): 12.6 against 9.7.  256 x 256 needs
// long sums and tiles for most CUs: 64 heads, 512 -> 256, 600 tokens (192
// tiles): 19.8 against 21.8, 4096 tokens: 133 against 159; 16 heads of those,
// 2048 tokens (128 tiles): 17.2 against 11.9, 3000 tokens (192): 19.5 against
// 20.8.  From 192 sums on down it loses more than it gains, at 1024 to 16384
// tokens: 64 heads, 192 -> 512: 10 to 30% slower at eight of ten lengths, 3%
// faster at best; 128 heads of those: 9% faster to 10% slower at nine, 21%
// faster at 8192; 64 heads, 128 -> 512: 5 to 29% slower; 128 heads of those: 1%
// faster to 11% slower at nine, but 351 against 440 us at 8192, a length at
// which the smaller tiles are slow for a reason not found (8000 tokens: 369,
// 12000: 556).
hipError_t launch_mla_project(const MlaProjectArgs &a, int dtype, hipStream_t st) {
    return mla_with_type(dtype, [&](auto t) {
        using T = decltype(t);
        if (a.tokens <= 32 || gemm_tile_count(a.n_out, a.tokens, 128, 32) * a.heads <= SMALL_TILES)
            return project<Gemm<T, false, 128, 32, 4, 4, 3, 2>>(a, st);
        if (a.n_in <= 192 || a.n_out <= 128 || gemm_tile_count(a.n_out, a.tokens, 256, 256) * a.heads < 192)
            return project<Gemm<T, false, 128, 128, 4, 2, 2, 2, true>>(a, st);
        return project<Gemm<T, false, 256, 256, 8, 2, 2, 1, true>>(a, st);
    });
}

hipError_t launch_mla_expand(const MlaExpandArgs &a, const coli_mla_dims &d, hipStream_t st) {
    return mla_with_type(d.dtype, [&](auto t) {
        using T = decltype(t);
        return d.kv_format == COLI_KV_E4M3 ? expand_by_size<T, true>(a, d.rank, st) : expand_by_size<T, false>(a, d.rank, st);
    });
}

}  // namespace coli

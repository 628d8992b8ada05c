// Products with the latent projections, out[t, o] = sum_k w[o, k] x[t, k]:
// project (a product a head) and expand (all heads at once, the rows x
// gathered out of the paged cache).
//
// Both keep their reduction dimension contiguous in both operands, so one
// tiled product serves them: a workgroup of four wavefronts takes TM output
// features by TN tokens, w as the A operand, so that a lane's results are four
// consecutive features of one token.  Steps of 32 along k go through a ring
// of three LDS stages, loaded straight from memory two steps ahead; the
// results go through LDS once more, to leave in whole rows.
#include "kernels.h"
#include "mla_mfma.h"

namespace coli {
namespace {

constexpr int STAGES = 3;

template <class T_, bool FP8_, int TM_, int TN_, int WM_>
struct Gemm {
    using T = T_;
    static constexpr bool FP8 = FP8_;
    static constexpr int TM = TM_, TN = TN_, WM = WM_, WN = 4 / WM_;
    static constexpr int FM = TM / WM / 32, FN = TN / WN / 32;       // 32 x 32 tiles of a wavefront
    static constexpr int BROW = FP8 ? 32 : 64;                       // bytes of a token's step
    static constexpr int ASTAGE = TM * 64, STAGE = ASTAGE + TN * BROW;
    static constexpr int LA = TM / 64;                               // 1 KiB loads a wavefront and step
    static constexpr int LB_ALL = TN * BROW / 1024, LB = LB_ALL < 4 ? 1 : LB_ALL / 4;
    static constexpr int OROW = 2 * TM + 16;                         // bytes of a result row in LDS
    static constexpr int LDS = STAGES * STAGE > TN * OROW ? STAGES * STAGE : TN * OROW;
};

// The product of one tile.  wp, xp: this lane's sources of its A and B loads
// at k = 0; dst: the tile's first feature of each token.
template <class D, class Row>
__device__ __forceinline__ void gemm_tile(const uint8_t *const (&wp)[D::LA], const uint8_t *const (&xp)[D::LB], int steps,
                                          int features, const float (&scale)[D::FN], Row row_of) {
    using T = typename D::T;
    const int tid = threadIdx.x, lane = tid & 63, wave = uniform(tid >> 6), n = lane & 31, hf = lane >> 5;
    const int wm = wave % D::WM, wn = wave / D::WM;
    auto issue = [&](int step) {
        const uint32_t base = step % STAGES * D::STAGE;
#pragma unroll
        for (int i = 0; i < D::LA; ++i) load_to_lds(wp[i] + step * 64, base + (wave * D::LA + i) * 1024);
#pragma unroll
        for (int i = 0; i < D::LB; ++i)   // fewer loads than wavefronts: some load the same once more
            load_to_lds(xp[i] + step * D::BROW, base + D::ASTAGE + (wave * D::LB + i) % D::LB_ALL * 1024);
    };
    f32x16 acc[D::FM][D::FN];
#pragma unroll
    for (int i = 0; i < D::FM; ++i)
#pragma unroll
        for (int j = 0; j < D::FN; ++j)
#pragma unroll
            for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.0f;
    const int f = (n >> 2) & 3;
    const uint32_t a_at = (wm * D::FM * 32 + n) * 64, b_at = D::ASTAGE + (wn * D::FN * 32 + n) * D::BROW;
    // Matrix step e of a stage takes k = 16 hf + 8 e + 0..7 on both sides: 16 bytes of codes then hold both steps.
    const uint32_t c0 = ((2 * hf) ^ f) << 4, c1 = ((2 * hf + 1) ^ f) << 4, c8 = (hf ^ ((n >> 3) & 1)) << 4;
    issue(0);
    if (steps > 1) issue(1);
    for (int step = 0; step < steps; ++step) {
        if (step + 1 < steps)
            wait_vm<D::LA + D::LB>();
        else
            wait_vm<0>();
        barrier_lds();
        if (step + 2 < steps) issue(step + 2);
        const uint32_t base = step % STAGES * D::STAGE;
        x8<T> av[2][D::FM], bv[2][D::FN];
#pragma unroll
        for (int j = 0; j < D::FN; ++j) {
            if (D::FP8) {
                const u32x4 c = lds_read<u32x4>(base + b_at + j * 32 * D::BROW + c8);
                bv[0][j] = widen8<T>(u32x2{c[0], c[1]});
                bv[1][j] = widen8<T>(u32x2{c[2], c[3]});
            } else {
                bv[0][j] = lds_read<x8<T>>(base + b_at + j * 32 * D::BROW + c0);
                bv[1][j] = lds_read<x8<T>>(base + b_at + j * 32 * D::BROW + c1);
            }
        }
#pragma unroll
        for (int i = 0; i < D::FM; ++i) {
            av[0][i] = lds_read<x8<T>>(base + a_at + i * 2048 + c0);
            av[1][i] = lds_read<x8<T>>(base + a_at + i * 2048 + c1);
        }
#pragma unroll
        for (int e = 0; e < 2; ++e)
#pragma unroll
            for (int i = 0; i < D::FM; ++i)
#pragma unroll
                for (int j = 0; j < D::FN; ++j) acc[i][j] = mfma32<T>(av[e][i], bv[e][j], acc[i][j]);
    }
    barrier_lds();
#pragma unroll
    for (int j = 0; j < D::FN; ++j)
#pragma unroll
        for (int i = 0; i < D::FM; ++i)
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                x4<T> v;
#pragma unroll
                for (int k = 0; k < 4; ++k) v[k] = (T)(acc[i][j][4 * q + k] * scale[j]);
                lds_write(((wn * D::FN + j) * 32 + n) * D::OROW + 2 * ((wm * D::FM + i) * 32 + 8 * q + 4 * hf), v);
            }
    barrier_lds();
    constexpr int CH = D::TM / 8;
#pragma unroll 4
    for (int i = tid; i < D::TN * CH; i += 256) {
        const int t = i / CH, c = i % CH;
        T *dst = row_of(t);
        if (dst && 8 * c < features) *reinterpret_cast<x8<T> *>(dst + 8 * c) = lds_read<x8<T>>(t * D::OROW + 16 * c);
    }
}

// Lane's place in a 1 KiB load: 16 rows of four chunks (32 of two for
// codes), swizzled so that sixteen rows' same chunk lies in sixteen bank groups.
__device__ __forceinline__ int load_row(int lane) { return lane >> 2; }
__device__ __forceinline__ int load_chunk(int lane) { return ((lane & 3) ^ ((lane >> 4) & 3)) << 4; }
__device__ __forceinline__ int load_row8(int lane) { return lane >> 1; }
__device__ __forceinline__ int load_chunk8(int lane) { return ((lane & 1) ^ ((lane >> 4) & 1)) << 4; }

// Work items to XCDs: workgroups go to the eight XCDs in turn; each XCD takes
// a contiguous run of items.
__device__ __forceinline__ int xcd_item(int block, int total) {
    const int share = (total + 7) / 8, rest = total - (share - 1) * 8, xcd = block & 7, nth = block >> 3;
    return xcd < rest ? xcd * share + nth : rest * share + (xcd - rest) * (share - 1) + nth;
}

template <class D>
__global__ __launch_bounds__(256, 2) void k_mla_project(MlaProjectArgs a, int m_tiles, int n_tiles) {
    using T = typename D::T;
    const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
    const int id = xcd_item(blockIdx.x, gridDim.x);
    const int h = id / (m_tiles * n_tiles), mt = id / n_tiles % m_tiles, nt = id % n_tiles;
    const int o0 = mt * D::TM, t0 = nt * D::TN;
    const uint8_t *wp[D::LA], *xp[D::LB];
#pragma unroll
    for (int i = 0; i < D::LA; ++i) {
        const int o = min(o0 + (wave * D::LA + i) * 16 + load_row(lane), a.n_out - 1);
        wp[i] = reinterpret_cast<const uint8_t *>(static_cast<const T *>(a.w) + ((int64_t)h * a.n_out + o) * a.n_in) + load_chunk(lane);
    }
#pragma unroll
    for (int i = 0; i < D::LB; ++i) {
        const int64_t t = min(t0 + (wave * D::LB + i) % D::LB_ALL * 16 + load_row(lane), a.tokens - 1);
        xp[i] = reinterpret_cast<const uint8_t *>(static_cast<const T *>(a.x) + t * a.x_ts + h * a.x_hs) + load_chunk(lane);
    }
    float scale[D::FN];
#pragma unroll
    for (int j = 0; j < D::FN; ++j) scale[j] = 1.0f;
    gemm_tile<D>(wp, xp, a.n_in / 32, a.n_out - o0, scale, [&](int t) -> T * {
        return t0 + t < a.tokens ? static_cast<T *>(a.out) + ((int64_t)(t0 + t) * a.heads + h) * a.n_out + o0 : nullptr;
    });
}

template <class D>
__global__ __launch_bounds__(256, 2) void k_mla_expand(MlaExpandArgs a, int rank, int m_tiles, int n_tiles) {
    using T = typename D::T;
    constexpr int GROUP = 8;   // feature tiles of a group: their weights stay in an XCD's L2 while the tokens pass
    const int tid = threadIdx.x, lane = tid & 63, wave = uniform(tid >> 6);
    const int id = xcd_item(blockIdx.x, gridDim.x);
    const int group = id / (GROUP * n_tiles), width = min(GROUP, m_tiles - group * GROUP);
    const int mt = group * GROUP + (id - group * GROUP * n_tiles) % width, nt = (id - group * GROUP * n_tiles) / width;
    const int o0 = mt * D::TM, t0 = nt * D::TN;
    const int rows = min(a.rows, a.cu_k[a.batch]);
    if (t0 >= rows) return;
    const int row_bytes = D::FP8 ? rank + 2 * MLA_ROPE : 2 * (rank + MLA_ROPE);
    // the sequence of the tile's first row: how many end at or before it
    int first = 0;
    for (int b = 0; b < a.batch; b += 64)
        first += __popcll(__ballot(b + lane < a.batch && a.cu_k[min(b + lane, a.batch - 1) + 1] <= t0));
    auto slot_of = [&](int t) -> int64_t {
        const int r = min(t0 + t, rows - 1);
        int b = min(first, a.batch - 1);
        while (b + 1 < a.batch && a.cu_k[b + 1] <= r) ++b;
        const int at = r - a.cu_k[b];
        if (at < 0 || at >= (int64_t)a.c.width * a.c.page) {
            raise_status(a.status, ST_BADPAGE);
            return 0;
        }
        return mla_slot(a.c, b, at, a.status);
    };
    const uint8_t *wp[D::LA], *xp[D::LB];
#pragma unroll
    for (int i = 0; i < D::LA; ++i) {
        const int o = min(o0 + (wave * D::LA + i) * 16 + load_row(lane), a.n_out - 1);
        wp[i] = reinterpret_cast<const uint8_t *>(static_cast<const T *>(a.w) + (int64_t)o * rank) + load_chunk(lane);
    }
#pragma unroll
    for (int i = 0; i < D::LB; ++i) {
        const int l = (wave * D::LB + i) % D::LB_ALL;
        xp[i] = D::FP8 ? a.c.pages + slot_of(l * 32 + load_row8(lane)) * row_bytes + load_chunk8(lane)
                       : a.c.pages + slot_of(l * 16 + load_row(lane)) * row_bytes + load_chunk(lane);
    }
    float scale[D::FN];
#pragma unroll
    for (int j = 0; j < D::FN; ++j)
        scale[j] = D::FP8 ? a.c.scale[slot_of((wave / D::WM * D::FN + j) * 32 + (lane & 31))] : 1.0f;
    if (mt == 0)   // one tile of features also copies the keys
        for (int i = tid; i < D::TN * 8; i += 256)
            if (t0 + i / 8 < rows)
                *reinterpret_cast<x8<T> *>(static_cast<T *>(a.k_pe) + (int64_t)(t0 + i / 8) * MLA_ROPE + i % 8 * 8) =
                    *reinterpret_cast<const x8<T> *>(a.c.pages + slot_of(i / 8) * row_bytes + row_bytes - 2 * MLA_ROPE + i % 8 * 16);
    gemm_tile<D>(wp, xp, rank / 32, a.n_out - o0, scale, [&](int t) -> T * {
        return t0 + t < rows ? static_cast<T *>(a.kv) + (int64_t)(t0 + t) * a.n_out + o0 : nullptr;
    });
}

template <class D>
hipError_t project(const MlaProjectArgs &a, hipStream_t st) {
    const int mt = (a.n_out + D::TM - 1) / D::TM, nt = (a.tokens + D::TN - 1) / D::TN;
    const hipError_t e = ensure_dyn_smem(reinterpret_cast<const void *>(&k_mla_project<D>), D::LDS);
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(k_mla_project<D>, dim3((uint32_t)mt * nt * a.heads), dim3(256), D::LDS, st, a, mt, nt);
    return hipGetLastError();
}

template <class D>
hipError_t expand(const MlaExpandArgs &a, int rank, hipStream_t st) {
    const int mt = (a.n_out + D::TM - 1) / D::TM, nt = (a.rows + D::TN - 1) / D::TN;
    const hipError_t e = ensure_dyn_smem(reinterpret_cast<const void *>(&k_mla_expand<D>), D::LDS);
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(k_mla_expand<D>, dim3((uint32_t)mt * nt), dim3(256), D::LDS, st, a, rank, mt, nt);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_mla_project(const MlaProjectArgs &a, int dtype, hipStream_t st) {
    return mla_with_type(dtype, [&](auto t) {
        using T = decltype(t);
        if (a.tokens <= 32) return project<Gemm<T, false, 128, 32, 4>>(a, st);
        if (a.n_out <= 128 || a.tokens <= 512) return project<Gemm<T, false, 128, 128, 2>>(a, st);
        return project<Gemm<T, false, 256, 128, 2>>(a, st);
    });
}

hipError_t launch_mla_expand(const MlaExpandArgs &a, const coli_mla_dims &d, hipStream_t st) {
    return mla_with_type(d.dtype, [&](auto t) {
        using T = decltype(t);
        const bool fp8 = d.kv_format == COLI_KV_E4M3;
        if (a.rows <= 32)
            return fp8 ? expand<Gemm<T, true, 128, 32, 4>>(a, d.rank, st) : expand<Gemm<T, false, 128, 32, 4>>(a, d.rank, st);
        return fp8 ? expand<Gemm<T, true, 256, 128, 2>>(a, d.rank, st) : expand<Gemm<T, false, 256, 128, 2>>(a, d.rank, st);
    });
}

}  // namespace coli

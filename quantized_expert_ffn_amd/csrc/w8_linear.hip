// Products of 8-bit codes with scales for each token and output channel
// (coli_w8_linear): out[t, o] = s_t s_o sum_k q_tk w_ok + bias_o, on the int8
// matrix cores, with the channels as rows and the tokens as columns, so that a
// lane's results are consecutive channels of one token.  Sums are exact, so
// how they are split changes nothing.
#include "kernels.h"
#include "mfma.h"
#include "mla_mfma.h"
#include "w8.h"

namespace coli {
namespace {

// Where chunks behind the end of a row read.
__device__ const uint4 w8_zeros[8] = {};

// A result.  One for binary32 is formed in 64 bits and rounded once; for the
// 16-bit types each step is rounded to binary32 first, 2^-24 beside their 2^-11
// and more, since the tiles' many results would wait for slower instructions.
template <class T>
__device__ __forceinline__ float finish(int32_t sum, float st, float so, float bias, bool has_bias) {
    if constexpr (sizeof(T) == 4) {
        const double v = (double)sum * st * so;
        return (float)(has_bias ? v + bias : v);
    } else {
        const float v = (float)sum * st * so;
        return has_bias ? v + bias : v;
    }
}

// Lane's place in a 1 KiB load: eight rows of eight chunks, swizzled so that
// sixteen rows' same chunk lies in sixteen groups of banks.
__device__ __forceinline__ int swz(int r) { return 4 * ((r >> 1) & 1) + 2 * ((r >> 2) & 1) + ((r >> 3) & 1); }

// ---------------------------------------------------------------- some tokens
// All tokens by 32 FM channels a workgroup, so that weights pass once and many
// workgroups share them out.  Steps of NW / 4 lines of 128 along k go through a
// ring of LDS stages, and each of the NW wavefronts multiplies 32 of every
// step; their sums meet in LDS at the end, BATCH tiles of 32 x 32 at a time.
//
// What bounds it is the memory's time to answer: weights and tokens on their
// way, about 64 KiB a CU of either, arrive after 1.2 us, 50 GB/s a CU, of which
// the tokens' part comes from the L2 over and over.  One token, 6144 -> 16384,
// 101 MB: 18.9 us, 5.3 TB/s, as a copy; 61 tokens, 16384 -> 6144: 29.3 (192
// workgroups of 1.5 MB); 133 tokens, 6144 -> 19393, binary32: 46.7.  What was
// tried, beside builds whose binary32 results were still formed in binary32: a
// ring for weights and one for tokens, each loaded by its half of the wavefronts,
// so that more weights are out, 20.2 -> 22.6, 30.8 -> 50.2 and 43.6 -> 49.2;
// nothing loaded for places without a token, 20.3 -> 22.7, 30.8 -> 34.1, 43.5 ->
// 45.0; rings twice as deep, one workgroup a CU, 30.8 -> 39.3.
template <class T_, int FM_, int FN_, int NW_, int STAGES_, int WGS_>
struct Split {
    using T = T_;
    static constexpr int FM = FM_, FN = FN_, NW = NW_, STAGES = STAGES_, WGS = WGS_, TM = 32 * FM, TN = 32 * FN, STEP = 32 * NW;
    static constexpr int LINE = (TM + TN) * 128, STAGE = LINE * NW / 4, LOADS = FM + FN;   // 1 KiB loads a wavefront and step
    static constexpr int OROW = 36 * 4, SUMS = NW * 4096, OUT = 32 * OROW;   // of a 32 x 32 tile's join
    static constexpr int ROOM = 160 * 1024 / WGS / (SUMS + OUT), TILES = FM * FN < 4 ? FM * FN : 4, BATCH = TILES < ROOM ? TILES : ROOM;
    static constexpr int RING = STAGES * STAGE, JOIN = BATCH * (SUMS + OUT), LDS = RING > JOIN ? RING : JOIN;
    static_assert(LDS * WGS <= 160 * 1024 && (STAGES - 2) * LOADS < 64, "LDS, loads that are out");
};

template <class D>
__global__ __launch_bounds__(64 * D::NW, D::WGS * D::NW / 4) void k_w8_split(W8LinearArgs a, int wide_out) {
    using T = typename D::T;
    const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6), n = lane & 31, hf = lane >> 5;
    const int o0 = blockIdx.x * D::TM, steps = (a.k + D::STEP - 1) / D::STEP;
    const int8_t *src[D::LOADS];
    int chunk[D::LOADS];
#pragma unroll
    for (int i = 0; i < D::LOADS; ++i) {
        constexpr int GROUPS = D::LINE / 1024;
        const int l = wave * D::LOADS + i, r = l % GROUPS * 8 + (lane >> 3);
        chunk[i] = l / GROUPS * 128 + (((lane & 7) ^ swz(r)) << 4);
        src[i] = (r < D::TM ? a.w + (int64_t)min(o0 + r, a.n_out - 1) * a.k : a.x + (int64_t)min(r - D::TM, a.tokens - 1) * a.x_stride) + chunk[i];
    }
    // Rows are often a power of two apart, or nearly so, and the lines of a step then lie in few channels of the L2: each
    // workgroup of an XCD begins elsewhere along k, and goes round (16384 -> 6144, one token: 25.0 us without, 20.6; 61
    // tokens: 33.7, 30.5; rows of 6144 alike with and without).
    const int turn = (int)((int64_t)(blockIdx.x >> 3) * steps / ((gridDim.x + 7) >> 3));
    int load = turn, load_slot = 0;
    auto issue = [&] {   // behind the last step nothing is read that counts
        const int k = load * D::STEP;
        const uint32_t base = load_slot * D::STAGE + wave * D::LOADS * 1024;
        if (k + D::STEP <= a.k) {
#pragma unroll
            for (int i = 0; i < D::LOADS; ++i) load_to_lds(src[i] + k, base + i * 1024);
        } else {   // a row that ends inside the step: zeros behind it
#pragma unroll
            for (int i = 0; i < D::LOADS; ++i)
                load_to_lds(k + chunk[i] < a.k ? src[i] + k : reinterpret_cast<const int8_t *>(w8_zeros), base + i * 1024);
        }
        load_slot = load_slot == D::STAGES - 1 ? 0 : load_slot + 1;
        load = load == steps - 1 ? 0 : load + 1;
    };
#pragma unroll
    for (int i = 0; i < D::STAGES - 1; ++i) issue();
    // this wavefront's 32 of a step: line wave / 4, chunks 2 (wave % 4) + hf
    const uint32_t at = wave / 4 * D::LINE + (n >> 3) * 1024 + (n & 7) * 128 + (((2 * (wave & 3) + hf) ^ swz(n)) << 4);
    i32x16 acc[D::FM][D::FN];
#pragma unroll
    for (int i = 0; i < D::FM; ++i)
#pragma unroll
        for (int j = 0; j < D::FN; ++j)
#pragma unroll
            for (int r = 0; r < 16; ++r) acc[i][j][r] = 0;
    int slot = 0;
    for (int k = 0; k < steps; ++k) {
        wait_vm<(D::STAGES - 2) * D::LOADS>();
        barrier_lds();
        issue();
        const uint32_t base = slot * D::STAGE + at;
        slot = slot == D::STAGES - 1 ? 0 : slot + 1;
        i32x4 av[D::FM], bv[D::FN];
#pragma unroll
        for (int i = 0; i < D::FM; ++i) av[i] = lds_read<i32x4>(base, i * 4096);
#pragma unroll
        for (int j = 0; j < D::FN; ++j) bv[j] = lds_read<i32x4>(base, (D::FM + j) * 4096);
#pragma unroll
        for (int i = 0; i < D::FM; ++i)
#pragma unroll
            for (int j = 0; j < D::FN; ++j) acc[i][j] = __builtin_amdgcn_mfma_i32_32x32x32_i8(av[i], bv[j], acc[i][j], 0, 0, 0);
    }
    wait_vm<0>();
    typedef T four __attribute__((ext_vector_type(4)));
#pragma unroll
    for (int p0 = 0; p0 < D::FM * D::FN; p0 += D::BATCH) {
        constexpr int ALL = D::FM * D::FN;
        const int count = p0 + D::BATCH < ALL ? D::BATCH : ALL - p0;
        barrier_lds();   // the ring, or the tiles before, are done with
#pragma unroll
        for (int x = 0; x < D::BATCH; ++x) {
            if (p0 + x >= ALL) continue;
            const i32x16 &c = acc[(p0 + x) / D::FN][(p0 + x) % D::FN];
#pragma unroll
            for (int q = 0; q < 4; ++q)
                lds_write(x * D::SUMS + (wave * 4 + q) * 1024 + 16 * lane, i32x4{c[4 * q], c[4 * q + 1], c[4 * q + 2], c[4 * q + 3]});
        }
        barrier_lds();
        for (int task = wave; task < 4 * count; task += D::NW) {   // eight of a tile's channels
            const int x = task >> 2, q = task & 3, i = (p0 + x) / D::FN, j = (p0 + x) % D::FN;
            i32x4 sum = lds_read<i32x4>(x * D::SUMS + q * 1024 + 16 * lane);
#pragma unroll
            for (int w = 1; w < D::NW; ++w) sum += lds_read<i32x4>(x * D::SUMS + (w * 4 + q) * 1024 + 16 * lane);
            const float st = a.x_scale[min(32 * j + n, a.tokens - 1)];
            f32x4 v;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int o = min(o0 + 32 * i + 8 * q + 4 * hf + k, a.n_out - 1);
                v[k] = finish<T>(sum[k], st, a.w_scale[o], a.bias ? a.bias[o] : 0.0f, a.bias != nullptr);
            }
            lds_write(D::BATCH * D::SUMS + x * D::OUT + n * D::OROW + 32 * q + 16 * hf, v);
        }
        barrier_lds();
        for (int task = wave; task < 4 * count; task += D::NW) {   // eight tokens' runs of 32 channels, eight lanes each
            const int x = task >> 2, i = (p0 + x) / D::FN, j = (p0 + x) % D::FN, r = 8 * (task & 3) + (lane >> 3);
            const int t = 32 * j + r, o = o0 + 32 * i + 4 * (lane & 7);
            const f32x4 v = lds_read<f32x4>(D::BATCH * D::SUMS + x * D::OUT + r * D::OROW + 16 * (lane & 7));
            if (t < a.tokens) {
                T *dst = static_cast<T *>(a.out) + (int64_t)t * a.o_stride + o;
                if (wide_out && o + 4 <= a.n_out) {
                    *reinterpret_cast<four *>(dst) = four{(T)v[0], (T)v[1], (T)v[2], (T)v[3]};
                } else {
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        if (o + k < a.n_out) dst[k] = (T)v[k];
                }
            }
        }
    }
}

// ---------------------------------------------------------------- tiles
// NW wavefronts in WM x NW / WM pieces of a tile of TM channels by TN tokens;
// WGS workgroups fit a CU.  Steps of 128 along k, a line of every row, form one
// stream over a workgroup's tiles, through a ring of LDS stages loaded straight
// from memory; results pass through the stage used last, to leave in whole lines.
//
// What bounds it: 8192 tokens, 6144 -> 16384, 739 to 763 us, 2.16 to 2.23 POP/s: matrix
// products alone, without loads, ran 512 us at the clock that their power left
// (1.5 to 1.8 GHz); 256 x 256 tiles read 6.4 GB through L2s that hold 79 % of
// it.  Steps of 64 in four stages, beginning elsewhere along k, and eight
// wavefronts as 4 x 2 gained nothing.
template <class T_, int TM_, int TN_, int NW_, int WM_, int STAGES_, int WGS_>
struct Tile {
    using T = T_;
    static constexpr int TM = TM_, TN = TN_, NW = NW_, WM = WM_, WN = NW_ / WM_, STAGES = STAGES_, WGS = WGS_;
    static constexpr int FM = TM / WM / 32, FN = TN / WN / 32;       // 32 x 32 tiles of a wavefront
    static constexpr int ASTAGE = TM * 128, STAGE = ASTAGE + TN * 128;
    static constexpr int LA = TM / 8 / NW, LB = TN / 8 / NW;         // 1 KiB loads a wavefront and step
    static constexpr int OF = sizeof(T) == 4 || FM < 2 ? 1 : 2;      // 32-channel tiles that leave together
    static constexpr int OROW = 32 * OF * sizeof(T) + 16, OUT = NW * 32 * OROW;
    static constexpr int L_SCALE = STAGES * STAGE;                   // float [TM]: channels' scales, then their biases
    static constexpr int LDS = L_SCALE + 8 * TM;
    static_assert(LA >= 1 && LB >= 1 && OUT <= STAGE && LDS * WGS <= 160 * 1024, "LDS");
};

// Work items to XCDs: workgroups go to the eight XCDs in turn; each XCD takes
// a contiguous run of items.
__device__ __forceinline__ int xcd_item(int block, int total) {
    const int share = (total + 7) / 8, rest = total - (share - 1) * 8, xcd = block & 7, nth = block >> 3;
    return xcd < rest ? xcd * share + nth : rest * share + (xcd - rest) * (share - 1) + nth;
}

template <class D>
__global__ __launch_bounds__(64 * D::NW, D::NW * D::WGS / 4) void k_w8_tiles(W8LinearArgs a, int m_tiles, int parts, int n_tiles, int wide_out) {
    using T = typename D::T;
    const int tid = threadIdx.x, lane = tid & 63, wave = uniform(tid >> 6), n = lane & 31, hf = lane >> 5;
    const int wm = wave % D::WM, wn = wave / D::WM;
    // An XCD has all parts of few token tiles: its L2 keeps those while the weights pass through it.
    const int id = xcd_item(blockIdx.x, gridDim.x);
    const int across = 4 * parts, run = id / across, wide = min(4, n_tiles - 4 * run);
    const int part = (id - run * across) / wide, t0 = (4 * run + (id - run * across) % wide) * D::TN;
    int mt = (int)((int64_t)part * m_tiles / parts);
    const int mt_end = (int)((int64_t)(part + 1) * m_tiles / parts), steps = (a.k + 127) / 128;
    // ---- the stream of loads
    const int8_t *wp[D::LA], *xp[D::LB];
    int load_mt = mt, load_k = 0, load_slot = 0;
    auto chunk = [&](int r) { return ((lane & 7) ^ swz(r)) << 4; };
#pragma unroll
    for (int i = 0; i < D::LB; ++i) {
        const int r = (wave * D::LB + i) * 8 + (lane >> 3);
        xp[i] = a.x + (int64_t)min(t0 + r, a.tokens - 1) * a.x_stride + chunk(r);
    }
    auto aim = [&] {
#pragma unroll
        for (int i = 0; i < D::LA; ++i) {
            const int r = (wave * D::LA + i) * 8 + (lane >> 3);
            wp[i] = a.w + (int64_t)min(load_mt * D::TM + r, a.n_out - 1) * a.k + chunk(r);
        }
    };
    // A step's loads in three parts, which stand between products: together they would hold the wavefronts up.  Behind the
    // last step they read its lines once more.
    auto issue = [&](int part) {
        const uint32_t base = load_slot * D::STAGE;
        const int k = load_k * 128;
        constexpr int ALL = D::LA + D::LB;
#pragma unroll
        for (int l = 0; l < ALL; ++l) {
            if (l * 3 / ALL != part) continue;
            const bool of_w = l < D::LA;
            const int g = of_w ? wave * D::LA + l : wave * D::LB + l - D::LA;
            const int8_t *src = (of_w ? wp[of_w ? l : 0] : xp[of_w ? 0 : l - D::LA]) + k;
            if (k + 128 > a.k && k + chunk(8 * g + (lane >> 3)) >= a.k) src = reinterpret_cast<const int8_t *>(w8_zeros);
            load_to_lds(src, base + (of_w ? 0 : D::ASTAGE) + g * 1024);
        }
        if (part < 2) return;
        load_slot = load_slot == D::STAGES - 1 ? 0 : load_slot + 1;
        if (++load_k == steps) {
            load_k = 0;
            load_mt = min(load_mt + 1, mt_end - 1);
            aim();
        }
    };
    aim();
#pragma unroll
    for (int i = 0; i < D::STAGES - 1; ++i)
#pragma unroll
        for (int part = 0; part < 3; ++part) issue(part);
    issue(0);
    // Matrix step e of a stage takes k = 32 e + 16 hf + 0..15 of both sides.
    uint32_t aa[4], ba[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const uint32_t at = (n >> 3) * 1024 + (n & 7) * 128 + (((2 * e + hf) ^ swz(n)) << 4);
        aa[e] = wm * D::FM * 4096 + at;
        ba[e] = D::ASTAGE + wn * D::FN * 4096 + at;
    }
    float st[D::FN];
#pragma unroll
    for (int j = 0; j < D::FN; ++j) st[j] = a.x_scale[min(t0 + (wn * D::FN + j) * 32 + n, a.tokens - 1)];
#pragma unroll
    for (int j = 0; j < D::FN; ++j) arrived(st[j]);
    // A step's four products a tile: operands are read one ahead, so that those of step 3 are in registers before it.  There
    // the barrier stands, for the next step's lines to have arrived and this one's stage to be free, and step 3's products
    // cover the first reads behind it.
    int slot = 0, ready = 0;   // steps whose loads are known to have arrived
    uint32_t base = 0;
    i32x4 av[2][D::FM], bv[2][D::FN];
    auto read = [&](int e) {
#pragma unroll
        for (int j = 0; j < D::FN; ++j) bv[e & 1][j] = lds_read<i32x4>(base + ba[e], j * 4096);
#pragma unroll
        for (int i = 0; i < D::FM; ++i) av[e & 1][i] = lds_read<i32x4>(base + aa[e], i * 4096);
    };
    wait_vm<0>();
    barrier_lds();
    read(0);
    for (; mt < mt_end; ++mt) {
        i32x16 acc[D::FM][D::FN];
#pragma unroll
        for (int i = 0; i < D::FM; ++i)
#pragma unroll
            for (int j = 0; j < D::FN; ++j)
#pragma unroll
                for (int r = 0; r < 16; ++r) acc[i][j][r] = 0;
        auto multiply = [&](int e) {
#pragma unroll
            for (int i = 0; i < D::FM; ++i)
#pragma unroll
                for (int j = 0; j < D::FN; ++j)
                    acc[i][j] = __builtin_amdgcn_mfma_i32_32x32x32_i8(av[e & 1][i], bv[e & 1][j], acc[i][j], 0, 0, 0);
        };
        uint32_t spent = 0;
        for (int k = 0; k < steps; ++k) {
#pragma unroll
            for (int e = 0; e < 3; ++e) {
                __builtin_amdgcn_sched_barrier(0);
                read(e + 1);
                multiply(e);
                if (e < 2) issue(e + 1);
            }
            __builtin_amdgcn_sched_barrier(0);
            if (ready > 0)
                --ready;
            else
                wait_vm<(D::STAGES - 2) * (D::LA + D::LB)>();
            barrier_lds();
            spent = base;
            slot = slot == D::STAGES - 1 ? 0 : slot + 1;
            base = slot * D::STAGE;
            read(0);
            multiply(3);
            if (k + 1 < steps) issue(0);
            __builtin_amdgcn_sched_barrier(0);
        }
        // The loads that are out, before the stores: a later count of loads must not wait for those.
        wait_vm<0>();
        ready = D::STAGES - 2;
        for (int i = tid; i < D::TM; i += 64 * D::NW) {
            const int o = min(mt * D::TM + i, a.n_out - 1);
            lds_write<float>(D::L_SCALE + 4 * i, a.w_scale[o]);
            lds_write<float>(D::L_SCALE + 4 * D::TM + 4 * i, a.bias ? a.bias[o] : 0.0f);
        }
        barrier_lds();
        const uint32_t at = spent + wave * 32 * D::OROW;
        constexpr int VEC = 16 / sizeof(T), PER = 32 * D::OF / VEC;   // channels of 16 bytes, lanes a token's run of them
        typedef T vec __attribute__((ext_vector_type(VEC)));
        typedef T four __attribute__((ext_vector_type(4)));
#pragma unroll
        for (int j = 0; j < D::FN; ++j)
#pragma unroll
            for (int i = 0; i < D::FM; i += D::OF) {
#pragma unroll
                for (int q = 0; q < 4 * D::OF; ++q) {
                    const uint32_t ch = D::L_SCALE + 4 * ((wm * D::FM + i) * 32 + 4 * hf);
                    const f32x4 so = lds_read<f32x4>(ch, 32 * q), b = lds_read<f32x4>(ch, 4 * D::TM + 32 * q);
                    four v;
#pragma unroll
                    for (int k = 0; k < 4; ++k) v[k] = (T)finish<T>(acc[i + q / 4][j][4 * (q % 4) + k], st[j], so[k], b[k], a.bias != nullptr);
                    lds_write(at + n * D::OROW + 4 * sizeof(T) * hf, v, 8 * sizeof(T) * q);
                }
                const int o = mt * D::TM + (wm * D::FM + i) * 32 + VEC * (lane % PER);
#pragma unroll
                for (int p = 0; p < PER / 2; ++p) {
                    const int r = p * (64 / PER) + lane / PER, t = t0 + (wn * D::FN + j) * 32 + r;
                    const vec v = lds_read<vec>(at + r * D::OROW + 16 * (lane % PER));
                    if (t < a.tokens) {
                        T *dst = static_cast<T *>(a.out) + (int64_t)t * a.o_stride + o;
                        if (wide_out && o + VEC <= a.n_out) {
                            *reinterpret_cast<vec *>(dst) = v;
                        } else {
#pragma unroll
                            for (int k = 0; k < VEC; ++k)
                                if (o + k < a.n_out) dst[k] = v[k];
                        }
                    }
                }
            }
        barrier_lds();   // the scales are read, and the stage is free
        issue(0);
    }
}

template <class D>
hipError_t tiles(const W8LinearArgs &a, hipStream_t st) {
    const int mt = (a.n_out + D::TM - 1) / D::TM, nt = (a.tokens + D::TN - 1) / D::TN;
    int64_t parts = 256 * D::WGS / nt;
    parts = parts < 1 ? 1 : parts < mt ? parts : mt;
    const hipError_t e = ensure_dyn_smem(reinterpret_cast<const void *>(&k_w8_tiles<D>), D::LDS);
    if (e != hipSuccess) return e;
    const int wide_out = reinterpret_cast<uintptr_t>(a.out) % 16 == 0 && a.o_stride * (int64_t)sizeof(typename D::T) % 16 == 0;
    hipLaunchKernelGGL(k_w8_tiles<D>, dim3((uint32_t)(parts * nt)), dim3(64 * D::NW), D::LDS, st, a, mt, (int)parts, nt, wide_out);
    return hipGetLastError();
}

template <class D>
hipError_t split(const W8LinearArgs &a, hipStream_t st) {
    const hipError_t e = ensure_dyn_smem(reinterpret_cast<const void *>(&k_w8_split<D>), D::LDS);
    if (e != hipSuccess) return e;
    constexpr int64_t four = 4 * sizeof(typename D::T);
    const int wide_out = reinterpret_cast<uintptr_t>(a.out) % four == 0 && a.o_stride * (int64_t)sizeof(typename D::T) % four == 0;
    hipLaunchKernelGGL(k_w8_split<D>, dim3((a.n_out + D::TM - 1) / D::TM), dim3(64 * D::NW), D::LDS, st, a, wide_out);
    return hipGetLastError();
}

// Channels of a workgroup where all tokens go with them: as few tiles of 32 as
// let all workgroups run at once, a CU each (96 tokens, 6144 -> 6144: 19.0 us
// with one, 26.5 with two; -> 12288: 34.2, 28.3 with two, 33.1 with three; ->
// 24576: 51.1, 48.7, 37.7).  One tile of tokens has two workgroups a CU at any
// size (32 tokens, 6144 -> 16384: 21.8 us with one, 21.4 with two).  Eight wavefronts where
// channels are few and the chain along k is what counts (one token, 6144 ->
// 2048: 6.6 us against 8.2; -> 8192: 11.6 against 11.3).
template <class T, int FN, int S1, int W1, int S2, int S3>
hipError_t split_by_channels(const W8LinearArgs &a, hipStream_t st) {
    if (a.n_out <= 32 * 256) return split<Split<T, 1, FN, 4, S1, W1>>(a, st);
    if (a.n_out <= 64 * 256) return split<Split<T, 2, FN, 4, S2, 1>>(a, st);
    return split<Split<T, 3, FN, 4, S3, 1>>(a, st);
}

}  // namespace

hipError_t launch_w8_linear(const W8LinearArgs &a, int dtype, hipStream_t st) {
    return w8_with_type(dtype, [&](auto t) {
        using T = decltype(t);
        if (a.tokens <= 32) return a.n_out <= 2048 ? split<Split<T, 1, 1, 8, 4, 2>>(a, st) : split<Split<T, 1, 1, 4, 9, 2>>(a, st);
        if (a.tokens <= 64) return split_by_channels<T, 2, 6, 2, 9, 7>(a, st);
        if (a.tokens <= 96) return split_by_channels<T, 3, 4, 2, 7, 6>(a, st);
        if (a.tokens <= 128) return split_by_channels<T, 4, 7, 1, 6, 5>(a, st);
        // up to 160, split or in tiles: 160 tokens, 6144 -> 6144, 26.5 us or 27.3; 16384 -> 6144, 54.0 or 60.9; 6144 -> 24576,
        // 46.4 or 51.3; 64 tokens, 6144 -> 6144, 15.6 or 29.2
        if (a.tokens <= 160) return split_by_channels<T, 5, 6, 1, 5, 4>(a, st);
        // More tokens: rounds of workgroups by what one takes, in 42 us at k = 6144: 128 x 64 tiles, two a CU, 1 (0.65 if one
        // a CU is enough); 256 x 128: 1.15; 256 x 256: 2.1.  Inputs in turn, codes evenly spread (which take more power than
        // activations'): 512 tokens, 6144 -> 6144: 43.7, 49.7 and 89.0 us; 1024 tokens: 80.8, 50.4, 90.6; 2048 tokens: 124,
        // 101, 92.4; 8192 tokens, -> 16384: 1264, 830, 769.
        auto tiles_of = [&](int64_t m, int64_t n) { return (a.n_out + m - 1) / m * ((a.tokens + n - 1) / n); };
        const int64_t small = tiles_of(128, 64);
        const double c64 = small <= 256 ? 0.65 : (double)((small + 511) / 512);
        const double c128 = 1.15 * (double)((tiles_of(256, 128) + 255) / 256), c256 = 2.1 * (double)((tiles_of(256, 256) + 255) / 256);
        if (c64 <= c128 && c64 <= c256) return tiles<Tile<T, 128, 64, 4, 4, 3, 2>>(a, st);
        if (c128 < c256) return tiles<Tile<T, 256, 128, 8, 4, 3, 1>>(a, st);
        return tiles<Tile<T, 256, 256, 8, 2, 2, 1>>(a, st);
    });
}

}  // namespace coli

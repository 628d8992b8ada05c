// Absorbed attention of a batch's new tokens over a prefix that all its
// sequences share, and the join with what they see of their own tokens.
//
// The query rows of all sequences are one product with the prefix's latents:
// s = scale (<q, c> + <p, k>), out = sum e^s c / sum e^s over tiles of 32
// tokens.  A workgroup takes 128 rows, a wavefront 32 of them with all columns,
// so that weights stay in the registers they are formed in: 256 accumulators
// and 144 registers of queries beside them.  With 64 rows, as where each
// sequence reads for itself, a token's 1152 bytes go through LDS twice as often
// for the same products.
//
// Tiles pass through a ring in LDS ahead of use, one barrier a tile.  A tile's
// scores are formed while the values of the one before wait, then its softmax
// in steps between those values' products, which leave it no time of its own.
// E4M3 codes come into LDS as they are and are widened there, a line between
// two pairs of the scores' products.
//
// What bounds it: matrix products at what the card's power allows, then their
// operands from LDS.  64 x 128 rows over 8192 tokens and up to 1024 of their
// own, rank 512, binary16: 179 to 183 us, 0.83 to 0.85 PFLOP/s, of which the join
// 14; its products alone, with nothing else in the kernel, ran 107 us (1.37
// PFLOP/s).  Leaving out any one of softmax, value reads, key reads or loads saved
// 8 to 12 us of it.  E4M3, 64 x 64 rows over 32768: 364 us, of which widening 45
// (by default a call of that size has its sequences read apart, 350 us).
//
// Weights are rounded to 16 bits before the values' product, since the matrix
// cores take both sides in the cache's type; their sum is of the weights before
// that rounding.  Beside a plain form that keeps 32 bits the error against 64 bits
// is an eighth larger: bf16 1.9e-3 against 1.7e-3 of the largest value, fp16
// 2.4e-4 against 2.1e-4.
#include "kernels.h"
#include "mla_mfma.h"

#include <type_traits>

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
    static constexpr int RING = FP8 ? 3 : 4;
    static constexpr int TILE = SHD_TILE * CB * 128;
    static constexpr int L_ID = RING * TILE;                    // int32 [4][4 wavefronts][64]: page ids of tiles to come
    // codes as they come, [2][4 wavefronts]: lines of 1 KiB, then 256 bytes of scales
    static constexpr int LINES = ROW / 128, RAW = LINES * 1024 + 256, L_RAW = L_ID + 4 * 1024;
    static constexpr int L_SCALE = L_RAW + (FP8 ? 8 * RAW : 0); // float [RING][32]: E4M3 scales
    static constexpr int L_EXP = L_SCALE + RING * 4 * SHD_TILE; // float [RING][32]: their exponents
    static constexpr int L_FRAC = L_EXP + RING * 4 * SHD_TILE;  // float [RING][32]: and fractions
    static constexpr int LDS = L_FRAC + RING * 4 * SHD_TILE;
    static constexpr int SLOT = SHD_ROWS * RANK + 2 * SHD_ROWS;
    static_assert(LDS <= 160 * 1024, "the LDS of a CU");
};

// Work is shared out evenly in units of one tile of one block of rows, blocks
// in order.  Where blocks are of one sequence each (`whole`), its own tokens are
// further tiles behind the prefix's, and blocks differ in length by sequence;
// else all blocks have the prefix's tiles and the own tokens are apart.  A group
// is the blocks of one length.
//
// A share that passes from one block to the next costs about as much as CROSS
// tiles: queries to load, a pipeline to fill and one more result to write (64
// blocks of 257 to 288 tiles: 206 us; each in four parts: 170).  Where that is
// no worse, every block is cut into `parts` of its own, one a workgroup.
constexpr int CROSS = 8;
// A workgroup has LEAST units or more, if there are as many: a result of 128
// rows takes 256 KiB to write and the join to read (64 x 1 x 16 rows behind
// 2047 tokens: 57.9 us with one, 57.6 with two, 52.2 with three, 50.6 with six;
// 128 rows behind 8192: 45.3, 37.1, 36.0, 38.0).
constexpr int LEAST = 3;
struct Units {
    int64_t total;
    int shares, parts;   // parts: 0, or of each block
    __device__ int64_t first(int g) const { return total * g / shares; }
    // the workgroup that has a unit
    __device__ int owner(int64_t unit) const { return (int)(((unit + 1) * shares - 1) / total); }
};
__host__ __device__ inline int tiles_of(int tokens) { return (tokens + SHD_TILE - 1) / SHD_TILE; }
__host__ __device__ inline int64_t blocks_of(int64_t rows) { return (rows + SHD_ROWS - 1) / SHD_ROWS; }
__host__ __device__ inline int64_t shares_of(int64_t units) { return (units + LEAST - 1) / LEAST; }
__host__ __device__ inline bool whole_blocks(int64_t rows_of_sequence) { return rows_of_sequence % SHD_ROWS == 0; }

// Most workgroups, each of which takes a CU.
int shd_shares(int64_t rows, int prefix, int max_kv) {
    const int64_t units = blocks_of(rows) * ((int64_t)tiles_of(prefix) + tiles_of(max_kv));
    return (int)(shares_of(units) < 256 ? shares_of(units) : 256);
}

// Behind the plan, the groups' first units and the parts of a block, come the
// partial results.
size_t shd_plan_bytes(int batch) { return (8 * ((size_t)batch + 2) + 255) & ~(size_t)255; }

__device__ __forceinline__ int64_t wave_scan64(int64_t v) {
    const int lane = threadIdx.x & 63;
    for (int o = 1; o < 64; o += o) {
        const int64_t u = __shfl_up(v, o);
        if (lane >= o) v += u;
    }
    return v;
}

__device__ __forceinline__ int64_t uniform64(int64_t v) {
    return (int64_t)(uint32_t)uniform((int)v) | (int64_t)uniform((int)(v >> 32)) << 32;
}

// A product whose sum stays in ordinary registers, beside accumulators that
// fill the others (left to the compiler they moved between both kinds, and
// spilled).  The first wait covers operands just written by vector
// instructions; whoever reads the sum waits for it (settled).
template <class T>
__device__ __forceinline__ void mfma_v(f32x16 &c, x8<T> a, x8<T> b) {
    if constexpr (std::is_same<T, __bf16>::value)
        asm volatile("s_nop 1\n\tv_mfma_f32_32x32x16_bf16 %0, %1, %2, %0" : "+v"(c) : "v"(a), "v"(b));
    else
        asm volatile("s_nop 1\n\tv_mfma_f32_32x32x16_f16 %0, %1, %2, %0" : "+v"(c) : "v"(a), "v"(b));
}
// Waits out a matrix instruction of up to sixteen passes.
__device__ __forceinline__ void settled(f32x16 &c) { asm volatile("s_nop 15\n\ts_nop 7" : "+v"(c)); }

// Accumulators by a factor, and out of their registers: eight at a time
// through one ordinary register each, since the compiler would bring them all
// over at once, for which there is no room.
template <int I>
__device__ __forceinline__ void acc_scale(f32x16 &c, float f) {
    float t, v0 = c[I], v1 = c[I + 1], v2 = c[I + 2], v3 = c[I + 3], v4 = c[I + 4], v5 = c[I + 5], v6 = c[I + 6], v7 = c[I + 7];
#define COLI_SCALE(r) "v_accvgpr_read_b32 %8, " r "\n\ts_nop 1\n\tv_mul_f32 %8, %8, %9\n\ts_nop 1\n\tv_accvgpr_write_b32 " r ", %8\n\t"
    asm volatile(COLI_SCALE("%0") COLI_SCALE("%1") COLI_SCALE("%2") COLI_SCALE("%3") COLI_SCALE("%4") COLI_SCALE("%5")
                     COLI_SCALE("%6") COLI_SCALE("%7") "s_nop 3"
                 : "+a"(v0), "+a"(v1), "+a"(v2), "+a"(v3), "+a"(v4), "+a"(v5), "+a"(v6), "+a"(v7), "=&v"(t)
                 : "v"(f));
#undef COLI_SCALE
    c[I] = v0, c[I + 1] = v1, c[I + 2] = v2, c[I + 3] = v3, c[I + 4] = v4, c[I + 5] = v5, c[I + 6] = v6, c[I + 7] = v7;
}
__device__ __forceinline__ f32x4 acc_read(float a, float b, float c, float d) {
    f32x4 v;
    float x, y, z, w;
    asm volatile("v_accvgpr_read_b32 %0, %4\n\tv_accvgpr_read_b32 %1, %5\n\tv_accvgpr_read_b32 %2, %6\n\tv_accvgpr_read_b32 %3, %7\n\ts_nop 1"
                 : "=&v"(x), "=&v"(y), "=&v"(z), "=&v"(w)
                 : "a"(a), "a"(b), "a"(c), "a"(d));
    v[0] = x, v[1] = y, v[2] = z, v[3] = w;
    return v;
}
// Waits out the matrix instructions before.
__device__ __forceinline__ void acc_settled() { asm volatile("s_nop 15\n\ts_nop 7" ::: "memory"); }

__device__ __forceinline__ int shd_swz(int t) { return 4 * ((t >> 1) & 1) + 2 * ((t >> 2) & 1) + ((t >> 3) & 1); }

// The tokens that a query row sees of its sequence's own, 0 or fewer where it
// ends in the prefix.
__device__ __forceinline__ int shd_seen(const MlaSharedArgs &a, int64_t row) {
    const int per = a.n_q * a.heads, b = (int)(row / per), j = (int)(row - (int64_t)b * per) / a.heads;
    return mla_len(a.kv_lens, b, a.max_kv, a.status) - a.n_q + 1 + j;
}

// The units a call has, those of workgroup g, and the group that they begin in.
struct Place {
    Units u;
    int64_t unit, end, group_first;
    int group;
};
__device__ __forceinline__ Place shd_units(const MlaSharedArgs &a, int groups, int blocks, int g) {
    const int lane = threadIdx.x & 63, prefix = tiles_of(a.prefix);
    auto tiles_at = [&](int b) { return b < groups ? prefix + (a.whole ? tiles_of(mla_len(a.kv_lens, b, a.max_kv, a.status)) : 0) : 0; };
    Place p{};
    int longest = 0;
    for (int b = 0; b < groups; b += 64) {
        const int t = tiles_at(b + lane);
        p.u.total += uniform64(__shfl(wave_scan64((int64_t)t * blocks), 63));
        for (int o = 32, v = t; o; o >>= 1) longest = max(longest, v = max(v, __shfl_xor(v, o)));
    }
    longest = uniform(longest);
    p.u.shares = (int)min(shares_of(p.u.total), (int64_t)a.shares);
    const int parts = (int)(p.u.shares / ((int64_t)groups * blocks));
    if (parts > 0 && parts <= prefix && (longest + parts - 1) / parts <= p.u.total / p.u.shares + CROSS) p.u.parts = parts;
    int64_t base = 0;
    p.group = -1;
    p.unit = p.u.first(min(g, p.u.shares));
    p.end = p.u.first(min(g + 1, p.u.shares));
    for (int b = 0; b < groups; b += 64) {
        const int64_t mine = (int64_t)tiles_at(b + lane) * blocks, incl = wave_scan64(mine);
        if (g == 0 && threadIdx.x < 64 && b + lane < groups) a.plan[b + lane] = base + incl - mine;
        const uint64_t hit = __ballot(b + lane < groups && base + incl > p.unit);
        if (p.group < 0 && hit) {
            const int l = __builtin_ctzll(hit);
            p.group = uniform(b + l);
            p.group_first = base + uniform64(__shfl(incl - mine, l));
        }
        base += uniform64(__shfl(incl, 63));
    }
    if (g == 0 && threadIdx.x == 0) {
        a.plan[groups] = base;
        a.plan[groups + 1] = p.u.parts;
    }
    if (p.u.parts) {
        const int blk = g / parts, part = g - blk * parts;
        p.group = blk / blocks;
        p.group_first = 0;
        const int64_t tiles = p.group < groups ? uniform(tiles_at(p.group)) : 0, at = (blk - p.group * blocks) * tiles;
        p.unit = at + tiles * part / parts;
        p.end = at + tiles * (part + 1) / parts;
    }
    return p;
}

template <class D>
__global__ __launch_bounds__(256, 1) void k_mla_shared(MlaSharedArgs a) {
    using T = typename D::T;
    constexpr int RANK = D::RANK, CT = D::CT, KS = D::KS;
    constexpr bool FP8 = D::FP8;
    constexpr float NEG = -__builtin_inff();
    constexpr float LIFT = WEIGHT_LIFT<T>, LAG = LIFT + MAX_LAG;
    const int tid = threadIdx.x, lane = tid & 63, wave = uniform(tid >> 6);
    const int n = lane & 31, hf = lane >> 5, g = blockIdx.x;
    const int64_t rows = (int64_t)a.batch * a.n_q * a.heads;
    const int groups = a.whole ? a.batch : 1, prefix_tiles = tiles_of(a.prefix);
    const int blocks = (int)(a.whole ? a.n_q * a.heads / SHD_ROWS : blocks_of(rows));   // of a group
    const Place mine = shd_units(a, groups, blocks, g);
    int64_t unit = mine.unit, group_first = mine.group_first;
    const int64_t end = mine.end;
    int group = mine.group;
    // the segment's own tokens, if it has any here: how many, the tile they begin with, their pages
    int own_len = 0, own_from = INT32_MAX;
    const int32_t *own_row = a.own_table;
    const float scale = a.scale * LOG2E;
    const uint32_t page_inv = 0xffffffffu / (uint32_t)a.c.page;
    bool bad_page = false;

    // ---- lane addresses inside a tile
    uint32_t ka, va;
    {
        const int x = lane & 15, cb = (lane >> 4) & 1, t8 = 4 * hf + (x >> 2);
        ka = (n >> 3) * D::CB * 1024 + (n & 7) * 128 + ((hf ^ shd_swz(n)) << 4);          // chunk 2 v + hf at ka ^ 32 v
        va = t8 * 128 + (((2 * cb + ((x & 3) >> 1)) ^ shd_swz(t8)) << 4) + 8 * (x & 1);   // odd column tiles at va ^ 64,
    }                                                                                     // tokens 8 .. 15 at va ^ 16 + 1 KiB lines
    // ---- the tiles on their way: a thread loads chunk lane % 8 of every line of token lt
    const int lt = 8 * wave + (lane >> 3), lf = shd_swz(lt), chunk = (lane & 7) ^ lf;
    auto slot_in_ring = [](int tile) { return (uint32_t)tile % (uint32_t)D::RING; };
    auto base_of = [&](int tile) { return slot_in_ring(tile) * D::TILE; };
    auto scale_of = [&](int tile) { return 4 * slot_in_ring(tile) * SHD_TILE; };
    struct Where {
        int page, in;
    };
    auto place = [&](int tile) {   // behind a part's end: its last token again
        const bool own = tile >= own_from;
        const int start = (own ? tile - own_from : tile) * SHD_TILE, last = (own ? own_len : a.prefix) - 1;
        const int t = min(start + lt, last), pi = div_by(t, a.c.page, page_inv);
        return Where{pi, t - pi * a.c.page};
    };
    auto table_of = [&](int tile) { return tile >= own_from ? own_row : a.c.table; };
    auto slot_of = [&](int id, const Where &p) {
        const bool bad = (uint32_t)id >= (uint32_t)a.c.n_pages;
        bad_page |= bad;
        return (int64_t)(bad ? 0 : id) * a.c.page + p.in;
    };
    // page ids go to LDS two tiles before the rows do
    const uint32_t id_at = D::L_ID + wave * 256;
    auto issue_id = [&](int tile) { load_word_to_lds(table_of(tile) + place(tile).page, id_at + (tile & 3) * 1024); };
    // plain rows go to their place in the ring, codes to one of two buffers
    constexpr int OPS = FP8 ? D::LINES + 1 : D::LINES;   // loads of a tile
    auto raw_of = [&](int tile) { return (uint32_t)(D::L_RAW + ((tile & 1) * 4 + wave) * D::RAW); };
    struct Aim {
        const uint8_t *src;
        const float *scale;
        uint32_t dst;
    };
    auto aim = [&](int tile) {
        const int id = lds_read<int>(id_at + (tile & 3) * 1024 + 4 * lane);
        const int64_t slot = slot_of(id, place(tile));
        return Aim{a.c.pages + slot * D::ROW + 16 * (FP8 ? lane & 7 : chunk), FP8 ? a.c.scale + slot : nullptr,
                   FP8 ? raw_of(tile) : base_of(tile) + wave * D::CB * 1024};
    };
    auto issue_op = [](const Aim &x, int op) {   // one of OPS
        switch (op) {
        case 0: load_to_lds<0>(x.src, x.dst); break;
        case 1: load_to_lds<128>(x.src, x.dst, 1024); break;
        case 2: load_to_lds<256>(x.src, x.dst, 2048); break;
        case 3:
            if constexpr (D::LINES > 3) load_to_lds<384>(x.src, x.dst, 3 * 1024);
            break;
        case 4:
            if constexpr (D::LINES > 3) load_to_lds<512>(x.src, x.dst, 4 * 1024);
            break;
        case 5:
            if constexpr (D::LINES > 5) load_to_lds<640>(x.src, x.dst, 5 * 1024);
            break;
        case 6:
            if constexpr (D::LINES > 5) load_to_lds<768>(x.src, x.dst, 6 * 1024);
            break;
        case 7:
            if constexpr (D::LINES > 5) load_to_lds<896>(x.src, x.dst, 7 * 1024);
            break;
        default:
            if constexpr (D::LINES > 5) load_to_lds<1024>(x.src, x.dst, 8 * 1024);
        }
    };
    auto issue_scale = [&](const Aim &x) {
        if constexpr (FP8) load_word_to_lds(x.scale, x.dst + D::LINES * 1024);
    };
    auto issue = [&](int tile) {
        const Aim x = aim(tile);
#pragma unroll
        for (int op = 0; op < D::LINES; ++op) issue_op(x, op);
        issue_scale(x);
    };
    // A line of a thread's codes, its own of the loads above, widened into the ring: sixteen codes are chunks 2 c and 2 c + 1
    // of a row, c = lane % 8 + 8 line.  The last line is the key, then the scale follows.
    auto raw_line = [&](int tile, int line) { return lds_read<u32x4>(raw_of(tile) + 16 * lane, 1024 * line); };
    auto widen = [&](int tile, int line, u32x4 v) {
        const uint32_t dst = base_of(tile) + wave * D::CB * 1024 + (lane >> 3) * 128;
        if (line < D::LINES - 1) {
            const uint32_t at = dst + ((lane & 7) >> 2) * 1024;
            lds_write(at + ((((2 * lane) & 7) ^ lf) << 4), widen8<T>(u32x2{v[0], v[1]}), 2048 * line);
            lds_write(at + ((((2 * lane + 1) & 7) ^ lf) << 4), widen8<T>(u32x2{v[2], v[3]}), 2048 * line);
        } else {
            lds_write(dst + (chunk << 4), v, (D::CB - 1) * 1024);
            const float sc = lds_read<float>(raw_of(tile) + D::LINES * 1024 + 4 * lane);
            const uint32_t at = scale_of(tile) + 4 * lt;
            lds_write<float>(D::L_SCALE + at, sc);
            lds_write<float>(D::L_FRAC + at, __builtin_amdgcn_frexp_mantf(sc));
            lds_write<float>(D::L_EXP + at, sc == 0.0f ? NEG : (float)__builtin_amdgcn_frexp_expf(sc));
        }
    };
    // A tile that some rows see only in part: values that are not finite would reach rows that do not see them.
    auto clear = [&](int tile, int from) {
        constexpr int CH = (D::CB - 1) * 8;
        for (int i = tid; i < (SHD_TILE - from) * CH; i += 256) {
            const int t = from + i / CH, c = i % CH;
            const uint32_t w = base_of(tile) + ((t >> 3) * D::CB + (c >> 3)) * 1024 + (t & 7) * 128 + ((c & 7) << 4);
            x8<T> v = lds_read<x8<T>>(w);
#pragma unroll
            for (int k = 0; k < 8; ++k)
                if (!finite_f32((float)v[k])) v[k] = (T)0.0f;
            lds_write(w, v);
        }
        barrier_lds();
    };

    while (unit < end) {
        own_len = a.whole ? uniform(mla_len(a.kv_lens, group, a.max_kv, a.status)) : 0;
        own_from = own_len > 0 ? prefix_tiles : INT32_MAX;
        own_row = a.own_table + (int64_t)group * a.own_width;
        const int tiles = prefix_tiles + tiles_of(own_len);
        const int in_group = (int)((unit - group_first) / tiles), lo = (int)(unit - group_first - (int64_t)in_group * tiles);
        const int hi = (int)min((int64_t)tiles, lo + end - unit);
        const int64_t blk = (int64_t)group * blocks + in_group;
        unit += hi - lo;
        const int64_t row = blk * SHD_ROWS + 32 * wave + n, wave_row = blk * SHD_ROWS + 32 * wave;
        const bool works = wave_row < rows;
        const int64_t at_row = row < rows ? row : rows - 1;
        issue_id(lo);
        issue_id(lo + 1);
        issue_id(lo + 2);
        issue_id(lo + 3);
        x8<T> qf[KS];
#pragma unroll
        for (int s = 0; s < KS; ++s)
            qf[s] = *reinterpret_cast<const x8<T> *>(s < RANK / 16
                                                         ? static_cast<const T *>(a.q_lat) + at_row * RANK + 16 * s + 8 * hf
                                                         : static_cast<const T *>(a.q_pe) + at_row * MLA_ROPE + 16 * (s - RANK / 16) + 8 * hf);
        // Tokens that a row sees of its own and of the prefix; the least of a wavefront's rows and of the block's.
        const int seen = shd_seen(a, at_row);
        int wave_seen = seen;
        for (int o = 16; o; o >>= 1) wave_seen = min(wave_seen, __shfl_xor(wave_seen, o));
        wave_seen = uniform(wave_seen);
        int block_seen = INT32_MAX;
        for (int64_t r = blk * SHD_ROWS + lane; r < min((blk + 1) * SHD_ROWS, rows); r += 64) block_seen = min(block_seen, shd_seen(a, r));
        for (int o = 32; o; o >>= 1) block_seen = min(block_seen, __shfl_xor(block_seen, o));
        block_seen = uniform(block_seen);
        // Of tile t, the first token that some row does not see though it exists; SHD_TILE if there is none.
        auto hidden = [&](int t) {
            const bool own = t >= prefix_tiles;
            const int least = own ? block_seen : a.prefix + min(0, block_seen), all = own ? own_len : a.prefix;
            const int from = max(0, least - (own ? t - prefix_tiles : t) * SHD_TILE);
            return least < all && from < SHD_TILE ? from : SHD_TILE;
        };
#pragma unroll
        for (int s = 0; s < KS; ++s) arrived(qf[s]);
        wait_vm<0>();
        issue(lo);
        issue(lo + 1);
        if constexpr (FP8) {
            wait_vm<0>();
#pragma unroll
            for (int line = 0; line < D::LINES; ++line) {
                widen(lo, line, raw_line(lo, line));
                widen(lo + 1, line, raw_line(lo + 1, line));
            }
        }
        issue(lo + 2);

        f32x16 o[CT];
#pragma unroll
        for (int c = 0; c < CT; ++c)
#pragma unroll
            for (int r = 0; r < 16; ++r) o[c][r] = 0.0f;
        float m = NEG, l = 0.0f, mv = NEG;
        f32x16 s;
        f32x4 frac, expo;   // E4M3: four tokens' scales
        float f = 1.0f, ref = 0.0f, refv = 0.0f;
        bool moved = false;
        x8<T> p[2], pn[2];

        // ---- scores of a tile.  Between the products the loads of the tile after the next go out (all of them at once would
        // hold the wavefront up; behind the last tile: rows that are not used), and the codes of the next are widened.
        auto score = [&](int tile, auto steady) {
            constexpr bool STEADY = decltype(steady)::value;
            Aim x{};
            if constexpr (STEADY) x = aim(tile + 2);
            const uint32_t base = base_of(tile);
            uint32_t kb[4];
#pragma unroll
            for (int v = 0; v < 4; ++v) kb[v] = base + (ka ^ 32 * v);
#pragma unroll
            for (int r = 0; r < 16; ++r) s[r] = 0.0f;
            // operands four reads before their products
            u32x4 w[6], raw{};
#pragma unroll
            for (int i = 0; i < 4; ++i) w[i] = lds_read<u32x4>(kb[i]);
            if (STEADY && FP8) raw = raw_line(tile + 1, 0);
#pragma unroll
            for (int k = 0; k < KS; k += 2) {
                __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                for (int i = k + 4; i < k + 6 && i < KS; ++i) w[i % 6] = lds_read<u32x4>(kb[i & 3], (i >> 2) * 1024);
                if (FP8 && k == RANK / 16) {
                    settled(s);
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const f32x4 v = lds_read<f32x4>(D::L_SCALE + 16 * hf + scale_of(tile), 32 * q);
#pragma unroll
                        for (int i = 0; i < 4; ++i) s[4 * q + i] *= v[i];
                    }
                }
#pragma unroll
                for (int i = k; i < k + 2; ++i) mfma_v<T>(s, __builtin_bit_cast(x8<T>, w[i % 6]), qf[i]);
                if (STEADY && k % 4 == 0 && k / 4 < D::LINES) {
                    issue_op(x, k / 4);
                    if (FP8) {
                        widen(tile + 1, k / 4, raw);
                        if (k / 4 + 1 < D::LINES) raw = raw_line(tile + 1, k / 4 + 1);
                    }
                }
            }
            __builtin_amdgcn_sched_barrier(0);
            if constexpr (STEADY) issue_scale(x);
            issue_id(tile + 4);
            __builtin_amdgcn_sched_barrier(0);
            const bool own = tile >= prefix_tiles;
            const int t0 = (own ? tile - prefix_tiles : tile) * SHD_TILE;
            if (t0 + SHD_TILE > (own ? wave_seen : a.prefix + min(0, wave_seen))) {
                settled(s);
                int rem = (own ? seen : a.prefix + min(0, seen)) - t0 - 4 * hf;
                arrived(rem);   // a branch, not selects that every tile would pay for
#pragma unroll
                for (int r = 0; r < 16; ++r)
                    if (8 * (r >> 2) + (r & 3) >= rem) s[r] = NEG;
            }
        };
        // ---- its softmax in CT steps, for the shadows of matrix instructions
        auto soften = [&](int tile, int step) {
            // The products of steps 0 and 1 stand between the scores' last one and this wait, which covers the end of it.
            if (step == 1) {
                settled(s);
                float top = fmaxf(fmaxf(s[0], s[1]), s[2]);
#pragma unroll
                for (int r = 3; r < 15; r += 2) top = fmaxf(fmaxf(top, s[r]), s[r + 1]);
                top = half_max(fmaxf(top, s[15])) * scale;
                bool grows = top > m + LAG;
                const float to = grows ? top - LIFT : m;
                f = m == to ? 1.0f : __builtin_amdgcn_exp2f(m - to);
                l *= f;
                m = to;
                ref = m == NEG ? 0.0f : m;
                if (FP8) {
                    float topv = NEG;
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const f32x4 e = lds_read<f32x4>(D::L_EXP + 16 * hf + scale_of(tile), 32 * q);
#pragma unroll
                        for (int i = 0; i < 4; ++i) topv = fmaxf(topv, __builtin_fmaf(s[4 * q + i], scale, e[i]));
                    }
                    topv = half_max(topv);
                    const bool growsv = topv > mv + LAG;
                    const float tov = growsv ? rintf(topv) - LIFT : mv;
                    f = mv == tov ? 1.0f : __builtin_amdgcn_exp2f(mv - tov);
                    mv = tov;
                    refv = mv == NEG ? 0.0f : mv;
                    grows |= growsv;
                }
                moved = __ballot(grows) != 0;
            } else if (step > 1) {
#pragma unroll
                for (int r = 0; r < 16; ++r)
                    if (r >= (step - 2) * 16 / (CT - 2) && r < (step - 1) * 16 / (CT - 2)) {
                        float w = __builtin_amdgcn_exp2f(__builtin_fmaf(s[r], scale, -ref));
                        l += w;
                        if (FP8) {
                            if (r % 4 == 0) {
                                const uint32_t at = 16 * hf + scale_of(tile);
                                frac = lds_read<f32x4>(D::L_FRAC + at, 8 * r);
                                expo = lds_read<f32x4>(D::L_EXP + at, 8 * r);
                            }
                            w = frac[r % 4] * __builtin_amdgcn_exp2f(__builtin_fmaf(s[r], scale, expo[r % 4]) - refv);
                            if (s[r] == NEG) w = 0.0f;   // not seen, whatever its scale
                        }
                        pn[r >> 3][r & 7] = (T)w;
                    }
            }
        };
        auto take = [&] {   // the weights formed are the ones to use
            p[0] = pn[0];
            p[1] = pn[1];
            if (moved) {
                acc_settled();
#pragma unroll
                for (int c = 0; c < CT; ++c) {
                    acc_scale<0>(o[c], f);
                    acc_scale<8>(o[c], f);
                }
            }
        };
        // ---- a tile's values by its weights; the next tile's softmax between the products
        auto values = [&](int tile, auto next) {
            const uint32_t base = base_of(tile);
            uint32_t vb[4];
#pragma unroll
            for (int v = 0; v < 4; ++v) vb[v] = base + (va ^ (64 * (v & 1) + 16 * (v >> 1))) + (v >> 1) * D::CB * 1024;
            auto read = [&](int c, int k) {
                const int imm = 2 * k * D::CB * 1024 + (c >> 1) * 1024;
                const u32x2 v0 = lds_read_tr16(vb[c & 1], imm), v1 = lds_read_tr16(vb[2 + (c & 1)], imm);
                return u32x4{v0[0], v0[1], v1[0], v1[1]};
            };
            // all columns by the first sixteen tokens, then by the others, so that no product waits for the one before it;
            // operands three reads ahead
            u32x4 w[4];
#pragma unroll
            for (int i = 0; i < 3; ++i) w[i] = read(i % CT, i / CT);
#pragma unroll
            for (int i = 0; i < 2 * CT; ++i) {
                if (i % 2 == 0) __builtin_amdgcn_sched_barrier(0);
                if (i + 3 < 2 * CT) w[(i + 3) & 3] = read((i + 3) % CT, (i + 3) / CT);
                o[i % CT] = mfma32<T>(__builtin_bit_cast(x8<T>, w[i & 3]), p[i / CT], o[i % CT]);
                if constexpr (decltype(next)::value)
                    if (i % 2) soften(tile + 1, i / 2);
            }
            __builtin_amdgcn_sched_barrier(0);
        };

        if constexpr (!FP8) wait_vm<2 * OPS>();
        barrier_lds();
        score(lo, std::false_type());
#pragma unroll
        for (int c = 0; c < CT; ++c) soften(lo, c);
        take();
        int i = lo;
        for (; i + 1 < hi; ++i) {
            // plain rows: tile i + 1 has come, i + 2 is out; codes: those of tile i + 2 have come
            wait_vm<FP8 ? 1 : OPS + 1>();
            barrier_lds();   // tile i + 1 is there, and every wavefront is done with tile i - 1
            if (const int from = hidden(i); from < SHD_TILE) clear(i, from);
            score(i + 1, std::true_type());
            values(i, std::true_type());
            take();
        }
        if (const int from = hidden(i); from < SHD_TILE) {
            barrier_lds();
            clear(i, from);
        }
        values(i, std::false_type());
        wait_vm<0>();
        barrier_lds();   // the ring is free
        acc_settled();

        // ---- the segment's result, divided by its sum
        l = half_sum(l);
        if (works) {
            const float half_off = FP8 && l != 0.0f ? __builtin_amdgcn_exp2f(0.5f * (mv - m)) : 1.0f;
            const float by = l == 0.0f ? 0.0f : half_off / l;
            float *dst = a.part + (g + blk) * D::SLOT, *at = dst + wave * CT * 1024 + 4 * lane;
#pragma unroll
            for (int c = 0; c < CT; ++c) {
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    __builtin_amdgcn_sched_barrier(0);
                    f32x4 v = acc_read(o[c][4 * q], o[c][4 * q + 1], o[c][4 * q + 2], o[c][4 * q + 3]);
#pragma unroll
                    for (int k = 0; k < 4; ++k) v[k] = FP8 ? v[k] * by * half_off : v[k] * by;
                    *reinterpret_cast<f32x4 *>(at + (c * 4 + q) * 256) = v;
                }
            }
            if (hf == 0) *reinterpret_cast<float2 *>(dst + SHD_ROWS * RANK + 2 * (32 * wave + n)) = make_float2(m, l);
        }
        if (hi == tiles && in_group + 1 == blocks) {
            group_first += (int64_t)blocks * tiles;
            ++group;
        }
    }
    if (bad_page) raise_status(a.status, ST_BADPAGE);
}

// Joins partial results: out = sum 2^{m_i - M} l_i o_i / sum 2^{m_i - M} l_i,
// those over the prefix in order, then those of the rows' sequences.  A
// wavefront has 32 rows by 8 COLS columns.  W > 1: a workgroup's wavefronts take every
// W-th partial each of one such piece, for few rows in many parts.
template <class T, int RANK, int W, int COLS>
__global__ __launch_bounds__(W > 1 ? 64 * W : 256) void k_mla_shared_join(MlaSharedArgs a) {
    constexpr int SLOT = SHD_ROWS * RANK + 2 * SHD_ROWS, PIECES = RANK / 8 / COLS;
    constexpr float NEG = -__builtin_inff();
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, n = lane & 31;
    const int64_t id = W > 1 ? blockIdx.x : (int64_t)blockIdx.x * 4 + wave;
    const int piece = (int)(id % PIECES), part = W > 1 ? wave : 0;
    const int64_t rows = (int64_t)a.batch * a.n_q * a.heads, row = id / PIECES * 32 + n;
    if (W == 1 && id / PIECES * 32 >= rows) return;
    const int64_t at_row = row < rows ? row : rows - 1;
    __shared__ f32x4 so[W > 1 ? W : 1][64];
    __shared__ float sm[W > 1 ? W : 1][64], sl[W > 1 ? W : 1][64];
    float m = NEG, l = 0.0f;
    f32x4 o[COLS];
#pragma unroll
    for (int c = 0; c < COLS; ++c) o[c] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    // AHEAD partials at a time; those past the last one again, with no weight
    constexpr int AHEAD = W > 1 ? 4 : 2;
    auto add = [&](int first, int count, auto at) {
        for (int i = first; i < count; i += AHEAD * W) {
            float2 ml[AHEAD];
            f32x4 v[AHEAD][COLS];
#pragma unroll
            for (int k = 0; k < AHEAD; ++k) {
                const float *base, *stats;
                at(min(i + k * W, count - 1), base, stats);
                ml[k] = *reinterpret_cast<const float2 *>(stats);
#pragma unroll
                for (int c = 0; c < COLS; ++c) v[k][c] = *reinterpret_cast<const f32x4 *>(base + 256 * c);
            }
            float to = m;
#pragma unroll
            for (int k = 0; k < AHEAD; ++k) to = fmaxf(to, ml[k].x);
            const float old = m == to ? 1.0f : __builtin_amdgcn_exp2f(m - to);
            m = to;
            l *= old;
#pragma unroll
            for (int c = 0; c < COLS; ++c)
#pragma unroll
                for (int j = 0; j < 4; ++j) o[c][j] *= old;
#pragma unroll
            for (int k = 0; k < AHEAD; ++k)
                if (i + k * W < count) {
                    const float f = ml[k].y * (ml[k].x == to ? 1.0f : __builtin_amdgcn_exp2f(ml[k].x - to));
                    l += f;
#pragma unroll
                    for (int c = 0; c < COLS; ++c)
#pragma unroll
                        for (int j = 0; j < 4; ++j) o[c][j] = __builtin_fmaf(v[k][c][j], f, o[c][j]);
                }
        }
    };
    {
        // the block's units, from the plan: a piece's rows are of one block
        const int64_t blk = uniform((int)(id / PIECES * 32 / SHD_ROWS));
        const int group = a.whole ? (int)(blk / (a.n_q * a.heads / SHD_ROWS)) : 0;
        const int groups = a.whole ? a.batch : 1, parts = (int)a.plan[groups + 1];
        int64_t g0 = blk * parts, g1 = g0 + parts - 1;
        if (!parts) {
            const int64_t blocks = a.whole ? a.n_q * a.heads / SHD_ROWS : blocks_of(rows), total = a.plan[groups];
            const Units u{total, (int)min(shares_of(total), (int64_t)a.shares), 0};
            const int64_t tiles = (a.plan[group + 1] - a.plan[group]) / blocks, unit = a.plan[group] + (blk - group * blocks) * tiles;
            g0 = u.owner(unit);
            g1 = u.owner(unit + tiles - 1);
        }
        const int r = (int)(row - blk * SHD_ROWS);
        const int col = (r / 32 * (RANK / 8) + piece * COLS) * 256 + 4 * lane, stat = SHD_ROWS * RANK + 2 * r;
        add(part, (int)(g1 - g0) + 1, [&](int i, const float *&base, const float *&stats) {
            const float *slot = a.part + (g0 + i + blk) * SLOT;
            base = slot + col;
            stats = slot + stat;
        });
    }
    if (a.own) {   // own tokens apart
        const int per = a.n_q * a.heads, b = (int)(at_row / per), w = (int)(at_row - (int64_t)b * per);
        const int block = w / a.p.rows, r = w - block * a.p.rows;
        const int32_t *plan = reinterpret_cast<const int32_t *>(a.own) + 2 * b;
        const int g0 = plan[0], g1 = plan[1];
        const int col = (r / 32 * (RANK / 8) + piece * COLS) * 256 + 4 * (r % 32 + 32 * (lane >> 5)), stat = a.p.rows * RANK + 2 * r;
        add(part, g1 - g0 + 1, [&](int i, const float *&base, const float *&stats) {
            const float *slot = g0 == g1 ? a.full + ((int64_t)b * a.p.blocks + block) * a.p.slot
                                         : a.own + a.p.first + (2 * ((int64_t)block * a.p.groups + g0 + i) + (i == 0 ? 1 : 0)) * a.p.slot;
            base = slot + col;
            stats = slot + stat;
        });
    }
    if constexpr (W > 1) {
        static_assert(COLS == 1, "one piece a workgroup");
        so[wave][lane] = o[0];
        sm[wave][lane] = m;
        sl[wave][lane] = l;
        __syncthreads();
        if (wave) return;
#pragma unroll
        for (int w = 1; w < W; ++w) m = fmaxf(m, sm[w][lane]);
        o[0] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        l = 0.0f;
#pragma unroll
        for (int w = 0; w < W; ++w) {
            const float f = sm[w][lane] == m ? 1.0f : __builtin_amdgcn_exp2f(sm[w][lane] - m);
            const f32x4 v = so[w][lane];
            l = __builtin_fmaf(sl[w][lane], f, l);
#pragma unroll
            for (int i = 0; i < 4; ++i) o[0][i] = __builtin_fmaf(v[i], f, o[0][i]);
        }
    }
    if (row >= rows) return;
    const float f = l == 0.0f ? 0.0f : 1.0f / l;
#pragma unroll
    for (int c = 0; c < COLS; ++c) {
        x4<T> v;
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = (T)(o[c][i] * f);
        *reinterpret_cast<x4<T> *>(static_cast<T *>(a.out) + row * RANK + 8 * (piece * COLS + c) + 4 * (lane >> 5)) = v;
    }
    if (a.lse && piece == 0 && lane < 32) a.lse[row] = l == 0.0f ? NEG : (m + __builtin_amdgcn_logf(l)) * LN2;
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

// A join of at most this many groups of 32 rows has sixteen wavefronts a piece
// (4 groups: 45 us for the whole call against 130; 16: 50 against 62; 32: 61
// against 58; 64: 72 against 58).
constexpr int JOIN_DEEP = 16, JOIN_COLS = 4;

// Which is faster, in us by what both measured (rank 512, 100 tokens of their
// own, sizes in batch x n_q x heads x prefix): tiles of 64 tokens a workgroup
// where sequences read the prefix apart, blocks of 32 rows if a sequence has no
// more, else of 64; tiles of 32 tokens a workgroup, and a third launch where
// blocks are not of one sequence, together.  Apart / together, plain:
//   4 x 1 x 16 x 8192     22.5 / 39.8     64 x 1 x 16 x 32768   240 / 112
//   64 x 1 x 16 x 8192    76.5 / 68.8     64 x 1 x 5 x 32768    241 / 71.2
//   64 x 1 x 64 x 8192     101 / 113      64 x 1 x 64 x 32768   318 / 292
//   16 x 1 x 128 x 8192   57.6 / 67.9     64 x 1 x 128 x 32768  570 / 517
// E4M3, whose codes are widened in registers there, here through LDS:
//   64 x 1 x 16 x 8192    87.2 / 76.2     64 x 1 x 16 x 32768   296 / 137
//   16 x 4 x 64 x 32768    350 / 364      64 x 1 x 128 x 32768  680 / 687
// Prefixes that no cache holds whole, 100 tokens of their own, E4M3 on the left
// (both ways come to the same, up to 2 x 128 rows a sequence too), plain on the right:
//   16 x 1 x 128 x 131072  673 / 685      16 x 1 x 128 x 131072   586 / 528
//   16 x 1 x 128 x 524288 2625 / 2617     16 x 1 x 128 x 524288  2346 / 2008
//   64 x 1 x 128 x 131072 2611 / 2613     64 x 1 x 128 x 131072  2251 / 2009
//   64 x 1 x 16 x 524288  4489 / 1420     64 x 1 x 16 x 524288   3958 / 1120
bool mla_prefix_by_sequence(const coli_mla_dims &d, int batch, int n_q, int prefix, int max_kv, int path) {
    const int64_t longest = (int64_t)prefix + max_kv;
    if (longest > COLI_MLA_MAX_LENGTH || batch * longest > COLI_MLA_MAX_TOKENS) return false;
    if (path) return path == 2;
    const int rows = n_q * d.n_heads, own = max_kv / 2;
    const bool fp8 = d.kv_format == COLI_KV_E4M3, few = rows <= 32, whole = whole_blocks(rows);
    const double size = d.rank == 512 ? 1.0 : 0.6, own_blocks = whole ? (double)batch * rows / SHD_ROWS : 0.0;
    const double apart = size / (64 * 256) * batch * ((rows + 63) / 64) * ((double)prefix + own);
    const double together = size / (32 * 256) * ((double)blocks_of((int64_t)batch * rows) * prefix + own_blocks * own);
    const double t_apart = few ? 13.0 + (fp8 ? 2.2 : 2.0) * apart : 20.0 + (fp8 ? 2.6 : 2.3) * apart;
    const double t_together = (whole ? 35.0 : 48.0) * (d.rank == 512 ? 1.0 : 0.8) + (fp8 ? 5.0 + 2.6 * together : 1.9 * together);
    return t_apart <= t_together;
}

size_t mla_shared_part_bytes(const coli_mla_dims &d, int batch, int n_q, int prefix, int max_kv) {
    // slots are counted by workgroup + block of rows: a bound that grows with each argument
    const int64_t rows = (int64_t)batch * n_q * d.n_heads;
    return shd_plan_bytes(batch) +
           4 * (size_t)(SHD_ROWS * d.rank + 2 * SHD_ROWS) * (size_t)(shd_shares(rows, prefix, max_kv) + blocks_of(rows));
}

MlaSharedArgs mla_shared_args(const coli_mla_dims &d, void *part, int batch, int n_q, int prefix, int max_kv) {
    MlaSharedArgs a{};
    a.plan = static_cast<int64_t *>(part);
    a.part = reinterpret_cast<float *>(static_cast<uint8_t *>(part) + shd_plan_bytes(batch));
    a.batch = batch;
    a.n_q = n_q;
    a.heads = d.n_heads;
    a.prefix = prefix;
    a.max_kv = max_kv;
    a.scale = d.softmax_scale;
    a.whole = whole_blocks((int64_t)n_q * d.n_heads);
    a.shares = shd_shares((int64_t)batch * n_q * d.n_heads, prefix, a.whole ? max_kv : 0);
    return a;
}

hipError_t launch_mla_shared(const MlaSharedArgs &a, const coli_mla_dims &d, hipStream_t st) {
    return with_shape(d, [&](auto shape) {
        using D = decltype(shape);
        const hipError_t e = ensure_dyn_smem(reinterpret_cast<const void *>(&k_mla_shared<D>), D::LDS);
        if (e != hipSuccess) return e;
        hipLaunchKernelGGL(k_mla_shared<D>, dim3(a.shares), dim3(256), D::LDS, st, a);
        return hipGetLastError();
    });
}

hipError_t launch_mla_shared_join(const MlaSharedArgs &a, const coli_mla_dims &d, hipStream_t st) {
    const int64_t rows = (int64_t)a.batch * a.n_q * a.heads;
    return with_shape(d, [&](auto shape) {
        using D = decltype(shape);
        const int64_t groups = (rows + 31) / 32, pieces = D::RANK / 8;
        // parts of a row: those of the prefix, and of its own tokens
        if (groups <= JOIN_DEEP)
            hipLaunchKernelGGL((k_mla_shared_join<typename D::T, D::RANK, 16, 1>), dim3((uint32_t)(groups * pieces)), dim3(1024), 0, st,
                               a);
        else
            hipLaunchKernelGGL((k_mla_shared_join<typename D::T, D::RANK, 1, JOIN_COLS>),
                               dim3((uint32_t)((groups * (pieces / JOIN_COLS) + 3) / 4)), dim3(256), 0, st, a);
        return hipGetLastError();
    });
}

}  // namespace coli

// Absorbed attention of a few new tokens a sequence over the paged latents:
//
//   s_rt = scale (<q_r, c_t> + <p_r, k_t>),  out_r = sum_t e^{s_rt} c_t / sum_t e^{s_rt}
//
// for the n_q * n_heads query rows r of a sequence.  Every row reads the same
// latents, so a sequence is one product [rows x (rank + 64)] x [tokens] and
// one [tokens] x [rank], of the same cached tile: read from memory once, used
// twice from LDS.
//
// What bounds it: up to 64 rows the cached bytes, and that a CU has no load out
// from a tile's end, which waits for all, until the next tile's scores (131071
// tokens, 64 heads, rank 512, bf16: 151 MB; 44 us and 12 us for the join from
// memory, 3.5 TB/s in the first; 33 and 9.5 where the last-level cache holds
// them); from 128 rows on a tile's own chain of scores, softmax and values,
// which one wavefront a SIMD runs through without overlap (registers: 144 of
// queries and 128 of accumulators): a four-token verify of 64 heads over
// 115700 E4M3 tokens takes 84.5 us and 9.6 us, 0.67 PFLOP/s, matrix cores 33%
// busy; reads from LDS, widening, softmax, loads and page bookkeeping, each
// taken out alone, saved 5 to 7 us.
#include "kernels.h"
#include "mla_mfma.h"

namespace coli {
namespace {

constexpr int DEC_TILE = 64;     // tokens a tile
constexpr float LOG2E = 1.44269504088896340736f, LN2 = 0.69314718055994530942f;
// The running maximum moves only when a score exceeds it by this many powers
// of two: weights then reach 2^8 (binary16, lifted by 2^7: 2^15), which both
// types hold, and most tiles spare the pass over the accumulators.
constexpr float MAX_LAG = 8.0f;

// E4M3 tokens have a scale each, f 2^e with 1/2 <= |f| < 1, and what is rounded
// to 16 bits is weight times scale.  That product has a reference of its own,
// the row's largest 2^{score + e} so far, lagging alike: a token whose scale is
// far above the others' takes their bits only as far as its weight lets it
// count, and one that a row does not see takes none.  The scale's exponent costs
// one rounding, of score + e; f stays outside, and the reference is a whole
// number, so that subtracting it costs none.

// Four wavefronts: RG groups of 32 rows, each of CG = 4 / RG wavefronts that
// share the output's columns.  Wavefronts 0 and 1 of a group score half of a
// tile's tokens each and hand their weights to the others through LDS.  Whole
// columns for a wavefront would spare that exchange, but 256 registers of
// accumulators beside 144 of queries spilled 330 and more.  Not built: eight
// wavefronts, a quarter of the columns and half of each score's sum apiece,
// which would read LDS as much as this in half the registers.
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
    static constexpr int QB = KS / 4;                         // blocks of eight chunks in a query row
    static constexpr int QUERY = ROWS * 128 * QB;
    // Queries pass through LDS on their way to registers: through the buffer of the tile before, which plain rows fill
    // alike, or, with codes, through a region of their own.
    static constexpr int L_OFF = 2 * TILE + (FP8 ? QUERY : 0);  // int64 [2][64]: row offsets of tiles to come
    static constexpr int L_SCALE = L_OFF + 2 * 8 * DEC_TILE;  // float [2][64]: E4M3 scales
    static constexpr int L_EXP = L_SCALE + 2 * 4 * DEC_TILE;  // float [2][64]: their exponents
    static constexpr int L_TOP = L_EXP + (FP8 ? 2 * 4 * DEC_TILE : 0);   // float [RG][2][32]: maxima, at the end sums
    static constexpr int TOPS = RG * 2 * 32 * 4;              // bytes of them; with codes, as many of score + exponent follow
    static constexpr int L_GROW = L_TOP + (FP8 ? 2 : 1) * TOPS;   // int: the last tile whose maxima had to move, counted from 1
    // weights: [RG][2][2][64 lanes] of 16 bytes (with codes, in the region of the queries, which are in registers then)
    static constexpr int L_P = FP8 ? 2 * TILE : L_GROW + 16;
    static constexpr int LDS = L_GROW + 16 + (FP8 ? 0 : RG * 2 * 2048);
    static_assert(LDS <= 160 * 1024, "the LDS of a CU");
    static constexpr int SLOT = ROWS * RANK + 2 * ROWS;       // floats of a partial result
};

// A sequence's tiles; one without tokens keeps an empty tile, whose owner
// writes its zeros.
__device__ __forceinline__ int dec_tiles(int len) { return len > 0 ? (len + DEC_TILE - 1) / DEC_TILE : 1; }

// Work is shared out evenly in units: a sequence of n tiles is n + 1 of them,
// unit 0 standing for its queries and its results, which cost about a tile,
// unit k > 0 for tile k - 1.  Workgroup g of `shares` has `per` units in order,
// the first `more` workgroups one more.
struct Shares {
    int per, more;
    __device__ __forceinline__ Shares(int units, int shares) : per((uint32_t)units / (uint32_t)shares), more(units - per * shares) {}
    __device__ __forceinline__ int first(int g) const { return g * per + min(g, more); }
    __device__ __forceinline__ int owner(int unit) const {
        const int t = unit - more * (per + 1);
        return t < 0 ? (uint32_t)unit / (uint32_t)(per + 1) : more + (uint32_t)t / (uint32_t)per;
    }
};

// Swizzle of a token's 16-byte chunks: LDS holds a tile as [8 tokens][8
// chunks] blocks of 1 KiB, which is what a wavefront's load writes, chunk c of
// token t at position (c ^ swz(t)) of its 128 bytes.  The same chunk of
// sixteen tokens, and what 32 lanes of a transposing read take (four tokens
// by four chunks, or eight tokens by two for codes), then lie in sixteen
// different groups of banks.
template <bool FP8>
__device__ __forceinline__ int dec_swz(int t) {
    const int b1 = (t >> 1) & 1, b2 = (t >> 2) & 1, b3 = (t >> 3) & 1;
    return FP8 ? 4 * b1 + b2 + 2 * b3 : 4 * b1 + 2 * b2 + b3;
}

// The tiles of a workgroup form one stream, whatever sequences they belong
// to: page ids are read three tiles ahead, row offsets stand in LDS two ahead,
// the tiles' loads run one ahead.
//
// A tile takes two barriers: one when it has arrived, one when its weights
// have.  The weights are formed with the maximum of the tiles before, and
// formed again (a third barrier) only where a score exceeds that by MAX_LAG.
template <class D>
__global__ __launch_bounds__(256, 1) void k_mla_decode(MlaDecodeArgs a, int groups) {
    using T = typename D::T;
    constexpr int RANK = D::RANK, CT = D::CT, KS = D::KS;
    constexpr bool FP8 = D::FP8;
    constexpr float NEG = -__builtin_inff();
    const int tid = threadIdx.x, lane = tid & 63, wave = uniform(tid >> 6);
    const int n = lane & 31, hf = lane >> 5;
    const int rg = wave / D::CG, cg = wave % D::CG, th = cg & 1;
    const int g = blockIdx.x, rows = a.n_q * a.heads;
    const int block_row = blockIdx.y * D::ROWS, wave_row = block_row + 32 * rg, row = wave_row + n;
    const bool has_rows = wave_row < rows;

    // ---- this workgroup's tiles: `total` of them from tile `tile` of sequence `seq`
    auto tiles_of = [&](int b) { return b < a.batch ? dec_tiles(mla_len(a.kv_lens, b, a.max_kv, a.status)) : 0; };
    int tiles = 0, mine = 0, incl = 0;
    for (int b = 0; b < a.batch; b += 64) {
        mine = tiles_of(b + lane);
        incl = wave_scan(mine);
        tiles += __builtin_amdgcn_readlane(incl, 63);
    }
    const int shares = min(groups, tiles);
    if (g >= shares) return;
    const Shares share(tiles + a.batch, shares);
    const int begin = share.first(g), end = share.first(g + 1);
    int seq = -1, tile = 0, total = 0;
    for (int b = 0, base = 0; b < a.batch; b += 64) {
        if (a.batch > 64) {
            mine = tiles_of(b + lane);
            incl = wave_scan(mine);
        }
        const bool real = b + lane < a.batch;
        const int f = base + incl - mine + b + lane;   // the sequence's unit 0
        if (g == 0 && blockIdx.y == 0 && wave == 0 && real) {   // for the join
            int32_t *plan = reinterpret_cast<int32_t *>(a.part) + 2 * (b + lane);
            plan[0] = share.owner(f + 1);
            plan[1] = share.owner(f + mine);
        }
        // its tiles here: those of the units in [begin, end)
        const int from = min(max(begin - f - 1, 0), mine), to = min(max(end - f - 1, 0), mine);
        const uint64_t hit = __ballot(real && to > from);
        if (seq < 0 && hit) {
            const int l = __builtin_ctzll(hit);
            seq = b + l;
            tile = __builtin_amdgcn_readlane(from, l);
        }
        total += __builtin_amdgcn_readlane(wave_scan(real ? to - from : 0), 63);
        base += __builtin_amdgcn_readlane(incl, 63);
    }
    if (total == 0) return;

    // ---- the stream of page ids, row offsets and loads: every wavefront carries all of it, a token a lane, in straight
    // lines that fill the shadows of matrix instructions
    const uint32_t page_inv = 0xffffffffu / (uint32_t)a.c.page;
    int lens_from = seq, lens = 0;   // lane i: the length of sequence lens_from + i
    auto load_lens = [&] {
        lens_from = seq;
        lens = min(max(a.kv_lens[min(seq + lane, a.batch - 1)], 0), a.max_kv);
    };
    load_lens();
    int next_seq = seq, next_tile = tile, next_len = __builtin_amdgcn_readlane(lens, 0);
    bool bad_page = false;
    struct Page {
        int id, in;   // of token `lane` of a tile
    };
    auto page_ids = [&](Page &p) {
        const int t = max(0, min(next_tile * DEC_TILE + lane, next_len - 1));   // behind the end: the last again
        const int pi = div_by(t, a.c.page, page_inv);
        p.in = t - pi * a.c.page;
        p.id = a.c.table[(int64_t)next_seq * a.c.width + pi];
        if (next_len == 0) p.id = 0;
        const bool cross = (next_tile + 1) * DEC_TILE >= next_len;
        next_tile = cross ? 0 : next_tile + 1;
        next_seq = cross ? min(next_seq + 1, a.batch - 1) : next_seq;   // behind the last tile: read and not used
        next_len = __builtin_amdgcn_readlane(lens, next_seq - lens_from);
    };
    float sc_next = 0.0f;
    auto put_offsets = [&](int it, const Page &p) {
        const bool bad = (uint32_t)p.id >= (uint32_t)a.c.n_pages;
        bad_page |= bad;
        const int64_t slot = (int64_t)(bad ? 0 : p.id) * a.c.page + p.in;
        lds_write<int64_t>(D::L_OFF + 8 * ((it & 1) * DEC_TILE + lane), slot * D::ROW);
        if (FP8) sc_next = a.c.scale[slot];
    };
    auto put_scales = [&](int it) {
        const uint32_t at = 4 * ((it & 1) * DEC_TILE + lane);
        lds_write<float>(D::L_SCALE + at, sc_next);
        lds_write<float>(D::L_EXP + at, sc_next == 0.0f ? NEG : (float)__builtin_amdgcn_frexp_expf(sc_next));
    };
    // what this thread loads: chunk (lane % 8) of tokens 16 wave + lane / 8 and + 8
    const int lt0 = 16 * wave + (lane >> 3), lt1 = lt0 + 8;
    const uint8_t *src0 = a.c.pages + (((lane & 7) ^ dec_swz<FP8>(lt0)) << 4);
    const uint8_t *src1 = a.c.pages + (((lane & 7) ^ dec_swz<FP8>(lt1)) << 4);
    auto source = [&](int it, int t) { return lds_read<int64_t>(D::L_OFF + 8 * ((it & 1) * DEC_TILE + t)); };
    auto lds_line = [](int c, const uint8_t *p, uint32_t d) {   // line c of a row, its block c
        switch (c) {
        case 0: load_to_lds<0>(p, d); break;
        case 1: load_to_lds<128>(p, d, 1024); break;
        case 2: load_to_lds<256>(p, d, 2048); break;
        case 3: load_to_lds<384>(p, d, 3 * 1024); break;
        case 4: load_to_lds<512>(p, d, 4 * 1024); break;
        case 5: load_to_lds<640>(p, d, 5 * 1024); break;
        case 6: load_to_lds<768>(p, d, 6 * 1024); break;
        case 7: load_to_lds<896>(p, d, 7 * 1024); break;
        default: load_to_lds<1024>(p, d, 8 * 1024); break;
        }
    };
    auto issue = [&](int it, int c, const uint8_t *p0, const uint8_t *p1) {
        const uint32_t d = (it & 1) * D::TILE + 2 * wave * D::CB * 1024;
        lds_line(c, p0, d);
        lds_line(c, p1, d + D::CB * 1024);
    };
    // A sequence's queries: whole rows into LDS, as a tile's, then every wavefront's operands out of it.
    x8<T> qf[KS];
    auto issue_q = [&](int b, uint32_t to) {
#pragma unroll
        for (int i = 0; i < D::RG; ++i) {
            const int grp = wave * D::RG + i, r8 = 8 * grp + (lane >> 3), r = block_row + r8 < rows ? block_row + r8 : 0;
            const int chunk = 8 * ((lane & 7) ^ dec_swz<false>(r8));
            const T *ql = static_cast<const T *>(a.q_lat) + ((int64_t)b * rows + r) * RANK + chunk;
            const T *qp = static_cast<const T *>(a.q_pe) + ((int64_t)b * rows + r) * MLA_ROPE + chunk;
#pragma unroll
            for (int c = 0; c < D::QB; ++c) load_to_lds(c < D::QB - 1 ? ql + 64 * c : qp, to + (grp * D::QB + c) * 1024);
        }
    };
    auto read_q = [&](uint32_t from) {
        const int r = 32 * rg + n, f = dec_swz<false>(r);
        uint32_t at[8];
#pragma unroll
        for (int v = 0; v < 8; ++v) at[v] = from + (r >> 3) * D::QB * 1024 + (r & 7) * 128 + ((v ^ f) << 4);
#pragma unroll
        for (int s = 0; s < KS; ++s) {
            // the chunk of this lane half: codes come sixteen to a read, two matrix steps
            if (FP8 && s < RANK / 16) {
                const int c = 4 * (s >> 1) + (s & 1);
                qf[s] = lds_read<x8<T>>(hf ? at[(c + 2) & 7] : at[c & 7], (c >> 3) * 1024);
            } else {
                qf[s] = lds_read<x8<T>>(hf ? at[(2 * s + 1) & 7] : at[2 * s & 7], (s >> 2) * 1024);
            }
        }
#pragma unroll
        for (int s = 0; s < KS; ++s) arrived_acc(qf[s]);
    };
    // Brings the lines of a sequence's queries into the L2: a word of each, ROWS / 256 threads a row.
    uint32_t touched[3] = {0, 0, 0};
    auto touch_q = [&](int b) {
        constexpr int PER = 256 / D::ROWS, LINES = RANK / 64 / PER;   // threads and latent lines: 4 and 2 or 1, 8 and 1 or 0
        const int r8 = tid / PER, r = block_row + r8 < rows ? block_row + r8 : 0;
        const uint8_t *ql = reinterpret_cast<const uint8_t *>(static_cast<const T *>(a.q_lat) + ((int64_t)b * rows + r) * RANK);
        const uint8_t *qp = reinterpret_cast<const uint8_t *>(static_cast<const T *>(a.q_pe) + ((int64_t)b * rows + r) * MLA_ROPE);
        touched[0] = *reinterpret_cast<const uint32_t *>(qp);
        touched[1] = *reinterpret_cast<const uint32_t *>(ql + tid % PER % (RANK / 64) * 128);
        if (LINES == 2) touched[2] = *reinterpret_cast<const uint32_t *>(ql + (tid % PER + PER) * 128);
    };
    Page pages;
    {
        Page p0, p1;
        page_ids(p0);
        page_ids(p1);
        page_ids(pages);
        arrived(p0.id);
        arrived(p1.id);
        arrived(pages.id);
        issue_q(seq, FP8 ? 2 * D::TILE : D::TILE);
        put_offsets(0, p0);
        const float sc0 = sc_next;
        put_offsets(1, p1);
        const float sc1 = sc_next;
        sc_next = sc0;
        if (FP8) put_scales(0);
        sc_next = sc1;
    }
    if (tid == 0) lds_write<int>(D::L_GROW, 0);
    barrier_lds();
    {
        const uint8_t *p0 = src0 + source(0, lt0), *p1 = src1 + source(0, lt1);
#pragma unroll
        for (int c = 0; c < D::CB; ++c) issue(0, c, p0, p1);
        wait_vm<2 * D::CB>();
        barrier_lds();   // the queries are there
        read_q(FP8 ? 2 * D::TILE : D::TILE);
        wait_vm<0>();
        arrived(pages.id);
        arrived(sc_next);
    }

    // ---- lane addresses inside a tile
    uint32_t ka[4], va[4];
    {
        const int t = 32 * th + n, f = dec_swz<FP8>(t);
#pragma unroll
        for (int v = 0; v < 4; ++v)
            ka[v] = (t >> 3) * D::CB * 1024 + (t & 7) * 128 + (((2 * v + hf) ^ f) << 4);
        const int x = lane & 15, cb = (lane >> 4) & 1;
#pragma unroll
        for (int v = 0; v < 4; ++v) {
            if (FP8) {      // va[ct & 3], matrix step s at + 2 s groups of tokens
                const int jr = x >> 1, t8 = 4 * hf + (jr & 3), fv = dec_swz<FP8>(8 * (jr >> 2) + t8);
                va[v] = (jr >> 2) * D::CB * 1024 + t8 * 128 + (((2 * v + cb) ^ fv) << 4) + 8 * (x & 1);
            } else {        // va[2 e + (ct & 1)], e the token group of a step
                const int e = v >> 1, t8 = 4 * hf + (x >> 2), fv = dec_swz<FP8>(8 * e + t8);
                va[v] = e * D::CB * 1024 + t8 * 128 + (((4 * (v & 1) + 2 * cb + ((x & 3) >> 1)) ^ fv) << 4) + 8 * (x & 1);
            }
        }
    }

    const float scale = a.scale * LOG2E;
    const uint32_t top_at = D::L_TOP + 4 * (64 * rg + n), p_at = D::L_P + 4096 * rg + 2048 * th + 16 * lane;
    const int block_j = block_row / a.heads, wave_j = wave_row / a.heads, row_j = row / a.heads;
    int it = 0;
    while (it < total) {
        // ---- a segment: tiles tile .. of one sequence
        const int len = __builtin_amdgcn_readlane(lens, seq - lens_from), n_tiles = dec_tiles(len);
        const int lo = tile, hi = min(n_tiles, lo + total - it);
        const int block_seen = len - a.n_q + 1 + block_j;          // tokens every row here sees,
        const int wave_seen = len - a.n_q + 1 + wave_j;            // every row of the wavefront
        const int seen = row < rows ? len - a.n_q + 1 + row_j : len;
        const bool works = has_rows && len > 0, scores = works && cg < 2;
        f32x16 o[CT];
#pragma unroll
        for (int c = 0; c < CT; ++c)
#pragma unroll
            for (int r = 0; r < 16; ++r) o[c][r] = 0.0f;
        constexpr float LIFT = WEIGHT_LIFT<T>, LAG = LIFT + MAX_LAG;
        float m = NEG, l = 0.0f;   // m: the running maximum less LIFT
        float mv = NEG;   // E4M3: the reference of weights times scales, and of the accumulators

        for (; tile < hi; ++tile, ++it) {
            const int buf = it & 1, t0 = tile * DEC_TILE, tw = t0 + 32 * th;
            const uint32_t base = buf * D::TILE;
            const bool more = it + 1 < total;
            barrier_lds();   // the tile is there, and every wavefront is done with the one before
            const uint8_t *p0 = src0, *p1 = src1;
            if (more) {
                p0 += source(it + 1, lt0);
                p1 += source(it + 1, lt1);
            }
            if (tile + 1 == hi && it + 1 < total) touch_q(seq + 1);
            f32x16 s;
            float sum = 0.0f;
            float sc[16], sv[16];   // E4M3: scales, from the scores on their fractions; score + exponent
            auto weigh = [&] {
                const float ref = m == NEG ? 0.0f : m, refv = mv == NEG ? 0.0f : mv;
                x8<T> p[2];
                sum = 0.0f;
#pragma unroll
                for (int r = 0; r < 16; ++r) {
                    float w = __builtin_amdgcn_exp2f(__builtin_fmaf(s[r], scale, -ref));
                    sum += w;
                    if (FP8) w = sc[r] * __builtin_amdgcn_exp2f(sv[r] - refv);
                    p[r >> 3][r & 7] = (T)w;
                }
                lds_write(p_at, p[0], 0);
                lds_write(p_at, p[1], 1024);
            };
            if (scores) {
#pragma unroll
                for (int r = 0; r < 16; ++r) s[r] = 0.0f;
                // operands four reads ahead of their products (no more: the compiler would hoist reads until it spills),
                // the next tile's loads between them
                u32x4 ahead[2][4];
                uint32_t kb[4];
#pragma unroll
                for (int v = 0; v < 4; ++v) kb[v] = base + ka[v];
                constexpr int READS = D::CB * 4;
#pragma unroll
                for (int i = 0; i < 4; ++i) ahead[0][i] = lds_read<u32x4>(kb[i]);
                if (FP8) {
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const f32x4 v = lds_read<f32x4>(D::L_SCALE + 16 * hf + 4 * (buf * DEC_TILE + 32 * th), 32 * q);
#pragma unroll
                        for (int i = 0; i < 4; ++i) sc[4 * q + i] = v[i];
                    }
                }
#pragma unroll
                for (int c = 0; c < READS; c += 4) {
                    __builtin_amdgcn_sched_barrier(0);
                    if (c + 4 < READS) {
#pragma unroll
                        for (int i = 0; i < 4; ++i) ahead[(c / 4 + 1) & 1][i] = lds_read<u32x4>(kb[i], (c / 4 + 1) * 1024);
                    }
                    if (more) issue(it + 1, c / 4, p0, p1);
                    if (FP8 && c == RANK / 32) {
#pragma unroll
                        for (int r = 0; r < 16; ++r) {
                            s[r] *= sc[r];
                            sc[r] = __builtin_amdgcn_frexp_mantf(sc[r]);
                        }
                    }
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const u32x4 w = ahead[(c / 4) & 1][i];
                        const int k = c + i;
                        if (FP8 && k < RANK / 32) {
                            s = mfma32<T>(widen8<T>(u32x2{w[0], w[1]}), qf[2 * k], s);
                            s = mfma32<T>(widen8<T>(u32x2{w[2], w[3]}), qf[2 * k + 1], s);
                        } else {
                            s = mfma32<T>(__builtin_bit_cast(x8<T>, w), qf[FP8 ? k + RANK / 32 : k], s);
                        }
                    }
                }
                __builtin_amdgcn_sched_barrier(0);
                if (tw + 32 > wave_seen) {
                    int rem = seen - tw - 4 * hf;
                    arrived(rem);   // a branch, not selects that every tile would pay for
#pragma unroll
                    for (int r = 0; r < 16; ++r)
                        if (8 * (r >> 2) + (r & 3) >= rem) {
                            s[r] = NEG;
                            sc[r] = 0.0f;
                        }
                }
                float top = fmaxf(fmaxf(s[0], s[1]), s[2]);
#pragma unroll
                for (int r = 3; r < 15; r += 2) top = fmaxf(fmaxf(top, s[r]), s[r + 1]);
                top = half_max(fmaxf(top, s[15])) * scale;
                lds_write<float>(top_at + 128 * th, top);
                bool grows = top > m + LAG;
                if (FP8) {
                    float topv = NEG;
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const f32x4 e = lds_read<f32x4>(D::L_EXP + 16 * hf + 4 * (buf * DEC_TILE + 32 * th), 32 * q);
#pragma unroll
                        for (int i = 0; i < 4; ++i) sv[4 * q + i] = __builtin_fmaf(s[4 * q + i], scale, e[i]);
                        topv = fmaxf(fmaxf(topv, sv[4 * q]), sv[4 * q + 1]);
                        topv = fmaxf(fmaxf(topv, sv[4 * q + 2]), sv[4 * q + 3]);
                    }
                    topv = half_max(topv);
                    lds_write<float>(top_at + D::TOPS + 128 * th, topv);
                    grows |= topv > mv + LAG;
                }
                if (__ballot(grows) && lane == 0) lds_write<int>(D::L_GROW, it + 1);
            } else if (more) {
#pragma unroll
                for (int c = 0; c < D::CB; ++c) issue(it + 1, c, p0, p1);
            }
            if (scores && tile > lo) weigh();   // a segment's first maximum moves: its weights come below
            // A tile that some rows see only in part, though its tokens exist: values that are not finite would reach
            // rows that do not see them as 0 * NaN; a row that does see them has them in its scores already.
            if (block_seen < len && t0 + DEC_TILE > block_seen) {
                barrier_lds();
                const int from = block_seen > t0 ? block_seen - t0 : 0;
                constexpr int CH = (D::CB - 1) * 8;
                for (int i = tid; i < (DEC_TILE - from) * CH; i += 256) {
                    const int t = from + i / CH, c = i % CH;
                    const uint32_t w = base + ((t >> 3) * D::CB + (c >> 3)) * 1024 + (t & 7) * 128 + ((c & 7) << 4);
                    if (FP8) {
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
            barrier_lds();   // the weights are there
            const int grow = lds_read<int>(D::L_GROW);
            x8<T> p[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) p[k] = lds_read<x8<T>>(p_at - 2048 * th, 1024 * k);
            if (tile == lo || uniform(grow) == it + 1) {
                barrier_lds();   // read by all
                if (works) {
                    const float top = fmaxf(lds_read<float>(top_at), lds_read<float>(top_at, 128));
                    const float to = top > m + LAG ? top - LIFT : m;
                    float f = m == to ? 1.0f : __builtin_amdgcn_exp2f(m - to);
                    l *= f;
                    m = to;
                    if (FP8) {
                        const float topv = fmaxf(lds_read<float>(top_at + D::TOPS), lds_read<float>(top_at + D::TOPS, 128));
                        const float tov = topv > mv + LAG ? rintf(topv) - LIFT : mv;
                        f = mv == tov ? 1.0f : __builtin_amdgcn_exp2f(mv - tov);
                        mv = tov;
                    }
#pragma unroll
                    for (int c = 0; c < CT; ++c)
#pragma unroll
                        for (int r = 0; r < 16; ++r) o[c][r] *= f;
                    if (scores) weigh();
                }
                barrier_lds();
#pragma unroll
                for (int k = 0; k < 4; ++k) p[k] = lds_read<x8<T>>(p_at - 2048 * th, 1024 * k);
            }
            l += sum;
            auto stream = [&](int part) {
                if (part == 0 && FP8) put_scales(it + 1);
                if (part == 1) put_offsets(it + 2, pages);
                if (part == 2) page_ids(pages);
            };
            if (works) {
                u32x4 ahead[2][4];   // a column tile's four matrix steps (E4M3: two words each)
                uint32_t vb[4];      // E4M3, where a wavefront has two column tiles: their low bits differ from c's
                const int col0 = cg * CT;
#pragma unroll
                for (int v = 0; v < 4; ++v)
                    vb[v] = base + (FP8 && CT % 4 ? va[0] ^ (((col0 + v) & 3) << 5) : va[v]) + (FP8 ? col0 >> 2 : col0 >> 1) * 1024;
                auto fetch = [&](int c, int k) {
                    const int imm = 2 * k * D::CB * 1024 + (FP8 ? c >> 2 : c >> 1) * 1024;
                    if (FP8) {
                        const u32x2 w = lds_read_tr8(vb[c & 3], imm);
                        return u32x4{w[0], w[1], 0, 0};
                    }
                    const u32x2 v0 = lds_read_tr16(vb[c & 1], imm), v1 = lds_read_tr16(vb[2 + (c & 1)], imm);
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
                        const x8<T> v = FP8 ? widen8<T>(u32x2{w[0], w[1]}) : __builtin_bit_cast(x8<T>, w);
                        o[c] = mfma32<T>(v, p[k], o[c]);
                    }
                    if (c < 3) stream(c);
                    if (CT == 2 && c == 1) stream(2);
                }
                __builtin_amdgcn_sched_barrier(0);
            } else {
                for (int part = 0; part < 3; ++part) stream(part);
            }
            wait_vm<0>();
            arrived(pages.id);
            arrived(sc_next);
#pragma unroll
            for (int i = 0; i < 3; ++i) arrived(touched[i]);
        }

        // ---- the segment's result: the sums of both halves of the tokens, then out or a partial result
        const uint32_t spent = ((it - 1) & 1) * D::TILE, q_at = FP8 ? 2 * D::TILE : spent;
        barrier_lds();
        if (it < total) issue_q(seq + 1, q_at);
        if (scores) lds_write<float>(top_at + 128 * th, half_sum(l));
        wait_vm<0>();
        barrier_lds();
        l = works ? lds_read<float>(top_at) + lds_read<float>(top_at, 128) : 0.0f;
        if (it < total) {
            read_q(q_at);
            barrier_lds();
        }
        // Results leave divided by the segment's sum; the difference of the references may pass binary32's exponents, half
        // of it does not.
        const float half_off = FP8 && l != 0.0f ? __builtin_amdgcn_exp2f(0.5f * (mv - m)) : 1.0f;
        const float f = l == 0.0f ? 0.0f : half_off / l;
        auto result = [&](int c, int r) { return FP8 ? o[c][r] * f * half_off : o[c][r] * f; };
        if (lo == 0 && hi == n_tiles) {
            // through the buffer of the last tile, 64 columns at a time, so that rows leave in whole lines
            const uint32_t at = spent + wave * 32 * 144;
#pragma unroll
            for (int c = 0; c < CT; c += 2) {
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    x4<T> v;
#pragma unroll
                    for (int k = 0; k < 4; ++k) v[k] = (T)result(c + i / 4, 4 * (i % 4) + k);
                    lds_write(at + n * 144 + 8 * hf, v, 64 * (i / 4) + 16 * (i % 4));
                }
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int r = 8 * i + (lane >> 3);
                    const x8<T> v = lds_read<x8<T>>(at + r * 144 + 16 * (lane & 7));
                    if (wave_row + r < rows)
                        *reinterpret_cast<x8<T> *>(static_cast<T *>(a.out) + ((int64_t)seq * rows + wave_row + r) * RANK +
                                                   (cg * CT + c) * 32 + 8 * (lane & 7)) = v;
                }
            }
            if (a.lse && row < rows && hf == 0 && cg == 0)
                a.lse[(int64_t)seq * rows + row] = l == 0.0f ? NEG : (m + __builtin_amdgcn_logf(l)) * LN2;
        } else if (has_rows) {
            // slot 0: the segment begins inside its sequence, slot 1: with it
            const int64_t slot = ((int64_t)blockIdx.y * groups + g) * 2 + (lo == 0 ? 1 : 0);
            float *dst = a.part + 2 * ((a.batch + 7) & ~7) + slot * D::SLOT;
            float *at = dst + (rg * (RANK / 32) + cg * CT) * 1024 + 4 * lane;
#pragma unroll
            for (int c = 0; c < CT; ++c)
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    f32x4 v;
#pragma unroll
                    for (int i = 0; i < 4; ++i) v[i] = result(c, 4 * q + i);
                    *reinterpret_cast<f32x4 *>(at + (c * 4 + q) * 256) = v;
                }
            if (hf == 0 && cg == 0)
                *reinterpret_cast<float2 *>(dst + D::ROWS * RANK + 2 * (32 * rg + n)) = make_float2(m, l);
        }
        tile = 0;
        ++seq;
        if (seq + 8 >= lens_from + 64 && it < total) load_lens();
    }
    if (bad_page) raise_status(a.status, ST_BADPAGE);
}

// Joins the partial results of a sequence, each divided by its own sum: out =
// sum_g 2^{m_g - M} l_g o_g / sum_g 2^{m_g - M} l_g, over the workgroups in
// order, 32 rows by 8 columns a wavefront.  DEEP: a workgroup's sixteen wavefronts take every sixteenth
// partial each of one such piece, for few sequences in many parts; else they
// take pieces of their own.
constexpr int JOIN_WAVES = 16;   // of a deep one; else four
template <class T, int RANK, int ROWS, bool DEEP>
__global__ __launch_bounds__(DEEP ? 64 * JOIN_WAVES : 256) void k_mla_join(MlaDecodeArgs a, int groups) {
    constexpr int SLOT = ROWS * RANK + 2 * ROWS, EVERY = DEEP ? JOIN_WAVES : 1;
    constexpr float NEG = -__builtin_inff();
    const int b = blockIdx.z, lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int32_t *plan = reinterpret_cast<const int32_t *>(a.part) + 2 * b;
    const int g0 = plan[0], g1 = plan[1];
    if (g0 == g1) return;
    __shared__ f32x4 so[DEEP ? JOIN_WAVES : 1][64];
    __shared__ float sm[DEEP ? JOIN_WAVES : 1][64], sl[DEEP ? JOIN_WAVES : 1][64];
    const int rgs = blockIdx.y, rb = rgs / (ROWS / 32), rg = rgs % (ROWS / 32), n = lane & 31;
    const int cq = DEEP ? blockIdx.x : blockIdx.x * 4 + wave;
    const float *part = a.part + 2 * ((a.batch + 7) & ~7) + (int64_t)rb * groups * 2 * SLOT;
    auto slot = [&](int g) { return part + (int64_t)(2 * g + (g == g0 ? 1 : 0)) * SLOT; };
    auto weight = [](float m, float to) { return m == to ? 1.0f : __builtin_amdgcn_exp2f(m - to); };
    float m = NEG, l = 0.0f;
    f32x4 o = {0.0f, 0.0f, 0.0f, 0.0f};
    constexpr int AHEAD = DEEP ? 8 : 4;   // partials read together
    for (int g = g0 + (DEEP ? wave : 0); g <= g1; g += AHEAD * EVERY) {
        float2 ml[AHEAD];
        f32x4 v[AHEAD];
#pragma unroll
        for (int i = 0; i < AHEAD; ++i) {
            const float *p = slot(min(g + i * EVERY, g1));
            ml[i] = *reinterpret_cast<const float2 *>(p + ROWS * RANK + 2 * (32 * rg + n));
            v[i] = *reinterpret_cast<const f32x4 *>(p + (rg * (RANK / 32) * 4 + cq) * 256 + 4 * lane);
        }
        float to = m;
#pragma unroll
        for (int i = 0; i < AHEAD; ++i) to = fmaxf(to, ml[i].x);
        const float old = weight(m, to);
        l *= old;
#pragma unroll
        for (int k = 0; k < 4; ++k) o[k] *= old;
        m = to;
#pragma unroll
        for (int i = 0; i < AHEAD; ++i)
            if (g + i * EVERY <= g1) {
                const float f = ml[i].y * weight(ml[i].x, m);
                l += f;
#pragma unroll
                for (int k = 0; k < 4; ++k) o[k] = __builtin_fmaf(v[i][k], f, o[k]);
            }
    }
    if (DEEP) {
        so[wave][lane] = o;
        sm[wave][lane] = m;
        sl[wave][lane] = l;
        __syncthreads();
        if (wave) return;
#pragma unroll
        for (int w = 1; w < JOIN_WAVES; ++w) m = fmaxf(m, sm[w][lane]);
        o = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        l = 0.0f;
#pragma unroll
        for (int w = 0; w < JOIN_WAVES; ++w) {
            const float f = weight(sm[w][lane], m);
            const f32x4 v = so[w][lane];
            l = __builtin_fmaf(sl[w][lane], f, l);
#pragma unroll
            for (int i = 0; i < 4; ++i) o[i] = __builtin_fmaf(v[i], f, o[i]);
        }
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

// A join of at most this many groups of 32 rows is a deep one (131071 tokens,
// 64 heads: 44.5 against 92 us for the whole call; 8 x 4096 tokens, 32 heads:
// 25.0 against 26.2; 16 x 2000 tokens, 16 heads: 28.6 against 23.2; the uneven
// batch of 64, 128 heads: 86 against 49).
constexpr int JOIN_DEEP = 8;

// Rows of a workgroup: 32 where they suffice (16 heads, 131071 tokens: 38.4 us
// against 40.6 with 64; 1023 tokens: 13.6 against 14.2), and how many
// workgroups share the batch's tiles: as many as fill the 256 CUs once (a
// workgroup's LDS and registers take one).
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
    if (groups > 1) {
        const int rgs = (rows + 31) / 32, pieces = D::RANK / 8;
        if ((int64_t)a.batch * rgs <= JOIN_DEEP)
            hipLaunchKernelGGL((k_mla_join<typename D::T, D::RANK, D::ROWS, true>), dim3(pieces, rgs, a.batch),
                               dim3(64 * JOIN_WAVES), 0, st, a, groups);
        else
            hipLaunchKernelGGL((k_mla_join<typename D::T, D::RANK, D::ROWS, false>), dim3(pieces / 4, rgs, a.batch),
                               dim3(256), 0, st, a, groups);
    }
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

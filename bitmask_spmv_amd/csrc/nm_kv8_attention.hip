// nm_kv8_attention.hip -- attention over the 8-bit key/value cache, over all keys or over blocks of 64 that each row selects.
//
// For query row i of a sequence (place p = kv_len - rows + i) and head h:
//     s_j = scale * sum_c q_c K_jc,  m = max_j s_j,  l = sum_j exp(s_j - m),
//     o_c = sum_j exp(s_j - m) V_jc / l,  lse = m + log l,
// over the keys j <= p, and j > p - window where there is a window, and j in the row's selected blocks where there are some.
//
// Row tiles.  The query rows of one key/value head (its query heads times the sequence's new tokens; with selected blocks
// times one token) form tiles of 16.  A wave takes one tile and walks blocks of 64 tokens:
//   S^T [64 x 16] = K [64 x D] . Q^T and O^T [D x 16] += V^T [D x 64] . P^T, both on the bf16 matrix instruction.  E4M3
//     numbers times a power of two are bf16 numbers, so keys and values are converted exactly, two an instruction, in the
//     order the page has them: K units are 16 channels of a token, V units 16 tokens of a channel, and S^T leaves a lane the
//     weights of just those tokens.  Nothing passes through LDS.  The scaled matrix instruction would take the bytes as they lie, but
//     it aligns the products of 8 neighbouring channels to 13 bits below the largest, too few for two E4M3 factors; the
//     conversions (128 a block and lane) hide behind the reads.
// Weights are rounded to bf16 for the second product (2^-8 of each at most, either way), as its operands are of one type and a value times the scale
// of its block is a bf16 number, but no fp16 one; scores, maxima, sums and O stay in fp32.  In a row tile the largest weight is 1, in
// prompts it is rounded as the others are, and its rounding is in the divisor too (see the end of `prompt`).  Weights as two bf16 pieces, a matrix
// product more, leave row tiles 0.0017 off 64-bit results, the rounding of these, instead of 0.0018 (root mean square), for 164.2 us instead of
// 163.0 (16 sequences to 64K), 65.5 instead of 64.7 (48 to 8K) and 90 instead of 82 (a chunk of 512 rows that chooses): not taken.
//
// Work split.  As the 4-bit kernels: all (sequence, key/value head, row tile, 64-token block) units of a call laid end to end and
// cut into equal runs, one a wave; pieces of rows cut between waves are joined in LDS, between workgroups by a second kernel, in
// a fixed order.  Selected blocks make the same units, so many to every row.
//
// Bound by reading the cache for single tokens: 16 sequences to 64K, 64 / 8 heads of 128, 987 MB in 163 us (6.1 TB/s; a plain read of 2 GiB
// 7.3), 48 to 8K 64 us; prompts by matrix and vector instructions that overlap in part: 3 of 4K behind 2K, 455 GFLOP in 481-503 us, matrix units
// busy for 42 % of the cycles, vector units for 51 %, both at once for 22 %, neither for 29 %.
#include "nm_kv_attention.h"
#include "nm_kv_rows.h"

namespace nmk {
namespace {

constexpr float kSlack = 8.f;   // prompts: O is rescaled only when a score passes the largest one so far by 2^kSlack
constexpr float kFar = 4096.f;  // reference (log2) up to which a rounded product of it is off by 2^-13 at most
// Context up to which each row tile may be one workgroup's, which needs no second launch (four times that where tiles fill a quarter of
// the machine): 1 x 1024 tokens, 8 heads, 10.1 us whole and 11.2 in runs, 1 x 2048 15.8 and 12.8; 24 x 2048 18.9 and 22.9.
constexpr int kWholeTokens = 1024;
// Row tiles of a call, one to so many waves at most, up to which prompts are walked by row tiles too: 32 / 8 heads behind 4K tokens, 256
// rows 40 us by row tiles and 96 by prompts' tiles, 512 rows 67 and 97, 1024 rows 103 and 100; 2 x 600 rows 67 and 56.
constexpr int kFewTiles = 2;
constexpr int kGroupsPerCu = 2;     // resident workgroups: 8 waves a CU
// Blocks that a wave walks in the time of a second launch: of one row and 8 heads 16 chosen blocks take 10.0 us by a workgroup and 10.6 by
// runs, 32 13.3 and 11.5, 64 20.8 and 13.4.
constexpr int kJoinBlocks = 4;

__device__ __forceinline__ uint32_t fp8_pair(uint32_t w, float s, bool high) {
    union { bf16x2 h; uint32_t u; } c;
    c.h = high ? __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, s, true) : __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, s, false);
    return c.u;
}

union Operand {  // eight bf16 numbers of a lane
    u32x4 u;
    uint32_t w[4];
    bf16x8 h;
};

// Eight E4M3 numbers times s.
__device__ __forceinline__ Operand eight(uint32_t a, uint32_t b, float s) {
    Operand x;
    x.w[0] = fp8_pair(a, s, false);
    x.w[1] = fp8_pair(a, s, true);
    x.w[2] = fp8_pair(b, s, false);
    x.w[3] = fp8_pair(b, s, true);
    return x;
}

// Eight channels of a query with the sign of the scale; zeros for a row that is none.  An infinity becomes NaN: a product with it could
// look like a key that is not seen.
__device__ __forceinline__ Operand read_query(const uint16_t *from, bool real, const Kv8Attention &a) {
    const uint32_t flip = a.minus ? 0x80008000u : 0u;
    Operand x;
    x.u = real ? *reinterpret_cast<const u32x4 *>(from) : (u32x4){0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t none = ((x.w[i] & 0x7F807F80u) + 0x00800080u) & 0x80008000u;  // exponents of all ones
        x.w[i] = a.zero ? (none >> 15) * 0x7FC0u : (x.w[i] ^ flip) | none >> 9;
    }
    return x;
}

// Where the blocks of one head lie: lane i holds the address and the scales of a block and its number, so that a walk reads the page table
// once for kAhead blocks.  Without a valid page, and without a place in [from, upto], those that some row sees, the address is that of
// page 0, so that loads need no branch, the scales are 1 (what was never written may be scales that are no numbers, and values of 0 times
// one are none either), and the block's bit in `valid` is clear.
struct Blocks {
    static constexpr int kAhead = 60;  // of 64: a walk looks up to three blocks ahead
    uint32_t lo, hi, scales;
    int block;
    uint64_t valid;
    __device__ void load(const Kv8Batch &b, const int32_t *row, int head, int mine, int from, int upto) {
        block = mine;
        const int per = b.f.blocks(), col = block >= 0 ? block / per : 0;
        int page = block >= 0 && col < b.cols ? row[col] : -1;
        const bool ok = page >= 0 && page < b.num_pages && block >= from >> 6 && block <= upto >> 6;
        if (!ok) page = 0;
        valid = __ballot(ok);
        const uint32_t at = (uint32_t)(head * per + (ok ? block & (per - 1) : 0));
        const uint8_t *p = b.cache + (uint64_t)page * (uint64_t)b.f.page_bytes();
        scales = ok ? *reinterpret_cast<const uint32_t *>(p + b.f.scales_at() + at * 4) : 0x7F7Fu;
        const uint64_t k = (uint64_t)(uintptr_t)p + (uint64_t)at * (uint32_t)b.f.block_bytes();
        lo = (uint32_t)k;
        hi = (uint32_t)(k >> 32);
    }
    __device__ const uint8_t *at(int i) const {
        const uint32_t l = __builtin_amdgcn_readlane((int)lo, i), h = __builtin_amdgcn_readlane((int)hi, i);
        return (const uint8_t *)(uintptr_t)((uint64_t)h << 32 | l);
    }
    __device__ float k_scale(int i) const { return __uint_as_float((__builtin_amdgcn_readlane((int)scales, i) & 255u) << 23); }
    __device__ float v_scale(int i) const { return __uint_as_float((__builtin_amdgcn_readlane((int)scales, i) & 0xFF00u) << 15); }
    __device__ int number(int i) const { return __builtin_amdgcn_readlane(block, i); }
    __device__ bool ok(int i) const { return (valid >> i) & 1; }
};

// The cache bytes of 64 tokens of one head that a lane multiplies.
template <int D>
struct Bytes {
    u32x4 k[D / 16], v[D / 16];
};

// Lane (col, g): K units g + 4 u of tokens 16 j + col, V units g of channels 16 c + col.
template <int D>
struct Lane {
    int col, g;
    uint32_t k_off, v_off;
    __device__ Lane(int lane) {
        col = lane & 15;
        g = lane >> 4;
        k_off = (g * 64 + col) * 16;
        v_off = 64 * D + (g * D + col) * 16;
    }
};

template <int D, bool NT>
__device__ __forceinline__ void load_block(Bytes<D> &x, const uint8_t *k, const Lane<D> &ln) {
#pragma unroll
    for (int i = 0; i < D / 16; ++i) x.k[i] = load_cache<NT, u32x4>(k + ln.k_off + (i >> 2) * 4096 + (i & 3) * 256);
#pragma unroll
    for (int i = 0; i < D / 16; ++i) x.v[i] = load_cache<NT, u32x4>(k + ln.v_off + i * 256);
}

// Scores of 64 tokens: s[j][i] is token 16 j + 4 g + i of the column's row.
template <int D>
__device__ __forceinline__ void scores(const Bytes<D> &x, const Operand (&q)[D / 32], float scale, f32x4 (&s)[4]) {
#pragma unroll
    for (int u = 0; u < D / 64; ++u)
#pragma unroll
        for (int e = 0; e < 2; ++e)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const u32x4 &w = x.k[u * 4 + j];
                const f32x4 zero = {0.f, 0.f, 0.f, 0.f};
                s[j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(eight(w[2 * e], w[2 * e + 1], scale).h, q[2 * u + e].h,
                                                               u + e ? s[j] : zero, 0, 0, 0);
            }
}

// O += V^T P for 64 tokens: lane's row i of tile c is channel 16 c + 4 g + i.
template <int D>
__device__ __forceinline__ void add_values(Tile<D> &t, const Bytes<D> &x, const f32x4 (&p)[4], float scale) {
#pragma unroll
    for (int s = 0; s < 2; ++s) {
        Operand b;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            b.w[2 * j] = pack_bf16(p[2 * s + j][0], p[2 * s + j][1]);
            b.w[2 * j + 1] = pack_bf16(p[2 * s + j][2], p[2 * s + j][3]);
        }
#pragma unroll
        for (int c = 0; c < D / 16; ++c)
            t.o[c] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(eight(x.v[c][2 * s], x.v[c][2 * s + 1], scale).h, b.h, t.o[c], 0, 0, 0);
    }
}

// Of four tokens from `tok` on, a byte each, those in [from, upto].
__device__ __forceinline__ uint32_t seen_bytes(int tok, int from, int upto) {
    const int lo = min(max(from - tok, 0), 4), hi = min(max(upto + 1 - tok, 0), 4);
    const uint32_t below_hi = hi == 4 ? ~0u : (1u << (8 * hi)) - 1, below_lo = lo == 4 ? ~0u : (1u << (8 * lo)) - 1;
    return below_hi & ~below_lo;
}

template <int D>
__device__ __forceinline__ void store_row(const Kv8Attention &a, int t, int h, int g, const Tile<D> &tl, float m, float l) {
    const float inv = l != 0.f ? 1.f / l : 0.f;
    uint16_t *p = a.out.p + t * a.out.ld + h * a.out.hd + 4 * g;
#pragma unroll
    for (int c = 0; c < D / 16; ++c) {
        uint2 w;
        w.x = pack_bf16(tl.o[c][0] * inv, tl.o[c][1] * inv);
        w.y = pack_bf16(tl.o[c][2] * inv, tl.o[c][3] * inv);
        *reinterpret_cast<uint2 *>(p + 16 * c) = w;
    }
    if (g == 0 && a.lse) a.lse[t * a.ld_lse + h] = l != 0.f ? (m + __builtin_amdgcn_logf(l)) * kLn2 : -INFINITY;
}

template <int D>
__device__ __forceinline__ void keep_part(Part<D> &p, const Tile<D> &t, float c, const Lane<D> &ln) {
#pragma unroll
    for (int i = 0; i < D / 16; ++i) *reinterpret_cast<f32x4 *>(&p.o[ln.col][16 * i + 4 * ln.g]) = t.o[i];
    const float l = cross_rows_sum(t.l);
    if (ln.g == 0) {
        p.m[ln.col] = t.m == -INFINITY ? -INFINITY : reference(t.m, c);
        p.l[ln.col] = l;
    }
}

// A row tile: rows r0 .. of the n * group of a sequence's (or of one token's) rows, and the keys they look at.
struct Rows {
    int s, q0, head, tile, rows;  // sequence, token row of row 0, key/value head, tile of 16 and its rows
    int place;                    // of row 0's token
    int see_end;                  // places below it hold keys
    int last;                     // place of the last token among the rows that masks are asked for
};

// Blocks b0 .. b1 of the tile's list: all from block `first` on, or a row's selected ones.
template <int D, bool NT, bool SEL, class L>
__device__ __forceinline__ void walk(const Kv8Attention &a, const Rows &r, int first, int b0, int b1, bool begins, bool ends, const Lane<D> &ln,
                                     int lane, int wave, Shared<D> *sh, L &&listed) {
    const int group = a.heads / a.b.f.n_kv;
    const int32_t *row = a.b.table + (int64_t)r.s * a.b.ld_table;
    // keys that any of the rows sees
    auto first_of = [&](int p) { return a.window > 0 && p >= a.window ? (int)(p - a.window + 1) : 0; };
    const int any_first = first_of(r.place), any_last = min(r.last, r.see_end - 1);
    Blocks lies;
    int held = b0;
    auto look = [&] {
        if constexpr (SEL) {
            const int b = listed(held + lane);
            lies.load(a.b, row, r.head, held + lane < b1 ? b : -1, any_first, any_last);
        } else {
            lies.load(a.b, row, r.head, first + held + lane, any_first, any_last);
        }
    };
    look();
    Bytes<D> x0, x1;
    load_block<D, NT>(x0, lies.at(0), ln);

    // queries of my column
    const int in = r.tile * kRows + ln.col;
    const int qi = SEL ? 0 : in / group, t = r.q0 + qi, h = r.head * group + (in - qi * group);
    const bool real = ln.col < r.rows && (uint32_t)t < (uint32_t)a.b.T;
    Operand q[D / 32];
    const uint16_t *from = a.q.p + t * a.q.ld + h * a.q.hd;
#pragma unroll
    for (int i = 0; i < D / 32; ++i) q[i] = read_query(from + 64 * (i >> 1) + 16 * ln.g + 8 * (i & 1), real, a);
    // keys that my row sees: [see_first, see_last]; that every row sees
    const int place = r.place + qi;
    const int see_last = real ? min(place, r.see_end - 1) : -1, see_first = first_of(place);
    const int all_first = first_of(r.last), all_last = min(r.place, r.see_end - 1);

    Tile<D> tl;
    clear(tl);
    auto add = [&](Bytes<D> &x, int i, int b) {
        const int j0 = (SEL ? lies.number(i) : first + b) * kBlock;
        f32x4 sc[4];
        scores<D>(x, q, lies.k_scale(i), sc);
        if (j0 < all_first || j0 + (kBlock - 1) > all_last) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int tok = j0 + 16 * j + 4 * ln.g + e;
                    if (tok > see_last || tok < see_first) sc[j][e] = -INFINITY;
                }
                // a weight of 0 times what an unseen place holds must be 0
                const uint32_t keep = seen_bytes(j0 + 16 * j + 4 * ln.g, any_first, any_last);
#pragma unroll
                for (int c = 0; c < D / 16; ++c) x.v[c][j] &= keep;
            }
        }
        weights(tl, sc, a.c);
        add_values<D>(tl, x, sc, lies.v_scale(i));
    };
    // Behind the last block the loads, which are not branched around, go to the cache's first bytes for all waves.
    for (int b = b0; b < b1; b += 2) {
        if (b - held == Blocks::kAhead) {
            held = b;
            look();
        }
        const int i = b - held;
        load_block<D, NT>(x1, b + 1 < b1 ? lies.at(i + 1) : a.b.cache, ln);
        if (lies.ok(i)) add(x0, i, b);
        if (b + 1 >= b1) break;
        load_block<D, NT>(x0, b + 2 < b1 ? lies.at(i + 2) : a.b.cache, ln);
        if (lies.ok(i + 1)) add(x1, i + 1, b + 1);
    }

    if (begins && ends) {
        const float l = cross_rows_sum(tl.l);
        if (real) store_row<D>(a, t, h, ln.g, tl, reference(tl.m, a.c), l);
    } else {
        const int slot = begins ? 1 : 0;
        keep_part(sh->part[wave][slot], tl, a.c, ln);
        if (lane == 0) sh->tag[wave][slot] = {ends ? kEnds : kThrough, r.q0, r.head, r.tile, r.rows, 0};
    }
}

// Workgroup `block` of `blocks`: its waves' runs of the units of all sequences.
template <int D, bool NT>
__device__ __forceinline__ void decode(Kv8Attention &a, Part<D> *parts, PartTag *tags, Shared<D> &sh, int block, int blocks) {
    a.b.f.dim = D;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int group = a.heads / a.b.f.n_kv, n_kv = a.b.f.n_kv;
    const Lane<D> ln(lane);
    const int64_t cap = (int64_t)a.b.cols * a.b.f.page;

    // my run of units
    SeqLane sl, behind;
    sl.load(a.b, lane);
    int64_t w = seq_from(a, group, sl.q0, sl.q1, sl.len).units(n_kv, a.whole);
    int64_t upto = units_scan(w, lane);
    int64_t total = lane64(upto, 63);
    for (int s0 = 64; s0 < a.b.S; s0 += 64) {
        if (s0 == 64) behind.load(a.b, s0 + lane);
        const SeqLane x = behind;
        behind.load(a.b, s0 + 64 + lane);
        total += lane64(units_scan(seq_from(a, group, x.q0, x.q1, x.len).units(n_kv, a.whole), lane), 63);
    }
    const int64_t waves = (int64_t)blocks * kWaves;
    const int64_t run = total < ((int64_t)1 << 31) ? (int64_t)(((uint32_t)total + (uint32_t)waves - 1) / (uint32_t)waves)
                                                   : (total + waves - 1) / waves;
    int64_t u = a.whole ? block : ((int64_t)block * kWaves + wave) * run;
    const int64_t stop = a.whole ? u + 1 : u + run;
    const int64_t end = stop < total ? stop : total;
    if (lane < 2) sh.tag[wave][lane].state = kNone;

    int s0 = 0;        // the 64 sequences that the lanes hold
    int64_t base = 0;  // units before them
    while (u < end) {
        // the sequence that unit u is in
        const uint64_t past = __ballot(base + upto > u);
        if (!past) {
            base += lane64(upto, 63);
            s0 += 64;
            sl.load(a.b, s0 + lane);
            w = seq_from(a, group, sl.q0, sl.q1, sl.len).units(n_kv, a.whole);
            upto = units_scan(w, lane);
            continue;
        }
        const int at = __builtin_ctzll(past);
        const Seq sq = seq_from(a, group, __builtin_amdgcn_readlane(sl.q0, at), __builtin_amdgcn_readlane(sl.q1, at),
                                __builtin_amdgcn_readlane(sl.len, at));
        const int64_t in = u - base - lane64(upto - w, at);
        int item, b0, b1;
        if (a.whole) {  // a unit is a row tile, a quarter of its blocks is mine (the last waves may have none)
            const int mine = (sq.blocks + kWaves - 1) / kWaves;
            item = (int)in;
            b0 = wave * mine;
            b1 = b0 + mine < sq.blocks ? b0 + mine : sq.blocks;
            u = end;
            if (b0 >= b1) break;
        } else {
            item = in < ((int64_t)1 << 31) ? (int)((uint32_t)in / (uint32_t)sq.blocks) : (int)(in / sq.blocks);
            b0 = (int)(in - (int64_t)item * sq.blocks);
            const int64_t room = end - u;
            b1 = (int)(room < sq.blocks - b0 ? b0 + room : sq.blocks);
            u += b1 - b0;
        }
        const int head = item / sq.tiles, tile = item - head * sq.tiles;
        const int64_t left = (int64_t)sq.n * group - (int64_t)tile * kRows;
        const Rows r = {s0 + at, sq.q0, head, tile, (int)(left < kRows ? left : kRows), sq.len - sq.n,
                        (int)(sq.len < cap ? sq.len : cap), sq.len - 1};
        walk<D, NT, false>(a, r, sq.first, b0, b1, b0 == 0, b1 == sq.blocks, ln, lane, wave, &sh, [](int) { return 0; });
    }
    __syncthreads();
    join_pieces<D>(a, parts, tags, sh, block);
}

template <int D, bool NT>
__global__ __launch_bounds__(kWaves *kWave, 2) void kv8_decode_kernel(Kv8Attention a, Part<D> *parts, PartTag *tags) {
    __shared__ Shared<D> sh;
    decode<D, NT>(a, parts, tags, sh, blockIdx.x, gridDim.x);
}

// Selected blocks: items are (key/value head, token, tile of 16 of its rows), units the `top` blocks of each.  kItem: an item is a
// workgroup's, each wave takes a quarter of the blocks that the row has.  kWave1: a wave's.  kRuns: units are cut into runs.
// With kWave1 workgroups that go to one XCD take neighbouring items, tokens of few heads, whose blocks its L2 holds.
enum : int { kItem = 0, kWave1 = 1, kRuns = 2 };

template <int D, int MODE>
__global__ __launch_bounds__(kWaves *kWave, 2) void kv8_selected_kernel(Kv8Attention a, Part<D> *parts, PartTag *tags) {
    __shared__ Shared<D> shared;
    Shared<D> *sh = MODE == kWave1 ? nullptr : &shared;
    a.b.f.dim = D;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int n_kv = a.b.f.n_kv, group = a.heads / n_kv, subs = (group + kRows - 1) / kRows;
    const Lane<D> ln(lane);
    const int64_t cap = (int64_t)a.b.cols * a.b.f.page;
    const int64_t items = (int64_t)a.b.T * n_kv * subs;
    const int me = MODE == kWave1 ? by_xcd(blockIdx.x, gridDim.x) : (int)blockIdx.x;
    int64_t u, end;
    if (MODE == kRuns) {
        const int64_t total = items * a.top, waves = (int64_t)gridDim.x * kWaves, run = (total + waves - 1) / waves;
        u = ((int64_t)me * kWaves + wave) * run;
        end = u + run < total ? u + run : total;
    } else {
        u = MODE == kItem ? me : (int64_t)me * kWaves + wave;
        end = u < items ? u + 1 : u;
    }
    if (MODE != kWave1 && lane < 2) sh->tag[wave][lane].state = kNone;
    while (u < end) {
        const int64_t item = MODE == kRuns ? u / a.top : u;
        const int ht = (int)(item / subs), tile = (int)(item - (int64_t)ht * subs);
        const int head = ht / a.b.T, t = ht - head * a.b.T;
        const int32_t *list = a.selected + (int64_t)t * a.ld_selected + (int64_t)head * a.top;
        int b0 = 0, b1, blocks = a.top;
        if (MODE == kRuns) {
            b0 = (int)(u - item * a.top);
            b1 = (int)(end - u < a.top - b0 ? b0 + (end - u) : a.top);
            u += b1 - b0;
        } else {
            u = end;
        }
        const int entry = list[min(b0 + lane, a.top - 1)];
        const RowSeq seq(a.b, t, lane);
        if (t < seq.q0 || t >= seq.q1) continue;
        if (MODE != kRuns) {
            blocks = 1;  // up to the last one that is named
            for (int i = 0; i < a.top; i += 64) {
                const int e = i ? list[min(i + lane, a.top - 1)] : entry;
                const uint64_t some = __ballot(i + lane < a.top && e >= 0);
                if (some) blocks = i + 64 - __clzll((long long)some);
            }
            const int mine = MODE == kItem ? (blocks + kWaves - 1) / kWaves : blocks;
            b0 = MODE == kItem ? wave * mine : 0;
            b1 = min(b0 + mine, blocks);
            if (b0 >= b1) continue;
        }
        const int place = seq.len - seq.q1 + t;
        const Rows r = {seq.s, t, head, tile, min(kRows, group - tile * kRows), place, (int)(seq.len < cap ? seq.len : cap), place};
        const int from = MODE == kRuns ? b0 : 0;  // entry is list[from + lane]
        walk<D, MODE != kWave1, true>(a, r, 0, b0, b1, b0 == 0, b1 == blocks, ln, lane, wave, sh, [&](int i) {
            if (b1 - from <= 64) return __shfl(entry, i - from);
            return (int)list[min(i, a.top - 1)];
        });
    }
    if (MODE == kWave1) return;
    __syncthreads();
    join_pieces<D>(a, parts, tags, *sh, me);
}

template <int D>
__global__ __launch_bounds__(256) void kv8_join_kernel(Kv8Attention a, const Part<D> *parts, const PartTag *tags) {
    join_groups<D>(a, parts, tags);
}

// ---- prompts ----
//
// Many rows of a sequence: a workgroup takes kPromptRows rows of one key/value head, 32 a wave, and walks the blocks of 64 tokens that
// the last of them sees, in 32 x 32 tiles.  Values are converted once for the 128 rows: a thread has the 16 + 16 tokens of one
// channel that one lane half of a score tile has, and leaves them in LDS in the operand order of the product (two buffers, one
// barrier a block).  Keys go the same way, a block further ahead.  The walk is a pipeline over tiles of 32 tokens, one step of which has the products of three of them, so that
// matrix and vector instructions alternate within a wave: see `step`.
constexpr int kPromptTile = 32;                       // rows of a wave
constexpr int kPromptRows = kWaves * kPromptTile;     // rows of a workgroup

// Lane (col, hh) = (lane % 32, lane / 32): column col is a query row, token rows of the scores are
// 8 (i / 4) + 4 hh + i % 4 of a tile of 32, channel rows of O 32 mt + 8 (i / 4) + 4 hh + i % 4.
template <int D>
struct Staged {  // two blocks' bf16 operands
    u32x4 k[2][2][D / 16][kWave];  // of a tile of 32 tokens: channels 32 (i / 2) + 16 hh + 8 (i % 2) ..
    u32x4 v[2][4][D / 32][kWave];
};

// Workgroup `block` of tiles * n_kv.
template <int D>
__device__ __forceinline__ void prompt(Kv8Attention &a, int tiles, Staged<D> &staged, int block) {
    constexpr int MT = D / 32, KU = D / 32;  // channel tiles of the values, K units of a lane
    a.b.f.dim = D;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int col = lane & 31, hh = lane >> 5;
    const int group = a.heads / a.b.f.n_kv;

    // Row tile: sequence s owns the tiles from q_start[s] * group / rows + s on, which are
    // enough for it.  Later rows, which see more, go first; the heads of a tile go to
    // neighbouring workgroups, that is to different XCDs, so an XCD reads few heads.
    const int head = block % a.b.f.n_kv;
    const int vt = tiles - 1 - block / a.b.f.n_kv;
    int s = 0;
    for (int n = a.b.S; n > 1;) {  // the last s whose first tile is at or before vt, 64 looks at a time
        const int step = (n + 63) >> 6, at = s + lane * step;
        const bool yes = lane * step < n && (uint32_t)(a.b.q_start[at] * group) / kPromptRows + at <= (uint32_t)vt;
        const uint64_t m = __ballot(yes);
        s += (m ? 63 - __clzll((long long)m) : 0) * step;
        n = min(step, a.b.S - s);
    }
    const int q0 = uniform_load(a.b.q_start + s), n = uniform_load(a.b.q_start + s + 1) - q0;
    const int len = uniform_load(a.b.kv_len + s);
    const int rows = n * group;  // at most 2^30, as all rows of a call together
    if (rows <= (a.b.S > 1 ? kDecodeRows : 0)) return;  // a lone sequence is all that there is
    const int r0 = (vt - (int)((uint32_t)(q0 * group) / kPromptRows) - s) * kPromptRows;
    if (r0 < 0 || r0 >= rows) return;

    const float c = a.c;
    const int64_t room = (int64_t)a.b.cols * a.b.f.page;
    const int cap = len < room ? len : (int)room;  // tokens that have a place
    const int place0 = len - n;                    // of the sequence's first row
    // The first and the last key that a row at some place sees; the same for places at the end of the keys.
    const int window = a.window > 0 && a.window < len ? (int)a.window : 0;
    auto first_of = [&](int place) { return window && place >= window ? place - window + 1 : 0; };
    auto last_of = [&](int place) { return place < cap ? place : cap - 1; };
    const int any_from = first_of(place0), any_upto = cap - 1;

    const int w0 = r0 + wave * kPromptTile;  // the wave's first row
    const int r = w0 + col;
    const int qi = (int)((uint32_t)r / (uint32_t)group), t = q0 + qi, h = head * group + (r - qi * group);
    const bool real = r < rows && (uint32_t)t < (uint32_t)a.b.T;
    Operand q[2 * KU];  // product 2 i + e: channels 32 i + 16 hh + 8 e ..
#pragma unroll
    for (int i = 0; i < 2 * KU; ++i) q[i] = read_query(a.q.p + t * a.q.ld + h * a.q.hd + 32 * (i >> 1) + 16 * hh + 8 * (i & 1), real, a);
    const int upto = real ? last_of(place0 + qi) : -1, from = first_of(place0 + qi);
    f32x16 o[MT];
#pragma unroll
    for (int i = 0; i < MT; ++i) o[i] = f32x16{};
    float top = -INFINITY, off = 0.f, l = 0.f;  // weights are 2^((score - top) c - off); their sum
    float most = -INFINITY;                     // the largest score so far
    // what follows from top and off: the score that asks for new ones, what is taken from scores times c, and
    // whether that is far from 0 for a row of the wave
    float limit = -INFINITY, less = 0.f;
    bool far = false;

    // blocks that the workgroup walks, and those that need no mask for the wave
    auto place_of = [&](int r) { return place0 + (int)((uint32_t)min(r, rows - 1) / (uint32_t)group); };
    const int b_first = first_of(place_of(r0)) / kBlock;
    const int see_last = last_of(place_of(r0 + kPromptRows - 1));
    const int b_end = see_last >= 0 ? see_last / kBlock + 1 : 0;
    const int w_all = last_of(place_of(w0)), w_all_from = first_of(place_of(w0 + kPromptTile - 1));

    const int32_t *row = a.b.table + (int64_t)s * a.b.ld_table;
    Blocks lies;
    int held = b_first;  // first of the blocks whose places are held
    lies.load(a.b, row, head, held + lane, any_from, any_upto);

    // this thread's share of a block's keys: token `lane`, units kUnits wave ..
    constexpr int kUnits = D / 64;
    const uint32_t k_off = (wave * kUnits * 64 + lane) * 16;
    u32x4 kx[kUnits];
    float kscale = 1.f;
    auto load_keys = [&](int b) {
        const uint8_t *kp = lies.at(b - held) + k_off;
        kscale = lies.k_scale(b - held);
#pragma unroll
        for (int i = 0; i < kUnits; ++i) kx[i] = load_cache<false, u32x4>(kp + i * 1024);
    };
    auto put_keys = [&](int i, const Operand (&x)[2], int b) {  // unit 2 ku + half of the block
        const int u = wave * kUnits + i;
#pragma unroll
        for (int e = 0; e < 2; ++e) staged.k[b & 1][lane >> 5][(u >> 1) * 2 + e][(u & 1) * 32 + col] = x[e].u;
    };

    // this thread's share of a block's values: channel vc of the lane half vh, tokens 16 j + 4 vh + {0..3, 8..11} for kShare of
    // the four j, from vj on
    constexpr int kShare = D / 32;
    const int vc = (D == 128 ? wave * 32 : (wave & 1) * 32) + col, vh = hh, vj = D == 128 ? 0 : (wave >> 1) * 2;
    const uint32_t v_off = 64 * D + (vh * D + vc) * 16 + vj * 4;
    uint32_t vx[2][kShare];  // units vh and vh + 2
    float vscale = 1.f;
    auto load_values = [&](int b) {
        const uint8_t *vp = lies.at(b - held) + v_off;
        vscale = lies.v_scale(b - held);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            if constexpr (D == 128) {
                const u32x4 w = load_cache<false, u32x4>(vp + i * 32 * D);
#pragma unroll
                for (int j = 0; j < 4; ++j) vx[i][j] = w[j];
            } else {
                typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
                const u32x2 w = load_cache<false, u32x2>(vp + i * 32 * D);
                vx[i][0] = w[0];
                vx[i][1] = w[1];
            }
        }
    };
    load_keys(b_first);
    load_values(b_first);
    // a weight of 0 times what an unseen place holds must be 0
    auto hide_values = [&](int b) {
        const int j0 = b * kBlock;
        const bool page = lies.ok(b - held);
        if (j0 < any_from || j0 + kBlock - 1 > any_upto || !page) {
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int j = 0; j < kShare; ++j)
                    vx[i][j] &= page ? seen_bytes(j0 + 16 * (vj + j) + 8 * i + 4 * vh, any_from, any_upto) : 0u;
        }
    };
    auto operand = [&](int j) {
        Operand x;
#pragma unroll
        for (int k = 0; k < 4; ++k) x.w[k] = fp8_pair(vx[k >> 1][j], vscale, k & 1);
        return x;
    };
    auto put_values = [&](int j, const Operand &x, int b) { staged.v[b & 1][vj + j][vc >> 5][vh * 32 + (vc & 31)] = x.u; };

    // Products of the scores: number i of a 32-token tile's 2 KU.
    auto dot = [&](int i, const u32x4 &w, f32x16 &acc) {
        const f32x16 zero = {};
        Operand x;
        x.u = w;
        acc = __builtin_amdgcn_mfma_f32_32x32x16_bf16(x.h, q[i].h, i ? acc : zero, 0, 0, 0);
    };
    constexpr int kDots = 2 * KU, kSums = 2 * MT;  // matrix products of a 32-token tile: scores, values
    auto sum = [&](int i, const u32x4 &v, const uint32_t (&w)[8]) {
        Operand x, y;
        x.u = v;
#pragma unroll
        for (int e = 0; e < 4; ++e) y.w[e] = w[4 * (i / MT) + e];
        o[i % MT] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(x.h, y.h, o[i % MT], 0, 0, 0);
    };
    // Scores of tile tt of block b: unseen ones to -infinity.
    auto hide = [&](int b, int tt, f32x16 &sc) {
        const int j0 = b * kBlock + 32 * tt;
        const bool page = lies.ok(b - held);
        if (j0 < w_all_from || j0 + 31 > w_all || !page) {
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const int tok = j0 + 8 * (i >> 2) + 4 * hh + (i & 3);
                if (tok > upto || tok < from || !page) sc[i] = -INFINITY;
            }
        }
    };
    auto largest = [&](const f32x16 &sc) {
        float x = __builtin_amdgcn_fmed3f(sc[0], sc[1], INFINITY), y = __builtin_amdgcn_fmed3f(sc[2], sc[3], INFINITY);
#pragma unroll
        for (int i = 4; i < 16; i += 4) {
            x = __builtin_amdgcn_fmed3f(__builtin_amdgcn_fmed3f(x, sc[i], INFINITY), sc[i + 1], INFINITY);
            y = __builtin_amdgcn_fmed3f(__builtin_amdgcn_fmed3f(y, sc[i + 2], INFINITY), sc[i + 3], INFINITY);
        }
        return halves_max(fmaxf(x, y));
    };
    // A new reference where a score has passed the old one.  The first is the largest score itself and kSlack,
    // so that a lone key's weight is a power of two; the next ones lie whole powers of two from it, so that
    // the weights w, which are rounded already and not yet multiplied, follow exactly; of one so far behind
    // that nothing remains, the largest score begins anew.
    auto raise = [&](float x, uint32_t (&w)[8]) {
        if (__any(x > limit)) {
            const float past = __builtin_fmaf(x - top, c, -off);  // NaN: neither has a key
            const float by = floorf(past) + kSlack;
            const bool anew = by > 150.f, mine = past > 0.f;
            const float keep = mine ? __builtin_ldexpf(1.f, (int)fmaxf(-by, -1000.f)) : 1.f;
#pragma unroll
            for (int i = 0; i < MT; ++i) o[i] *= keep;
#pragma unroll
            for (int i = 0; i < 8; ++i) w[i] = pack_bf16(bf16_lo(w[i]) * keep, bf16_hi(w[i]) * keep);
            l *= keep;
            if (mine) off = anew ? kSlack : off + by;
            if (mine && anew) top = x;
            less = __builtin_fmaf(top == -INFINITY ? 0.f : top, c, off);
            far = __any(fabsf(less) > kFar);
            if (far) less = off;
            limit = __builtin_fmaf(off, __builtin_amdgcn_rcpf(c), top);  // not above its exact value:
            if (top != -INFINITY) limit = __builtin_fmaf(fabsf(limit), -0x1p-21f, limit);
        }
    };
    // Where a reference is far from 0 the product of a score, rounded to be subtracted, would be off by more than the
    // weights' own rounding: there scores become differences first.
    auto relative = [&](f32x16 &sc) {
        if (__builtin_expect(far, 0)) {
            const float base = top == -INFINITY ? 0.f : top;
#pragma unroll
            for (int i = 0; i < 16; ++i) sc[i] -= base;
        }
    };

    // Tile t = 2 b + tt: between them, product by product, the values of tile t (weights w are ready), the scores
    // of tile t + 2 (into n), the softmax of tile t + 1 (scores sc to weights wn) and half of the conversions: of
    // block b + 1's values and block b + 2's keys.
    auto step = [&](int b, int tt, uint32_t (&w)[8], uint32_t (&wn)[8], f32x16 &sc, f32x16 &n) {
        const u32x4 *values = &staged.v[b & 1][2 * tt][0][lane], *keys = &staged.k[(b + 1) & 1][tt][0][lane];
        hide(tt ? b + 1 : b, tt ^ 1, sc);
        const float x = largest(sc);
        most = fmaxf(most, x);
        raise(x, w);
        relative(sc);
        const float mc = less;
        if (tt == 0) hide_values(b + 1);

        constexpr int kRead = 3;  // operands read ahead
        u32x4 v[kRead], kk[kRead];
#pragma unroll
        for (int i = 0; i < kRead - 1; ++i) {
            v[i] = values[i * kWave];
            kk[i] = keys[i * kWave];
        }
        constexpr int kMine = kShare / 2;  // operands of values converted in a step
        Operand cv[kMine], ck[2];
        float part = 0.f;
        __builtin_amdgcn_s_setprio(1);  // ahead of the wave that loads or rescales (499 -> 495 us)
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            if (k + kRead - 1 < kSums) v[(k + kRead - 1) % kRead] = values[(k + kRead - 1) * kWave];
            if (k + kRead - 1 < kDots) kk[(k + kRead - 1) % kRead] = keys[(k + kRead - 1) * kWave];
            if (k < kSums) sum(k, v[k % kRead], w);
            if (k < kDots) dot(k, kk[k % kRead], n);
            const float e0 = __builtin_amdgcn_exp2f(__builtin_fmaf(sc[2 * k], c, -mc));
            const float e1 = __builtin_amdgcn_exp2f(__builtin_fmaf(sc[2 * k + 1], c, -mc));
            wn[k] = pack_bf16(e0, e1);
            part += e0 + e1;
            if (k < 4 * kMine) cv[k / 4].w[k % 4] = fp8_pair(vx[k % 4 / 2][kMine * tt + k / 4], vscale, k & 1);
            if (tt < kUnits) ck[k / 4].w[k % 4] = fp8_pair(kx[tt < kUnits ? tt : 0][k / 2], kscale, k & 1);
            __builtin_amdgcn_sched_group_barrier(0x100, 2, 0);
            __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
            __builtin_amdgcn_sched_group_barrier(0x002, 5, 0);
            __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
            __builtin_amdgcn_sched_group_barrier(0x002, 9, 0);
            __builtin_amdgcn_sched_barrier(0);
        }
        __builtin_amdgcn_s_setprio(0);
        // this step's work: not to be put off to where it is used
        asm volatile("" : "+v"(n));
#pragma unroll
        for (int k = 0; k < 8; ++k) asm volatile("" : "+v"(wn[k]));
        l += part;
#pragma unroll
        for (int j = 0; j < kMine; ++j) put_values(kMine * tt + j, cv[j], b + 1);
        if (tt < kUnits) put_keys(tt, ck, b + 2);
        if (tt == 1) load_values(b + 2);
        if (tt == 1) load_keys(b + 3);
    };

    if (b_first < b_end) {
        // fill the pipeline: values of the first block, keys of the first two, scores of the first's two tiles, weights of one
        uint32_t wa[8], wb[8];
        f32x16 sa, sb;
        auto convert_keys = [&](int b) {
#pragma unroll
            for (int i = 0; i < kUnits; ++i) {
                const Operand x[2] = {eight(kx[i][0], kx[i][1], kscale), eight(kx[i][2], kx[i][3], kscale)};
                put_keys(i, x, b);
            }
        };
        hide_values(b_first);
#pragma unroll
        for (int j = 0; j < kShare; ++j) put_values(j, operand(j), b_first);
        load_values(b_first + 1);
        convert_keys(b_first);
        load_keys(b_first + 1);
        convert_keys(b_first + 1);
        load_keys(b_first + 2);
        __syncthreads();
#pragma unroll
        for (int tt = 0; tt < 2; ++tt)
#pragma unroll
            for (int i = 0; i < kDots; ++i) dot(i, staged.k[b_first & 1][tt][i][lane], tt ? sb : sa);
        hide(b_first, 0, sa);
        {
#pragma unroll
            for (int k = 0; k < 8; ++k) wa[k] = 0;
            most = largest(sa);
            raise(most, wa);
            relative(sa);
            const float mc = less;
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const float e0 = __builtin_amdgcn_exp2f(__builtin_fmaf(sa[2 * k], c, -mc));
                const float e1 = __builtin_amdgcn_exp2f(__builtin_fmaf(sa[2 * k + 1], c, -mc));
                wa[k] = pack_bf16(e0, e1);
                l += e0 + e1;
            }
        }
        __syncthreads();
        int b = b_first;
        do {
            if (b - held == Blocks::kAhead) {
                held = b;
                lies.load(a.b, row, head, held + lane, any_from, any_upto);
            }
            step(b, 0, wa, wb, sb, sa);
            step(b, 1, wb, wa, sa, sb);
            __syncthreads();
        } while (++b < b_end);
    }
    l = halves_sum(l);
    if (!real) return;
    // Results are divided by the weights' sum with the largest one as it was multiplied, in bf16: its rounding, which in a row with a dominant
    // key all of the result would have, cancels (0.0023 off the 64-bit result -> 0.0021, root mean square; all weights so: the same, but
    // 485 us -> 517).
    const float heavy = __builtin_amdgcn_exp2f(__builtin_fmaf(far && top != -INFINITY ? most - top : most, c, -less));
    const float inv = l != 0.f ? 1.f / (l + (bf16_lo(pack_bf16(heavy, 0.f)) - heavy)) : 0.f;
    uint16_t *out = a.out.p + t * a.out.ld + h * a.out.hd + 4 * hh;
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            uint2 w;
            w.x = pack_bf16(o[mt][4 * i] * inv, o[mt][4 * i + 1] * inv);
            w.y = pack_bf16(o[mt][4 * i + 2] * inv, o[mt][4 * i + 3] * inv);
            *reinterpret_cast<uint2 *>(out + 32 * mt + 8 * i) = w;
        }
    if (hh == 0 && a.lse) a.lse[t * a.ld_lse + h] = l != 0.f ? (__builtin_fmaf(top, c, off) + __builtin_amdgcn_logf(l)) * kLn2 : -INFINITY;
}

// The first `groups` workgroups walk the sequences of few rows, the others take the prompts: while the ones
// wait for memory the others multiply.
template <int D>
__global__ __launch_bounds__(kWaves *kWave, 2) void kv8_mixed_kernel(Kv8Attention a, Part<D> *parts, PartTag *tags,
                                                                     int groups, int tiles) {
    __shared__ union {
        Shared<D> sh;
        Staged<D> staged;
    } lds;
    if ((int)blockIdx.x < groups)
        decode<D, false>(a, parts, tags, lds.sh, blockIdx.x, groups);
    else
        prompt<D>(a, tiles, lds.staged, (int)blockIdx.x - groups);
}

// Few and short: a workgroup to each row tile (sequence s has none but its own of
// q_start[s] * group / rows + s on, so their number is bounded), nothing to join.
int64_t whole_tiles(int64_t T, int64_t S, int heads, int n_kv) { return (T * (heads / n_kv) / kRows + S) * n_kv; }
bool whole(int64_t tiles, int groups, int64_t room) {
    return tiles <= groups && room <= (4 * tiles < groups ? kWholeTokens : 4 * kWholeTokens);
}

// The same of selected blocks: their number is known.  A wave to each item where there are items for all of them, or a workgroup, or, where
// that would leave many blocks to few, equal runs and a second launch.
int64_t selected_items(int64_t T, int heads, int n_kv) { return T * n_kv * ((heads / n_kv + kRows - 1) / kRows); }
int selected_mode(int64_t items, int groups, int top) {
    if (items >= groups) return kWave1;
    const int64_t whole = (top + kWaves - 1) / kWaves, runs = (items * top + groups * kWaves - 1) / (groups * kWaves);
    return whole <= runs + kJoinBlocks ? kItem : kRuns;
}

template <int D>
hipError_t launch(Kv8Attention a, int64_t max_q, void *ws, hipStream_t st) {
    const int group = a.heads / a.b.f.n_kv;
    const int groups = device_cus() * kGroupsPerCu;
    Part<D> *parts = (Part<D> *)ws;
    PartTag *tags = (PartTag *)(parts + 2 * (size_t)groups);
    // Without a workspace (kv8_attention_workspace) nothing may be split between workgroups.
    if (a.selected) {
        const int64_t items = selected_items(a.b.T, a.heads, a.b.f.n_kv);
        const int mode = selected_mode(items, groups, a.top);
        a.whole = mode != kRuns;
        if (mode == kWave1) {
            kv8_selected_kernel<D, kWave1><<<(unsigned)((items + kWaves - 1) / kWaves), kWaves * kWave, 0, st>>>(a, parts, tags);
        } else if (mode == kItem) {
            kv8_selected_kernel<D, kItem><<<(unsigned)items, kWaves * kWave, 0, st>>>(a, parts, tags);
        } else {
            kv8_selected_kernel<D, kRuns><<<groups, kWaves * kWave, 0, st>>>(a, parts, tags);
            kv8_join_kernel<D><<<groups, 256, 0, st>>>(a, parts, tags);
        }
        return hipGetLastError();
    }
    const int64_t row_tiles = whole_tiles(a.b.T, a.b.S, a.heads, a.b.f.n_kv);
    a.whole = whole(row_tiles, groups, (int64_t)a.b.cols * a.b.f.page);
    // Where no sequence has many rows, or all rows make few row tiles for the machine's waves, every sequence is
    // walked by row tiles, split over its keys; else each is taken as its own rows ask for.
    a.prompts = !a.whole && max_q * group > kDecodeRows && (int64_t)a.b.T * a.heads > (int64_t)groups * kWaves * kRows / kFewTiles;
    if (a.prompts) {
        const int64_t tiles = (int64_t)a.b.T * group / kPromptRows + a.b.S;
        const int first = a.b.S > 1 ? groups / kGroupsPerCu : 0;  // a lone sequence is a prompt whatever its rows
        kv8_mixed_kernel<D><<<(unsigned)(first + tiles * a.b.f.n_kv), kWaves * kWave, 0, st>>>(a, parts, tags, first, (int)tiles);
        if (first) kv8_join_kernel<D><<<first, 256, 0, st>>>(a, parts, tags);
        return hipGetLastError();
    }
    const int grid = a.whole ? (int)row_tiles : groups;
    if (max_q * group <= kRows)
        kv8_decode_kernel<D, true><<<grid, kWaves * kWave, 0, st>>>(a, parts, tags);
    else
        kv8_decode_kernel<D, false><<<grid, kWaves * kWave, 0, st>>>(a, parts, tags);
    if (!a.whole) kv8_join_kernel<D><<<groups, 256, 0, st>>>(a, parts, tags);
    return hipGetLastError();
}

}  // namespace

size_t kv8_attention_workspace(int64_t T, int64_t S, int heads, int n_kv, int dim, int64_t room, int top) {
    const int groups = device_cus() * kGroupsPerCu;
    if (top > 0 ? selected_mode(selected_items(T, heads, n_kv), groups, top) != kRuns : whole(whole_tiles(T, S, heads, n_kv), groups, room)) return 0;
    return dim == 128 ? decode_workspace<128>(groups) : decode_workspace<64>(groups);
}

hipError_t launch_kv8_attention(const Kv8Attention &a, int64_t max_q, void *ws, hipStream_t st) {
    return a.b.f.dim == 128 ? launch<128>(a, max_q, ws, st) : launch<64>(a, max_q, ws, st);
}

}  // namespace nmk

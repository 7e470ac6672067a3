// nm_kv4_attention.hip -- attention over the 4-bit key/value cache.
//
// For query row i of a sequence (place p = kv_len - rows + i) and head h:
//     s_j = scale * sum_c q_c K_jc,  m = max_j s_j,  l = sum_j exp(s_j - m),
//     o_c = sum_j exp(s_j - m) V_jc / l,  lse = m + log l,
// over the keys j <= p, and j > p - window where there is a window.
//
// Decode.  The query rows of one key/value head (its query heads times the sequence's new
// tokens) form tiles of 16.  A wave takes one tile and walks blocks of 64 tokens:
//   S^T [64 x 16] = K [64 x D] . Q^T: the scaled matrix instruction reads the 4-bit keys and
//     their scales as they lie in the page (16 tokens x 128 channels an instruction), so
//     keys cost no conversion at all.  Queries are sums of four 6-bit (E2M3) pieces, so
//     the scores are those of the bf16 queries.
//   O^T [D x 16] += V^T [D x 64] . P^T: S^T leaves a lane four consecutive tokens of one
//     query row, which is what the bf16 product over tokens takes; V units of 4 tokens x 8
//     channels give the same lane its 8 tokens of 8 channels with one conversion and one
//     byte permute per two values, nothing passes through LDS.
// Weights are rounded to bf16 for that product (off by 2^-8 of each at most, either way, so
// much of it cancels over keys); scores, maxima, sums and O stay in fp32.
//
// Work split.  All (sequence, key/value head, row tile, 64-token block) units of a call
// are laid end to end, in that order, and cut into equal runs, one per wave: lengths need
// not be alike, nor known to the host.  A wave finishes the rows whose blocks are all its own;
// pieces of rows cut between waves are joined in LDS, those cut between workgroups in fp32
// through the workspace by a second kernel, in a fixed order.
//
// Bound: reading the cache.  16 sequences of up to 64K tokens, 64 and 8 heads: 525 MB, 93 us a call among others (traced alone
// this kernel takes 90, 5.8 TB/s, and the join 6); 48 of up to 8K, 40 and 8 heads: 183 MB, 42 us (39 and 5).  A plain read of
// a large buffer reaches 6.9.  Until half of the waves are through, 28 us after the start of the smaller one, the
// walk itself reads 7.6 TB/s; the rest is the way to the first block (6 us: lengths, page table and bytes, each
// waits for the one before), the waves that had to wait for the other one of their SIMD, and the join.
#include <atomic>

#include "nm_device.h"
#include "nm_kv.h"

namespace nmk {
namespace {

constexpr float kLn2 = 0.6931471805599453f;
constexpr int kBlock = 64;      // tokens a wave takes at a time
constexpr int kRows = 16;       // query rows of a tile
// Prompts: O is rescaled only when a score passes the largest one so far by 2^kSlack; weights are kept
// relative to that point, so that they stay at or below 1.  Row tiles, which
// wait for memory, follow every new largest score at no cost: its weight is then 1, which bf16 holds
// exactly (48 sequences of up to 8K tokens: 0.0019 off the 64-bit result, 0.0023 with the slack).
constexpr float kSlack = 8.f;
constexpr float kFar = 4096.f;  // reference (log2) up to which a rounded product of it is off by 2^-13 at most
constexpr int kWaves = 4;       // waves per workgroup
// Context up to which each row tile may be one workgroup's, which needs no second launch: 8 sequences of up to
// 1000 tokens, 32 and 8 heads, 10.5 us against 11.8 split, of 2000 13.2 against 12.3; four times that where there are row
// tiles for a quarter of the workgroups: 20 of up to 4000 20.2 against 20.4, 32 21.4 against 24.2, 32 of 8000 36 against 32.
constexpr int kWholeTokens = 1024;
constexpr int kDecodeRows = 64; // query rows of a head up to which a sequence among others is walked by row tiles
// Row tiles of a call, one to so many waves at most, up to which prompts are walked by row tiles too: a
// workgroup that takes a prompt walks all keys of its rows, so a short prompt behind a long context would keep a few
// CUs busy for long (32 query, 8 key heads: 40 rows behind 20K tokens 416 us there and 49 in row tiles, 512 behind
// nothing 24 and 20, 640 behind 3K 88 and 94, 1024 behind nothing 35 and 44).
constexpr int kFewTiles = 2;
constexpr int kGroupsPerCu = 2; // resident workgroups: 8 waves a CU, 8.7 KB of cache in flight each

typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef float f32x32 __attribute__((ext_vector_type(32)));
typedef uint32_t u32x6 __attribute__((ext_vector_type(6)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x32 __attribute__((ext_vector_type(32)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

// A read with a wave-uniform address of data that no kernel in flight writes: through the
// scalar cache, so it does not enter the order in which a wave's vector loads return.
__device__ __forceinline__ int32_t uniform_load(const int32_t *p) {
    return *(const __attribute__((address_space(4))) int32_t *)(uintptr_t)p;
}

__device__ __forceinline__ float pow2_byte(uint32_t byte) { return __uint_as_float(byte << 23); }

// Scale i of a dword's four for the conversion instruction, which reads the exponent field
// alone: what lands in the sign and fraction does not matter.
__device__ __forceinline__ float scale_field(uint32_t dword, int i) {
    return __uint_as_float(i < 3 ? dword << (23 - 8 * i) : dword >> 1);
}

__device__ __forceinline__ float rows_max(float v) {  // over the four lanes of a column
    const uint32_t u = __float_as_uint(v);
    const auto p = __builtin_amdgcn_permlane16_swap(u, u, false, false);
    const float w = fmaxf(__uint_as_float(p[0]), __uint_as_float(p[1]));
    const uint32_t x = __float_as_uint(w);
    const auto q = __builtin_amdgcn_permlane32_swap(x, x, false, false);
    return fmaxf(__uint_as_float(q[0]), __uint_as_float(q[1]));
}

__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
    union { bf16x2 h; uint32_t u; } c;
    c.h = __builtin_convertvector((f32x2){a, b}, bf16x2);
    return c.u;
}

__device__ __forceinline__ uint32_t fp4_pair(uint32_t w, float s, int byte) {
    union { bf16x2 h; uint32_t u; } c;
    switch (byte) {
    case 0: c.h = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 0); break;
    case 1: c.h = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 1); break;
    case 2: c.h = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 2); break;
    default: c.h = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 3); break;
    }
    return c.u;
}

// A lane's 32 query channels as four 6-bit (E2M3) pieces with a scale each: 2^-2, 2^-6,
// 2^-11 and 2^-16 of the power of two at or below the largest of them.  What is left is at
// most 2^-20 of that, and nothing of numbers within 2^-8 of it.  The instruction aligns the products of 8
// neighbouring channels to about 13 bits below the largest of them: those of 4-bit and 6-bit
// numbers always fit, those of 4-bit and 8-bit (E4M3) ones do not (two 8-bit pieces, at the
// same matrix time, were measured 2^-17 of |q| |k| off).  Of a block with an infinity or NaN the
// scales are NaN, and so is what its row gets.  `at`: the pieces' scales, a byte each, for what is multiplied: queries
// times 2^fold (of a score what is below 2^-127 of its key's largest channel may be lost).
struct Pieces {
    u32x6 p[4];
    uint32_t at[4];
};

union Channels {  // 32 of them
    u32x4 u[4];
    uint32_t w[16];
    bf16x32 h;
};

__device__ __forceinline__ Channels read_query(const uint16_t *from, bool real) {
    Channels x;
#pragma unroll
    for (int i = 0; i < 4; ++i) x.u[i] = real ? *reinterpret_cast<const u32x4 *>(from + i * 8) : (u32x4){0, 0, 0, 0};
    return x;
}

__device__ __forceinline__ Pieces split_query(Channels x, const Kv4Attention &a) {
    const uint32_t keep = a.zero ? 0u : ~0u, flip = a.minus ? 0x80008000u : 0u;
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        top = max(top, max(x.w[i] & 0x7FFFu, (x.w[i] >> 16) & 0x7FFFu));
        x.w[i] = (x.w[i] & keep) ^ flip;
    }
    const uint32_t e = max(top >> 7, (uint32_t)(20 - a.fold));  // biased exponent of the largest magnitude
    Pieces q;
    q.at[0] = e - 2;
    q.at[1] = e - 6;
    q.at[2] = e - 11;
    q.at[3] = e - 16;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const float s = pow2_byte(q.at[k]);
        q.p[k] = __builtin_amdgcn_cvt_scalef32_pk32_fp6_bf16(x.h, s);
        if (k < 3) {  // what is left is a bf16 number: the bits that the piece did not take
            const f32x32 d = __builtin_amdgcn_cvt_scalef32_pk32_f32_fp6(q.p[k], s);
#pragma unroll
            for (int i = 0; i < 16; ++i)
                x.w[i] = pack_bf16(bf16_lo(x.w[i]) - d[2 * i], bf16_hi(x.w[i]) - d[2 * i + 1]);
        }
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) q.at[k] = e == 255u ? 255u : q.at[k] + a.fold;
    return q;
}

// The pieces of a decode tile's row.  At dim 64 the instruction's upper 64 channels multiply the
// same keys again: lanes 32.. hold the second and fourth piece.
template <int D>
struct Query {
    static constexpr int kSteps = D / 32;
    u32x6 p[kSteps];
    uint32_t scales;  // a byte for each of p
};

template <int D>
__device__ __forceinline__ Query<D> load_query(const uint16_t *row, bool real, const Kv4Attention &a, int g) {
    const Pieces x = split_query(read_query(row + (D == 128 ? g : (g & 1)) * 32, real), a);
    Query<D> q;
    if constexpr (D == 128) {
#pragma unroll
        for (int k = 0; k < 4; ++k) q.p[k] = x.p[k];
        q.scales = x.at[0] | x.at[1] << 8 | x.at[2] << 16 | x.at[3] << 24;
    } else {
#pragma unroll
        for (int k = 0; k < 2; ++k) q.p[k] = g < 2 ? x.p[2 * k] : x.p[2 * k + 1];
        q.scales = g < 2 ? x.at[0] | x.at[2] << 8 : x.at[1] | x.at[3] << 8;
    }
    return q;
}

// Of the scaled matrix instruction's operands 4-bit formats are read from four registers
// and 6-bit ones from six; the rest of the type is never read.
__device__ __forceinline__ i32x8 wide(u32x6 v) {
    return (i32x8)__builtin_shufflevector(v, v, 0, 1, 2, 3, 4, 5, -1, -1);
}
__device__ __forceinline__ i32x8 wide(u32x4 v) {
    return (i32x8)__builtin_shufflevector(v, v, 0, 1, 2, 3, -1, -1, -1, -1);
}

// What a sequence asks of a call.
struct Seq {
    int q0, n, len;      // first row, rows, tokens
    int tiles;           // row tiles per key/value head
    int first, blocks;   // first 64-token block and how many (at least one)
    __device__ int64_t units(int n_kv, bool whole) const { return (int64_t)tiles * n_kv * (whole ? 1 : blocks); }
};

__device__ __forceinline__ Seq seq_from(const Kv4Attention &a, int group, int q0, int q1, int len) {
    Seq q = {q0, q1 - q0, len, 0, 0, 1};
    if (q.n <= 0 || (a.prompts && (int64_t)q.n * group > kDecodeRows)) {
        q.n = 0;
        return q;
    }
    q.tiles = (int)(((int64_t)q.n * group + kRows - 1) / kRows);
    const int64_t cap = (int64_t)a.b.cols * a.b.f.page;
    const int64_t end = q.len < cap ? q.len : cap;
    int64_t lo = a.window > 0 ? (int64_t)q.len - q.n - a.window + 1 : 0;
    if (lo < 0) lo = 0;
    q.first = (int)(lo / kBlock);
    const int64_t last = (end + kBlock - 1) / kBlock;
    q.blocks = last > q.first ? (int)(last - q.first) : 1;
    return q;
}

// Sixty-four sequences, one a lane (behind the last one: without rows), and the inclusive
// prefix sums of their units.
struct SeqLane {
    int q0, q1, len;
    __device__ void load(const Kv4Batch &b, int s) {
        q0 = q1 = len = 0;
        if (s < b.S) {
            q0 = b.q_start[s];
            q1 = b.q_start[s + 1];
            len = b.kv_len[s];
        }
    }
};

template <int kCtrl, int kRowMask>
__device__ __forceinline__ uint32_t dpp_scan_add(uint32_t v) {
    return v + (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, kCtrl, kRowMask, 0xF, false);
}

__device__ __forceinline__ int64_t units_scan(int64_t w, int lane) {
    if (__builtin_expect(__any(w >> 25) == 0, 1)) {  // 64 of them fit in 31 bits
        uint32_t v = (uint32_t)w;
        v = dpp_scan_add<0x111, 0xF>(v);  // shifts within rows of 16 lanes
        v = dpp_scan_add<0x112, 0xF>(v);
        v = dpp_scan_add<0x114, 0xF>(v);
        v = dpp_scan_add<0x118, 0xF>(v);
        v = dpp_scan_add<0x142, 0xA>(v);  // last lane of rows 0 and 2 to rows 1 and 3
        v = dpp_scan_add<0x143, 0xC>(v);  // lane 31 to the upper half
        return v;
    }
    for (int d = 1; d < 64; d <<= 1) {
        const int64_t u = __shfl_up(w, d);
        if (lane >= d) w += u;
    }
    return w;
}

// A value that is the same in all lanes, or lane i's, in scalar registers.
__device__ __forceinline__ int64_t lane64(int64_t v, int i) {
    const uint32_t lo = __builtin_amdgcn_readlane((int)(uint32_t)v, i);
    const uint32_t hi = __builtin_amdgcn_readlane((int)(uint32_t)((uint64_t)v >> 32), i);
    return (int64_t)(((uint64_t)hi << 32) | lo);
}

// Where the 64-token blocks of one head lie: lane i holds the address of block `first` + i of
// a sequence, so that a walk reads the page table once for kAhead blocks and turns a page into
// an address off its critical path.  Without a valid page the address is that of page 0,
// so that loads need no branch (a branch around them would make the wave wait for all it has in
// flight), and the block's bit in `valid` is clear.
struct Blocks {
    static constexpr int kAhead = 60;  // of 64: a walk looks up to three blocks ahead
    uint32_t lo, hi;
    uint64_t valid;
    __device__ void load(const Kv4Batch &b, const int32_t *row, int head, int first, int lane) {
        const int per = b.f.page / kBlock, block = first + lane;
        const int col = block / per;
        int page = col < b.cols ? row[col] : -1;
        const bool ok = page >= 0 && page < b.num_pages;
        if (!ok) page = 0;
        valid = __ballot(ok);
        const uint64_t at = (uint64_t)(uintptr_t)b.cache + (uint64_t)page * (uint64_t)b.f.page_bytes() +
                            (uint64_t)head * (uint64_t)b.f.head_bytes() +
                            (uint64_t)((block & (per - 1)) * (kBlock / 2)) * b.f.dim;
        lo = (uint32_t)at;
        hi = (uint32_t)(at >> 32);
    }
    // K values of block i of the 64 (V values v_at behind them); places that scales differ
    // by are in scales_at.
    __device__ const uint8_t *at(int i) const {
        const uint32_t l = __builtin_amdgcn_readlane((int)lo, i), h = __builtin_amdgcn_readlane((int)hi, i);
        return (const uint8_t *)(uintptr_t)((uint64_t)h << 32 | l);
    }
    __device__ bool ok(int i) const { return (valid >> i) & 1; }
};

// From a block's K values to its K scales: the tokens before it in the page count D / 32
// scale bytes, not D / 2 value bytes.
__device__ __forceinline__ int scales_at(const Kv4Format &f, int block) {
    const int tok0 = (block & (f.page / kBlock - 1)) * kBlock;
    return f.ks_at() - tok0 * (f.dim / 2 - f.dim / 32);
}

// One tile's running softmax in registers: column c = lane % 16 is query row c, the four
// lanes of a column share m and hold their own tokens' part of l and D/4 channels of O.
template <int D>
struct Tile {
    f32x4 o[D / 16];
    float m, l;  // m: the raw score that weights are relative to
};

template <int D>
__device__ __forceinline__ void clear(Tile<D> &t) {
#pragma unroll
    for (int i = 0; i < D / 16; ++i) t.o[i] = (f32x4){0.f, 0.f, 0.f, 0.f};
    t.m = -INFINITY;
    t.l = 0.f;
}

// The cache bytes of 64 tokens of one head that a lane multiplies.
template <int D>
struct Bytes {
    u32x4 k[4], v[4];
    uint32_t ks, vs[4];
};

template <int D>
struct Lane {
    int col, g;
    uint32_t k_off, ks_off, v_off, vs_off;  // byte places of this lane within a block of 64 tokens
    __device__ Lane(int lane) {
        col = lane & 15;
        g = lane >> 4;
        const int kb = D == 128 ? g : (g & 1);
        k_off = col * (D / 2) + kb * 16;
        ks_off = (col * (D / 32) + kb) * 4;
        const int c8 = D == 128 ? col : col >> 1;
        v_off = (g * (D / 8) + c8) * 16;
        vs_off = (g * (D / 32) + (c8 >> 2)) * 4;
    }
};

// Cache bytes at an address put together from its halves: said to be global memory (a load that might be
// from LDS as well counts among the LDS operations too, and waits for one would wait for it).
// NT: bytes that are read once (one row tile per head) stay out of the caches' way.
template <bool NT, class T>
__device__ __forceinline__ T load_cache(const uint8_t *p) {
    typedef const __attribute__((address_space(1))) T *Global;
    return NT ? __builtin_nontemporal_load((Global)(uintptr_t)p) : *(Global)(uintptr_t)p;
}

template <int D, bool NT>
__device__ __forceinline__ void load_block(Bytes<D> &x, const uint8_t *k, const Kv4Format &f, int block,
                                           const Lane<D> &ln) {
    const uint8_t *v = k + f.v_at(), *ks = k + scales_at(f, block), *vs = ks + f.page * (D / 32);
#pragma unroll
    for (int j = 0; j < 4; ++j) x.k[j] = load_cache<NT, u32x4>(k + ln.k_off + j * 8 * D);
    x.ks = load_cache<NT, uint32_t>(ks + ln.ks_off);
#pragma unroll
    for (int j = 0; j < 4; ++j) x.v[j] = load_cache<NT, u32x4>(v + ln.v_off + j * 8 * D);
#pragma unroll
    for (int j = 0; j < 4; ++j) x.vs[j] = load_cache<NT, uint32_t>(vs + ln.vs_off + j * (D / 2));
}

// Scores of 64 tokens: s[j][i] is token 16 j + 4 g + i of the column's row.
template <int D>
__device__ __forceinline__ void scores(const Bytes<D> &x, const Query<D> &q, f32x4 (&s)[4]) {
    const f32x4 zero = {0.f, 0.f, 0.f, 0.f};
    const int sc = (int)q.scales, ks = (int)x.ks;
#define NM_KV4_DOT(J, P, C) \
    s[J] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(wide(x.k[J]), wide(q.p[P]), C, 4, 2, J, ks, P, sc)
    NM_KV4_DOT(0, 0, zero); NM_KV4_DOT(1, 0, zero); NM_KV4_DOT(2, 0, zero); NM_KV4_DOT(3, 0, zero);
    NM_KV4_DOT(0, 1, s[0]); NM_KV4_DOT(1, 1, s[1]); NM_KV4_DOT(2, 1, s[2]); NM_KV4_DOT(3, 1, s[3]);
    if constexpr (D == 128) {
        NM_KV4_DOT(0, 2, s[0]); NM_KV4_DOT(1, 2, s[1]); NM_KV4_DOT(2, 2, s[2]); NM_KV4_DOT(3, 2, s[3]);
        NM_KV4_DOT(0, 3, s[0]); NM_KV4_DOT(1, 3, s[1]); NM_KV4_DOT(2, 3, s[2]); NM_KV4_DOT(3, 3, s[3]);
    }
#undef NM_KV4_DOT
}

// Values are multiplied as 2^-spare(keys) of what they are: weights are at most 1, so O stays below the largest
// value, and in range whatever the values are; the factor leaves with the sum of the weights.
__device__ __forceinline__ int spare(int keys) { return keys > 0 ? 32 - __clz(keys) : 0; }
__device__ __forceinline__ float pow2(int e) { return __uint_as_float((uint32_t)(127 + e) << 23); }

// What weights are relative to, as a power of two.
__device__ __forceinline__ float reference(float m, float c) { return m == -INFINITY ? 0.f : m * c; }

// Scores -> weights; O and l follow the reference.  The difference is taken before the product with c: the
// product of a large score, rounded to be subtracted, would be off by more than a power of two (a subtraction more per
// weight: 42.3 us against 41.9 for 48 sequences of up to 8K tokens; in a branch for large scores, as in prompts, 42.2).
template <int D>
__device__ __forceinline__ void weights(Tile<D> &t, f32x4 (&s)[4], float c) {
    float mx = fmaxf(fmaxf(s[0][0], s[0][1]), fmaxf(s[0][2], s[0][3]));
#pragma unroll
    for (int j = 1; j < 4; ++j) mx = fmaxf(mx, fmaxf(fmaxf(s[j][0], s[j][1]), fmaxf(s[j][2], s[j][3])));
    const float mn = fmaxf(t.m, rows_max(mx));
    if (__any(mn > t.m)) {
        const float keep = t.m == -INFINITY ? 0.f : __builtin_amdgcn_exp2f((t.m - mn) * c);
#pragma unroll
        for (int i = 0; i < D / 16; ++i) t.o[i] *= keep;
        t.l *= keep;
        t.m = mn;
    }
    const float base = t.m == -INFINITY ? 0.f : t.m;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
#pragma unroll
        for (int i = 0; i < 4; ++i) s[j][i] = __builtin_amdgcn_exp2f((s[j][i] - base) * c);
        t.l += (s[j][0] + s[j][1]) + (s[j][2] + s[j][3]);
    }
}

// O += V^T P for 64 tokens, values times `down`.
template <int D>
__device__ __forceinline__ void add_values(Tile<D> &t, const Bytes<D> &x, const f32x4 (&p)[4], float down, int col) {
#pragma unroll
    for (int s = 0; s < 2; ++s) {
        union { uint32_t w[4]; bf16x8 h; } b;
        b.w[0] = pack_bf16(p[2 * s][0], p[2 * s][1]);
        b.w[1] = pack_bf16(p[2 * s][2], p[2 * s][3]);
        b.w[2] = pack_bf16(p[2 * s + 1][0], p[2 * s + 1][1]);
        b.w[3] = pack_bf16(p[2 * s + 1][2], p[2 * s + 1][3]);
        uint32_t w[8];
        float f[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            w[e] = x.v[2 * s + (e >> 2)][e & 3];
            if (D == 64) w[e] >>= (col & 1) * 16;
            f[e] = scale_field(x.vs[2 * s + (e >> 2)], e & 3) * down;
        }
#pragma unroll
        for (int by = 0; by < D / 32; ++by) {
            uint32_t c[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) c[e] = fp4_pair(w[e], f[e], by);
            union { uint32_t w[4]; bf16x8 h; } lo, hi;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                lo.w[e] = __builtin_amdgcn_perm(c[2 * e + 1], c[2 * e], 0x05040100u);
                hi.w[e] = __builtin_amdgcn_perm(c[2 * e + 1], c[2 * e], 0x07060302u);
            }
            t.o[2 * by] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(lo.h, b.h, t.o[2 * by], 0, 0, 0);
            t.o[2 * by + 1] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(hi.h, b.h, t.o[2 * by + 1], 0, 0, 0);
        }
    }
}

// Lane's channel of o[mt][i]: (D/4) g + (D/16) i + mt.
template <int D>
__device__ __forceinline__ void store_row(const Kv4Attention &a, int t, int h, int g, const float *o, float m, float l,
                                          float up, bool with_lse) {
    const float inv = l != 0.f ? up / l : 0.f;
    uint16_t *p = a.out.p + t * a.out.ld + h * a.out.hd + g * (D / 4);
#pragma unroll
    for (int i = 0; i < D / 32; ++i) {
        u32x4 w;
#pragma unroll
        for (int j = 0; j < 4; ++j) w[j] = pack_bf16(o[8 * i + 2 * j] * inv, o[8 * i + 2 * j + 1] * inv);
        *reinterpret_cast<u32x4 *>(p + 8 * i) = w;
    }
    if (with_lse && a.lse) a.lse[t * a.ld_lse + h] = l != 0.f ? (m + __builtin_amdgcn_logf(l)) * kLn2 : -INFINITY;
}

// Pieces of rows cut between waves (LDS) or workgroups (workspace): unnormalised O by
// row, the maximum (log2 units, scaled) and the sum.  The rows' stride keeps the 16 columns
// of a wave on different banks.
template <int D>
struct Part {
    float o[kRows][D + 4];
    float m[kRows], l[kRows];
};

enum : int { kNone = 0, kEnds = 1, kThrough = 2 };  // the item's last block is in / behind the piece

struct PartTag {
    int state;                  // kNone, kEnds, kThrough
    int q0, head, tile, rows;   // the sequence's first row, the row tile and its rows
    int spare;                  // O is 2^-spare of what it is
};

template <int D>
struct Shared {
    Part<D> part[kWaves][2];
    PartTag tag[kWaves][2];
};

template <int D>
__device__ __forceinline__ void keep_part(Part<D> &p, const Tile<D> &t, float c, const Lane<D> &ln) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int q = 0; q < D / 64; ++q) {
            const f32x4 w = {t.o[4 * q][i], t.o[4 * q + 1][i], t.o[4 * q + 2][i], t.o[4 * q + 3][i]};
            *reinterpret_cast<f32x4 *>(&p.o[ln.col][(D / 4) * ln.g + (D / 16) * i + 4 * q]) = w;
        }
    const float l = cross_rows_sum(t.l);
    if (ln.g == 0) {
        p.m[ln.col] = t.m == -INFINITY ? -INFINITY : reference(t.m, c);
        p.l[ln.col] = l;
    }
}

__device__ __forceinline__ float weight_of(float m, float top) {
    return m == -INFINITY ? 0.f : __builtin_amdgcn_exp2f(m - top);
}

// Threads of a workgroup over a part: 16 rows x 16 threads of D/16 channels.
template <int D>
struct Join {
    static constexpr int N = D / 16;
    float o[N], m, l;
    __device__ Join() : m(-INFINITY), l(0.f) {
#pragma unroll
        for (int i = 0; i < N; ++i) o[i] = 0.f;
    }
    __device__ void add(const Part<D> &p, int row, int c) {
        const float pm = p.m[row], mn = fmaxf(m, pm);
        const float mine = weight_of(m, mn), its = weight_of(pm, mn);
        l = l * mine + p.l[row] * its;
#pragma unroll
        for (int i = 0; i < N; ++i) o[i] = o[i] * mine + p.o[row][c * N + i] * its;
        m = mn;
    }
    __device__ void put(Part<D> &p, int row, int c) const {
#pragma unroll
        for (int i = 0; i < N; ++i) p.o[row][c * N + i] = o[i];
        if (c == 0) {
            p.m[row] = m;
            p.l[row] = l;
        }
    }
    __device__ void finish(const Kv4Attention &a, const PartTag &tag, int group, int row, int c) const {
        if (row >= tag.rows) return;
        const int r = tag.tile * kRows + row;
        const int t = tag.q0 + r / group, h = tag.head * group + r % group;
        if ((uint32_t)t >= (uint32_t)a.b.T) return;
        const float inv = l != 0.f ? pow2(tag.spare) / l : 0.f;
        uint32_t *p = reinterpret_cast<uint32_t *>(a.out.p + t * a.out.ld + h * a.out.hd + c * N);
#pragma unroll
        for (int i = 0; i < N / 2; ++i) p[i] = pack_bf16(o[2 * i] * inv, o[2 * i + 1] * inv);
        if (c == 0 && a.lse) a.lse[t * a.ld_lse + h] = l != 0.f ? (m + __builtin_amdgcn_logf(l)) * kLn2 : -INFINITY;
    }
};

// Workgroup `block` of `blocks`.
template <int D, bool NT>
__device__ __forceinline__ void decode(Kv4Attention &a, Part<D> *parts, PartTag *tags, Shared<D> &sh, int block,
                                       int blocks) {
    a.b.f.dim = D;
    const Kv4Format &f = a.b.f;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int group = a.heads / f.n_kv;
    const Lane<D> ln(lane);
    const float c = a.c;
    const int64_t cap = (int64_t)a.b.cols * f.page;

    // my run of units
    SeqLane sl, behind;
    sl.load(a.b, lane);
    int64_t w = seq_from(a, group, sl.q0, sl.q1, sl.len).units(f.n_kv, a.whole);
    int64_t upto = units_scan(w, lane);
    int64_t total = lane64(upto, 63);
    for (int s0 = 64; s0 < a.b.S; s0 += 64) {
        if (s0 == 64) behind.load(a.b, s0 + lane);
        const SeqLane x = behind;
        behind.load(a.b, s0 + 64 + lane);
        total += lane64(units_scan(seq_from(a, group, x.q0, x.q1, x.len).units(f.n_kv, a.whole), lane), 63);
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
            w = seq_from(a, group, sl.q0, sl.q1, sl.len).units(f.n_kv, a.whole);
            upto = units_scan(w, lane);
            continue;
        }
        const int at = __builtin_ctzll(past), s = s0 + at;
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

        // two blocks in flight: the next one's loads are under way while one is multiplied
        const int32_t *row = a.b.table + (int64_t)s * a.b.ld_table;
        Blocks lies;
        int held = b0;  // first of the blocks whose places are held
        lies.load(a.b, row, head, sq.first + held, lane);
        Bytes<D> x0, x1;
        load_block<D, NT>(x0, lies.at(0), f, sq.first + b0, ln);

        // queries of my column
        const int64_t r = (int64_t)tile * kRows + ln.col;
        const int qi = (int)r / group, t = sq.q0 + qi, h = head * group + ((int)r - qi * group);
        const bool real = r < (int64_t)sq.n * group && (uint32_t)t < (uint32_t)a.b.T;
        const Query<D> q = load_query<D>(a.q.p + t * a.q.ld + h * a.q.hd, real, a, ln.g);
        // keys that my row sees: [from, upto]
        const int64_t place = (int64_t)sq.len - sq.n + qi;
        const int see_last = real ? (int)(place < cap ? place : cap - 1) : -1;
        const int see_first = a.window > 0 && place - a.window + 1 > 0 ? (int)(place - a.window + 1) : 0;
        // tokens that every row of the sequence sees (their blocks need no mask), and that any of them sees
        const int all_first = a.window > 0 && sq.len > a.window ? (int)(sq.len - a.window) : 0;
        const int all_last = (int)((int64_t)sq.len - sq.n < cap ? (int64_t)sq.len - sq.n : cap - 1);
        const int64_t some = (int64_t)sq.len - sq.n - a.window + 1;
        const int any_first = a.window > 0 && some > 0 ? (int)some : 0;
        const int any_last = (int)((int64_t)sq.len < cap ? (int64_t)sq.len : cap) - 1;
        const int bits = spare(any_last + 1);
        const float down = pow2(-bits);

        Tile<D> tl;
        clear(tl);
        auto add = [&](Bytes<D> &x, int b) {
            const int j0 = (sq.first + b) * kBlock;
            f32x4 sc[4];
            scores(x, q, sc);
            if (j0 < all_first || j0 + (kBlock - 1) > all_last) {
#pragma unroll
                for (int j = 0; j < 4; ++j)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int tok = j0 + 16 * j + 4 * ln.g + i;
                        if (tok > see_last || tok < see_first) sc[j][i] = -INFINITY;
                        // a weight of 0 times what an unseen place holds must be 0
                        if (tok > any_last || tok < any_first) x.vs[j] &= ~(255u << (8 * i));
                    }
            }
            weights(tl, sc, c);
            add_values(tl, x, sc, down, ln.col);
        };
        // Behind the last block the loads, which are not branched around, go to the cache's first
        // bytes for all waves: a block more of each run's own would be a tenth more traffic at 10 blocks a run (48
        // sequences of up to 8K tokens: 44.4 -> 43.2 us).
        for (int b = b0; b < b1; b += 2) {
            if (b - held == Blocks::kAhead) {
                held = b;
                lies.load(a.b, row, head, sq.first + held, lane);
            }
            const int i = b - held;
            load_block<D, NT>(x1, b + 1 < b1 ? lies.at(i + 1) : a.b.cache, f, sq.first + b + 1, ln);
            if (lies.ok(i)) add(x0, b);
            if (b + 1 >= b1) break;
            load_block<D, NT>(x0, b + 2 < b1 ? lies.at(i + 2) : a.b.cache, f, sq.first + b + 2, ln);
            if (lies.ok(i + 1)) add(x1, b + 1);
        }

        const bool begins = b0 == 0, ends = b1 == sq.blocks;
        if (begins && ends) {
            float o[D / 4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int m = 0; m < D / 16; ++m) o[(D / 16) * i + m] = tl.o[m][i];
            const float l = cross_rows_sum(tl.l);
            if (real) store_row<D>(a, t, h, ln.g, o, reference(tl.m, c), l, pow2(bits), ln.g == 0);
        } else {
            const int slot = begins ? 1 : 0;
            keep_part(sh.part[wave][slot], tl, c, ln);
            const int64_t left = (int64_t)sq.n * group - (int64_t)tile * kRows;
            if (lane == 0)
                sh.tag[wave][slot] = {ends ? kEnds : kThrough, sq.q0, head, tile, (int)(left < kRows ? left : kRows), bits};
        }
    }
    __syncthreads();

    // Join the pieces.  Slot 0 of a wave belongs to a row that began before it, slot 1 to
    // one that begins in it and goes on behind it.
    const int row = threadIdx.x >> 4, cc = threadIdx.x & 15;
    const int64_t me = block;
    PartTag out0 = {kNone}, out1 = {kNone};
    for (int first = -1; first < kWaves; ++first) {  // -1: the chain that enters this workgroup
        PartTag tag = first < 0 ? sh.tag[0][0] : sh.tag[first][1];
        if (tag.state == kNone) continue;
        Join<D> j;
        if (first >= 0) j.add(sh.part[first][1], row, cc);
        int state = kThrough;
        for (int w = first + 1; w < kWaves && state == kThrough; ++w) {
            if (sh.tag[w][0].state == kNone) break;
            j.add(sh.part[w][0], row, cc);
            state = sh.tag[w][0].state;
        }
        tag.state = state;
        if (first >= 0 && state == kEnds) {
            j.finish(a, tag, group, row, cc);
        } else {
            if (row < tag.rows) j.put(parts[me * 2 + (first < 0 ? 0 : 1)], row, cc);
            if (first < 0) out0 = tag; else out1 = tag;
        }
    }
    if (threadIdx.x == 0 && !a.whole) {
        tags[me * 2] = out0;
        tags[me * 2 + 1] = out1;
    }
}

template <int D, bool NT>
__global__ __launch_bounds__(kWaves *kWave, 2) void kv4_decode_kernel(Kv4Attention a, Part<D> *parts, PartTag *tags) {
    __shared__ Shared<D> sh;
    decode<D, NT>(a, parts, tags, sh, blockIdx.x, gridDim.x);
}

// Rows cut between workgroups: the workgroup in which a row begins owns it; the pieces
// follow in the slots 0 of the next ones, up to one in which the row ends.
template <int D>
__global__ __launch_bounds__(256) void kv4_join_kernel(Kv4Attention a, const Part<D> *parts, const PartTag *tags) {
    const int w = blockIdx.x, lane = threadIdx.x & 63, last = (int)gridDim.x - 1;
    // what follows is asked for beside the row itself: most chains end within 64 workgroups
    int state = tags[2 * min(w + 1 + lane, last)].state;
    const PartTag tag = tags[2 * w + 1];
    if (tag.state != kThrough) return;
    int n = 0;  // pieces behind the first
    for (int k = w + 1;;) {
        const uint64_t stop = __ballot(k + lane > last || state != kThrough);
        if (stop) {
            const int at = __builtin_ctzll(stop);
            n += at + (k + at <= last && __builtin_amdgcn_readlane(state, at) == kEnds);
            break;
        }
        n += 64;
        k += 64;
        state = tags[2 * min(k + lane, last)].state;
    }
    const int row = threadIdx.x >> 4, cc = threadIdx.x & 15;
    if (row >= tag.rows) return;
    // Pieces eight at a time, all their loads under way at once; behind the last one the last again, with weight 0.
    constexpr int kAtOnce = 8, N = Join<D>::N;
    Join<D> j;
    for (int k0 = 0; k0 <= n; k0 += kAtOnce) {
        float m[kAtOnce], l[kAtOnce], o[kAtOnce][N], top = j.m;
#pragma unroll
        for (int i = 0; i < kAtOnce; ++i) {
            const int k = min(k0 + i, n);
            const Part<D> &p = parts[k ? 2 * (w + k) : 2 * w + 1];
            m[i] = p.m[row];
            l[i] = p.l[row];
#pragma unroll
            for (int e = 0; e < N; ++e) o[i][e] = p.o[row][cc * N + e];
        }
#pragma unroll
        for (int i = 0; i < kAtOnce; ++i) top = fmaxf(top, m[i]);
        const float keep = weight_of(j.m, top);
        j.l *= keep;
#pragma unroll
        for (int e = 0; e < N; ++e) j.o[e] *= keep;
        j.m = top;
#pragma unroll
        for (int i = 0; i < kAtOnce; ++i) {
            const float its = k0 + i <= n ? weight_of(m[i], top) : 0.f;
            j.l += l[i] * its;
#pragma unroll
            for (int e = 0; e < N; ++e) j.o[e] += o[i][e] * its;
        }
    }
    j.finish(a, tag, a.heads / a.b.f.n_kv, row, cc);
}

// ---- prompts ----
//
// Many rows of a sequence: a workgroup takes kPromptRows rows of one key/value head, 32 a
// wave, and walks the blocks of 64 tokens that the last of them sees.  Each wave converts a
// quarter of the next block's values into the operand order of the product and leaves them
// in LDS (two buffers, one barrier a block), so a value is converted once for 128 rows and
// read from LDS without bank conflicts; keys go from the page into the matrix
// instruction as in decode.  Here 32 x 32 tiles: a matrix instruction keeps the vector unit
// from issuing for about 8 cycles whatever its size, and softmax needs that unit for
// about as long as the matrix unit is busy (four vector instructions to every 16 x 16 x 32
// product: 23.6 ns in 16 x 16 tiles, 18.9 ns in 32 x 32 ones; 15 ns without them).
//
// Both units run at once only where a wave alternates between them: a burst of products
// keeps the other wave of the SIMD from issuing vector instructions (two halves of a workgroup that
// took turns at products and softmax, a barrier between: 1250 cycles of products and 1200 of
// softmax a block took 2500 together).  So the walk is a pipeline over tiles of 32 tokens, one step
// of which has the products of three of them: see `step`.  A block takes 3760 cycles against 4110 for
// scores, softmax and values one after the other; the clock falls by 4 % (2.14 GHz: the
// card's power is the bound), so 3 prompts of up to 4K rows behind 2K, 455 GFLOP, took 464 us against 475 on one card when the two were
// compared; with all that keeps sums and scores in range 476 to 502 by card (905 to 955 TFLOP/s).
constexpr int kPromptTile = 32;                       // rows of a wave
constexpr int kPromptRows = kWaves * kPromptTile;     // rows of a workgroup

typedef float f32x16 __attribute__((ext_vector_type(16)));

// Lane (col, hh) = (lane % 32, lane / 32): column col is a query row, token rows of the scores are
// 8 (i / 4) + 4 hh + i % 4 of a tile of 32.  Channels: row m of channel tile mt is channel
// 8 c8 + b with (c8, b) = (m % 16, 2 mt + m / 16) at dim 128, (m % 8, 4 mt + m / 8) at
// dim 64, so that the 8 channels of a V unit end up in one lane.
template <int D>
struct PromptQuery {
    u32x6 p[D / 64][4];       // 64 channels each: this lane's 32 of them
    uint32_t scales[D / 64];  // a byte for each piece
};

__device__ __forceinline__ float halves_max(float v) {
    const auto p = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    return fmaxf(__uint_as_float(p[0]), __uint_as_float(p[1]));
}
__device__ __forceinline__ float halves_sum(float v) {
    const auto p = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    return __uint_as_float(p[0]) + __uint_as_float(p[1]);
}

template <int D>
using Values = u32x4[2][4][D / 32][kWave];

// Workgroup `block` of tiles * n_kv.
template <int D>
__device__ __forceinline__ void prompt(Kv4Attention &a, int tiles, Values<D> &values, int block) {
    constexpr int MT = D / 32, CH = D / 64;  // channel tiles of the values, chunks of the keys
    a.b.f.dim = D;
    const Kv4Format &f = a.b.f;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int col = lane & 31, hh = lane >> 5;
    const int group = a.heads / f.n_kv;

    // Row tile: sequence s owns the tiles from q_start[s] * group / rows + s on, which are
    // enough for it.  Later rows, which see more, go first; the heads of a tile go to
    // neighbouring workgroups, that is to different XCDs, so an XCD reads few heads.
    const int head = block % f.n_kv;
    const int vt = tiles - 1 - block / f.n_kv;
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
    const int64_t room = (int64_t)a.b.cols * f.page;
    const int cap = len < room ? len : (int)room;  // tokens that have a place
    const int place0 = len - n;                    // of the sequence's first row
    // The first and the last key that a row at some place sees; the same for places at the end of the keys.
    const int window = a.window > 0 && a.window < len ? (int)a.window : 0;
    auto first_of = [&](int place) { return window && place >= window ? place - window + 1 : 0; };
    auto last_of = [&](int place) { return place < cap ? place : cap - 1; };
    const int any_from = first_of(place0), any_upto = cap - 1;
    const float down = pow2(-spare(cap));

    const int w0 = r0 + wave * kPromptTile;  // the wave's first row
    const int r = w0 + col;
    const int qi = (int)((uint32_t)r / (uint32_t)group), t = q0 + qi, h = head * group + (r - qi * group);
    const bool real = r < rows && (uint32_t)t < (uint32_t)a.b.T;
    Channels raw[CH];  // split into pieces once the first block's bytes are on their way
#pragma unroll
    for (int k = 0; k < CH; ++k) raw[k] = read_query(a.q.p + t * a.q.ld + h * a.q.hd + k * 64 + hh * 32, real);
    const int upto = real ? last_of(place0 + qi) : -1, from = first_of(place0 + qi);
    f32x16 o[MT];
#pragma unroll
    for (int i = 0; i < MT; ++i) o[i] = f32x16{};
    float top = -INFINITY, off = 0.f, l = 0.f;  // weights are 2^((score - top) c - off); their sum
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
    lies.load(a.b, row, head, held, lane);

    // keys: token 32 tt + col, block 2 k + hh; their scales lie by token % 16
    const uint32_t k_off = col * (D / 2) + hh * 16;
    const uint32_t ks_off = ((col & 15) * (D / 32) + hh) * 4;
    u32x4 kx[2][CH];
    uint32_t ks[2][CH];
    auto load_keys = [&](int b, int tt) {
        const uint8_t *kp = lies.at(b - held), *sp = kp + scales_at(f, b);
#pragma unroll
        for (int k = 0; k < CH; ++k) {
            kx[tt][k] = load_cache<false, u32x4>(kp + k_off + (tt * 16 * D + k * 32));
            ks[tt][k] = load_cache<false, uint32_t>(sp + ks_off + k * 8);
        }
    };

    // this wave's share of a block's values: tokens 16 vu + 4 vh + {0..3, 8..11} of unit column c8,
    // bytes byte0 .. of their words (a byte is two channels)
    constexpr int kBytes = D / 64;
    const int vg = lane >> 4, vh = vg & 1, vu = 2 * (wave >> 1) + (vg >> 1);
    const int c8 = D == 128 ? (lane & 15) : (lane & 7);
    const int byte0 = D == 128 ? 2 * (wave & 1) : (2 * (wave & 1) + ((lane >> 3) & 1));
    const uint32_t v_off = ((4 * vu + vh) * (D / 8) + c8) * 16, vs_off = ((4 * vu + vh) * (D / 32) + (c8 >> 2)) * 4;
    u32x4 vx[2];
    uint32_t vs[2];
    auto load_values = [&](int b) {
        const uint8_t *kp = lies.at(b - held), *vp = kp + f.v_at(), *sp = kp + scales_at(f, b) + f.page * (D / 32);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            vx[i] = load_cache<false, u32x4>(vp + v_off + i * 4 * D);
            vs[i] = load_cache<false, uint32_t>(sp + vs_off + i * (D / 4));
        }
    };
    load_keys(b_first, 0);
    load_keys(b_first, 1);
    load_values(b_first);
    PromptQuery<D> q;
#pragma unroll
    for (int k = 0; k < CH; ++k) {
        const Pieces x = split_query(raw[k], a);
#pragma unroll
        for (int i = 0; i < 4; ++i) q.p[k][i] = x.p[i];
        q.scales[k] = x.at[0] | x.at[1] << 8 | x.at[2] << 16 | x.at[3] << 24;
    }
    // a weight of 0 times what an unseen place holds must be 0
    auto hide_values = [&](int b) {
        const int j0 = b * kBlock;
        const bool page = lies.ok(b - held);
        if (j0 < any_from || j0 + kBlock - 1 > any_upto || !page) {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const int tok = j0 + 16 * vu + 8 * (e >> 2) + 4 * vh + (e & 3);
                if (tok > any_upto || tok < any_from || !page) vs[e >> 2] &= ~(255u << (8 * (e & 3)));
            }
        }
    };
    // token e of the eight, byte byte0 + by of its word; then the channels 2 (byte0 + by) and the next of all of them
    auto convert = [&](int by, int e) {
        return fp4_pair(vx[e >> 2][e & 3] >> (8 * byte0), scale_field(vs[e >> 2], e & 3) * down, by);
    };
    auto put_values = [&](int by, const u32x4 &even, const u32x4 &odd, u32x4 (*to)[MT][kWave]) {
        if constexpr (D == 128) {
            to[vu][byte0 + by][vh * 32 + c8] = even;
            to[vu][byte0 + by][vh * 32 + 16 + c8] = odd;
        } else {
            u32x4 *p = &to[vu][byte0 >> 1][vh * 32 + 16 * (byte0 & 1) + c8];
            p[0] = even;
            p[8] = odd;
        }
    };
    auto even_of = [](uint32_t hi, uint32_t lo) { return __builtin_amdgcn_perm(hi, lo, 0x05040100u); };
    auto odd_of = [](uint32_t hi, uint32_t lo) { return __builtin_amdgcn_perm(hi, lo, 0x07060302u); };

    // Products of the scores: number i of a 32-token tile's 4 CH, that of chunk i / 4 and piece i % 4.  Of a
    // scale dword's four tokens 16 j + col % 16 this lane's are j = col / 16 and that + 2.
    auto dot = [&](int tt, int i, f32x16 &acc) {
        const f32x16 zero = {};
        const int sk = (int)(ks[tt][i / 4] >> ((col >> 4) * 8));
#define NM_KV4_DOT(T, P)                                                                                                  \
    acc = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(wide(kx[T][i / 4]), wide(q.p[i / 4][P]), i ? acc : zero, 4, 2,  \
                                                          2 * T, sk, P, (int)q.scales[i / 4])
        switch (4 * tt + i % 4) {
        case 0: NM_KV4_DOT(0, 0); break;
        case 1: NM_KV4_DOT(0, 1); break;
        case 2: NM_KV4_DOT(0, 2); break;
        case 3: NM_KV4_DOT(0, 3); break;
        case 4: NM_KV4_DOT(1, 0); break;
        case 5: NM_KV4_DOT(1, 1); break;
        case 6: NM_KV4_DOT(1, 2); break;
        default: NM_KV4_DOT(1, 3); break;
        }
#undef NM_KV4_DOT
    };
    constexpr int kDots = 4 * CH, kSums = 2 * MT;  // matrix products of a 32-token tile: scores, values
    auto sum = [&](int i, const u32x4 &v, const uint32_t (&w)[8]) {
        union { u32x4 u; bf16x8 h; } x;
        union { uint32_t w[4]; bf16x8 h; } y;
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
    // of tile t + 2 (into n), the softmax of tile t + 1 (scores sc to weights wn) and half of the conversion of
    // block b + 1.
    auto step = [&](int b, int tt, uint32_t (&w)[8], uint32_t (&wn)[8], f32x16 &sc, f32x16 &n) {
        const u32x4 *from_lds = &values[b & 1][2 * tt][0][lane];
        hide(tt ? b + 1 : b, tt ^ 1, sc);
        raise(largest(sc), w);
        relative(sc);
        const float mc = less;
        if (tt == 0) hide_values(b + 1);

        constexpr int kRead = 3;  // value operands read ahead
        u32x4 v[kRead];
#pragma unroll
        for (int i = 0; i < kRead - 1; ++i) v[i] = from_lds[i * kWave];
        uint32_t cv[8];
        u32x4 even, odd;
        float part = 0.f;
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            if (k + kRead - 1 < kSums) v[(k + kRead - 1) % kRead] = from_lds[(k + kRead - 1) * kWave];
            if (k < kSums) sum(k, v[k % kRead], w);
            if (k < kDots) dot(tt, k, n);
            const float e0 = __builtin_amdgcn_exp2f(__builtin_fmaf(sc[2 * k], c, -mc));
            const float e1 = __builtin_amdgcn_exp2f(__builtin_fmaf(sc[2 * k + 1], c, -mc));
            wn[k] = pack_bf16(e0, e1);
            part += e0 + e1;
            if (tt < kBytes) {
                cv[k] = convert(tt, k);
                if (k & 1) {
                    even[k / 2] = even_of(cv[k], cv[k - 1]);
                    odd[k / 2] = odd_of(cv[k], cv[k - 1]);
                }
            }
            __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
            __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
            __builtin_amdgcn_sched_group_barrier(0x002, 5, 0);
            __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
            __builtin_amdgcn_sched_group_barrier(0x002, 9, 0);
            __builtin_amdgcn_sched_barrier(0);
        }
        // this step's work: not to be put off to where it is used
        asm volatile("" : "+v"(n));
#pragma unroll
        for (int k = 0; k < 8; ++k) asm volatile("" : "+v"(wn[k]));
        l += part;
        if (tt < kBytes) put_values(tt, even, odd, values[(b + 1) & 1]);
        if (tt == kBytes - 1) load_values(b + 2);
        load_keys(b + 2, tt);
    };

    if (b_first < b_end) {
        // fill the pipeline: values of the first block, scores of its two tiles, weights of the first
        uint32_t wa[8], wb[8];
        f32x16 sa, sb;
        hide_values(b_first);
#pragma unroll
        for (int by = 0; by < kBytes; ++by) {
            u32x4 even, odd;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const uint32_t lo = convert(by, 2 * e), hi = convert(by, 2 * e + 1);
                even[e] = even_of(hi, lo);
                odd[e] = odd_of(hi, lo);
            }
            put_values(by, even, odd, values[b_first & 1]);
        }
        load_values(b_first + 1);
#pragma unroll
        for (int i = 0; i < kDots; ++i) dot(0, i, sa);
#pragma unroll
        for (int i = 0; i < kDots; ++i) dot(1, i, sb);
        load_keys(b_first + 1, 0);
        load_keys(b_first + 1, 1);
        hide(b_first, 0, sa);
        {
#pragma unroll
            for (int k = 0; k < 8; ++k) wa[k] = 0;
            raise(largest(sa), wa);
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
                lies.load(a.b, row, head, held, lane);
            }
            step(b, 0, wa, wb, sb, sa);
            step(b, 1, wb, wa, sa, sb);
            __syncthreads();
        } while (++b < b_end);
    }
    l = halves_sum(l);
    if (!real) return;
    const float inv = l != 0.f ? pow2(spare(cap)) / l : 0.f;
    uint16_t *out = a.out.p + t * a.out.ld + h * a.out.hd;
    // the lane's rows m = 8 i + 4 hh + j of every channel tile
#pragma unroll
    for (int i = 0; i < (D == 128 ? 2 : 1); ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            u32x4 w;
            if constexpr (D == 128) {  // unit column 8 i + 4 hh + j; channels 2 mt (rows below 16) and 2 mt + 1
#pragma unroll
                for (int mt = 0; mt < MT; ++mt) w[mt] = pack_bf16(o[mt][4 * i + j] * inv, o[mt][4 * (i + 2) + j] * inv);
            } else {  // unit column 4 hh + j; channels 4 mt + row / 8
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    w[k] = pack_bf16(o[k >> 1][4 * (2 * (k & 1)) + j] * inv, o[k >> 1][4 * (2 * (k & 1) + 1) + j] * inv);
            }
            *reinterpret_cast<u32x4 *>(out + (8 * i + 4 * hh + j) * 8) = w;
        }
    if (hh == 0 && a.lse) a.lse[t * a.ld_lse + h] = l != 0.f ? (__builtin_fmaf(top, c, off) + __builtin_amdgcn_logf(l)) * kLn2 : -INFINITY;
}

// The first `groups` workgroups walk the sequences of few rows, the others take the prompts: while the ones
// wait for memory the others multiply.  One of the former to a CU leaves room for the latter beside them: 64 sequences of
// up to 4000 tokens and a prompt of 2048, 32 and 8 heads, 86 us, with two to a CU 107 and in two launches
// 106; 16 of up to 60000 and a prompt of 600, 64 and 8 heads, 122, 129 and 142.
template <int D>
__global__ __launch_bounds__(kWaves *kWave, 2) void kv4_mixed_kernel(Kv4Attention a, Part<D> *parts, PartTag *tags,
                                                                     int groups, int tiles) {
    __shared__ union {
        Shared<D> sh;
        Values<D> values;
    } lds;
    if ((int)blockIdx.x < groups)
        decode<D, false>(a, parts, tags, lds.sh, blockIdx.x, groups);
    else
        prompt<D>(a, tiles, lds.values, (int)blockIdx.x - groups);
}

int device_cus() {
    static std::atomic<int> known[64];
    int dev = 0, cu = 0;
    if (hipGetDevice(&dev) != hipSuccess || dev < 0 || dev >= 64) {
        (void)hipGetLastError();
        return 256;
    }
    if ((cu = known[dev].load(std::memory_order_relaxed)) > 0) return cu;
    if (hipDeviceGetAttribute(&cu, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess || cu <= 0) {
        (void)hipGetLastError();
        return 256;
    }
    known[dev].store(cu, std::memory_order_relaxed);
    return cu;
}

template <int D>
size_t decode_workspace(int groups) {
    return (size_t)groups * 2 * (sizeof(Part<D>) + sizeof(PartTag));
}

// Few and short: a workgroup to each row tile (sequence s has none but its own of
// q_start[s] * group / rows + s on, so their number is bounded), nothing to join.
int64_t whole_tiles(int64_t T, int64_t S, int heads, int n_kv) { return (T * (heads / n_kv) / kRows + S) * n_kv; }
bool whole(int64_t tiles, int groups, int64_t room) {
    return tiles <= groups && room <= (4 * tiles < groups ? kWholeTokens : 4 * kWholeTokens);
}

template <int D>
hipError_t launch(Kv4Attention a, int64_t max_q, void *ws, hipStream_t st) {
    const int group = a.heads / a.b.f.n_kv;
    const int groups = device_cus() * kGroupsPerCu;
    // Without a workspace (kv4_attention_workspace) nothing may be split between workgroups.
    const int64_t row_tiles = whole_tiles(a.b.T, a.b.S, a.heads, a.b.f.n_kv);
    a.whole = whole(row_tiles, groups, (int64_t)a.b.cols * a.b.f.page);
    // Where no sequence has many rows, or all rows make few row tiles for the machine's waves, every sequence is
    // walked by row tiles, split over its keys; else each is taken as its own rows ask for.
    a.prompts = !a.whole && max_q * group > kDecodeRows && (int64_t)a.b.T * a.heads > (int64_t)groups * kWaves * kRows / kFewTiles;
    Part<D> *parts = (Part<D> *)ws;
    PartTag *tags = (PartTag *)(parts + 2 * (size_t)groups);
    if (a.prompts) {
        const int64_t tiles = (int64_t)a.b.T * group / kPromptRows + a.b.S;
        const int first = a.b.S > 1 ? groups / kGroupsPerCu : 0;  // a lone sequence is a prompt whatever its rows
        kv4_mixed_kernel<D><<<(unsigned)(first + tiles * a.b.f.n_kv), kWaves * kWave, 0, st>>>(a, parts, tags, first, (int)tiles);
        if (first) kv4_join_kernel<D><<<first, 256, 0, st>>>(a, parts, tags);
        return hipGetLastError();
    }
    const int grid = a.whole ? (int)row_tiles : groups;
    if (max_q * group <= kRows)
        kv4_decode_kernel<D, true><<<grid, kWaves * kWave, 0, st>>>(a, parts, tags);
    else
        kv4_decode_kernel<D, false><<<grid, kWaves * kWave, 0, st>>>(a, parts, tags);
    if (!a.whole) kv4_join_kernel<D><<<groups, 256, 0, st>>>(a, parts, tags);
    return hipGetLastError();
}

}  // namespace

size_t kv4_attention_workspace(int64_t T, int64_t S, int heads, int n_kv, int dim, int64_t room) {
    const int groups = device_cus() * kGroupsPerCu;
    if (whole(whole_tiles(T, S, heads, n_kv), groups, room)) return 0;
    return dim == 128 ? decode_workspace<128>(groups) : decode_workspace<64>(groups);
}

hipError_t launch_kv4_attention(const Kv4Attention &a, int64_t max_q, void *ws, hipStream_t st) {
    return a.b.f.dim == 128 ? launch<128>(a, max_q, ws, st) : launch<64>(a, max_q, ws, st);
}

}  // namespace nmk

// nm_kv8_select.hip -- which blocks of 64 cached tokens a row looks at.
//
// For a row (place p) and key/value head, over the blocks b <= p / 64 that have a page:
//     score_b = sum_h sum_c max(q_hc most_bc, q_hc least_bc) = sum_c (sum_h max(q_hc, 0)) most_bc + (sum_h min(q_hc, 0)) least_bc,
// h the query heads of the key/value head, most and least the bounds that the cache keeps of a block's keys: no key of
// the block has a larger sum of scores.  Taken are the first and the last blocks asked for and then those of the largest
// scores, of equal ones the lowest, `top` in all.
//
// The choice is that of scores in 64 bits (but for those closer than 2^-48), which are formed where they decide alone.  First all blocks get a
// score from the bf16 matrix instruction: sums of queries, as multiples of the power of two of the largest, are three bf16 pieces (24 bits), bounds
// are bf16 numbers, products are exact, sums are off by at most `slack`.  The `top`-th largest of these and the slack decide for all
// blocks but those next to it; if there are several of them and not all are taken, they get scores in 64 bits.
//
// Single rows: a workgroup takes a row and head, the three pieces are three columns of the instruction.  Many rows of a sequence: 16 rows a
// workgroup are its columns, and a block's bounds are read once for them.  One wave has the scores of up to 1024 blocks in registers
// and searches for the last one taken: it counts the scores at or above one after another that it interpolates between one with more above
// it and one with fewer, until as many are above as are asked for, without a barrier; behind more blocks a workgroup does the same, its counts meet
// in LDS.  What that leaves to scores in 64 bits is ranked directly, up to 64 blocks; more of them, as where many are alike, and rows whose queries
// are not finite go by the bits that keys differ in: one at a time by one wave (choose), 8 at a time by a workgroup (choose_among_many).
// Bound by the chain of reads (lengths, page, bounds) and of the choice's steps; by the bytes of the bounds, 2 D + 4 for every 128 D of keys
// and values, where there are rows enough for all compute units.  Traced, 8 heads: 16 rows to 64K tokens 20.7 us for 17 MB; one row of 32K 12.1;
// 512 rows of up to 264 blocks by sixteens 26.9 (in a graph 24.9; up to 256 blocks, of which a lane holds four and not eight, 21.8).
#include <atomic>

#include "nm_kv_rows.h"

namespace nmk {
namespace {

typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));

constexpr int kMaxWaves = 16;
constexpr int kFew = 64;          // candidates that one wave ranks
constexpr int kOneWave = 1024;    // blocks that one wave chooses from: 16 a lane
constexpr int kTileRows = 16;

template <int kCtrl>
__device__ __forceinline__ double lane_add(double v) {
    const int lo = __builtin_amdgcn_update_dpp(0, __double2loint(v), kCtrl, 0xF, 0xF, false);
    const int hi = __builtin_amdgcn_update_dpp(0, __double2hiint(v), kCtrl, 0xF, 0xF, false);
    return v + __hiloint2double(hi, lo);
}

// Over a wave; in all lanes.
template <bool OR>
__device__ __forceinline__ uint32_t wave_bits(uint32_t v) {
    auto op = [](uint32_t a, uint32_t b) { return OR ? a | b : a & b; };
    v = op(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0xB1, 0xF, 0xF, false));
    v = op(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x4E, 0xF, 0xF, false));
    v = op(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x141, 0xF, 0xF, false));
    v = op(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x140, 0xF, 0xF, false));
    const auto p = __builtin_amdgcn_permlane16_swap(v, v, false, false);
    v = op((uint32_t)p[0], (uint32_t)p[1]);
    const auto q = __builtin_amdgcn_permlane32_swap(v, v, false, false);
    return __builtin_amdgcn_readfirstlane((int)op((uint32_t)q[0], (uint32_t)q[1]));
}
template <bool OR>
__device__ __forceinline__ uint64_t wave_bits64(uint64_t v) {
    return (uint64_t)wave_bits<OR>((uint32_t)(v >> 32)) << 32 | wave_bits<OR>((uint32_t)v);
}

__device__ __forceinline__ uint32_t wave_max(uint32_t v) {
    auto op = [](uint32_t a, uint32_t b) { return max(a, b); };
    v = op(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0xB1, 0xF, 0xF, false));
    v = op(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x4E, 0xF, 0xF, false));
    v = op(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x141, 0xF, 0xF, false));
    v = op(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x140, 0xF, 0xF, false));
    const auto p = __builtin_amdgcn_permlane16_swap(v, v, false, false);
    v = op((uint32_t)p[0], (uint32_t)p[1]);
    const auto q = __builtin_amdgcn_permlane32_swap(v, v, false, false);
    return __builtin_amdgcn_readfirstlane((int)op((uint32_t)q[0], (uint32_t)q[1]));
}

__device__ __forceinline__ uint32_t wave_total(uint32_t v) {
    v += (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0xB1, 0xF, 0xF, false);
    v += (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x4E, 0xF, 0xF, false);
    v += (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x141, 0xF, 0xF, false);
    v += (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x140, 0xF, 0xF, false);
    const auto p = __builtin_amdgcn_permlane16_swap(v, v, false, false);
    v = (uint32_t)p[0] + (uint32_t)p[1];
    const auto q = __builtin_amdgcn_permlane32_swap(v, v, false, false);
    return __builtin_amdgcn_readfirstlane((int)((uint32_t)q[0] + (uint32_t)q[1]));
}

// A score as a whole number with the same order; 0 is none, kAsked a block that is taken in any case.  First scores
// are the upper half of a key, the lower half is 1.
constexpr uint64_t kAsked = ~0ull;
__device__ __forceinline__ uint64_t ordered(double v) {
    const uint64_t u = (uint64_t)__double_as_longlong(v + 0.0);
    return u ^ ((u >> 63) ? ~0ull : 1ull << 63);
}
__device__ __forceinline__ uint32_t ordered(float v) {
    const uint32_t u = __float_as_uint(v + 0.f);
    return u ^ ((u >> 31) ? ~0u : 1u << 31);
}
__device__ __forceinline__ float number(uint32_t u) { return __uint_as_float(u ^ ((u >> 31) ? 1u << 31 : ~0u)); }
constexpr uint64_t kAlike = 1ull << 63;  // every score of a row with queries that are not finite

// How far a first score may be off.  The sum of the magnitudes of its products is at most 448 times `size`, the sum of the magnitudes of the query
// sums.  Each of the eight instructions (dim 64: four) that multiply the first pieces is taken to cut its sum four times by a unit in the last place
// (2^-23): 2^-18.  Those of the second and the third pieces, 2^-8 and 2^-16 as large, cut as much of that less, whether they have columns of their own
// or, in a tile, go into the same sum, the smallest first; adding the columns is off by 2^-23: with them less than 2^-18 (1 + 2^-4) (2^-20.9 is
// the most that 80 million random sums were off).  Query sums of `group` heads may be off by group 2^-24; and whatever is below 2^-126.
__device__ __forceinline__ float slack(float size, int group, int scale) {
    return __builtin_ldexpf(__builtin_fmaf(size, 448.f * __builtin_fmaf((float)group, 0x1p-24f, 0x1.1p-18f), 0x1p-100f), scale - 127);
}

__device__ __forceinline__ float channel(const u32x4 &w, int i) { return i & 1 ? bf16_hi(w[i >> 1]) : bf16_lo(w[i >> 1]); }

// What a row asks for.
struct Ask {
    int n, mine, first, last;  // blocks up to its own that the table has; its own
    __device__ Ask(const Kv8Select &a, int place) : mine(place >> 6), first(a.first), last(a.last) {
        n = place < 0 ? 0 : (int)min((int64_t)mine + 1, (int64_t)a.b.cols * a.b.f.blocks());
    }
    __device__ bool asked(int block) const { return block < first || block > mine - last; }
};

// One wave, keys of n <= 64 R blocks.
template <int R>
__device__ __forceinline__ void choose(const uint64_t *key, int n, int top, int32_t *out, int lane) {
    uint64_t k[R], any = 0, all = ~0ull;
    int forced = 0, count = 0;
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const int i = r * 64 + lane;
        k[r] = i < n ? key[i] : 0ull;
        const bool asked = k[r] == kAsked, free = !asked && k[r] != 0;
        any |= free ? k[r] : 0ull;
        all &= free ? k[r] : ~0ull;
        forced += __popcll(__ballot(asked));
        count += __popcll(__ballot(free));
    }
    // Taken: keys of `from` and above, and of those equal to `tie` the first `ties`.
    int left = top - forced, ties = 0;
    uint64_t from = 1, tie = 0;
    auto above = [&](uint64_t c) {
        int m = -forced;
#pragma unroll
        for (int r = 0; r < R; ++r) m += __popcll(__ballot(k[r] >= c));
        return m;
    };
    if (left <= 0) {
        from = kAsked;
    } else if (count > left) {
        any = wave_bits64<true>(any);
        all = wave_bits64<false>(all);
        uint64_t pre = all;
        bool exact = false;
        if (any != all) {
            int d = 63 - __builtin_clzll(any ^ all);
            pre = d == 63 ? 0ull : all >> (d + 1) << (d + 1);
            for (; d >= 0 && !exact; --d) {
                const uint64_t c = pre | 1ull << d;
                const int m = above(c);
                if (m >= left) pre = c;
                exact = m == left;
            }
        }
        from = pre;
        if (!exact) {
            from = pre + 1;
            tie = pre;
            ties = left - above(from);
        }
    }
    int over = 0, on = 0;
    const uint64_t below = (1ull << lane) - 1;
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const bool is_over = k[r] >= from, is_on = ties > 0 && k[r] == tie;
        const uint64_t o = __ballot(is_over), e = __ballot(is_on);
        const int e_before = on + __popcll(e & below), to = over + __popcll(o & below) + min(e_before, ties);
        if ((is_over || (is_on && e_before < ties)) && to < top) out[to] = r * 64 + lane;
        over += __popcll(o);
        on += __popcll(e);
    }
    for (int i = over + min(on, ties) + lane; i < top; i += 64) out[i] = -1;
}

// Where one row's blocks lie and what is asked of them.
struct RowBlocks {
    const uint16_t *q;     // the first query head's channels
    int64_t hd;
    int group, head, per;
    const int32_t *table;
    const Kv8Batch *b;
    const double *sums;    // of positive, then of negative parts of the channels' queries; null: not kept
};

// Blocks that first scores do not decide about.
struct Doubts {
    int at[kFew];
    uint64_t key[kFew];
};

// Positive (or negative) parts of the queries of a head's group, summed: 16 channels from `from` on.
__device__ __forceinline__ void add_queries(double (&q)[16], const uint16_t *from, int64_t hd, int group, bool low) {
#pragma unroll
    for (int i = 0; i < 16; ++i) q[i] = 0.0;
    for (int h0 = 0; h0 < group; h0 += 4) {
        u32x4 w[4][2];
#pragma unroll
        for (int h = 0; h < 4; ++h)
#pragma unroll
            for (int i = 0; i < 2; ++i) w[h][i] = *reinterpret_cast<const u32x4 *>(from + (int64_t)min(h0 + h, group - 1) * hd + 8 * i);
#pragma unroll
        for (int h = 0; h < 4; ++h) {
            if (h0 + h >= group) break;
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const float x = channel(w[h][i >> 3], i & 7);
                q[i] += (double)(low ? fminf(x, 0.f) : fmaxf(x, 0.f));
            }
        }
    }
}

// Scores in 64 bits: a lane has 16 channels of the largest or the smallest keys, 16 lanes (dim 64: 8) a block.
template <int D>
struct Exact {
    static constexpr int kLanes = D / 8, kAtOnce = kWave / kLanes;
    double q[16];
    int part, sub;
    __device__ Exact(const RowBlocks &r, int lane) : part(lane % kLanes), sub(lane / kLanes) {
        const bool low = part >= D / 16;
        if (r.sums) {
#pragma unroll
            for (int i = 0; i < 16; ++i) q[i] = r.sums[part * 16 + i];
        } else {
            add_queries(q, r.q + (low ? part - D / 16 : part) * 16, r.hd, r.group, low);
        }
    }
    __device__ uint64_t key(const RowBlocks &r, int block) const {  // of a block that has a page; the same in all its lanes
        const Kv8Batch &b = *r.b;
        const uint8_t *p = b.cache + (int64_t)r.table[block / r.per] * b.f.page_bytes();
        const int at = r.head * r.per + (block & (r.per - 1));
        const u32x4 w = *reinterpret_cast<const u32x4 *>(p + b.f.bounds_at() + at * 2 * D + part * 16);
        const int scale = p[b.f.scales_at() + at * 4];
        double v = 0.0, v1 = 0.0;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const f32x2 x = __builtin_amdgcn_cvt_pk_f32_fp8((int)w[j], false), y = __builtin_amdgcn_cvt_pk_f32_fp8((int)w[j], true);
            v = __builtin_fma(q[4 * j], (double)x[0], v);
            v1 = __builtin_fma(q[4 * j + 1], (double)x[1], v1);
            v = __builtin_fma(q[4 * j + 2], (double)y[0], v);
            v1 = __builtin_fma(q[4 * j + 3], (double)y[1], v1);
        }
        v = lane_add<0x141>(lane_add<0x4E>(lane_add<0xB1>(v + v1)));
        if (D == 128) v = lane_add<0x140>(v);
        return ordered(__builtin_ldexp(v, scale - 127));
    }
};

// One wave: first scores of n <= 64 R blocks, 64 r + lane a lane's, 0 behind the last, `off` how far they may be off.  `key`: room for n.
template <int D, int R>
__device__ __forceinline__ void choose_first(const uint32_t (&k)[R], uint64_t *key, int n, int top, float off, const RowBlocks &rb, Doubts &few,
                                             int32_t *out, int lane) {
    uint32_t most = 0, least = ~0u;
    int forced = 0, count = 0;
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const bool asked = k[r] == ~0u, free = !asked && k[r] != 0;
        most = free ? max(most, k[r]) : most;
        least = free ? min(least, k[r]) : least;
        forced += __popcll(__ballot(asked));
        count += __popcll(__ballot(free));
    }
    auto from_on = [&](uint32_t c) {  // free blocks of key c and above
        int m = -forced;
#pragma unroll
        for (int r = 0; r < R; ++r) m += __popcll(__ballot(k[r] >= c));
        return m;
    };
    const int left = top - forced;
    uint32_t near = 1, sure = 1;  // above `sure`: taken; below `near`: not
    uint64_t taken = ~0ull;       // of those between, in their order
    if (left <= 0) {
        near = sure = ~0u;
    } else if (count > left) {
        // a key with as many at or above it as are left: between two with more and fewer, where it should lie if the logarithm of the
        // number above fell evenly, as it does at the upper end of most distributions; each fourth time halfway
        uint32_t lo = ~wave_max(~least), hi = wave_max(most) + 1;
        int above_lo = count, above_hi = 0;
        const float want = __builtin_amdgcn_logf((float)left + 0.25f);
        for (int turns = 1; above_lo != left && hi - lo > 1; ++turns) {
            uint32_t c = lo + (hi - lo) / 2;
            if (turns & 3) {
                const float a = number(lo), b = number(hi);
                const float la = __builtin_amdgcn_logf((float)above_lo + 0.5f), lb = __builtin_amdgcn_logf((float)above_hi + 0.5f);
                const float at = a + (b - a) * ((la - want) * __builtin_amdgcn_rcpf(la - lb));
                c = min(max((uint32_t)__builtin_amdgcn_readfirstlane((int)ordered(at)), lo + 1), hi - 1);
            }
            const int m = from_on(c);
            if (m >= left) {
                lo = c;
                above_lo = m;
            } else {
                hi = c;
                above_hi = m;
            }
        }
        if (above_lo == left) {  // the smallest of them: the left-th largest
            least = ~0u;
#pragma unroll
            for (int r = 0; r < R; ++r) least = k[r] >= lo ? min(least, k[r]) : least;
            lo = ~wave_max(~least);
        }
        const float t = number(lo);
        near = max(ordered(t - 2.f * off), 1u);  // in pages that were never written scores may be NaN: blocks without one stay out
        sure = min(ordered(t + 2.f * off), ~1u);
        const int some = from_on(near), sures = from_on(sure + 1), doubts = some - sures;
        if (some > left && doubts <= kFew) {  // one wave ranks them by scores in 64 bits
            int at = 0;
#pragma unroll
            for (int r = 0; r < R; ++r) {
                const bool doubt = k[r] >= near && k[r] <= sure;
                const uint64_t m = __ballot(doubt);
                if (doubt) few.at[at + __popcll(m & ((1ull << lane) - 1))] = r * 64 + lane;
                at += __popcll(m);
            }
            const Exact<D> exact(rb, lane);
            for (int i = 0; i < doubts; i += Exact<D>::kAtOnce) {
                const uint64_t x = exact.key(rb, few.at[min(i + exact.sub, doubts - 1)]);
                if (exact.part == 0 && i + exact.sub < doubts) few.key[i + exact.sub] = x;
            }
            const uint64_t x = lane < doubts ? few.key[lane] : 0ull;
            int ahead = 0;
            for (int j = 0; j < doubts; ++j) {
                const uint64_t y = (uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)(x >> 32), j) << 32 |
                                   (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)x, j);
                ahead += y > x || (y == x && j < lane);
            }
            taken = __ballot(lane < doubts && ahead < left - sures);
        } else if (some > left) {  // many, alike for instance: keys in 64 bits take their place
            bool doubt[R];
#pragma unroll
            for (int r = 0; r < R; ++r) {
                const int i = r * 64 + lane;
                doubt[r] = k[r] >= near && k[r] <= sure;
                if (i < n && !doubt[r]) key[i] = k[r] > sure ? kAsked : 0ull;
            }
            const Exact<D> exact(rb, lane);
#pragma unroll
            for (int r = 0; r < R; ++r) {
                const uint64_t all = __ballot(doubt[r]);
                uint64_t m = all;
                while (m) {  // kAtOnce of them
                    int mine = -1;
#pragma unroll
                    for (int s = 0; s < Exact<D>::kAtOnce; ++s) {
                        const int at = m ? __builtin_ctzll(m) : -1;
                        if (s == exact.sub) mine = at;
                        m &= m - 1;
                    }
                    const uint64_t x = exact.key(rb, r * 64 + (mine >= 0 ? mine : __builtin_ctzll(all)));
                    if (mine >= 0 && exact.part == 0) key[r * 64 + mine] = x;
                }
            }
            choose<R>(key, n, top, out, lane);
            return;
        }
    }
    int over = 0, at = 0;
    const uint64_t below = (1ull << lane) - 1;
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const bool doubt = k[r] >= near && k[r] <= sure;
        const uint64_t m = __ballot(doubt);
        const int place = at + __popcll(m & below);
        const bool is_over = k[r] > sure || (doubt && (place >= kFew || (taken >> place & 1)));
        const uint64_t o = __ballot(is_over);
        const int to = over + __popcll(o & below);
        if (is_over && to < top) out[to] = r * 64 + lane;
        over += __popcll(o);
        at += __popcll(m);
    }
    for (int i = over + lane; i < top; i += 64) out[i] = -1;
}

template <int D, int R>
__device__ __forceinline__ void choose_from(uint64_t *key, int n, int top, float off, const RowBlocks &rb, Doubts &few, int32_t *out, int lane) {
    uint32_t k[R];
#pragma unroll
    for (int r = 0; r < R; ++r) k[r] = r * 64 + lane < n ? (uint32_t)(key[r * 64 + lane] >> 32) : 0u;
    choose_first<D>(k, key, n, top, off, rb, few, out, lane);
}

template <int D>
__device__ __forceinline__ void choose_up_to_1024(uint64_t *key, int n, int top, float off, bool none, const RowBlocks &rb, Doubts &few,
                                                  int32_t *out, int lane) {
    if (none)
        choose<kOneWave / 64>(key, n, top, out, lane);
    else if (n <= 256)
        choose_from<D, 4>(key, n, top, off, rb, few, out, lane);
    else if (n <= 512)
        choose_from<D, 8>(key, n, top, off, rb, few, out, lane);
    else
        choose_from<D, kOneWave / 64>(key, n, top, off, rb, few, out, lane);
}

// ---- more blocks than one wave holds ----

struct Board {
    uint64_t any[kMaxWaves], all[kMaxWaves];
    int count[kMaxWaves], forced[kMaxWaves];
    int bins[256];
    int bin, above, inside;  // what the scan of the bins found
    int listed, sum[8];
    uint32_t least;
    uint64_t list[kFew];
    int at[kFew];
};

// The 8-bit pass over bits lo .. d of keys whose bits above d are `pre`.
struct Digits {
    int d, lo;
    uint64_t pre;
    __device__ bool of(uint64_t k) const { return k != 0 && k != kAsked && (d == 63 || k >> (d + 1) == pre); }
};

// How many keys there are, and the bits that they share.  The whole workgroup.
struct Survey {
    uint64_t any = 0, all = ~0ull;
    int count = 0, forced = 0;
    __device__ Survey(const uint64_t *key, int n, Board &sh) {
        const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), waves = blockDim.x >> 6;
        for (int i0 = 0; i0 < n; i0 += blockDim.x) {
            const uint64_t k = i0 + threadIdx.x < n ? key[i0 + threadIdx.x] : 0ull;
            const bool asked = k == kAsked, free = !asked && k != 0;
            any |= free ? k : 0ull;
            all &= free ? k : ~0ull;
            forced += __popcll(__ballot(asked));
            count += __popcll(__ballot(free));
        }
        any = wave_bits64<true>(any);
        all = wave_bits64<false>(all);
        if (lane == 0) {
            sh.any[wave] = any;
            sh.all[wave] = all;
            sh.count[wave] = count;
            sh.forced[wave] = forced;
        }
        __syncthreads();
        any = 0, all = ~0ull, count = 0, forced = 0;
        for (int w = 0; w < waves; ++w) {
            any |= sh.any[w];
            all &= sh.all[w];
            count += sh.count[w];
            forced += sh.forced[w];
        }
        __syncthreads();
    }
};

// Which bin of the pass the `left`-th largest of its keys is in, how many are in larger ones and in it.  The whole workgroup.
__device__ __forceinline__ void count_digits(const uint64_t *key, int n, int left, const Digits &g, Board &sh) {
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    for (int i = threadIdx.x; i < 256; i += blockDim.x) sh.bins[i] = 0;
    __syncthreads();
    for (int i = threadIdx.x; i < n; i += blockDim.x) {
        const uint64_t k = key[i];
        if (g.of(k)) atomicAdd(&sh.bins[(k >> g.lo) & ((2u << (g.d - g.lo)) - 1)], 1);
    }
    __syncthreads();
    if (wave == 0) {  // lane l has bins 255 - 4 l and the three below
        int own[4], sum = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            own[j] = sh.bins[255 - 4 * lane - j];
            sum += own[j];
        }
        int upto = sum;
        for (int m = 1; m < 64; m <<= 1) {
            const int o = __shfl_up(upto, m);
            if (lane >= m) upto += o;
        }
        int before = upto - sum;
        if (before < left && upto >= left) {
            int j = 0;
            while (before + own[j] < left) before += own[j++];
            sh.bin = 255 - 4 * lane - j;
            sh.above = before;
            sh.inside = own[j];
        }
    }
    __syncthreads();
}

// The whole workgroup.
__device__ __forceinline__ void choose_among_many(uint64_t *key, int n, int top, int32_t *out, Board &sh) {
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), waves = blockDim.x >> 6;
    if (threadIdx.x == 0) sh.listed = 0;
    const Survey v(key, n, sh);
    const uint64_t any = v.any, all = v.all;
    const int count = v.count, forced = v.forced;
    // Taken are keys above the border, and of those on it (k >> border == edge) the first `left`.
    int left = max(top - forced, 0), border = 0;
    uint64_t edge = 0;
    if (count <= left) {
        left = 0;  // all of them: 0 is none's alone
    } else if (left == 0) {
        edge = ~0ull;  // none of them
    } else if (any == all) {
        edge = any;
    } else {
        Digits g;
        g.d = 63 - __clzll((long long)(any ^ all));
        g.pre = g.d == 63 ? 0 : any >> (g.d + 1);
        for (;;) {
            g.lo = max(g.d - 7, 0);
            count_digits(key, n, left, g, sh);
            left -= sh.above;
            const int inside = sh.inside;
            g.pre = (g.d == 63 ? 0 : g.pre << (g.d - g.lo + 1)) | (uint64_t)sh.bin;
            border = g.lo;
            edge = g.pre;
            if (inside == left || g.lo == 0) break;
            g.d = g.lo - 1;
            if (inside <= kFew) {  // one wave ranks them
                for (int i = threadIdx.x; i < n; i += blockDim.x) {
                    const uint64_t k = key[i];
                    if (g.of(k)) {
                        const int to = atomicAdd(&sh.listed, 1);
                        sh.list[to] = k;
                        sh.at[to] = i;
                    }
                }
                __syncthreads();
                if (threadIdx.x < inside) {
                    const uint64_t k = sh.list[threadIdx.x];
                    const int i = sh.at[threadIdx.x];
                    int ahead = 0;
                    for (int j = 0; j < inside; ++j) ahead += sh.list[j] > k || (sh.list[j] == k && sh.at[j] < i);
                    key[i] = ahead < left ? kAsked : 0ull;
                }
                left = 0;
                __syncthreads();
                break;
            }
            __syncthreads();  // bins and what the scan found are used again
        }
    }

    // out in the order of the blocks
    int over = 0, on = 0;  // those before this round's
    for (int i0 = 0; i0 < n; i0 += blockDim.x) {
        const int i = i0 + threadIdx.x;
        const uint64_t k = i < n ? key[i] : 0;
        const uint64_t digits = k >> border;
        const bool is_over = k == kAsked || (k != 0 && digits > edge), is_on = k != 0 && k != kAsked && digits == edge;
        const uint64_t o = __ballot(is_over), e = __ballot(is_on), below = (1ull << lane) - 1;
        __syncthreads();  // counts are read before they are used again
        if (lane == 0) {
            sh.count[wave] = __popcll(o);
            sh.forced[wave] = __popcll(e);
        }
        __syncthreads();
        int o_before = over, e_before = on;
        for (int w = 0; w < waves; ++w) {
            if (w == wave) {
                o_before = over;
                e_before = on;
            }
            over += sh.count[w];
            on += sh.forced[w];
        }
        o_before += __popcll(o & below);
        e_before += __popcll(e & below);
        const int to = o_before + min(e_before, left);
        if ((is_over || (is_on && e_before < left)) && to < top) out[to] = i;
    }
    for (int i = over + min(on, left) + threadIdx.x; i < top; i += blockDim.x) out[i] = -1;
}

// The whole workgroup: first scores in `key`, `off` how far they may be off.  As choose_first, a key a thread and round; counts meet in LDS.
template <int D>
__device__ __forceinline__ void choose_together(uint64_t *key, int n, int top, float off, bool none, const RowBlocks &rb, Doubts &few, int32_t *out,
                                                Board &sh) {
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), waves = blockDim.x >> 6;
    uint32_t most = 0, least = ~0u;
    int forced = 0, count = 0;
    for (int i0 = 0; i0 < n; i0 += blockDim.x) {
        const uint32_t k = i0 + threadIdx.x < n ? (uint32_t)(key[i0 + threadIdx.x] >> 32) : 0u;
        const bool asked = k == ~0u, free = !asked && k != 0;
        most = free ? max(most, k) : most;
        least = free ? min(least, k) : least;
        forced += __popcll(__ballot(asked));
        count += __popcll(__ballot(free));
    }
    most = wave_max(most);
    least = ~wave_max(~least);
    if (lane == 0) {
        sh.any[wave] = (uint64_t)most << 32 | least;
        sh.all[wave] = (uint64_t)(uint32_t)forced << 32 | (uint32_t)count;
    }
    if (threadIdx.x < 8) sh.sum[threadIdx.x] = 0;
    if (threadIdx.x == 0) sh.least = ~0u;
    __syncthreads();
    {
        const uint64_t x = lane < waves ? sh.any[lane] : 0xFFFFFFFFull, y = lane < waves ? sh.all[lane] : 0ull;
        most = wave_max((uint32_t)(x >> 32));
        least = ~wave_max(~(uint32_t)x);
        forced = (int)wave_total((uint32_t)(y >> 32));
        count = (int)wave_total((uint32_t)y);
    }
    int turn = 0;
    auto round = [&](auto &&f) {  // of all keys
        for (int i0 = 0; i0 < n; i0 += blockDim.x) f(i0 + threadIdx.x < n ? (uint32_t)(key[i0 + threadIdx.x] >> 32) : 0u);
    };
    auto from_on = [&](uint32_t c) {  // free blocks of key c and above
        int m = 0;
        round([&](uint32_t k) { m += __popcll(__ballot(k >= c)); });
        if (lane == 0) atomicAdd(&sh.sum[turn & 3], m);
        if (threadIdx.x == 0) sh.sum[(turn + 2) & 3] = 0;  // the one after the next, which everyone has read
        __syncthreads();
        return sh.sum[turn++ & 3] - forced;
    };
    const int left = top - forced;
    if (!none && left > 0 && count > left) {
        uint32_t lo = least, hi = most + 1;
        int above_lo = count, above_hi = 0;
        const float want = __builtin_amdgcn_logf((float)left + 0.25f);
        for (int turns = 1; above_lo != left && hi - lo > 1; ++turns) {
            uint32_t c = lo + (hi - lo) / 2;
            if (turns & 3) {
                const float a = number(lo), b = number(hi);
                const float la = __builtin_amdgcn_logf((float)above_lo + 0.5f), lb = __builtin_amdgcn_logf((float)above_hi + 0.5f);
                const float at = a + (b - a) * ((la - want) * __builtin_amdgcn_rcpf(la - lb));
                c = min(max((uint32_t)__builtin_amdgcn_readfirstlane((int)ordered(at)), lo + 1), hi - 1);
            }
            const int m = __builtin_amdgcn_readfirstlane(from_on(c));
            if (m >= left) {
                lo = c;
                above_lo = m;
            } else {
                hi = c;
                above_hi = m;
            }
        }
        if (above_lo == left) {  // the smallest of them: the left-th largest
            uint32_t x = ~0u;
            round([&](uint32_t k) { x = k >= lo ? min(x, k) : x; });
            x = ~wave_max(~x);
            if (lane == 0) atomicMin(&sh.least, x);
            __syncthreads();
            lo = sh.least;
        }
        const float t = number(lo);
        const uint32_t near = max(ordered(t - 2.f * off), 1u), sure = min(ordered(t + 2.f * off), ~1u);  // above `sure`: taken; below `near`: not
        const int some = __builtin_amdgcn_readfirstlane(from_on(near)), sures = __builtin_amdgcn_readfirstlane(from_on(sure + 1));
        const int doubts = some - sures;
        const bool all = some == left, rank = !all && doubts <= kFew;
        if (threadIdx.x == 0) sh.listed = 0;
        __syncthreads();
        for (int i0 = wave * 64; i0 < n; i0 += waves * 64) {
            const int i = i0 + lane;
            const uint32_t k = i < n ? (uint32_t)(key[i] >> 32) : 0u;
            const bool doubt = k >= near && k <= sure && k != 0u && k != ~0u;
            if (i < n && !doubt) key[i] = k > sure ? kAsked : 0ull;
            if (doubt && all) key[i] = kAsked;
            if (doubt && rank) few.at[atomicAdd(&sh.listed, 1)] = i;
        }
        if (rank) {  // each wave's share in 64 bits, ranked by one
            __syncthreads();
            const int own = wave * Exact<D>::kAtOnce;
            if (own < doubts) {
                const Exact<D> exact(rb, lane);
                for (int i = own; i < doubts; i += waves * Exact<D>::kAtOnce) {
                    const uint64_t x = exact.key(rb, few.at[min(i + exact.sub, doubts - 1)]);
                    if (exact.part == 0 && i + exact.sub < doubts) few.key[i + exact.sub] = x;
                }
            }
            __syncthreads();
            if (wave == 0) {
                const uint64_t x = lane < doubts ? few.key[lane] : 0ull;
                const int i = lane < doubts ? few.at[lane] : 0;
                int ahead = 0;
                for (int j = 0; j < doubts; ++j) {
                    const uint64_t y = (uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)(x >> 32), j) << 32 |
                                       (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)x, j);
                    ahead += y > x || (y == x && __builtin_amdgcn_readlane(i, j) < i);
                }
                if (lane < doubts) key[i] = ahead < left - sures ? kAsked : 0ull;
            }
        } else if (!all) {  // many, alike for instance: keys in 64 bits take their place
            const Exact<D> exact(rb, lane);
            for (int i0 = wave * 64; i0 < n; i0 += waves * 64) {
                const uint64_t kept = i0 + lane < n ? key[i0 + lane] : 0ull;
                const uint64_t every = __ballot(kept != 0 && kept != kAsked);
                uint64_t m = every;
                while (m) {  // kAtOnce of them
                    int mine = -1;
#pragma unroll
                    for (int s = 0; s < Exact<D>::kAtOnce; ++s) {
                        const int at = m ? __builtin_ctzll(m) : -1;
                        if (s == exact.sub) mine = at;
                        m &= m - 1;
                    }
                    const uint64_t x = exact.key(rb, i0 + (mine >= 0 ? mine : __builtin_ctzll(every)));
                    if (mine >= 0 && exact.part == 0) key[i0 + mine] = x;
                }
            }
            __syncthreads();
            choose_among_many(key, n, top, out, sh);
            return;
        }
        __syncthreads();
    } else if (none) {
        __syncthreads();  // what was found above is read
        choose_among_many(key, n, top, out, sh);
        return;
    }
    // out in the order of the blocks: what is asked for by now, or all there are
    const bool every = count <= left;
    int before = 0;
    for (int i0 = 0; i0 < n; i0 += blockDim.x) {
        const int i = i0 + threadIdx.x;
        const uint64_t k = i < n ? key[i] : 0ull;
        const bool is = k == kAsked || (every && k != 0);
        const uint64_t m = __ballot(is);
        if (i0) __syncthreads();  // counts are read before they are used again
        if (lane == 0) sh.count[wave] = __popcll(m);
        __syncthreads();
        const int c = lane < waves ? sh.count[lane] : 0;
        const int to = before + (int)wave_total(lane < wave ? (uint32_t)c : 0u) + __popcll(m & ((1ull << lane) - 1));
        before += (int)wave_total((uint32_t)c);
        if (is && to < top) out[to] = i;
    }
    for (int i = before + threadIdx.x; i < top; i += blockDim.x) out[i] = -1;
}

// Up to 1024 blocks one wave is faster than all of them (512 blocks, 8 rows and heads: 13.4 us a call against 17.6).
template <int D, int CAP>
__device__ __forceinline__ void choose_any(uint64_t *key, int n, int top, float off, bool none, const RowBlocks &rb, Doubts &few, int32_t *out) {
    if (n <= kOneWave) {
        if (threadIdx.x < kWave) choose_up_to_1024<D>(key, n, top, off, none, rb, few, out, (int)threadIdx.x);
    } else if constexpr (CAP > kOneWave) {
        __shared__ Board board;
        choose_together<D>(key, n, top, off, none, rb, few, out, board);
    }
}

// ---- first scores ----

// The bounds of a block as 8 bf16 operands: lane (col, g) has numbers 64 i + 16 g .. of the 2 D for operands 2 i and 2 i + 1.
union Operand {
    uint32_t w[4];
    bf16x8 h;
    u32x4 u;
};
__device__ __forceinline__ uint32_t fp8_pair(uint32_t w, bool high) {
    union { bf16x2 h; uint32_t u; } c;
    c.h = high ? __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, 1.f, true) : __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, 1.f, false);
    return c.u;
}
__device__ __forceinline__ bf16x8 eight(uint32_t a, uint32_t b) {
    Operand x;
    x.w[0] = fp8_pair(a, false);
    x.w[1] = fp8_pair(a, true);
    x.w[2] = fp8_pair(b, false);
    x.w[3] = fp8_pair(b, true);
    return x.h;
}

// A sum of queries, between -2 and 2, as three bf16 pieces: 24 bits.
__device__ __forceinline__ void split(double x, uint32_t (&piece)[3]) {
#pragma unroll
    for (int i = 0; i < 3; ++i) {
        piece[i] = f32_to_bf16_rne((float)x);
        x -= (double)__uint_as_float(piece[i] << 16);
    }
}
// What brings the largest of some sums, of which the upper word is given, to between 1 and 2.
__device__ __forceinline__ int to_one(uint32_t top) { return 1023 - (int)(top >> 20); }
constexpr uint32_t kNotFinite = 0x7FF00000u;  // upper word of what is not

// What the first of two launches leaves for the second: a row's first scores, 0 for none and ~0 for a block that is taken in any
// case, the largest scale byte of each of its parts and how large its query sums are (NaN: not finite).
struct Left {
    uint32_t *key;      // [items][parts * kPart]
    uint32_t *largest;  // [items][parts]
    float *size;        // [items]
    int parts;
};
constexpr int kPart = 256;

// SPLIT: a workgroup takes kPart of a row's blocks and leaves their scores.
template <int D, int CAP, bool SPLIT>
__global__ __launch_bounds__(SPLIT ? kPart : kMaxWaves *kWave) void kv8_select_kernel(Kv8Select a, Left to) {
    __shared__ uint64_t key[CAP];
    __shared__ uint16_t pieces[4][2 * D];  // the last of zeros: for the columns behind the third
    __shared__ uint32_t tops[kMaxWaves], scales[kMaxWaves];
    __shared__ float sizes[kMaxWaves];
    __shared__ double sums[2 * D];
    __shared__ Doubts few;
    a.b.f.dim = D;
    const Kv8Batch &b = a.b;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), waves = blockDim.x >> 6;
    const int col = lane & 15, g = lane >> 4;
    const int n_kv = b.f.n_kv, group = a.heads / n_kv;
    // the heads of a row to one XCD: their bounds lie side by side, and their scales in one cache line
    const int item = SPLIT ? blockIdx.x / to.parts : by_xcd(blockIdx.x, gridDim.x), part = SPLIT ? blockIdx.x - item * to.parts : 0;
    const int t = item / n_kv, head = item - t * n_kv;

    // sums of the positive and of the negative parts of a channel's queries, a thread each
    const uint16_t *queries = a.q.p + (int64_t)t * a.q.ld + (int64_t)head * group * a.q.hd;
    double sum = 0.0;
    uint32_t top = 0;
    const bool mine = threadIdx.x < 2 * D;
    if (mine) {
        const uint16_t *p = queries + threadIdx.x % D;
        for (int h0 = 0; h0 < group; h0 += 8) {
            uint32_t x[8];
#pragma unroll
            for (int h = 0; h < 8; ++h) x[h] = p[(int64_t)min(h0 + h, group - 1) * a.q.hd];
#pragma unroll
            for (int h = 0; h < 8; ++h) {
                const float f = __uint_as_float(x[h] << 16);
                if ((x[h] & 0x7F80u) == 0x7F80u) top = kNotFinite;
                if (h0 + h < group) sum += (double)(threadIdx.x < D ? fmaxf(f, 0.f) : fminf(f, 0.f));
            }
        }
        top = max(top, (uint32_t)__double2hiint(sum) & 0x7FFFFFFFu);
        sums[threadIdx.x] = sum;
    }
    const RowSeq seq(b, t, lane);
    if (t < seq.q0 || t >= seq.q1) return;
    const Ask ask(a, seq.len - seq.q1 + t);
    const int per = b.f.blocks(), n = SPLIT ? min(ask.n, (part + 1) * kPart) : ask.n, begin = part * (kPart / 16);  // blocks, tiles
    if (SPLIT && part > 0 && n <= part * kPart) return;
    const RowBlocks rb = {queries, a.q.hd, group, head, per, b.table + (int64_t)seq.s * b.ld_table, &b, sums};

    // the first 64 blocks of a wave, 16 a tile: tile wave + waves * i is i's 16 lanes'
    auto block_of = [&](int tile0) { return (tile0 + g * waves) * 16 + col; };
    auto look = [&](int tile0) { return n > 0 ? rb.table[min(block_of(tile0), n - 1) / per] : -1; };
    int page = look(begin + wave);
    top = wave_max(top);
    if (lane == 0) tops[wave] = top;
    __syncthreads();
    top = 0;
    for (int w = 0; w < min(waves, 2 * D / kWave); ++w) top = max(top, tops[w]);
    const bool none = top >= kNotFinite;
    float size = 0.f;
    if (mine) {
        const double x = none ? 0.0 : __builtin_ldexp(sum, to_one(top));
        uint32_t piece[3];
        split(x, piece);
#pragma unroll
        for (int i = 0; i < 3; ++i) pieces[i][threadIdx.x] = (uint16_t)piece[i];
        pieces[3][threadIdx.x] = 0;
        size = (float)(x < 0.0 ? -x : x);
    }
    size = wave_sum(size);
    if (lane == 0) sizes[wave] = size;
    __syncthreads();
    size = 0.f;
    for (int w = 0; w < min(waves, 2 * D / kWave); ++w) size += sizes[w];
    Operand q[D / 16];
#pragma unroll
    for (int i = 0; i < D / 16; ++i) q[i].u = *reinterpret_cast<const u32x4 *>(&pieces[min(col, 3)][64 * (i >> 1) + 16 * g + 8 * (i & 1)]);

    uint32_t largest = 0;
    for (int tile0 = begin + wave; tile0 * 16 < n; tile0 += 4 * waves) {
        const int own = block_of(tile0), k = min(own, n - 1);
        const bool ok = page >= 0 && page < b.num_pages;
        const int at = head * per + (k & (per - 1));
        const uint8_t *p = b.cache + (int64_t)(ok ? page : 0) * b.f.page_bytes();
        const int scale = p[b.f.scales_at() + at * 4];
        const uint64_t bounds = (uint64_t)(uintptr_t)(p + b.f.bounds_at() + at * 2 * D);
        page = look(tile0 + 4 * waves);
        float score = 0.f;
        u32x4 w[D / 32], ahead[D / 32];
        auto load = [&](int i) {
            const uint32_t lo = (uint32_t)__shfl((int)(uint32_t)bounds, i * 16 + col), hi = (uint32_t)__shfl((int)(uint32_t)(bounds >> 32), i * 16 + col);
            const u32x4 *from = reinterpret_cast<const u32x4 *>((uintptr_t)((uint64_t)hi << 32 | lo) + 16 * g);
#pragma unroll
            for (int j = 0; j < D / 32; ++j) ahead[j] = from[4 * j];
        };
        const int tiles = min(4, ((n + 15) / 16 - tile0 + waves - 1) / waves);
        load(0);
        // Not unrolled: the code is run once, and read from memory (512 blocks, 8 heads: 4.6 -> 2.3 us).
#pragma unroll 1
        for (int i = 0; i < tiles; ++i) {
#pragma unroll
            for (int j = 0; j < D / 32; ++j) w[j] = ahead[j];
            load(min(i + 1, 3));
            f32x4 acc = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int j = 0; j < D / 16; ++j)
                acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(eight(w[j >> 1][2 * (j & 1)], w[j >> 1][2 * (j & 1) + 1]), q[j].h, acc, 0, 0, 0);
            // row 4 g + r of the tile in columns 0 .. 2, column 3 is 0: the quad's sum, kept by the lane that has the block
#pragma unroll
            for (int r = 0; r < 4; ++r) acc[r] = dpp_add<0x4E>(dpp_add<0xB1>(acc[r]));
            const int from = (col >> 2) * 16;  // block col of the tile: row col % 4 of lane group col / 4
            float v[4];
#pragma unroll
            for (int r = 0; r < 4; ++r) v[r] = __shfl(acc[r], from);  // by all lanes
            const float even = col & 2 ? v[2] : v[0], odd = col & 2 ? v[3] : v[1];
            score = g == i ? (col & 1 ? odd : even) : score;
        }
        if (own < n) {
            const uint32_t first = ordered(__builtin_ldexpf(score, scale - 127));
            if (SPLIT)
                to.key[((int64_t)item * to.parts * kPart) + own] = !ok ? 0u : ask.asked(own) ? ~0u : first;
            else
                key[own] = !ok ? 0ull : ask.asked(own) ? kAsked : none ? kAlike : (uint64_t)first << 32 | 1;
            if (ok) largest = max(largest, (uint32_t)scale);
        }
    }
    largest = wave_max(largest);
    if (lane == 0) scales[wave] = largest;
    __syncthreads();
    largest = wave_max(lane < waves ? scales[lane] : 0u);
    if constexpr (SPLIT) {
        if (threadIdx.x == 0) {
            to.largest[(int64_t)item * to.parts + part] = largest;
            if (part == 0) to.size[item] = none ? NAN : size;
        }
    } else {
        int32_t *out = a.out + (int64_t)t * a.ld_out + (int64_t)head * a.top;
        choose_any<D, CAP>(key, n, a.top, slack(size, group, (int)largest), none, rb, few, out);
    }
}

// The second of two launches: a workgroup to each row and head.
template <int D, int CAP>
__global__ __launch_bounds__(kMaxWaves *kWave) void kv8_choose_kernel(Kv8Select a, Left from) {
    __shared__ uint64_t key[CAP];
    __shared__ Doubts few;
    a.b.f.dim = D;
    const Kv8Batch &b = a.b;
    const int lane = threadIdx.x & 63;
    const int n_kv = b.f.n_kv, group = a.heads / n_kv;
    const int item = blockIdx.x, t = item / n_kv, head = item - t * n_kv;
    const float size = from.size[item];
    uint32_t largest = lane < from.parts ? from.largest[(int64_t)item * from.parts + lane] : 0u;  // at most 64 parts
    const RowSeq seq(b, t, lane);
    if (t < seq.q0 || t >= seq.q1) return;
    const Ask ask(a, seq.len - seq.q1 + t);
    const int n = ask.n;
    const bool none = size != size;
    if (lane * kPart >= n) largest = 0;
    const float off = slack(size, group, (int)wave_max(largest));
    const uint32_t *scores = from.key + (int64_t)item * from.parts * kPart;
    for (int i = threadIdx.x; i < n; i += blockDim.x) {
        const uint32_t x = scores[i];
        key[i] = x == 0 ? 0ull : x == ~0u ? kAsked : none ? kAlike : (uint64_t)x << 32 | 1;
    }
    __syncthreads();
    const RowBlocks rb = {a.q.p + (int64_t)t * a.q.ld + (int64_t)head * group * a.q.hd, a.q.hd, group, head, b.f.blocks(),
                          b.table + (int64_t)seq.s * b.ld_table, &b, nullptr};
    choose_any<D, CAP>(key, n, a.top, off, none, rb, few, a.out + (int64_t)t * a.ld_out + (int64_t)head * a.top);
}

// ---- sixteen rows of a sequence and a head ----

constexpr int kTileWaves = 8;  // two rows' choices a wave (with 16 waves registers spill: 512 rows behind 16K tokens 29 us in a graph, not 25)

// What the rows of a tile keep in LDS before their keys.
template <int D>
struct TileShared {
    uint16_t pieces[3][kTileRows][2 * D + 8];  // rows on different banks
    float size[kTileRows];
    int none[kTileRows];
    uint32_t scales[kTileWaves];
    Doubts few[kTileWaves];
};

// Sequence s owns the tiles from q_start[s] / 16 + s on.  The columns of the matrix instruction are rows.
template <int D>
__global__ __launch_bounds__(kTileWaves *kWave) void kv8_select_tile_kernel(Kv8Select a, int room) {
    extern __shared__ uint64_t keys[];  // [kTileRows][room]
    __shared__ TileShared<D> sh;
    a.b.f.dim = D;
    const Kv8Batch &b = a.b;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int col = lane & 15, g = lane >> 4;
    const int n_kv = b.f.n_kv, group = a.heads / n_kv;
    const int vt = blockIdx.x / n_kv, head = blockIdx.x - vt * n_kv;
    int s = 0;
    for (int n = b.S; n > 1;) {  // the last s whose first tile is at or before vt, 64 looks at a time
        const int step = (n + 63) >> 6, at = s + lane * step;
        const bool yes = lane * step < n && b.q_start[at] / kTileRows + at <= vt;
        const uint64_t m = __ballot(yes);
        s += (m ? 63 - __clzll((long long)m) : 0) * step;
        n = min(step, b.S - s);
    }
    s = __builtin_amdgcn_readfirstlane(s);
    const int q0 = b.q_start[s], q1 = b.q_start[s + 1], len = b.kv_len[s];
    const int t0 = q0 + (vt - q0 / kTileRows - s) * kTileRows;
    const int rows = min(min(q1, b.T) - t0, kTileRows);
    if (t0 < q0 || rows <= 0) return;
    const int place0 = len - q1 + t0;
    const int per = b.f.blocks();
    RowBlocks rb = {a.q.p + (int64_t)t0 * a.q.ld + (int64_t)head * group * a.q.hd, a.q.hd, group, head, per, b.table + (int64_t)s * b.ld_table, &b, nullptr};

    // Sums of queries, 16 threads (or 8) a row, 8 channels each, positive parts and negative ones: in fp32, of the power of two of the
    // row's largest query, which costs first scores group 2^-24 more (in 64 bits this took 3.9 us of a tile's 17).
    const int row = threadIdx.x >> 4, c8 = threadIdx.x & 15;
    if (row < kTileRows) {  // whole waves
        const bool mine = c8 < D / 8 && row < rows;
        const uint16_t *p = rb.q + (int64_t)min(row, rows - 1) * a.q.ld + min(c8, D / 8 - 1) * 8;
        auto heads = [&](auto &&f) {  // four loads at once
            for (int h0 = 0; h0 < group; h0 += 4) {
                u32x4 w[4];
#pragma unroll
                for (int h = 0; h < 4; ++h) w[h] = *reinterpret_cast<const u32x4 *>(p + (int64_t)min(h0 + h, group - 1) * a.q.hd);
#pragma unroll
                for (int h = 0; h < 4; ++h)
                    if (h0 + h < group) f(w[h]);
            }
        };
        u16x2 most = {0, 0};
        heads([&](const u32x4 &w) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                union { uint32_t u; u16x2 h; } x;
                x.u = w[i] & 0x7FFF7FFFu;
                most = __builtin_elementwise_max(most, x.h);
            }
        });
        uint32_t top = mine ? max(most[0], most[1]) : 0;
#define NM_KV8_ROW_MAX(C) top = max(top, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)top, C, 0xF, 0xF, false))
        NM_KV8_ROW_MAX(0xB1);
        NM_KV8_ROW_MAX(0x4E);
        NM_KV8_ROW_MAX(0x141);
        NM_KV8_ROW_MAX(0x140);
#undef NM_KV8_ROW_MAX
        const bool none = top >= 0x7F80u;
        const int down = none || !mine ? -1000 : 127 - (int)(top >> 7);  // zeros for what is not finite or not there
        float sum[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) sum[i] = 0.f;
        heads([&](const u32x4 &w) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float x = none ? 0.f : __builtin_ldexpf(channel(w, i), down);
                sum[i] += fmaxf(x, 0.f);
                sum[8 + i] += fminf(x, 0.f);
            }
        });
        float size = 0.f;
#pragma unroll
        for (int i = 0; i < 16; ++i) size += fabsf(sum[i]);
        size = dpp_add<0x140>(dpp_add<0x141>(dpp_add<0x4E>(dpp_add<0xB1>(size))));
#pragma unroll
        for (int k = 0; k < 3; ++k)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                u32x4 w;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    float &lo = sum[8 * i + 2 * e], &hi = sum[8 * i + 2 * e + 1];
                    union { bf16x2 h; uint32_t u; } x;
                    x.h = __builtin_convertvector((f32x2){lo, hi}, bf16x2);
                    w[e] = x.u;
                    lo -= bf16_lo(x.u);
                    hi -= bf16_hi(x.u);
                }
                if (c8 < D / 8) *reinterpret_cast<u32x4 *>(&sh.pieces[k][row][i * D + c8 * 8]) = w;
            }
        if (c8 == 0) {
            sh.size[row] = size;
            sh.none[row] = none;
        }
    }
    __syncthreads();
    Operand q[3][D / 16];
#pragma unroll
    for (int k = 0; k < 3; ++k)
#pragma unroll
        for (int i = 0; i < D / 16; ++i)
            q[k][i].u = *reinterpret_cast<const u32x4 *>(&sh.pieces[k][col][64 * (i >> 1) + 16 * g + 8 * (i & 1)]);
    const bool none = sh.none[col];
    const Ask mine(a, place0 + col), most(a, place0 + rows - 1);
    auto look = [&](int base) { return most.n > 0 ? rb.table[min(base + col, most.n - 1) / per] : -1; };
    int page = look(wave * 16);
    uint32_t largest = 0;
    for (int base = wave * 16; base < most.n; base += kTileWaves * 16) {
        const int k = min(base + col, most.n - 1);
        const bool ok = page >= 0 && page < b.num_pages;
        const int at = head * per + (k & (per - 1));
        const uint8_t *p = b.cache + (int64_t)(ok ? page : 0) * b.f.page_bytes();
        page = look(base + kTileWaves * 16);
        const u32x4 *from = reinterpret_cast<const u32x4 *>(p + b.f.bounds_at() + at * 2 * D + 16 * g);
        u32x4 w[D / 32];
#pragma unroll
        for (int i = 0; i < D / 32; ++i) w[i] = from[4 * i];
        const int scale = p[b.f.scales_at() + at * 4] | (ok ? 0 : 256);
        f32x4 acc = {0.f, 0.f, 0.f, 0.f};
        bf16x8 x[D / 16];
#pragma unroll
        for (int i = 0; i < D / 16; ++i) x[i] = eight(w[i >> 1][2 * (i & 1)], w[i >> 1][2 * (i & 1) + 1]);
#pragma unroll
        for (int k = 2; k >= 0; --k)
#pragma unroll
            for (int i = 0; i < D / 16; ++i) acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(x[i], q[k][i].h, acc, 0, 0, 0);
#pragma unroll
        for (int r = 0; r < 4; ++r) {  // block base + 4 g + r, row col
            const int block = base + 4 * g + r, sc = __shfl(scale, 4 * g + r);
            if (col < rows && block < mine.n)
                keys[col * room + block] = sc >= 256 ? 0ull : mine.asked(block) ? kAsked : none ? kAlike : (uint64_t)ordered(__builtin_ldexpf(acc[r], sc - 127)) << 32 | 1;
        }
        largest = max(largest, (uint32_t)scale & 255u);
    }
    largest = wave_max(largest);
    if (lane == 0) sh.scales[wave] = largest;
    __syncthreads();
    largest = wave_max(lane < kTileWaves ? sh.scales[lane] : 0u);
    for (int r = wave; r < rows; r += kTileWaves) {
        const Ask ask(a, place0 + r);
        rb.q = a.q.p + (int64_t)(t0 + r) * a.q.ld + (int64_t)head * group * a.q.hd;
        choose_up_to_1024<D>(keys + r * room, ask.n, a.top, slack(sh.size[r], group, (int)largest), sh.none[r], rb, sh.few[wave],
                             a.out + (int64_t)(t0 + r) * a.ld_out + (int64_t)head * a.top, lane);
    }
}

// Few rows behind long contexts: one compute unit reads bounds at about 30 GB/s, so their blocks go to many and the choice to a second launch.
constexpr int kFewItems = 512, kSplitBlocks = 2048;
bool split(int64_t items, int64_t room) { return items <= kFewItems && room > kSplitBlocks; }

// Sixteen rows a workgroup where there are that many of a sequence and more choices than the machine makes side by side.  By single rows
// and by tiles in a graph, 8 heads: 16 sequences of 5 rows behind 16K tokens 13.1 and 16.6 us, of 16 (2048 choices) 19.6 and 20.4, of 24 26.9 and
// 21.2; a lone one's 128 rows 16.6 and 20.8, 512 rows 44.1 and 22.5; 64 sequences of 12 rows behind 8K 34.0 and 37.1, of 16 43.7 and 40.8.
constexpr int kTileItems = 2048;
bool by_tiles(int64_t T, int64_t S, int64_t items, int64_t room) { return room <= kOneWave && T >= kTileRows * S && items > kTileItems; }

// Dynamic LDS beyond 64 KB has to be asked for, once a device: for the widest table, so that calls of other host threads need no less.
template <int D>
hipError_t allow_tile_lds(size_t bytes) {
    static std::atomic<uint64_t> done{0};
    if (bytes + sizeof(TileShared<D>) <= 64 * 1024) return hipSuccess;
    int dev = 0;
    hipError_t e = hipGetDevice(&dev);
    if (e != hipSuccess) return e;
    const uint64_t bit = 1ull << (dev & 63);
    if (done.load(std::memory_order_acquire) & bit) return hipSuccess;
    e = hipFuncSetAttribute((const void *)kv8_select_tile_kernel<D>, hipFuncAttributeMaxDynamicSharedMemorySize,
                            kTileRows * kOneWave * (int)sizeof(uint64_t));
    if (e == hipSuccess) done.fetch_or(bit, std::memory_order_acq_rel);
    return e;
}

template <int D>
hipError_t launch(const Kv8Select &a, void *ws, hipStream_t st) {
    const int64_t room = (int64_t)a.b.cols * a.b.f.blocks();
    const int64_t items = (int64_t)a.b.T * a.b.f.n_kv;
    if (by_tiles(a.b.T, a.b.S, items, room)) {
        const int64_t tiles = a.b.T / kTileRows + a.b.S;
        const size_t lds = (size_t)kTileRows * room * sizeof(uint64_t);
        const hipError_t e = allow_tile_lds<D>(lds);
        if (e != hipSuccess) return e;
        kv8_select_tile_kernel<D><<<(unsigned)(tiles * a.b.f.n_kv), kTileWaves * kWave, lds, st>>>(a, (int)room);
        return hipGetLastError();
    }
    Left left = {};
    if (split(items, room)) {
        left.parts = (int)((room + kPart - 1) / kPart);
        left.key = (uint32_t *)ws;
        left.largest = left.key + items * left.parts * kPart;
        left.size = (float *)(left.largest + items * left.parts);
        kv8_select_kernel<D, 1, true><<<(unsigned)(items * left.parts), kPart, 0, st>>>(a, left);
        kv8_choose_kernel<D, kMaxSelectBlocks><<<(unsigned)items, kMaxWaves * kWave, 0, st>>>(a, left);
        return hipGetLastError();
    }
    // more waves to a row where there are few rows and blocks enough (48 rows and 8 heads of up to 128 blocks: 24.8 us with 16 waves, 9.7 with 4)
    const dim3 block((items <= kFewItems && room > 256 ? kMaxWaves : 4) * kWave);
    if (room <= kOneWave)
        kv8_select_kernel<D, kOneWave, false><<<(unsigned)items, block, 0, st>>>(a, left);
    else if (room <= 4 * kOneWave)
        kv8_select_kernel<D, 4 * kOneWave, false><<<(unsigned)items, block, 0, st>>>(a, left);
    else
        kv8_select_kernel<D, kMaxSelectBlocks, false><<<(unsigned)items, block, 0, st>>>(a, left);
    return hipGetLastError();
}

}  // namespace

size_t kv8_select_workspace(int64_t T, int64_t S, int n_kv, int64_t blocks) {
    const int64_t items = T * n_kv, parts = (blocks + kPart - 1) / kPart;
    if (!split(items, blocks)) return 0;
    return (size_t)(items * (parts * kPart + parts + 1)) * sizeof(uint32_t);
}

hipError_t launch_kv8_select(const Kv8Select &a, void *ws, hipStream_t st) {
    return a.b.f.dim == 128 ? launch<128>(a, ws, st) : launch<64>(a, ws, st);
}

}  // namespace nmk

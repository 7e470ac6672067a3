// nm_kv8.hip -- tokens into the 8-bit key/value cache, keys and queries rotated by their places on the way, and back.
//
// A block of 64 tokens of one head has one scale for its keys and one for its values:
//     byte = clamp(E(amax) - 8 + (significand(amax) > 1.75), 63, 182),  x ~ e4m3 * 2^(byte - 127),
// E the biased exponent of the largest magnitude, which lands in (224, 448], 448 the largest E4M3 number.  A scale never
// shrinks while tokens of the block are there: new tokens that need a larger one have the earlier ones
// rounded again to it, which is exact but for numbers that become subnormal.  The ends 63 and 182 keep magnitudes below 2^64, so that
// sums over any number of keys and values stay in range.  Rotated keys and queries are products and one sum in 64 bits, rounded once.
//
// A workgroup takes one block and head: the block's largest magnitude has to be known before any of it is stored, and
// then everything it stores is in its registers.  Keys: a thread has 16 channels of one token (two runs of 8 where the pairs
// of the rotation lie half the rotated channels apart); values: a thread has two channels of 16 tokens (D = 64: of 8), whole 16-byte
// units of the cache.  Memory-bound for prompts (3 of 4K rows, 32 / 8 heads of 128: 275 MB past the L2s in 59 to 64 us), a chain of dependent reads
// (lengths, page, scales) for single tokens (48 of them 7.0 us).
#include "nm_kv_rows.h"

namespace nmk {
namespace {

constexpr int kThreads = 256;
constexpr int kLow = 63, kHigh = 182;  // scale bytes
constexpr uint32_t kNaN8 = 0x7F;
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

__device__ __forceinline__ float pow2_byte(uint32_t byte) { return __uint_as_float(byte << 23); }

// fp64 -> fp32 cut after 20 bits of fraction, the last of them set where something is lost: rounding that to fewer
// bits gives what rounding the 64 bits would.
__device__ __forceinline__ float narrowed(double d) {
    const uint32_t lo = (uint32_t)__double2loint(d), hi = (uint32_t)__double2hiint(d);
    return (float)__hiloint2double((int)(hi | (lo != 0u)), 0);
}

__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
    union { bf16x2 h; uint32_t u; } c;
    c.h = __builtin_convertvector((f32x2){a, b}, bf16x2);
    return c.u;
}

__device__ __forceinline__ int scale_byte(uint32_t top) {  // bits of the largest magnitude, fp32
    return min(max((int)(top >> 23) - 8 + ((top & 0x7FFFFFu) > 0x600000u ? 1 : 0), kLow), kHigh);
}

// Two numbers times s -> two E4M3 codes in the low or the high half of `old`.
template <bool HIGH>
__device__ __forceinline__ uint32_t codes(float a, float b, float s, uint32_t old) {
    a = __builtin_amdgcn_fmed3f(a * s, -448.f, 448.f);
    b = __builtin_amdgcn_fmed3f(b * s, -448.f, 448.f);
    return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(a, b, (int)old, HIGH);
}

// Four codes rounded again, as s times what they are.
__device__ __forceinline__ uint32_t again(uint32_t w, float s) {
    const f32x2 a = __builtin_amdgcn_cvt_pk_f32_fp8((int)w, false), b = __builtin_amdgcn_cvt_pk_f32_fp8((int)w, true);
    uint32_t r = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(a[0] * s, a[1] * s, 0, false);
    r = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(b[0] * s, b[1] * s, (int)r, true);
    return r & ~(((r & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u);  // the conversions may give a NaN either sign: kept as 0x7F
}

__device__ __forceinline__ uint32_t wave_max(uint32_t m) {
#define NM_KV8_MAX(C) m = max(m, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)m, C, 0xF, 0xF, false))
    NM_KV8_MAX(0xB1);
    NM_KV8_MAX(0x4E);
    NM_KV8_MAX(0x141);
    NM_KV8_MAX(0x140);
#undef NM_KV8_MAX
    const auto p = __builtin_amdgcn_permlane16_swap(m, m, false, false);
    m = max((uint32_t)p[0], (uint32_t)p[1]);
    const auto q = __builtin_amdgcn_permlane32_swap(m, m, false, false);
    return max((uint32_t)q[0], (uint32_t)q[1]);
}

// The largest (or smallest) over the lanes of a wave that have the same channels, `kSlots` lanes apart.
template <int kSlots, bool MOST>
__device__ __forceinline__ float over_tokens(float v) {
    auto pick = [](float a, float b) { return MOST ? fmaxf(a, b) : fminf(a, b); };
    if (kSlots == 4) v = pick(v, __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0x124, 0xF, 0xF, false)));  // row_ror:4
    v = pick(v, __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0x128, 0xF, 0xF, false)));                   // row_ror:8
    const uint32_t u = __float_as_uint(v);
    const auto p = __builtin_amdgcn_permlane16_swap(u, u, false, false);
    const uint32_t w = __float_as_uint(pick(__uint_as_float(p[0]), __uint_as_float(p[1])));
    const auto q = __builtin_amdgcn_permlane32_swap(w, w, false, false);
    return pick(__uint_as_float(q[0]), __uint_as_float(q[1]));
}

// The block of 64 tokens that a workgroup takes: rows t .. of the token arrays are its tokens lo .. hi.  Sequence s owns the blocks from
// q_start[s] / 64 + 2 s on, which are enough for it.
struct Unit {
    int s, block, lo, hi, t;
    uint8_t *page;  // null: no place
    int in_page;    // block of the page
};

template <class B>
__device__ __forceinline__ bool find_unit(const B &b, int slot, int lane, Unit &u) {
    int s = 0, q0, n, len;
    if (b.S <= kWave) {  // all of them read at once
        const int i = min(lane, b.S - 1);
        const int from = b.q_start[i], to = b.q_start[i + 1], l = b.kv_len[i];
        const uint64_t m = __ballot(lane < b.S && (from >> 6) + 2 * lane <= slot);
        s = m ? 63 - __clzll((long long)m) : 0;
        q0 = __builtin_amdgcn_readlane(from, s);
        n = __builtin_amdgcn_readlane(to, s) - q0;
        len = __builtin_amdgcn_readlane(l, s);
    } else {
        for (int left = b.S; left > 1;) {  // the last s whose first block is at or before the slot, 64 looks at a time
            const int step = (left + 63) >> 6, at = s + lane * step;
            const bool yes = lane * step < left && (b.q_start[at] >> 6) + 2 * at <= slot;
            const uint64_t m = __ballot(yes);
            s += (m ? 63 - __clzll((long long)m) : 0) * step;
            left = min(step, b.S - s);
        }
        s = __builtin_amdgcn_readfirstlane(s);
        q0 = b.q_start[s];
        n = b.q_start[s + 1] - q0;
        len = b.kv_len[s];
    }
    const int begin = len - n;
    if (n <= 0) return false;
    u.s = s;
    u.block = (begin >> 6) + slot - (q0 >> 6) - 2 * s;  // rounded down, also below 0
    const int at = u.block * 64;
    u.lo = max(begin - at, 0);
    u.t = q0 + max(at - begin, 0);
    u.hi = min(min(len - at, 64), u.lo + b.T - u.t);
    if (u.hi <= u.lo) return false;
    u.page = nullptr;
    const int per = b.f.blocks();
    if (u.block >= 0 && u.block / per < b.cols) {
        const int page = b.table[(int64_t)s * b.ld_table + u.block / per];
        if (page >= 0 && page < b.num_pages) u.page = b.cache + (int64_t)page * b.f.page_bytes();
    }
    u.in_page = u.block & (per - 1);
    return true;
}

// Cosines and sines of pairs 8 slot .. 8 slot + 7 of a place.
struct Turn {
    f32x4 x[4];  // cos, sin, cos, sin
    __device__ __forceinline__ void load(const KvRotation &r, int64_t place, int slot) {
        const f32x4 *p = reinterpret_cast<const f32x4 *>(r.cos_sin + place * r.ld + slot * 16);
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = p[i];
    }
};

// 16 channels: two runs of 8.
struct Runs {
    int a, b;
    bool turned;
    __device__ Runs(const KvRotation &r, int slot) {
        turned = slot * 16 < r.dim;
        const bool half = turned && !r.interleaved;
        a = half ? slot * 8 : slot * 16;
        b = half ? r.dim / 2 + slot * 8 : slot * 16 + 8;
    }
};

__device__ __forceinline__ float channel(const u32x4 &w, int i) { return i & 1 ? bf16_hi(w[i >> 1]) : bf16_lo(w[i >> 1]); }

// x[0..7] of run a, x[8..15] of run b -> rotated.
template <class F>
__device__ __forceinline__ void rotate(const u32x4 &a, const u32x4 &b, const Turn &t, bool interleaved, F &&put) {
#pragma unroll
    for (int p = 0; p < 8; ++p) {
        const int i = interleaved ? 2 * p : p, j = interleaved ? 2 * p + 1 : p + 8;
        const double x = i < 8 ? channel(a, i & 7) : channel(b, i & 7), y = j < 8 ? channel(a, j & 7) : channel(b, j & 7);
        const double c = t.x[p >> 1][2 * (p & 1)], s = t.x[p >> 1][2 * (p & 1) + 1];
        put(i, __builtin_elementwise_fma(x, c, -(y * s)));
        put(j, __builtin_elementwise_fma(y, c, x * s));
    }
}

template <int D>
struct AppendShared {
    uint32_t top[2][4];
    uint32_t bad[4];           // tokens of a wave's with a value that is not finite
    float most[4][D], least[4][D];
};

// What a block's new tokens need, and what its earlier ones are multiplied with: 1 unless the scale grows.
struct Scales {
    int kbyte, vbyte, kwas;
    float kdown, vdown, kmore, vmore;
    template <int D>
    __device__ __forceinline__ Scales(const AppendShared<D> &sh, bool had, uint32_t was) {
        const uint32_t ktop = max(max(sh.top[0][0], sh.top[0][1]), max(sh.top[0][2], sh.top[0][3]));
        const uint32_t vtop = max(max(sh.top[1][0], sh.top[1][1]), max(sh.top[1][2], sh.top[1][3]));
        kwas = min((int)(was & 255u), kHigh);
        const int vwas = min((int)(was >> 8 & 255u), kHigh);
        kbyte = had ? max(scale_byte(ktop), kwas) : scale_byte(ktop);
        vbyte = had ? max(scale_byte(vtop), vwas) : scale_byte(vtop);
        kdown = pow2_byte(254 - kbyte);
        vdown = pow2_byte(254 - vbyte);
        kmore = had ? pow2_byte(max(127 + kwas - kbyte, 0)) : 1.f;
        vmore = had ? pow2_byte(max(127 + vwas - vbyte, 0)) : 1.f;
    }
};

// Tokens before `lo` of the block's keys, times `more`: a unit of 16 channels a thread.
template <int D>
__device__ __forceinline__ void earlier_keys(uint8_t *block, int lo, float more) {
    for (int i = threadIdx.x; i < D / 16 * lo; i += kThreads) {
        u32x4 *p = reinterpret_cast<u32x4 *>(block + ((i / lo) * 64 + i % lo) * 16);
        u32x4 w = *p;
#pragma unroll
        for (int e = 0; e < 4; ++e) w[e] = again(w[e], more);
        *p = w;
    }
}

// Of the four tokens from `tok` on, a byte each, those before `lo` times `more`.
__device__ __forceinline__ uint32_t earlier_values(uint32_t w, int tok, int lo, float more) {
    const int n = min(max(lo - tok, 0), 4);
    const uint32_t early = n == 4 ? ~0u : (1u << (8 * n)) - 1;
    return (again(w, more) & early) | (w & ~early);
}

// Bounds of a block: of the new tokens (in LDS, by wave) and, if there were some, what it has.
template <int D>
__device__ __forceinline__ void store_bounds(const AppendShared<D> &sh, const Scales &sc, bool had, uint8_t *bounds, uint8_t *scales) {
    if (threadIdx.x < D) {  // two bounds of a channel
        const int c = threadIdx.x;
        float a = fmaxf(fmaxf(sh.most[0][c], sh.most[1][c]), fmaxf(sh.most[2][c], sh.most[3][c]));
        float d = fminf(fminf(sh.least[0][c], sh.least[1][c]), fminf(sh.least[2][c], sh.least[3][c]));
        if (had) {
            const float scale = pow2_byte((uint32_t)sc.kwas);
            a = fmaxf(a, __builtin_amdgcn_cvt_f32_fp8((int)bounds[c], 0) * scale);
            d = fminf(d, __builtin_amdgcn_cvt_f32_fp8((int)bounds[D + c], 0) * scale);
        }
        const uint32_t w = codes<false>(a, d, sc.kdown, 0);
        bounds[c] = (uint8_t)w;
        bounds[D + c] = (uint8_t)(w >> 8);
    }
    if (threadIdx.x == 0) *reinterpret_cast<uint32_t *>(scales) = (uint32_t)sc.kbyte | (uint32_t)sc.vbyte << 8;
}

// Few new tokens of a block and head: a lane has two channels of a token, the workgroup few_at_once of them, PASSES times.  Little code,
// which is run once and read from memory.  Calls of 48 sequences, 32 / 8 heads of 128, by the code for many tokens and by 2, 4 and 8
// passes of this: 1 token each 13.2 us and 7.0 (2), 7.5 (4); 16 tokens 14.6 and 10.3 (4), 10.9 (8); 32 tokens 16.5 and 14.3 (8);
// 512 sequences of 32 tokens 121 and 123 (8).
constexpr int few_at_once(int dim) { return kThreads / (dim / 2); }
template <int D, int PASSES>
__device__ __forceinline__ void append_few(const Kv8Batch &b, const KvRows &k, const KvRows &v, const KvRotation &r, const Unit &u, int head,
                                           AppendShared<D> &sh) {
    constexpr int kLanes = D / 2, kAtOnce = few_at_once(D), kPasses = PASSES;  // lanes to a token, tokens of the workgroup
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int at = head * b.f.blocks() + u.in_page;
    uint8_t *block = u.page + at * b.f.block_bytes();
    uint8_t *bounds = u.page + b.f.bounds_at() + at * 2 * D, *scales = u.page + b.f.scales_at() + at * 4;
    const bool had = u.lo > 0;
    const uint32_t was = had ? *reinterpret_cast<const uint32_t *>(scales) : 0u;
    const int c = 2 * (lane % kLanes), first = u.lo + (int)(threadIdx.x / kLanes);
    // the channels that mine are turned with, the pair of the first and whether mine are the second of theirs
    const bool turned = c < r.dim, second = !r.interleaved && c >= r.dim / 2;
    const int other = !turned || r.interleaved ? c : second ? c - r.dim / 2 : c + r.dim / 2;
    const int pair = r.interleaved ? c / 2 : second ? c - r.dim / 2 : c;

    uint32_t kx[kPasses], ko[kPasses], vx[kPasses];
    f32x2 t0[kPasses], t1[kPasses];
#pragma unroll
    for (int p = 0; p < kPasses; ++p) {
        const int tok = first + p * kAtOnce;
        kx[p] = ko[p] = vx[p] = 0;
        t0[p] = t1[p] = (f32x2){1.f, 0.f};
        if (tok < u.hi) {
            const int64_t t = u.t + tok - u.lo;
            const uint16_t *from = k.p + t * k.ld + head * k.hd;
            kx[p] = *reinterpret_cast<const uint32_t *>(from + c);
            ko[p] = *reinterpret_cast<const uint32_t *>(from + other);
            vx[p] = *reinterpret_cast<const uint32_t *>(v.p + t * v.ld + head * v.hd + c);
            if (turned) {
                const f32x2 *turn = reinterpret_cast<const f32x2 *>(r.cos_sin + ((int64_t)u.block * 64 + tok) * r.ld);
                t0[p] = turn[pair];
                t1[p] = r.interleaved ? t0[p] : turn[pair + 1];
            }
        }
    }
    float y[kPasses][2];
    uint32_t ktop = 0, vtop = 0;
    bool lost[kPasses];
#pragma unroll
    for (int p = 0; p < kPasses; ++p) {
        const float x0 = bf16_lo(kx[p]), x1 = bf16_hi(kx[p]);
        y[p][0] = x0;
        y[p][1] = x1;
        if (turned) {
            const float o0 = r.interleaved ? x1 : bf16_lo(ko[p]), o1 = r.interleaved ? x0 : bf16_hi(ko[p]);
            const double s0 = second ? (double)t0[p][1] : -(double)t0[p][1], s1 = second || r.interleaved ? (double)t1[p][1] : -(double)t1[p][1];
            y[p][0] = narrowed(__builtin_fma((double)x0, (double)t0[p][0], (double)o0 * s0));
            y[p][1] = narrowed(__builtin_fma((double)x1, (double)t1[p][0], (double)o1 * s1));
        }
        if (first + p * kAtOnce >= u.hi) y[p][0] = y[p][1] = 0.f;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const uint32_t m = __float_as_uint(y[p][i]) & 0x7FFFFFFFu;
            ktop = max(ktop, m < 0x7F800000u ? m : 0u);
        }
        const uint32_t lo = vx[p] << 16 & 0x7FFFFFFFu, hi = vx[p] & 0x7FFF0000u;
        vx[p] &= (lo >= 0x7F800000u ? 0xFFFF0000u : ~0u) & (hi >= 0x7F800000u ? 0xFFFFu : ~0u);
        const uint64_t m = __ballot(lo >= 0x7F800000u || hi >= 0x7F800000u);
        lost[p] = D == 128 ? m != 0 : (lane < 32 ? (uint32_t)m : (uint32_t)(m >> 32)) != 0;
        vtop = max(vtop, max(vx[p] << 16 & 0x7FFFFFFFu, vx[p] & 0x7FFF0000u));
    }
    ktop = wave_max(ktop);
    vtop = wave_max(vtop);
    if (lane == 0) {
        sh.top[0][wave] = ktop;
        sh.top[1][wave] = vtop;
    }
    __syncthreads();
    const Scales sc(sh, had, was);
    if (sc.kmore != 1.f) earlier_keys<D>(block, u.lo, sc.kmore);
    if (sc.vmore != 1.f) {
        for (int i = threadIdx.x; i < 4 * D; i += kThreads) {
            u32x4 *p = reinterpret_cast<u32x4 *>(block + 64 * D + i * 16);
            u32x4 w = *p;
#pragma unroll
            for (int j = 0; j < 4; ++j) w[j] = earlier_values(w[j], 16 * j + 4 * (i / D), u.lo, sc.vmore);
            *p = w;
        }
        __syncthreads();  // new tokens have bytes in the same units
    }
    float most[2] = {-INFINITY, -INFINITY}, least[2] = {INFINITY, INFINITY};
#pragma unroll
    for (int p = 0; p < kPasses; ++p) {
        const int tok = first + p * kAtOnce;
        if (tok >= u.hi) break;
        uint32_t w = codes<false>(y[p][0], y[p][1], sc.kdown, 0);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            if ((__float_as_uint(y[p][i]) & 0x7FFFFFFFu) >= 0x7F800000u) {
                w = (w & ~(255u << (8 * i))) | kNaN8 << (8 * i);
                y[p][i] = 0.f;
            }
            most[i] = fmaxf(most[i], y[p][i]);
            least[i] = fminf(least[i], y[p][i]);
        }
        if (c == 0 && lost[p]) w = (w & ~255u) | kNaN8;
        *reinterpret_cast<uint16_t *>(block + b.f.k_byte(tok, c)) = (uint16_t)w;
        const uint32_t x = codes<false>(bf16_lo(vx[p]), bf16_hi(vx[p]), sc.vdown, 0);
        uint8_t *to = block + b.f.v_byte(tok, c);
        to[0] = (uint8_t)x;
        to[16] = (uint8_t)(x >> 8);
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        if (D == 64) {  // two tokens a wave
            const uint32_t a = __float_as_uint(most[i]), d = __float_as_uint(least[i]);
            const auto p = __builtin_amdgcn_permlane32_swap(a, a, false, false);
            const auto q = __builtin_amdgcn_permlane32_swap(d, d, false, false);
            most[i] = fmaxf(__uint_as_float(p[0]), __uint_as_float(p[1]));
            least[i] = fminf(__uint_as_float(q[0]), __uint_as_float(q[1]));
        }
        sh.most[wave][c + i] = most[i];
        sh.least[wave][c + i] = least[i];
    }
    __syncthreads();
    store_bounds(sh, sc, had, bounds, scales);
}

template <int D>
__device__ __forceinline__ void append(const Kv8Batch &b, const KvRows &k, const KvRows &v, const KvRotation &r, const Unit &u, int head,
                                       AppendShared<D> &sh) {
    constexpr int kSlots = D / 16, kTokens = kThreads / kSlots, kPasses = 64 / kTokens;  // D 128: 32 tokens in 2 passes
    constexpr int kJ = D / 32;  // of the four j of a V unit, those that a thread has
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int at = head * b.f.blocks() + u.in_page;
    uint8_t *block = u.page + at * b.f.block_bytes();
    uint8_t *bounds = u.page + b.f.bounds_at() + at * 2 * D, *scales = u.page + b.f.scales_at() + at * 4;
    const bool had = u.lo > 0;
    const uint32_t was = had ? *reinterpret_cast<const uint32_t *>(scales) : 0u;

    // keys: token kTokens p + tk, 16 channels
    const int ks = threadIdx.x % kSlots, tk = threadIdx.x / kSlots;
    const Runs run(r, ks);
    u32x4 ka[kPasses], kb[kPasses];
    Turn turn[kPasses];
#pragma unroll
    for (int p = 0; p < kPasses; ++p) {
        const int tok = kTokens * p + tk;
        ka[p] = kb[p] = (u32x4){0, 0, 0, 0};
        if (tok >= u.lo && tok < u.hi) {
            const uint16_t *from = k.p + (int64_t)(u.t + tok - u.lo) * k.ld + head * k.hd;
            ka[p] = *reinterpret_cast<const u32x4 *>(from + run.a);
            kb[p] = *reinterpret_cast<const u32x4 *>(from + run.b);
            if (run.turned) turn[p].load(r, (int64_t)u.block * 64 + tok, ks);
        }
    }
    // values: channels 2 vc, 2 vc + 1 of tokens 16 (vj + j) + 4 wave + i
    const int vc = lane % (D / 2), vj = D == 128 ? 0 : (lane >> 5) * 2;
    uint32_t x[kJ][4];
    uint32_t mine = 0;  // which of them there are
#pragma unroll
    for (int j = 0; j < kJ; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int tok = 16 * (vj + j) + 4 * wave + i;
            x[j][i] = 0;
            if (tok >= u.lo && tok < u.hi) {
                mine |= 1u << (4 * j + i);
                x[j][i] = *reinterpret_cast<const uint32_t *>(v.p + (int64_t)(u.t + tok - u.lo) * v.ld + head * v.hd + 2 * vc);
            }
        }

    float y[kPasses][16];
    uint32_t ktop = 0;
#pragma unroll
    for (int p = 0; p < kPasses; ++p) {
        if (run.turned && r.interleaved) {
            rotate(ka[p], kb[p], turn[p], true, [&](int i, double d) { y[p][i] = narrowed(d); });
        } else if (run.turned) {
            rotate(ka[p], kb[p], turn[p], false, [&](int i, double d) { y[p][i] = narrowed(d); });
        } else {
#pragma unroll
            for (int i = 0; i < 16; ++i) y[p][i] = channel(i < 8 ? ka[p] : kb[p], i & 7);
        }
        const int tok = kTokens * p + tk;
        const bool there = tok >= u.lo && tok < u.hi;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            if (!there) y[p][i] = 0.f;  // what was loaded of a turn there is nothing
            const uint32_t m = __float_as_uint(y[p][i]) & 0x7FFFFFFFu;
            ktop = max(ktop, m < 0x7F800000u ? m : 0u);
        }
    }
    uint32_t vtop = 0, bad = 0;
#pragma unroll
    for (int j = 0; j < kJ; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t lo = x[j][i] << 16 & 0x7FFFFFFFu, hi = x[j][i] & 0x7FFF0000u;
            if (lo >= 0x7F800000u || hi >= 0x7F800000u) {
                bad |= 1u << (4 * (vj + j) + i);
                x[j][i] &= (lo >= 0x7F800000u ? 0xFFFF0000u : ~0u) & (hi >= 0x7F800000u ? 0xFFFFu : ~0u);
            }
            vtop = max(vtop, max(x[j][i] << 16 & 0x7FFFFFFFu, x[j][i] & 0x7FFF0000u));
        }
    if (__any(bad)) {  // seldom
        uint32_t all = 0;
        for (int i = 0; i < 16; ++i)
            if (__any(bad >> i & 1)) all |= 1u << i;
        bad = all;
    }
    ktop = wave_max(ktop);
    vtop = wave_max(vtop);
    if (lane == 0) {
        sh.top[0][wave] = ktop;
        sh.top[1][wave] = vtop;
        sh.bad[wave] = bad;
    }
    __syncthreads();
    const Scales sc(sh, had, was);
    const float kdown = sc.kdown, vdown = sc.vdown, vmore = sc.vmore;
    if (sc.kmore != 1.f) earlier_keys<D>(block, u.lo, sc.kmore);
    float most[16], least[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        most[i] = -INFINITY;
        least[i] = INFINITY;
    }
#pragma unroll
    for (int p = 0; p < kPasses; ++p) {
        const int tok = kTokens * p + tk;
        if (tok < u.lo || tok >= u.hi) continue;
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            w[i] = codes<false>(y[p][4 * i], y[p][4 * i + 1], kdown, 0);
            w[i] = codes<true>(y[p][4 * i + 2], y[p][4 * i + 3], kdown, w[i]);
        }
        // what is not a number: its own code, and 0 for the bounds
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            if ((__float_as_uint(y[p][i]) & 0x7FFFFFFFu) >= 0x7F800000u) {
                w[i >> 2] = (w[i >> 2] & ~(255u << (8 * (i & 3)))) | kNaN8 << (8 * (i & 3));
                y[p][i] = 0.f;
            }
            most[i] = fmaxf(most[i], y[p][i]);
            least[i] = fminf(least[i], y[p][i]);
        }
        if (ks == 0 && (sh.bad[tok >> 2 & 3] >> (4 * (tok >> 4) + (tok & 3)) & 1)) w[0] = (w[0] & ~255u) | kNaN8;
        uint2 a = {w[0], w[1]}, c = {w[2], w[3]};
        *reinterpret_cast<uint2 *>(block + b.f.k_byte(tok, run.a)) = a;
        *reinterpret_cast<uint2 *>(block + b.f.k_byte(tok, run.b)) = c;
    }
    // rounding keeps order: the bounds of what is stored are the bounds, rounded
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        const float a = over_tokens<kSlots, true>(most[i]), c = over_tokens<kSlots, false>(least[i]);
        if (lane < kSlots) {
            const int ch = i < 8 ? run.a + i : run.b + i - 8;
            sh.most[wave][ch] = a;
            sh.least[wave][ch] = c;
        }
    }
    // values: a unit is 16 tokens of a channel; bytes of others than the new tokens stay, or are rounded again
    constexpr uint32_t kAll = (1u << (4 * kJ)) - 1;
    if (mine || vmore != 1.f) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            uint32_t w[kJ];
#pragma unroll
            for (int j = 0; j < kJ; ++j) {
                float f[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) f[i] = e ? bf16_hi(x[j][i]) : bf16_lo(x[j][i]);
                w[j] = codes<true>(f[2], f[3], vdown, codes<false>(f[0], f[1], vdown, 0));
            }
            uint32_t *p = reinterpret_cast<uint32_t *>(block + 64 * D + (wave * D + 2 * vc + e) * 16 + vj * 4);
            if (mine != kAll) {
#pragma unroll
                for (int j = 0; j < kJ; ++j) {
                    const uint32_t m = mine >> (4 * j) & 15u;
                    const uint32_t keep = (m & 1 ? 0u : 255u) | (m & 2 ? 0u : 255u << 8) | (m & 4 ? 0u : 255u << 16) | (m & 8 ? 0u : 255u << 24);
                    uint32_t old = p[j];
                    if (vmore != 1.f) old = earlier_values(old, 16 * (vj + j) + 4 * wave, u.lo, vmore);
                    w[j] = (w[j] & ~keep) | (old & keep);
                }
            }
            if constexpr (D == 128) {
                *reinterpret_cast<u32x4 *>(p) = (u32x4){w[0], w[1], w[2], w[3]};
            } else {
                *reinterpret_cast<uint2 *>(p) = uint2{w[0], w[1]};
            }
        }
    }
    __syncthreads();
    store_bounds(sh, sc, had, bounds, scales);
}

// Queries: a wave takes a token, its lanes 16 channels each of several heads at once.
template <int D>
__device__ __forceinline__ void turn_queries(const Kv8Batch &b, const KvRotation &r, const KvRows &q, const KvRows &out, int heads, int t) {
    constexpr int kSlots = D / 16, kAtOnce = kWave / kSlots;
    const int lane = threadIdx.x & 63;
    if (t >= b.T || t >= b.q_start[b.S]) return;
    const int s = find_seq(b.q_start, b.S, t, lane);
    const int q1 = b.q_start[s + 1];
    if (t < b.q_start[s] || t >= q1) return;
    const int64_t place = (int64_t)b.kv_len[s] - q1 + t;
    if (place < 0 || place >= (int64_t)b.cols * b.f.page) return;
    const int slot = lane % kSlots;
    const Runs run(r, slot);
    Turn turn;
    if (run.turned) turn.load(r, place, slot);
    const uint16_t *from = q.p + (int64_t)t * q.ld;
    uint16_t *to = out.p + (int64_t)t * out.ld;
    for (int h = lane / kSlots; h < heads; h += kAtOnce) {
        u32x4 a = *reinterpret_cast<const u32x4 *>(from + h * q.hd + run.a), c = *reinterpret_cast<const u32x4 *>(from + h * q.hd + run.b);
        if (run.turned) {
            float w[16];
            auto put = [&](int i, double d) { w[i] = narrowed(d); };
            if (r.interleaved)
                rotate(a, c, turn, true, put);
            else
                rotate(a, c, turn, false, put);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                a[i] = pack_bf16(w[2 * i], w[2 * i + 1]);
                c[i] = pack_bf16(w[8 + 2 * i], w[9 + 2 * i]);
            }
        }
        *reinterpret_cast<u32x4 *>(to + h * out.hd + run.a) = a;
        *reinterpret_cast<u32x4 *>(to + h * out.hd + run.b) = c;
    }
}

// The first `blocks` workgroups store blocks, the others turn the queries of four tokens each.
template <int D>
__global__ __launch_bounds__(kThreads) void kv8_append_kernel(Kv8Batch b, KvRows k, KvRows v, KvRotation r, KvRows q, KvRows out, int heads,
                                                              int blocks) {
    __shared__ AppendShared<D> sh;
    b.f.dim = D;
    const int i = blockIdx.x;
    if (i < blocks) {
        Unit u;
        if (!find_unit(b, i / b.f.n_kv, threadIdx.x & 63, u) || !u.page) return;  // the whole workgroup
        if (u.hi - u.lo <= 2 * few_at_once(D))
            append_few<D, 2>(b, k, v, r, u, i % b.f.n_kv, sh);
        else if (u.hi - u.lo <= 4 * few_at_once(D))
            append_few<D, 4>(b, k, v, r, u, i % b.f.n_kv, sh);
        else if (u.hi - u.lo <= 8 * few_at_once(D) && u.hi - u.lo < 64)
            append_few<D, 8>(b, k, v, r, u, i % b.f.n_kv, sh);
        else
            append<D>(b, k, v, r, u, i % b.f.n_kv, sh);
    } else {
        const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
        turn_queries<D>(b, r, q, out, heads, (i - blocks) * 4 + wave);
    }
}

// The rows of one block and head out of the cache, threads as above.
template <int D>
__global__ __launch_bounds__(kThreads) void kv8_unpack_kernel(Kv8Batch b, KvRows k, KvRows v) {
    constexpr int kSlots = D / 16, kTokens = kThreads / kSlots, kPasses = 64 / kTokens, kJ = D / 32;
    b.f.dim = D;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int head = blockIdx.x % b.f.n_kv;
    Unit u;
    if (!find_unit(b, blockIdx.x / b.f.n_kv, lane, u)) return;
    const int at = head * b.f.blocks() + u.in_page;
    const uint8_t *block = u.page + at * b.f.block_bytes();
    const uint32_t scales = u.page ? *reinterpret_cast<const uint32_t *>(u.page + b.f.scales_at() + at * 4) : 0x7F7Fu;
    const float kscale = pow2_byte(scales & 255u), vscale = pow2_byte(scales >> 8 & 255u);
    auto pair = [](uint32_t w, bool high, float s) {
        union { decltype(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(0u, 1.f, false)) h; uint32_t u; } c;
        c.h = high ? __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, s, true) : __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, s, false);
        return c.u;
    };
    const int ks = threadIdx.x % kSlots, tk = threadIdx.x / kSlots;
#pragma unroll
    for (int p = 0; p < kPasses; ++p) {
        const int tok = kTokens * p + tk;
        if (tok < u.lo || tok >= u.hi) continue;
        u32x4 w = {0, 0, 0, 0};
        if (u.page) w = *reinterpret_cast<const u32x4 *>(block + b.f.k_byte(tok, 16 * ks));
        u32x4 *to = reinterpret_cast<u32x4 *>(k.p + (int64_t)(u.t + tok - u.lo) * k.ld + head * k.hd + 16 * ks);
        to[0] = (u32x4){pair(w[0], false, kscale), pair(w[0], true, kscale), pair(w[1], false, kscale), pair(w[1], true, kscale)};
        to[1] = (u32x4){pair(w[2], false, kscale), pair(w[2], true, kscale), pair(w[3], false, kscale), pair(w[3], true, kscale)};
    }
    const int vc = lane % (D / 2), vj = D == 128 ? 0 : (lane >> 5) * 2;
    bool some = false;
#pragma unroll
    for (int j = 0; j < kJ; ++j)
        some |= 16 * (vj + j) + 4 * wave < u.hi && 16 * (vj + j) + 4 * wave + 3 >= u.lo;
    if (!some) return;
    uint32_t w[2][kJ] = {};
    if (u.page) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const uint32_t *p = reinterpret_cast<const uint32_t *>(block + 64 * D + (wave * D + 2 * vc + e) * 16 + vj * 4);
#pragma unroll
            for (int j = 0; j < kJ; ++j) w[e][j] = p[j];
        }
    }
#pragma unroll
    for (int j = 0; j < kJ; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int tok = 16 * (vj + j) + 4 * wave + i;
            if (tok < u.lo || tok >= u.hi) continue;
            const uint32_t lo = pair(w[0][j], i >> 1, vscale), hi = pair(w[1][j], i >> 1, vscale);
            *reinterpret_cast<uint32_t *>(v.p + (int64_t)(u.t + tok - u.lo) * v.ld + head * v.hd + 2 * vc) =
                i & 1 ? __builtin_amdgcn_perm(hi, lo, 0x07060302u) : __builtin_amdgcn_perm(hi, lo, 0x05040100u);
        }
}

int64_t slots(const Kv8Batch &b) { return (b.T >> 6) + 2 * (int64_t)b.S; }

}  // namespace

hipError_t launch_kv8_append(const Kv8Batch &b, const KvRows &k, const KvRows &v, const KvRotation &r, const KvRows &q, int heads,
                             const KvRows &q_out, hipStream_t st) {
    const int blocks = (int)(slots(b) * b.f.n_kv);
    const unsigned grid = (unsigned)blocks + (q.p ? (unsigned)((b.T + 3) / 4) : 0u);
    if (b.f.dim == 128)
        kv8_append_kernel<128><<<grid, kThreads, 0, st>>>(b, k, v, r, q, q_out, heads, blocks);
    else
        kv8_append_kernel<64><<<grid, kThreads, 0, st>>>(b, k, v, r, q, q_out, heads, blocks);
    return hipGetLastError();
}

hipError_t launch_kv8_unpack(const Kv8Batch &b, const KvRows &k, const KvRows &v, hipStream_t st) {
    const unsigned grid = (unsigned)(slots(b) * b.f.n_kv);
    if (b.f.dim == 128)
        kv8_unpack_kernel<128><<<grid, kThreads, 0, st>>>(b, k, v);
    else
        kv8_unpack_kernel<64><<<grid, kThreads, 0, st>>>(b, k, v);
    return hipGetLastError();
}

}  // namespace nmk

// nm_kv8_select.hip -- which blocks of 64 cached tokens a row looks at.
//
// For a row (place p) and key/value head, over the blocks b <= p / 64 that have a page:
//     score_b = sum_h sum_c max(q_hc most_bc, q_hc least_bc) = sum_c (sum_h max(q_hc, 0)) most_bc + (sum_h min(q_hc, 0)) least_bc,
// h the query heads of the key/value head, most and least the bounds that the cache keeps of a block's keys: no key of
// the block has a larger sum of scores.  Taken are the first and the last blocks asked for and then those of the largest
// scores, of equal ones the lowest, `top` in all.
//
// Scores are formed in 64 bits, so that the choice is that of the definition but for scores closer than 2^-48.  A workgroup takes
// one row and head: a lane has 16 channels of the largest or the smallest keys and their sums of queries in
// registers, 16 lanes (dim 64: 8) read the bounds of a block side by side.  The choice: the scores as whole numbers that are
// ordered alike lie in LDS; histograms of 8 bits at a time, from the first bit that differs, find the smallest score taken.
// Bound by the bytes of the bounds, 2 D + 4 for every 128 D of keys and values, where contexts are long; by the chain of reads
// and barriers where they are short.
#include "nm_kv_rows.h"

namespace nmk {
namespace {

typedef float f32x2 __attribute__((ext_vector_type(2)));

__device__ __forceinline__ double lane_add(double v, int ctrl) {
    const int lo = __double2loint(v), hi = __double2hiint(v);
    int l, h;
    switch (ctrl) {
    case 0: l = __builtin_amdgcn_update_dpp(0, lo, 0xB1, 0xF, 0xF, false); h = __builtin_amdgcn_update_dpp(0, hi, 0xB1, 0xF, 0xF, false); break;
    case 1: l = __builtin_amdgcn_update_dpp(0, lo, 0x4E, 0xF, 0xF, false); h = __builtin_amdgcn_update_dpp(0, hi, 0x4E, 0xF, 0xF, false); break;
    case 2: l = __builtin_amdgcn_update_dpp(0, lo, 0x141, 0xF, 0xF, false); h = __builtin_amdgcn_update_dpp(0, hi, 0x141, 0xF, 0xF, false); break;
    default: l = __builtin_amdgcn_update_dpp(0, lo, 0x140, 0xF, 0xF, false); h = __builtin_amdgcn_update_dpp(0, hi, 0x140, 0xF, 0xF, false); break;
    }
    return v + __hiloint2double(h, l);
}

// A score as a whole number with the same order; 0 is none, ~0 a block that is taken in any case.
__device__ __forceinline__ uint64_t ordered(double v) {
    const uint64_t u = (uint64_t)__double_as_longlong(v + 0.0);
    return u ^ ((u >> 63) ? ~0ull : 1ull << 63);
}

constexpr int kMaxWaves = 16;
constexpr int kFew = 64;  // candidates that one wave ranks

template <int CAP>
struct SelectShared {
    uint64_t key[CAP];
    uint64_t any[kMaxWaves], all[kMaxWaves];
    int count[kMaxWaves], forced[kMaxWaves];
    int bins[256];
    int bin, above, inside;  // what the scan of the bins found
    int listed;
    uint64_t list[kFew];
    int at[kFew];
};

// The 8-bit pass over bits lo .. d of keys whose bits above d are `pre`.
struct Digits {
    int d, lo;
    uint64_t pre;
    __device__ bool of(uint64_t k) const { return k != 0 && k != ~0ull && (d == 63 || k >> (d + 1) == pre); }
};

template <int D, int CAP>
__global__ __launch_bounds__(kMaxWaves *kWave) void kv8_select_kernel(Kv8Select a) {
    __shared__ SelectShared<CAP> sh;
    constexpr int kLanes = D / 8, kAtOnce = kWave / kLanes;  // lanes to a block, blocks of a wave at once
    a.b.f.dim = D;
    const Kv8Batch &b = a.b;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), waves = blockDim.x >> 6;
    const int n_kv = b.f.n_kv, group = a.heads / n_kv;
    const int t = blockIdx.x / n_kv, head = blockIdx.x - t * n_kv;
    if (t >= b.q_start[b.S]) return;
    const int s = find_seq(b.q_start, b.S, t, lane);
    const int q1 = b.q_start[s + 1];
    if (t < b.q_start[s] || t >= q1) return;
    const int place = b.kv_len[s] - q1 + t, mine = place >> 6;
    const int per = b.f.blocks();
    const int n = place < 0 ? 0 : (int)min((int64_t)mine + 1, (int64_t)b.cols * per);
    int32_t *out = a.out + (int64_t)t * a.ld_out + (int64_t)head * a.top;

    // the sums of the queries' positive (or negative) parts in this lane's channels
    const int part = lane % kLanes;
    const bool low = part >= D / 16;
    double q[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) q[i] = 0.0;
    bool bad = false;
    const uint16_t *from = a.q.p + (int64_t)t * a.q.ld + (int64_t)head * group * a.q.hd + (low ? part - D / 16 : part) * 16;
    for (int h = 0; h < group; ++h) {
        const u32x4 *p = reinterpret_cast<const u32x4 *>(from + (int64_t)h * a.q.hd);
        const u32x4 w[2] = {p[0], p[1]};
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const uint32_t pair = w[i >> 3][i >> 1 & 3];
            const float x = i & 1 ? bf16_hi(pair) : bf16_lo(pair);
            bad |= (__float_as_uint(x) & 0x7F800000u) == 0x7F800000u;
            q[i] += (double)(low ? fminf(x, 0.f) : fmaxf(x, 0.f));
        }
    }
    const bool none = __any(bad);  // the same in all waves: each has all channels

    const int32_t *row = b.table + (int64_t)s * b.ld_table;
    // Page numbers of a wave's rounds, then their bounds, are asked for together.
    constexpr int kRounds = 4;
    for (int i0 = wave * kAtOnce * kRounds; i0 < n; i0 += waves * kAtOnce * kRounds) {
        int page[kRounds], scale[kRounds];
        u32x4 w[kRounds];
        uint32_t ok = 0;
#pragma unroll
        for (int r = 0; r < kRounds; ++r) page[r] = row[min(i0 + r * kAtOnce + lane / kLanes, n - 1) / per];
#pragma unroll
        for (int r = 0; r < kRounds; ++r) {
            const int k = min(i0 + r * kAtOnce + lane / kLanes, n - 1);
            const bool there = page[r] >= 0 && page[r] < b.num_pages;
            ok |= (uint32_t)there << r;
            const uint8_t *p = b.cache + (int64_t)(there ? page[r] : 0) * b.f.page_bytes();
            const int at = head * per + (k & (per - 1));
            w[r] = *reinterpret_cast<const u32x4 *>(p + b.f.bounds_at() + at * 2 * D + part * 16);
            scale[r] = p[b.f.scales_at() + at * 4];
        }
#pragma unroll
        for (int r = 0; r < kRounds; ++r) {
            double v = 0.0, v1 = 0.0;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const f32x2 x = __builtin_amdgcn_cvt_pk_f32_fp8((int)w[r][j], false), y = __builtin_amdgcn_cvt_pk_f32_fp8((int)w[r][j], true);
                v = __builtin_fma(q[4 * j], (double)x[0], v);
                v1 = __builtin_fma(q[4 * j + 1], (double)x[1], v1);
                v = __builtin_fma(q[4 * j + 2], (double)y[0], v);
                v1 = __builtin_fma(q[4 * j + 3], (double)y[1], v1);
            }
            v += v1;
#pragma unroll
            for (int c = 0; c < (D == 128 ? 4 : 3); ++c) v = lane_add(v, c);
            const int block = i0 + r * kAtOnce + lane / kLanes;
            if (part == 0 && block < n) {
                const bool asked = block < a.first || block > mine - a.last;
                sh.key[block] = !(ok >> r & 1) ? 0ull : asked ? ~0ull : none ? 1ull << 63 : ordered(__builtin_ldexp(v, scale[r] - 127));
            }
        }
    }
    if (threadIdx.x == 0) sh.listed = 0;
    __syncthreads();

    // how many there are, and the bits that they share
    uint64_t any = 0, all = ~0ull;
    int count = 0, forced = 0;
    for (int i = threadIdx.x; i < n; i += blockDim.x) {
        const uint64_t k = sh.key[i];
        if (k == ~0ull) {
            ++forced;
        } else if (k) {
            any |= k;
            all &= k;
            ++count;
        }
    }
    for (int m = 1; m < 64; m <<= 1) {
        any |= (uint64_t)__shfl_xor((long long)any, m);
        all &= (uint64_t)__shfl_xor((long long)all, m);
        count += __shfl_xor(count, m);
        forced += __shfl_xor(forced, m);
    }
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
    // Taken are keys above the border, and of those on it (k >> border == edge) the first `left`.
    int left = max(a.top - forced, 0), border = 0;
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
            for (int i = threadIdx.x; i < 256; i += blockDim.x) sh.bins[i] = 0;
            __syncthreads();
            for (int i = threadIdx.x; i < n; i += blockDim.x) {
                const uint64_t k = sh.key[i];
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
            left -= sh.above;
            const int inside = sh.inside;
            g.pre = (g.d == 63 ? 0 : g.pre << (g.d - g.lo + 1)) | (uint64_t)sh.bin;
            border = g.lo;
            edge = g.pre;
            if (inside == left || g.lo == 0) break;
            g.d = g.lo - 1;
            if (inside <= kFew) {  // one wave ranks them
                for (int i = threadIdx.x; i < n; i += blockDim.x) {
                    const uint64_t k = sh.key[i];
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
                    sh.key[i] = ahead < left ? ~0ull : 0ull;
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
        const uint64_t k = i < n ? sh.key[i] : 0;
        const uint64_t digits = k >> border;
        const bool is_over = k == ~0ull || (k != 0 && digits > edge), is_on = k != 0 && k != ~0ull && digits == edge;
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
        if ((is_over || (is_on && e_before < left)) && to < a.top) out[to] = i;
    }
    for (int i = over + min(on, left) + threadIdx.x; i < a.top; i += blockDim.x) out[i] = -1;
}

// Waves to a row and head: more where there are few of them.
template <int D, int CAP>
hipError_t launch(const Kv8Select &a, hipStream_t st) {
    const int64_t items = (int64_t)a.b.T * a.b.f.n_kv;
    const int waves = items <= 512 ? kMaxWaves : 4;
    kv8_select_kernel<D, CAP><<<(unsigned)items, waves * kWave, 0, st>>>(a);
    return hipGetLastError();
}

constexpr int kShort = 4096;  // blocks whose keys leave room for several workgroups a CU

template <int D>
hipError_t launch(const Kv8Select &a, hipStream_t st) {
    return (int64_t)a.b.cols * a.b.f.blocks() <= kShort ? launch<D, kShort>(a, st) : launch<D, kMaxSelectBlocks>(a, st);
}

}  // namespace

hipError_t launch_kv8_select(const Kv8Select &a, hipStream_t st) {
    return a.b.f.dim == 128 ? launch<128>(a, st) : launch<64>(a, st);
}

}  // namespace nmk

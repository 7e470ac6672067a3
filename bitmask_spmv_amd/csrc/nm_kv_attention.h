// nm_kv_attention.h -- what the attention kernels over the 4-bit and the 8-bit key/value cache share: how a ragged batch is
// laid out as work, the running softmax of a row tile, and the joining of rows that were cut between waves and workgroups.
// A is the arguments of a call (Kv4Attention, Kv8Attention).
#pragma once

#include <atomic>

#include "nm_device.h"
#include "nm_kv.h"

namespace nmk {
namespace {

constexpr float kLn2 = 0.6931471805599453f;
constexpr int kBlock = 64;      // tokens a wave takes at a time
constexpr int kRows = 16;       // query rows of a tile
constexpr int kWaves = 4;       // waves per workgroup
constexpr int kDecodeRows = 64; // query rows of a head up to which a sequence among others is walked by row tiles

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

// A read with a wave-uniform address of data that no kernel in flight writes: through the
// scalar cache, so it does not enter the order in which a wave's vector loads return.
__device__ __forceinline__ int32_t uniform_load(const int32_t *p) {
    return *(const __attribute__((address_space(4))) int32_t *)(uintptr_t)p;
}

__device__ __forceinline__ float pow2_byte(uint32_t byte) { return __uint_as_float(byte << 23); }

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

__device__ __forceinline__ float halves_max(float v) {
    const auto p = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    return fmaxf(__uint_as_float(p[0]), __uint_as_float(p[1]));
}
__device__ __forceinline__ float halves_sum(float v) {
    const auto p = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    return __uint_as_float(p[0]) + __uint_as_float(p[1]);
}

// What a sequence asks of a call.
struct Seq {
    int q0, n, len;      // first row, rows, tokens
    int tiles;           // row tiles per key/value head
    int first, blocks;   // first 64-token block and how many (at least one)
    __device__ int64_t units(int n_kv, bool whole) const { return (int64_t)tiles * n_kv * (whole ? 1 : blocks); }
};

template <class A>
__device__ __forceinline__ Seq seq_from(const A &a, int group, int q0, int q1, int len) {
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
    template <class B>
    __device__ void load(const B &b, int s) {
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

// Cache bytes at an address put together from its halves: said to be global memory (a load that might be
// from LDS as well counts among the LDS operations too, and waits for one would wait for it).
// NT: bytes that are read once (one row tile per head) stay out of the caches' way.
template <bool NT, class T>
__device__ __forceinline__ T load_cache(const uint8_t *p) {
    typedef const __attribute__((address_space(1))) T *Global;
    return NT ? __builtin_nontemporal_load((Global)(uintptr_t)p) : *(Global)(uintptr_t)p;
}

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
    template <class A>
    __device__ void finish(const A &a, const PartTag &tag, int group, int row, int c) const {
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

// The pieces that the waves of workgroup `block` left: rows that begin and end in it are finished, the others go to the workspace.
template <int D, class A>
__device__ __forceinline__ void join_pieces(const A &a, Part<D> *parts, PartTag *tags, Shared<D> &sh, int block) {
    const int group = a.heads / a.b.f.n_kv;
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

// Rows cut between workgroups: the workgroup in which a row begins owns it; the pieces
// follow in the slots 0 of the next ones, up to one in which the row ends.
template <int D, class A>
__device__ __forceinline__ void join_groups(const A &a, const Part<D> *parts, const PartTag *tags) {
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
        j.m = top;
#pragma unroll
        for (int i = 0; i < kAtOnce; ++i) {
            const float its = k0 + i <= n ? weight_of(m[i], top) : 0.f;
            // Which of the first two products is rounded is said here: else it is the compiler's choice, and differs between kernels.
            j.l = __builtin_fmaf(l[i], its, i ? j.l : j.l * keep);
#pragma unroll
            for (int e = 0; e < N; ++e) j.o[e] = i ? __builtin_fmaf(o[i][e], its, j.o[e]) : __builtin_fmaf(j.o[e], keep, o[0][e] * its);
        }
    }
    j.finish(a, tag, a.heads / a.b.f.n_kv, row, cc);
}

inline int device_cus() {
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

}  // namespace
}  // namespace nmk

// nm_kv4.hip -- tokens into the 4-bit key/value cache and back.
//
// A block of 32 channels of one token is stored as E2M1 numbers times a power of two:
//     byte = clamp(E(amax) - 2 + (significand(amax) > 1.75), 16, 252),  x ~ e2m1 * 2^(byte - 127),
// E the biased exponent of the largest magnitude: that magnitude lands in (3.5, 7], where
// rounding to nearest (6 the largest) is off by at most one unit of the scale.  The ends
// 16 and 252 keep every stored value a normal, finite bf16.
#include "nm_device.h"
#include "nm_kv.h"

namespace nmk {
namespace {

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

// Sequence that row t belongs to: the last s with q_start[s] <= t.  Called by a whole wave
// with one t: 64 lanes look at 64 places at once, so 4096 sequences take two looks.
__device__ __forceinline__ int find_seq(const int32_t *q_start, int S, int t, int lane) {
    int lo = 0, n = S;  // the answer is in [lo, lo + n)
    while (n > 1) {
        const int step = (n + 63) >> 6;
        const int at = lo + lane * step;
        const bool yes = lane * step < n && q_start[at] <= t;
        const uint64_t m = __ballot(yes);
        const int last = m ? 63 - __clzll((long long)m) : 0;
        lo += last * step;
        n = min(step, S - lo);
    }
    return lo;
}

// The same for a lane's row t < q_start[S], from the sequence s of the wave's first row t0.  Most rows are of s as well, or of
// the sequence as far behind it as the row is (single tokens): both are looked at at once.  Else in steps that
// double, and back: a few looks however many sequences without rows lie between.
__device__ __forceinline__ int seq_of_row(const int32_t *q_start, int S, int s, int t0, int t) {
    const int guess = min(s + (t - t0), S - 1);
    const int next = q_start[s + 1], from = q_start[guess], end = q_start[guess + 1];
    if (t < next) return s;
    if (from <= t && t < end) return guess;
    int step = 1;
    while (step < S - s && q_start[s + step] <= t) {
        s += step;
        step *= 2;
    }
    for (; step > 0; step >>= 1)
        if (step < S - s && q_start[s + step] <= t) s += step;
    return s;
}

// Where row t is kept: the head-0 block of its page and its token within the page; null
// where the sequence has no place or no valid page for it.
__device__ __forceinline__ uint8_t *place_of(const Kv4Batch &b, int s, int t, int &tok) {
    const int q0 = b.q_start[s], q1 = b.q_start[s + 1];
    const int64_t pos = (int64_t)b.kv_len[s] - q1 + t;
    if (t < q0 || t >= q1 || pos < 0) return nullptr;
    const int64_t col = pos / b.f.page;
    tok = (int)(pos - col * b.f.page);
    if (col >= b.cols) return nullptr;
    const int page = b.table[(int64_t)s * b.ld_table + col];
    if (page < 0 || page >= b.num_pages) return nullptr;
    return b.cache + (int64_t)page * b.f.page_bytes();
}

__device__ __forceinline__ float scale_of(uint32_t byte) { return __uint_as_float(byte << 23); }

__device__ __forceinline__ bf16x2 as_bf16x2(uint32_t u) {
    union { uint32_t u; bf16x2 h; } c;
    c.u = u;
    return c.h;
}

// Eight channels of a lane -> eight E2M1 codes; the block's scale byte in every lane of it.
__device__ __forceinline__ uint32_t quantize8(u32x4 x, uint32_t &byte) {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) m = max(m, max(x[i] & 0x7FFFu, (x[i] >> 16) & 0x7FFFu));
    m = max(m, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)m, 0xB1, 0xF, 0xF, false));  // lanes of 4
    m = max(m, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)m, 0x4E, 0xF, 0xF, false));
    const int e = (int)(m >> 7) - 2 + ((m & 127u) > 96u ? 1 : 0);
    byte = (uint32_t)min(max(e, 16), 252);
    const float s = scale_of(byte);
    uint32_t r = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(0, as_bf16x2(x[0]), s, 0);
    r = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(r, as_bf16x2(x[1]), s, 1);
    r = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(r, as_bf16x2(x[2]), s, 2);
    return __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(r, as_bf16x2(x[3]), s, 3);
}

__device__ __forceinline__ u32x4 dequantize8(uint32_t w, float s) {
    union { bf16x2 h[4]; u32x4 u; } c;
    c.h[0] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 0);
    c.h[1] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 1);
    c.h[2] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 2);
    c.h[3] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 3);
    return c.u;
}

constexpr int kThreads = 256;
constexpr int kFewWaves = 4096;
constexpr int kHeads = 4;  // heads whose rows a wave has in flight

// A lane takes 8 channels of one token and head, K and V.  The lanes of a wave cover one
// head of 4 (dim 128) or 8 (dim 64) consecutive tokens: four tokens of a sequence fill the
// 16-byte units of V.  A wave goes through `per` heads of them, so that the search for the
// token's place is paid once; rows are loaded before that search, which they do not need.
// Memory-bound: 4 bytes read and 1.06 written per channel.
template <int D, bool WRITE>
__global__ __launch_bounds__(kThreads) void kv4_rows_kernel(Kv4Batch b, Kv4Rows k, Kv4Rows v, int per) {
    constexpr int C8 = D / 8, ROWS = kWave / C8;
    b.f.dim = D;
    const int lane = threadIdx.x & 63;
    const uint32_t wave = __builtin_amdgcn_readfirstlane((blockIdx.x * kThreads + threadIdx.x) >> 6);
    const uint32_t parts = (b.f.n_kv + per - 1) / per;
    const int t0 = (int)(wave / parts) * ROWS, h0 = (int)(wave % parts) * per;
    if (t0 >= b.T) return;
    const int h1 = min(h0 + per, b.f.n_kv);
    const int t = t0 + lane / C8, c8 = lane % C8;
    uint16_t *kt = k.p + t * k.ld + c8 * 8, *vt = v.p + t * v.ld + c8 * 8;
    u32x4 kx[kHeads], vx[kHeads];
    auto load = [&](int h) {
#pragma unroll
        for (int i = 0; i < kHeads; ++i)
            if (h + i < h1 && t < b.T) {
                kx[i] = *reinterpret_cast<u32x4 *>(kt + (h + i) * k.hd);
                vx[i] = *reinterpret_cast<u32x4 *>(vt + (h + i) * v.hd);
            }
    };
    if (WRITE) load(h0);
    const int s0 = find_seq(b.q_start, b.S, t0, lane);
    if (t >= b.T || t >= b.q_start[b.S]) return;
    const int s = seq_of_row(b.q_start, b.S, s0, t0, t);
    int tok = 0;
    uint8_t *page = place_of(b, s, t, tok);
    if (WRITE && !page) return;  // all lanes of a row leave together
    const int k_at = b.f.k_byte(tok) + c8 * 4, v_at = b.f.v_word(tok, c8);
    const int ks_at = b.f.k_scale(tok, c8 >> 2), vs_at = b.f.v_scale(tok, c8 >> 2);
    for (int h = h0; h < h1; h += kHeads) {
        if constexpr (WRITE) {
            if (h > h0) load(h);
#pragma unroll
            for (int i = 0; i < kHeads; ++i) {
                if (h + i >= h1) break;
                uint8_t *p = page + (int64_t)(h + i) * b.f.head_bytes();
                uint32_t kb, vb;
                const uint32_t kw = quantize8(kx[i], kb), vw = quantize8(vx[i], vb);
                *reinterpret_cast<uint32_t *>(p + k_at) = kw;
                *reinterpret_cast<uint32_t *>(p + v_at) = vw;
                if ((c8 & 3) == 0) {
                    p[ks_at] = (uint8_t)kb;
                    p[vs_at] = (uint8_t)vb;
                }
            }
        } else {
            uint32_t kw[kHeads], vw[kHeads], ks[kHeads], vs[kHeads];
#pragma unroll
            for (int i = 0; i < kHeads; ++i) {
                kw[i] = vw[i] = 0;
                ks[i] = vs[i] = 127;
                if (h + i < h1 && page) {
                    const uint8_t *p = page + (int64_t)(h + i) * b.f.head_bytes();
                    kw[i] = *reinterpret_cast<const uint32_t *>(p + k_at);
                    vw[i] = *reinterpret_cast<const uint32_t *>(p + v_at);
                    ks[i] = p[ks_at];
                    vs[i] = p[vs_at];
                }
            }
#pragma unroll
            for (int i = 0; i < kHeads; ++i) {
                if (h + i >= h1) break;
                *reinterpret_cast<u32x4 *>(kt + (h + i) * k.hd) = dequantize8(kw[i], scale_of(ks[i]));
                *reinterpret_cast<u32x4 *>(vt + (h + i) * v.hd) = dequantize8(vw[i], scale_of(vs[i]));
            }
        }
    }
}

// Few rows: a wave to each head, for latency; many: the heads in turn once there are
// waves for every place on the machine (prompts of 9.4K rows in and out: 31 us a wave to each
// head, 25 us in turn).
template <bool WRITE>
hipError_t launch_rows(const Kv4Batch &b, const Kv4Rows &k, const Kv4Rows &v, hipStream_t st) {
    const int rows = kWave * 8 / b.f.dim;
    const int64_t groups = ((int64_t)b.T + rows - 1) / rows;
    const int per = groups * b.f.n_kv <= kFewWaves ? 1 : groups * ((b.f.n_kv + kHeads - 1) / kHeads) <= kFewWaves ? kHeads
                                                                                                         : b.f.n_kv;
    const int64_t waves = groups * ((b.f.n_kv + per - 1) / per);
    const dim3 grid((unsigned)((waves + 3) / 4));
    if (b.f.dim == 128)
        kv4_rows_kernel<128, WRITE><<<grid, kThreads, 0, st>>>(b, k, v, per);
    else
        kv4_rows_kernel<64, WRITE><<<grid, kThreads, 0, st>>>(b, k, v, per);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_kv4_append(const Kv4Batch &b, const Kv4Rows &k, const Kv4Rows &v, hipStream_t st) {
    return launch_rows<true>(b, k, v, st);
}

hipError_t launch_kv4_unpack(const Kv4Batch &b, const Kv4Rows &k, const Kv4Rows &v, hipStream_t st) {
    return launch_rows<false>(b, k, v, st);
}

}  // namespace nmk

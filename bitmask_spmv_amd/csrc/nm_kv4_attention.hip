// nm_kv4_attention.hip -- attention over the 4-bit key/value cache.
//
// For query row i of a sequence (place p = kv_len - rows + i) and head h:
//     s_j = scale * sum_c q_c K_jc,  m = max_j s_j,  l = sum_j exp(s_j - m),
//     o_c = sum_j exp(s_j - m) V_jc / l,  lse = m + log l,
// over the keys j <= p, and j > p - window where there is a window.
#include "nm_device.h"
#include "nm_kv.h"

namespace nmk {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

__device__ __forceinline__ float e2m1(uint32_t code) {
    const uint32_t e = (code >> 1) & 3u, m = code & 1u;
    const float a = e ? __uint_as_float(((e + 126u) << 23) | (m << 22)) : 0.5f * (float)m;
    return (code & 8u) ? -a : a;
}

__device__ __forceinline__ float pow2_byte(uint32_t byte) { return __uint_as_float(byte << 23); }

// One wave per row and head.  Lanes take one key each for the scores, then two channels
// each (one at dim 64) for the values.
template <int D>
__global__ __launch_bounds__(64) void kv4_attention_row_kernel(Kv4Attention a) {
    __shared__ float sq[D], sp[64];
    Kv4Batch &b = a.b;
    b.f.dim = D;
    const int lane = threadIdx.x, t = blockIdx.x, h = blockIdx.y;
    if (t >= b.q_start[b.S]) return;
    int lo = 0, hi = b.S;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (b.q_start[mid] <= t) lo = mid; else hi = mid;
    }
    const int s = lo;
    const int q0 = b.q_start[s], q1 = b.q_start[s + 1];
    if (t < q0 || t >= q1) return;
    const int64_t pos = (int64_t)b.kv_len[s] - q1 + t;
    const int64_t first = a.window > 0 && pos - a.window + 1 > 0 ? pos - a.window + 1 : 0;
    const int kvh = h / (a.heads / b.f.n_kv);
    const float c = a.scale * kLog2e;
    for (int i = lane; i < D; i += 64) sq[i] = bf16_lo(a.q.p[t * a.q.ld + h * a.q.hd + i]) * c;
    __syncthreads();
    float m = -INFINITY, l = 0.f, o[D / 64] = {};
    for (int64_t j0 = first & ~(int64_t)63; j0 <= pos; j0 += 64) {
        const int64_t col = j0 / b.f.page;
        if (col >= b.cols) break;
        const int page = b.table[(int64_t)s * b.ld_table + col];
        if (page < 0 || page >= b.num_pages) continue;
        const uint8_t *p = b.cache + (int64_t)page * b.f.page_bytes() + (int64_t)kvh * b.f.head_bytes();
        const int tok0 = (int)(j0 - col * b.f.page), tok = tok0 + lane;
        float x = -INFINITY;
        if (j0 + lane <= pos && j0 + lane >= first) {
            x = 0.f;
            for (int g = 0; g < D / 32; ++g) {
                float y = 0.f;
                for (int i = 0; i < 16; ++i) {
                    const uint32_t w = p[b.f.k_byte(tok) + g * 16 + i];
                    y += e2m1(w & 15u) * sq[g * 32 + 2 * i] + e2m1(w >> 4) * sq[g * 32 + 2 * i + 1];
                }
                x += y * pow2_byte(p[b.f.k_scale(tok, g)]);
            }
        }
        float top = x;
        for (int d = 32; d; d >>= 1) top = fmaxf(top, __shfl_xor(top, d));
        const float mn = fmaxf(m, top);
        if (mn == -INFINITY) continue;
        const float keep = exp2f(m - mn), pr = exp2f(x - mn);
        m = mn;
        l = l * keep + wave_sum(pr);
        sp[lane] = pr;
        __syncthreads();
        for (int i = 0; i < D / 64; ++i) o[i] *= keep;
        for (int j = 0; j < 64; ++j) {
            const float w = sp[j];
            if (w == 0.f) continue;  // masked places hold anything
            for (int i = 0; i < D / 64; ++i) {
                const int ch = lane + 64 * i;
                const uint32_t byte = p[b.f.v_word(tok0 + j, ch >> 3) + ((ch & 7) >> 1)];
                o[i] += w * e2m1((ch & 1) ? byte >> 4 : byte & 15u) * pow2_byte(p[b.f.v_scale(tok0 + j, ch >> 5)]);
            }
        }
        __syncthreads();
    }
    const float inv = l > 0.f ? 1.f / l : 0.f;
    for (int i = 0; i < D / 64; ++i)
        a.out.p[t * a.out.ld + h * a.out.hd + lane + 64 * i] = f32_to_bf16_rne(o[i] * inv);
    if (a.lse && lane == 0) a.lse[t * a.ld_lse + h] = l > 0.f ? (m + log2f(l)) * kLn2 : -INFINITY;
}

}  // namespace

size_t kv4_attention_workspace(int64_t, int64_t, int, int, int, int64_t) { return 0; }

hipError_t launch_kv4_attention(const Kv4Attention &a, int64_t, void *, hipStream_t st) {
    const dim3 grid((unsigned)a.b.T, (unsigned)a.heads);
    if (a.b.f.dim == 128)
        kv4_attention_row_kernel<128><<<grid, 64, 0, st>>>(a);
    else
        kv4_attention_row_kernel<64><<<grid, 64, 0, st>>>(a);
    return hipGetLastError();
}

}  // namespace nmk

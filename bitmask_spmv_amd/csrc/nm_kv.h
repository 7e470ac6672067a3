// nm_kv.h -- the 4-bit key/value cache: page format and launch interface shared by the
// C ABI (api.cpp) and the kernels (nm_kv4.hip, nm_kv4_attention.hip, nm_kv_pages.hip).
#pragma once

#include <hip/hip_runtime.h>
#include <math.h>
#include <stddef.h>
#include <stdint.h>

namespace nmk {

// Byte places of one head's block within a page: K values, V values, K scales, V scales.
// K values are token rows of D/2 bytes.  V values are units of 16 bytes, 4 tokens x 8
// channels, so a lane that multiplies over tokens finds the four of them side by side.
// K scales of 64 tokens are [16][D/32][4]: the dword of lane (r, b) holds the scales of
// tokens r, 16 + r, 32 + r, 48 + r, the four rows a wave's lane multiplies.  V scales of
// 4 tokens and one 32-channel block are one dword.
struct Kv4Format {
    int page = 64;     // tokens per page
    int n_kv = 1;      // key/value heads
    int dim = 128;     // channels per head (64 or 128)
    __host__ __device__ int v_at() const { return page * (dim / 2); }
    __host__ __device__ int ks_at() const { return page * dim; }
    __host__ __device__ int vs_at() const { return page * dim + page * (dim / 32); }
    __host__ __device__ int head_bytes() const { return page * dim + page * (dim / 32) * 2; }
    __host__ __device__ int64_t page_bytes() const { return (int64_t)n_kv * head_bytes(); }
    __host__ __device__ int k_byte(int t) const { return t * (dim / 2); }
    __host__ __device__ int v_word(int t, int c8) const { return v_at() + (((t >> 2) * (dim >> 3) + c8) * 4 + (t & 3)) * 4; }
    __host__ __device__ int k_scale(int t, int b) const {
        return ks_at() + (((t >> 6) * 16 + (t & 15)) * (dim / 32) + b) * 4 + ((t >> 4) & 3);
    }
    __host__ __device__ int v_scale(int t, int b) const { return vs_at() + ((t >> 2) * (dim / 32) + b) * 4 + (t & 3); }
};

// A ragged batch over a cache: sequence s owns rows q_start[s] .. q_start[s + 1] of the
// token arrays, and row i of them is at place kv_len[s] - rows + i of the sequence.
struct Kv4Batch {
    Kv4Format f;
    uint8_t *cache = nullptr;
    int64_t num_pages = 0;
    const int32_t *table = nullptr;
    int64_t ld_table = 0;
    int cols = 0;
    const int32_t *kv_len = nullptr;
    const int32_t *q_start = nullptr;
    int S = 0;
    int T = 0;
};

// Token arrays [T][heads][dim] with element strides of tokens and heads.
struct Kv4Rows {
    uint16_t *p = nullptr;
    int64_t ld = 0;
    int64_t hd = 0;
};

struct Kv4Attention {
    Kv4Batch b;
    Kv4Rows q, out;
    float *lse = nullptr;
    int64_t ld_lse = 0;
    int heads = 0;
    // Scores are (2^fold q . K) times c / log2(e), c / log2(e) in [1, 2) times a scale above 1: products stay in
    // range wherever the scores do.
    float c = 0.f;
    int16_t fold = 0;
    bool minus = false, zero = false;  // a scale below 0, of 0
    int64_t window = 0;  // keys a query looks back over, itself among them; 0: all
    bool whole = false;    // a workgroup to each row tile
    bool prompts = false;  // sequences of many rows are taken 128 rows at a time
    void set_scale(float scale) {
        const float size = fabsf(scale);
        minus = scale < 0.f;
        zero = scale == 0.f;
        fold = size > 0.f && size < 1.f ? (int16_t)ilogbf(size) : 0;
        c = (zero ? 1.f : ldexpf(size, -fold)) * 1.4426950408889634f;
    }
};

hipError_t launch_kv4_append(const Kv4Batch &b, const Kv4Rows &k, const Kv4Rows &v, hipStream_t st);
hipError_t launch_kv4_unpack(const Kv4Batch &b, const Kv4Rows &k, const Kv4Rows &v, hipStream_t st);
size_t kv4_attention_workspace(int64_t T, int64_t S, int heads, int n_kv, int dim, int64_t room);
hipError_t launch_kv4_attention(const Kv4Attention &a, int64_t max_q, void *ws, hipStream_t st);

// Page keeping.  Tables int32 [S][ld], lengths int32 [S], reference counts int32 [N].
struct KvBook {
    int32_t *table = nullptr;
    int64_t ld = 0;
    int cols = 0;
    int32_t *kv_len = nullptr;
    int S = 0;
    int32_t *refs = nullptr;
    int N = 0;
    int page = 64;
};
size_t kv_pages_workspace(int64_t S, int64_t n_pairs, int64_t num_pages, int64_t cols);
hipError_t launch_kv_fork(const KvBook &b, const int32_t *parent, const int32_t *child, int n, int32_t *moves,
                          int32_t *missing, void *ws, hipStream_t st);
hipError_t launch_kv_resize(const KvBook &b, const int32_t *new_len, int32_t *moves, int32_t *missing, void *ws,
                            hipStream_t st);
hipError_t launch_kv_compact(const KvBook &b, int32_t *moves, int cap, int32_t *used, void *ws, hipStream_t st);
hipError_t launch_kv_copy_pages(uint8_t *cache, int64_t num_pages, int64_t page_bytes, int64_t layers,
                                int64_t layer_stride, const int32_t *moves, int n, hipStream_t st);

}  // namespace nmk

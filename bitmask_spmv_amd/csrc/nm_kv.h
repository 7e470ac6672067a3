// nm_kv.h -- the 4-bit and the 8-bit key/value cache: page formats and launch interface shared by the
// C ABI (api.cpp) and the kernels (nm_kv4*.hip, nm_kv8*.hip, nm_kv_pages.hip).
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

// Byte places within a page of the 8-bit cache, in blocks of 64 tokens of one head: all values, then all
// bounds (the largest and the smallest key of the block in each channel), then all scales (a dword a block: byte 0 of the
// keys, byte 1 of the values).  K values are units of 16 channels of one token, a lane's bytes for the
// product over channels; V values units of one channel of the 16 tokens 16 j + 4 g + i, those that lane group
// g of a score tile has.  Rounded up to whole cache lines.
struct Kv8Format {
    int page = 64;
    int n_kv = 1;
    int dim = 128;
    __host__ __device__ int blocks() const { return page >> 6; }
    __host__ __device__ int block_bytes() const { return 128 * dim; }
    __host__ __device__ int bounds_at() const { return n_kv * blocks() * 128 * dim; }
    __host__ __device__ int scales_at() const { return n_kv * blocks() * 130 * dim; }
    __host__ __device__ int64_t page_bytes() const { return ((int64_t)scales_at() + n_kv * blocks() * 4 + 127) & ~(int64_t)127; }
    __host__ __device__ int k_byte(int t, int c) const { return ((c >> 4) * 64 + t) * 16 + (c & 15); }
    __host__ __device__ int v_byte(int t, int c) const { return 64 * dim + ((t >> 2 & 3) * dim + c) * 16 + (t >> 4) * 4 + (t & 3); }
};

// A ragged batch over a cache: sequence s owns rows q_start[s] .. q_start[s + 1] of the
// token arrays, and row i of them is at place kv_len[s] - rows + i of the sequence.
template <class F>
struct KvBatch {
    F f;
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

using Kv4Batch = KvBatch<Kv4Format>;
using Kv8Batch = KvBatch<Kv8Format>;

// Token arrays [T][heads][dim] with element strides of tokens and heads.
struct KvRows {
    uint16_t *p = nullptr;
    int64_t ld = 0;
    int64_t hd = 0;
};

using Kv4Rows = KvRows;

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

struct Kv8Attention {
    Kv8Batch b;
    KvRows q, out;
    float *lse = nullptr;
    int64_t ld_lse = 0;
    int heads = 0;
    float c = 0.f;                      // scores are (q . K) c / log2(e), c > 0
    bool minus = false, zero = false;  // a scale below 0, of 0
    int64_t window = 0;
    bool whole = false;
    bool prompts = false;
    const int32_t *selected = nullptr;  // [T][n_kv][top] blocks of 64 tokens that a row looks at; null: all
    int64_t ld_selected = 0;            // entries from a row to the next
    int top = 0;
    void set_scale(float scale) {
        minus = scale < 0.f;
        zero = scale == 0.f;
        c = (zero ? 1.f : fabsf(scale)) * 1.4426950408889634f;
    }
};

// Position rotation: cosine and sine of every place and pair of channels, fp32 [positions][ld].
struct KvRotation {
    const float *cos_sin = nullptr;  // null: none
    int64_t ld = 0;
    int dim = 0;  // channels that are rotated, the first of each head
    bool interleaved = false;
};

constexpr int kMaxSelectBlocks = 16384;  // blocks of a table row that a choice goes through: 2^20 tokens
struct Kv8Select {
    Kv8Batch b;
    KvRows q;
    int heads = 0;
    int top = 0, first = 0, last = 0;
    int32_t *out = nullptr;  // [T][n_kv][top]
    int64_t ld_out = 0;
};

hipError_t launch_kv8_append(const Kv8Batch &b, const KvRows &k, const KvRows &v, const KvRotation &r, const KvRows &q,
                             int heads, const KvRows &q_out, hipStream_t st);
hipError_t launch_kv8_unpack(const Kv8Batch &b, const KvRows &k, const KvRows &v, hipStream_t st);
size_t kv8_attention_workspace(int64_t T, int64_t S, int heads, int n_kv, int dim, int64_t room, int top);
hipError_t launch_kv8_attention(const Kv8Attention &a, int64_t max_q, void *ws, hipStream_t st);
size_t kv8_select_workspace(int64_t T, int64_t S, int n_kv, int64_t blocks);
hipError_t launch_kv8_select(const Kv8Select &a, void *ws, hipStream_t st);

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

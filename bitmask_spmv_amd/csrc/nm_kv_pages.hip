// nm_kv_pages.hip -- keeping the pages of a cache: fork, resize (reserve, truncate, free),
// compact, and the copying of page bytes that they ask for.
//
// State: a table row of page numbers per sequence (entries behind its last page are -1),
// its length in tokens, and a reference count per page (0: free).  Every operator is a
// function of that state alone: free pages are handed out lowest first, in the order of
// the requests, so results do not depend on the order in which workgroups run.
//
// Steps of fork and resize, one launch each (the counts of one step are the input of the
// next): pages given back; free pages counted per chunk of 4096, beside them the prefix
// sums of what is asked; pages handed out -- the free page of rank k goes to the request
// whose share of the prefix sums holds k.
#include "nm_device.h"
#include "nm_kv.h"

namespace nmk {
namespace {

constexpr int kThreads = 256;
constexpr int kChunk = 4096;  // pages per workgroup: 64 words of 64, one per lane of the first wave

__host__ __device__ inline int chunks_of(int64_t N) { return (int)((N + kChunk - 1) / kChunk); }

// What a request asks: `need` pages from column `col` on; `tail` >= 0: the first of them
// replaces that page and gets its bytes.  `row` < 0: nothing is done for it.
struct Request {
    int32_t need, col, tail, row;
};

struct Workspace {
    uint64_t *free_bits;   // [chunks * 64] one bit per page
    int32_t *chunk_count;  // [chunks]
    int32_t *prefix;       // [n] inclusive sums of need
    Request *req;          // [n]
    int32_t *valid;        // [n]
};

__host__ __device__ inline Workspace split_ws(void *ws, int64_t n, int64_t N) {
    Workspace w;
    const int64_t chunks = (N + kChunk - 1) / kChunk;
    char *p = (char *)ws;
    w.free_bits = (uint64_t *)p;
    p += chunks * 64 * 8;
    w.req = (Request *)p;
    p += n * sizeof(Request);
    w.chunk_count = (int32_t *)p;
    p += chunks * 4;
    w.prefix = (int32_t *)p;
    p += n * 4;
    w.valid = (int32_t *)p;
    return w;
}

__device__ __forceinline__ int pages_for(int64_t tokens, int page, int cols) {
    if (tokens <= 0) return 0;
    const int64_t n = (tokens + page - 1) / page;
    return n < cols ? (int)n : cols;
}

__device__ __forceinline__ bool in_pool(int page, int N) { return page >= 0 && page < N; }

__device__ int block_sum(int v, int *shared) {
    for (int d = 32; d; d >>= 1) v += __shfl_xor(v, d);
    if ((threadIdx.x & 63) == 0) shared[threadIdx.x >> 6] = v;
    __syncthreads();
    v = 0;
    for (int i = 0; i < kThreads / 64; ++i) v += shared[i];
    __syncthreads();
    return v;
}

// Gives back columns [keep, have) of a table row.
__device__ void release_row(const KvBook &b, int row, int keep, int have) {
    int32_t *t = b.table + (int64_t)row * b.ld;
    for (int c = keep + (int)threadIdx.x; c < have; c += kThreads) {
        const int page = t[c];
        if (in_pool(page, b.N)) atomicSub(&b.refs[page], 1);
        t[c] = -1;
    }
}

__global__ __launch_bounds__(kThreads) void resize_release_kernel(KvBook b, const int32_t *new_len) {
    const int s = blockIdx.x, want = new_len[s];
    if (want < 0) return;
    release_row(b, s, pages_for(want, b.page, b.cols), pages_for(b.kv_len[s], b.page, b.cols));
}

// A pair is carried out if its slots exist and differ, its child is not the child of an
// earlier pair, and its parent is nobody's child in this call.
__global__ __launch_bounds__(kThreads) void fork_release_kernel(KvBook b, const int32_t *parent, const int32_t *child,
                                                                int n, Workspace w) {
    const int i = blockIdx.x, p = parent[i], c = child[i];
    int ok = p >= 0 && p < b.S && c >= 0 && c < b.S && p != c;
    if (ok)
        for (int j = threadIdx.x; j < n; j += kThreads) {
            const int cj = child[j];
            if ((cj == c && j < i) || cj == p) ok = 0;
        }
    ok = __syncthreads_and(ok);
    if (threadIdx.x == 0) w.valid[i] = ok;
    if (ok) release_row(b, c, 0, pages_for(b.kv_len[c], b.page, b.cols));
}

// Workgroups 0 .. chunks - 1: which pages of the chunk are free, and how many.
__device__ void count_chunk(const int32_t *refs, int N, const Workspace &w, bool want_used) {
    __shared__ int part[kThreads / 64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    int total = 0;
    for (int i = wave; i < 64; i += kThreads / 64) {
        const int64_t page = (int64_t)blockIdx.x * kChunk + i * 64 + lane;
        const bool bit = page < N && (refs[page] > 0) == want_used;
        const uint64_t m = __ballot(bit);
        if (lane == 0) w.free_bits[(int64_t)blockIdx.x * 64 + i] = m;
        total += __popcll(m);
    }
    if (lane == 0) part[wave] = total;
    __syncthreads();
    if (threadIdx.x == 0) {
        total = 0;
        for (int i = 0; i < kThreads / 64; ++i) total += part[i];
        w.chunk_count[blockIdx.x] = total;
    }
}

// The last workgroup: inclusive prefix sums of the requests' needs.
template <class F>
__device__ void scan_requests(int n, const Workspace &w, F request) {
    __shared__ int part[kThreads / 64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    int base = 0;
    for (int i0 = 0; i0 < n; i0 += kThreads) {
        const int i = i0 + (int)threadIdx.x;
        Request r = {0, 0, -1, -1};
        if (i < n) r = request(i);
        int v = r.need;
        for (int d = 1; d < 64; d <<= 1) {
            const int u = __shfl_up(v, d);
            if (lane >= d) v += u;
        }
        if (lane == 63) part[wave] = v;
        __syncthreads();
        int before = base;
        for (int k = 0; k < kThreads / 64; ++k) {
            if (k < wave) before += part[k];
            base += part[k];
        }
        if (i < n) {
            w.req[i] = r;
            w.prefix[i] = before + v;
        }
        __syncthreads();
    }
}

__global__ __launch_bounds__(kThreads) void resize_count_kernel(KvBook b, const int32_t *new_len, Workspace w) {
    if ((int)blockIdx.x < (int)gridDim.x - 1) {
        count_chunk(b.refs, b.N, w, false);
        return;
    }
    scan_requests(b.S, w, [&](int s) {
        Request r = {0, 0, -1, -1};
        const int want = new_len[s], old = b.kv_len[s] > 0 ? b.kv_len[s] : 0;
        if (want < 0 || (int64_t)want > (int64_t)b.cols * b.page) return r;
        r.row = s;
        const int have = pages_for(old, b.page, b.cols), need = pages_for(want, b.page, b.cols);
        r.col = have;
        if (want > old && old % b.page != 0 && have > 0) {  // writes into its last page: shared pages are copied first
            const int tail = b.table[(int64_t)s * b.ld + have - 1];
            if (in_pool(tail, b.N) && b.refs[tail] > 1) {
                r.tail = tail;
                r.col = have - 1;
            }
        }
        r.need = need > r.col ? need - r.col : 0;
        if (want <= old) r.need = 0;
        return r;
    });
}

__global__ __launch_bounds__(kThreads) void fork_count_kernel(KvBook b, const int32_t *parent, const int32_t *child,
                                                              int n, Workspace w) {
    if ((int)blockIdx.x < (int)gridDim.x - 1) {
        count_chunk(b.refs, b.N, w, false);
        return;
    }
    scan_requests(n, w, [&](int i) {
        Request r = {0, 0, -1, -1};
        if (!w.valid[i]) return r;
        const int64_t cap = (int64_t)b.cols * b.page;
        const int64_t len = b.kv_len[parent[i]];
        r.row = child[i];
        if (len <= 0 || len > cap) return r;
        r.col = (int)(len / b.page);
        if (len % b.page) {
            const int tail = b.table[(int64_t)parent[i] * b.ld + r.col];
            r.need = 1;
            r.tail = in_pool(tail, b.N) ? tail : -1;
        }
        return r;
    });
}

// Sum of the chunk counts, and of those before this chunk.
__device__ int sum_chunks(const int32_t *count, int chunks, int upto, int &before) {
    __shared__ int sh[kThreads / 64];
    int all = 0, pre = 0;
    for (int i = threadIdx.x; i < chunks; i += kThreads) {
        const int c = count[i];
        all += c;
        if (i < upto) pre += c;
    }
    before = block_sum(pre, sh);
    return block_sum(all, sh);
}

// Hands out the free pages of one chunk.
__device__ void assign_chunk(const KvBook &b, int chunk, int chunks, int n, const Workspace &w, int32_t *moves) {
    int before;
    const int nfree = sum_chunks(w.chunk_count, chunks, chunk, before);
    const int asked = n > 0 ? w.prefix[n - 1] : 0;
    if (before >= asked) return;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    for (int i = 0; i < 64; ++i) {
        const uint64_t m = w.free_bits[(int64_t)chunk * 64 + i];
        const int k = before + __popcll(m & ((1ull << lane) - 1));
        before += __popcll(m);
        if (i % (kThreads / 64) != wave || !((m >> lane) & 1) || k >= asked) continue;
        int lo = 0, hi = n - 1;  // the first request whose prefix sum is above k
        while (lo < hi) {
            const int mid = (lo + hi) >> 1;
            if (w.prefix[mid] > k) hi = mid; else lo = mid + 1;
        }
        const Request r = w.req[lo];
        if (w.prefix[lo] > nfree || r.row < 0) continue;
        const int idx = k - (w.prefix[lo] - r.need), page = chunk * kChunk + i * 64 + lane;
        b.table[(int64_t)r.row * b.ld + r.col + idx] = page;
        b.refs[page] = 1;
        if (idx == 0 && r.tail >= 0) {
            moves[2 * lo] = r.tail;
            moves[2 * lo + 1] = page;
        }
    }
}

__global__ __launch_bounds__(kThreads) void resize_assign_kernel(KvBook b, const int32_t *new_len, Workspace w,
                                                                 int32_t *moves, int32_t *missing) {
    const int chunks = chunks_of(b.N);
    if ((int)blockIdx.x < chunks) {
        assign_chunk(b, blockIdx.x, chunks, b.S, w, moves);
        return;
    }
    int before;
    const int nfree = sum_chunks(w.chunk_count, chunks, 0, before);
    const int s = ((int)blockIdx.x - chunks) * kThreads + (int)threadIdx.x;
    if (s == 0) *missing = w.prefix[b.S - 1] > nfree ? w.prefix[b.S - 1] - nfree : 0;
    if (s >= b.S) return;
    const Request r = w.req[s];
    const bool ok = r.row >= 0 && (r.need == 0 || w.prefix[s] <= nfree);
    if (ok) b.kv_len[s] = new_len[s];
    if (!ok || r.need == 0 || r.tail < 0)
        moves[2 * s] = moves[2 * s + 1] = -1;
    else
        atomicSub(&b.refs[r.tail], 1);
}

__global__ __launch_bounds__(kThreads) void fork_assign_kernel(KvBook b, const int32_t *parent, int n, Workspace w,
                                                               int32_t *moves, int32_t *missing) {
    const int chunks = chunks_of(b.N);
    if ((int)blockIdx.x < chunks) {
        assign_chunk(b, blockIdx.x, chunks, n, w, moves);
        return;
    }
    int before;
    const int nfree = sum_chunks(w.chunk_count, chunks, 0, before);
    const int i = (int)blockIdx.x - chunks;
    if (i == 0 && threadIdx.x == 0) *missing = w.prefix[n - 1] > nfree ? w.prefix[n - 1] - nfree : 0;
    const Request r = w.req[i];
    const bool ok = r.row >= 0 && (r.need == 0 || w.prefix[i] <= nfree);
    if (threadIdx.x == 0) {
        if (!ok || r.need == 0 || r.tail < 0) moves[2 * i] = moves[2 * i + 1] = -1;
        if (r.row >= 0) b.kv_len[r.row] = ok && (r.col > 0 || r.need) ? b.kv_len[parent[i]] : 0;
    }
    if (r.row < 0) return;
    const int32_t *from = b.table + (int64_t)parent[i] * b.ld;
    int32_t *to = b.table + (int64_t)r.row * b.ld;
    for (int c = threadIdx.x; c < b.cols; c += kThreads) {
        if (ok && r.need && c == r.col) continue;  // written where its page is handed out
        int page = -1;
        if (ok && c < r.col) {
            page = from[c];
            if (in_pool(page, b.N)) atomicAdd(&b.refs[page], 1);
        }
        to[c] = page;
    }
}

// Compaction.  U pages are used: the j-th used page at or behind U moves into the j-th
// free page before it.
__global__ __launch_bounds__(kThreads) void compact_count_kernel(KvBook b, Workspace w) {
    count_chunk(b.refs, b.N, w, true);
}

// Used pages before page U, U being their number.
__device__ int used_before_u(const Workspace &w, int chunks, int &U, int &before) {
    U = sum_chunks(w.chunk_count, chunks, blockIdx.x, before);
    int rank;
    const int cu = U / kChunk;
    (void)sum_chunks(w.chunk_count, chunks, cu, rank);
    const int in = U - cu * kChunk;
    if (cu < chunks)
        for (int i = 0; i * 64 < in; ++i) {
            const uint64_t m = w.free_bits[(int64_t)cu * 64 + i];
            const int left = in - i * 64;
            rank += __popcll(left >= 64 ? m : m & ((1ull << left) - 1));
        }
    return rank;
}

__global__ __launch_bounds__(kThreads) void compact_match_kernel(KvBook b, Workspace w, int32_t *to_move,
                                                                 int32_t *moves, int cap, int32_t *used) {
    const int chunks = chunks_of(b.N);
    int U, rank;
    const int rank_u = used_before_u(w, chunks, U, rank);
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    if (blockIdx.x == 0 && threadIdx.x == 0) *used = U;
    for (int i = 0; i < 64; ++i) {
        const uint64_t m = w.free_bits[(int64_t)blockIdx.x * 64 + i];
        const int k = rank + __popcll(m & ((1ull << lane) - 1)), page = (int)blockIdx.x * kChunk + i * 64 + lane;
        rank += __popcll(m);
        if (i % (kThreads / 64) != wave || page >= b.N) continue;
        if ((m >> lane) & 1) {
            if (page >= U) {
                const int j = k - rank_u;
                to_move[page] = j;
                if (j < cap) moves[2 * j] = page;
            }
        } else if (page < U) {
            const int j = page - k;
            if (j < cap) moves[2 * j + 1] = page;
        }
    }
    // the list behind the moves
    const int made = min(U - rank_u, cap);
    for (int64_t j = made + (int64_t)blockIdx.x * kThreads + threadIdx.x; j < cap; j += (int64_t)gridDim.x * kThreads)
        moves[2 * j] = moves[2 * j + 1] = -1;
}

__global__ __launch_bounds__(kThreads) void compact_apply_kernel(KvBook b, Workspace w, const int32_t *to_move,
                                                                 const int32_t *moves, int cap, const int32_t *used) {
    const int U = *used;
    if ((int)blockIdx.x < b.S) {
        const int s = blockIdx.x, have = pages_for(b.kv_len[s], b.page, b.cols);
        int32_t *t = b.table + (int64_t)s * b.ld;
        for (int c = threadIdx.x; c < have; c += kThreads) {
            const int page = t[c];
            if (page < U || page >= b.N || !((w.free_bits[page >> 6] >> (page & 63)) & 1)) continue;
            const int j = to_move[page];
            if (j < cap) t[c] = moves[2 * j + 1];
        }
        return;
    }
    for (int64_t j = (int64_t)((int)blockIdx.x - b.S) * kThreads + threadIdx.x; j < cap;
         j += (int64_t)((int)gridDim.x - b.S) * kThreads) {
        const int of = moves[2 * j], to = moves[2 * j + 1];
        if (of < 0) break;
        b.refs[to] = b.refs[of];
        b.refs[of] = 0;
    }
}

// Page bytes: each workgroup takes pieces of 16 KiB, four 16-byte loads in flight per
// thread.  Moves whose pages are not in the pool are left out.
constexpr int kPiece = 16384;

__global__ __launch_bounds__(kThreads) void copy_pages_kernel(uint8_t *cache, int64_t num_pages, int64_t page_bytes,
                                                              int64_t layers, int64_t layer_stride,
                                                              const int32_t *moves, int n) {
    const int pieces = (int)((page_bytes + kPiece - 1) / kPiece);
    const int64_t units = (int64_t)n * layers * pieces;
    for (int64_t u = blockIdx.x; u < units; u += gridDim.x) {
        const int64_t i = u / (layers * pieces);
        const int rest = (int)(u - i * layers * pieces);
        const int layer = rest / pieces, piece = rest - layer * pieces;
        const int src = moves[2 * i], dst = moves[2 * i + 1];
        if (src < 0 || dst < 0 || src >= num_pages || dst >= num_pages || src == dst) continue;
        const int64_t at = (int64_t)layer * layer_stride + (int64_t)piece * kPiece;
        const int64_t left = page_bytes - (int64_t)piece * kPiece;
        const int words = (int)((left < kPiece ? left : kPiece) / 16);
        const u32x4 *from = reinterpret_cast<const u32x4 *>(cache + at + src * page_bytes);
        u32x4 *to = reinterpret_cast<u32x4 *>(cache + at + dst * page_bytes);
        u32x4 x[4];
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if ((int)threadIdx.x + k * kThreads < words) x[k] = __builtin_nontemporal_load(from + threadIdx.x + k * kThreads);
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if ((int)threadIdx.x + k * kThreads < words) __builtin_nontemporal_store(x[k], to + threadIdx.x + k * kThreads);
    }
}

size_t compact_base(int64_t N) {
    const int64_t chunks = chunks_of(N);
    return (size_t)(chunks * 64 * 8 + ((chunks * 4 + 15) & ~(int64_t)15));
}

}  // namespace

size_t kv_pages_workspace(int64_t requests, int64_t num_pages) {
    const size_t chunks = (size_t)chunks_of(num_pages);
    const size_t ask = chunks * 64 * 8 + (size_t)requests * sizeof(Request) + chunks * 4 + (size_t)requests * 8;
    const size_t compact = compact_base(num_pages) + (size_t)num_pages * 4;
    return ask > compact ? ask : compact;
}

hipError_t launch_kv_fork(const KvBook &b, const int32_t *parent, const int32_t *child, int n, int32_t *moves,
                          int32_t *missing, void *ws, hipStream_t st) {
    const Workspace w = split_ws(ws, n, b.N);
    const int chunks = chunks_of(b.N);
    fork_release_kernel<<<n, kThreads, 0, st>>>(b, parent, child, n, w);
    fork_count_kernel<<<chunks + 1, kThreads, 0, st>>>(b, parent, child, n, w);
    fork_assign_kernel<<<chunks + n, kThreads, 0, st>>>(b, parent, n, w, moves, missing);
    return hipGetLastError();
}

hipError_t launch_kv_resize(const KvBook &b, const int32_t *new_len, int32_t *moves, int32_t *missing, void *ws,
                            hipStream_t st) {
    const Workspace w = split_ws(ws, b.S, b.N);
    const int chunks = chunks_of(b.N);
    resize_release_kernel<<<b.S, kThreads, 0, st>>>(b, new_len);
    resize_count_kernel<<<chunks + 1, kThreads, 0, st>>>(b, new_len, w);
    resize_assign_kernel<<<chunks + (b.S + kThreads - 1) / kThreads, kThreads, 0, st>>>(b, new_len, w, moves, missing);
    return hipGetLastError();
}

hipError_t launch_kv_compact(const KvBook &b, int32_t *moves, int cap, int32_t *used, void *ws, hipStream_t st) {
    const Workspace w = split_ws(ws, 0, b.N);
    int32_t *to_move = (int32_t *)((char *)ws + compact_base(b.N));
    const int chunks = chunks_of(b.N);
    compact_count_kernel<<<chunks, kThreads, 0, st>>>(b, w);
    compact_match_kernel<<<chunks, kThreads, 0, st>>>(b, w, to_move, moves, cap, used);
    const int more = (int)(((int64_t)cap + kThreads - 1) / kThreads);
    compact_apply_kernel<<<b.S + (more < 64 ? more : 64), kThreads, 0, st>>>(b, w, to_move, moves, cap, used);
    return hipGetLastError();
}

hipError_t launch_kv_copy_pages(uint8_t *cache, int64_t num_pages, int64_t page_bytes, int64_t layers,
                                int64_t layer_stride, const int32_t *moves, int n, hipStream_t st) {
    const int64_t units = (int64_t)n * layers * ((page_bytes + kPiece - 1) / kPiece);
    copy_pages_kernel<<<(unsigned)(units < 4096 ? units : 4096), kThreads, 0, st>>>(cache, num_pages, page_bytes, layers,
                                                                                  layer_stride, moves, n);
    return hipGetLastError();
}

}  // namespace nmk

// nm_kv_pages.hip -- keeping the pages of a cache: fork, resize (reserve, truncate, free),
// compact, and the copying of page bytes that they ask for.
//
// State: a table row of page numbers per sequence (entries behind its last page are -1),
// its length in tokens, and a reference count per page (0: free).  Every operator is a
// function of that state alone: free pages are handed out lowest first, in the order of
// the requests, so results do not depend on the order in which workgroups run.
//
// Steps of fork and resize: pages given back; free pages counted, beside them the prefix
// sums of what is asked; pages handed out -- the free page of rank k goes to the request
// whose share of the prefix sums holds k.  Small pools and few requests go through all
// steps in one workgroup and need no workspace (one launch: 4-6 us; three launches: 12-17 us);
// larger ones take a launch for each step, a workgroup to each 4096 pages.
#include "nm_device.h"
#include "nm_kv.h"

namespace nmk {
namespace {

constexpr int kThreads = 1024;
constexpr int kWavesPerGroup = kThreads / kWave;
constexpr int kChunk = 4096;         // pages per workgroup: 64 words of 64
constexpr int kSmallPages = 16384;   // one workgroup: 256 words of 64 pages in LDS,
constexpr int kSmallRequests = 64;   // pairs, a wave to each in turn (4: 6 us against 13; 224: 60 us against 14),
constexpr int kSmallRows = 256;      // sequences, a thread to each and a wave to their rows in turn,
constexpr int kSmallEntries = 65536; // and their entries
constexpr int kPrefixLds = 4096;     // requests whose prefix sums a workgroup searches in LDS

__host__ __device__ inline int chunks_of(int64_t N) { return (int)((N + kChunk - 1) / kChunk); }

// What a request asks: `need` pages from column `col` on; `tail` >= 0: the first of them
// replaces that page and gets its bytes.  `row` < 0: nothing is done for it.
struct Request {
    int32_t need, col, tail, row;
};

struct Workspace {
    uint64_t *bits;        // [chunks * 64] one bit per page: free (fork, resize) or used (compact)
    Request *req;          // [n]
    int32_t *chunk_count;  // [chunks]
    int32_t *prefix;       // [n] inclusive sums of need
    int32_t *valid;        // [n]
};

inline Workspace split_ws(void *ws, int64_t n, int64_t N) {
    Workspace w;
    const int64_t chunks = chunks_of(N);
    char *p = (char *)ws;
    w.bits = (uint64_t *)p;
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

// A count that other lanes have just changed by atomics: read where they were made.
__device__ __forceinline__ int fresh(const int32_t *p) {
    return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

// A barrier behind which atomics and stores of the workgroup have been carried out: each wave waits for its own,
// and what reads their results reads where they were made (`fresh`).  A fence for the whole device
// would also write the caches back, for readers that a single workgroup does not have (resize of 16
// sequences 8.5 -> 5.6 us, of it a part by reading last pages before the barrier).
__device__ __forceinline__ void done_in_group() {
    __builtin_amdgcn_s_waitcnt(0);
    __syncthreads();
}

__device__ __forceinline__ uint64_t below(int lane) { return (1ull << lane) - 1; }

// Inclusive sum over the lanes of a wave.
template <int kCtrl, int kRowMask>
__device__ __forceinline__ int dpp_scan_step(int v) {
    return v + __builtin_amdgcn_update_dpp(0, v, kCtrl, kRowMask, 0xF, false);
}
__device__ __forceinline__ int wave_scan(int v) {
    v = dpp_scan_step<0x111, 0xF>(v);
    v = dpp_scan_step<0x112, 0xF>(v);
    v = dpp_scan_step<0x114, 0xF>(v);
    v = dpp_scan_step<0x118, 0xF>(v);
    v = dpp_scan_step<0x142, 0xA>(v);
    return dpp_scan_step<0x143, 0xC>(v);
}

// Inclusive sum over the threads of a workgroup; `total` is that of all of them.
__device__ __forceinline__ int group_scan(int v, int *part, int &total) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    v = wave_scan(v);
    if (lane == 63) part[wave] = v;
    __syncthreads();
    const int p = wave_scan(lane < kWavesPerGroup ? part[lane] : 0);
    total = __shfl(p, kWavesPerGroup - 1);
    const int before = __shfl(p, wave ? wave - 1 : 0);
    __syncthreads();
    return v + (wave ? before : 0);
}

// ---- steps ----

// Gives back columns [keep, have) of a table row; `lane` of `lanes` threads.
__device__ __forceinline__ void release_row(const KvBook &b, int row, int keep, int have, int lane, int lanes) {
    int32_t *t = b.table + (int64_t)row * b.ld;
    for (int c = keep + lane; c < have; c += lanes) {
        const int page = t[c];
        if (in_pool(page, b.N)) atomicSub(&b.refs[page], 1);
        t[c] = -1;
    }
}

// A pair is carried out if its slots exist and differ, its child is not the child of an
// earlier pair, and its parent is nobody's child in this call.
__device__ __forceinline__ bool slots_exist(const KvBook &b, int p, int c) {
    return p >= 0 && p < b.S && c >= 0 && c < b.S && p != c;
}

// The page that a sequence of `len` tokens writes next into, if its last page is partly filled; else -1.
__device__ __forceinline__ int tail_page(const KvBook &b, int s, int64_t len) {
    if (len <= 0 || len > (int64_t)b.cols * b.page || len % b.page == 0) return -1;
    const int tail = b.table[(int64_t)s * b.ld + len / b.page];
    return in_pool(tail, b.N) ? tail : -1;
}

// old: the length now; tail: its tail_page, which `holders` sequences hold.
__device__ __forceinline__ Request resize_request(const KvBook &b, int s, int want, int old, int tail, int holders) {
    Request r = {0, 0, -1, -1};
    if (old < 0) old = 0;
    if (want < 0 || (int64_t)want > (int64_t)b.cols * b.page) return r;
    r.row = s;
    const int have = pages_for(old, b.page, b.cols), pages = pages_for(want, b.page, b.cols);
    r.col = have;
    if (want <= old) return r;
    if (tail >= 0 && holders > 1) {  // writes into its last page: shared pages are copied first
        r.tail = tail;
        r.col = have - 1;
    }
    r.need = pages > r.col ? pages - r.col : 0;
    return r;
}

__device__ __forceinline__ Request fork_request(const KvBook &b, int c, int64_t len, int tail) {
    Request r = {0, 0, -1, c};
    if (len <= 0 || len > (int64_t)b.cols * b.page) return r;
    r.col = (int)(len / b.page);
    if (len % b.page) {
        r.need = 1;
        r.tail = tail;
    }
    return r;
}

// The free page of rank k to its request.  `prefix` and `req` may be in LDS or not.
__device__ __forceinline__ void hand_out(const KvBook &b, int page, int k, int n, int nfree, const int32_t *prefix,
                                         const Request *req, int32_t *moves) {
    int lo = 0, hi = n - 1;  // the first request whose prefix sum is above k
    while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (prefix[mid] > k) hi = mid; else lo = mid + 1;
    }
    const int upto = prefix[lo];
    const Request r = req[lo];
    if (upto > nfree || r.row < 0) return;
    const int idx = k - (upto - r.need);
    b.table[(int64_t)r.row * b.ld + r.col + idx] = page;
    b.refs[page] = 1;
    if (idx == 0 && r.tail >= 0) {
        moves[2 * lo] = r.tail;
        moves[2 * lo + 1] = page;
    }
}

// What is left to do for a sequence or a pair; `ok`: it got its pages.
__device__ __forceinline__ void resize_row(const KvBook &b, int s, const Request &r, bool ok, int want,
                                           int32_t *moves) {
    if (ok) b.kv_len[s] = want;
    if (!ok || r.need == 0 || r.tail < 0)
        moves[2 * s] = moves[2 * s + 1] = -1;
    else
        atomicSub(&b.refs[r.tail], 1);
}

__device__ __forceinline__ void fork_row(const KvBook &b, int i, int p, const Request &r, bool ok, int32_t *moves,
                                         int lane, int lanes) {
    if (lane == 0) {
        if (!ok || r.need == 0 || r.tail < 0) moves[2 * i] = moves[2 * i + 1] = -1;
        if (r.row >= 0) b.kv_len[r.row] = ok && (r.col > 0 || r.need) ? b.kv_len[p] : 0;
    }
    if (r.row < 0) return;
    const int32_t *from = b.table + (int64_t)p * b.ld;
    int32_t *to = b.table + (int64_t)r.row * b.ld;
    for (int c = lane; c < b.cols; c += lanes) {
        if (ok && r.need && c == r.col) continue;  // written where its page is handed out
        int page = -1;
        if (ok && c < r.col) {
            page = from[c];
            if (in_pool(page, b.N)) atomicAdd(&b.refs[page], 1);
        }
        to[c] = page;
    }
}

// ---- one workgroup ----

struct SmallPool {
    uint64_t bits[kSmallPages / 64];
    int base[kSmallPages / 64];  // set bits before each word
    int part[kWavesPerGroup];
};

// Bits of pages that are free (or used) and their ranks; the number of them.
__device__ int small_bits(SmallPool &p, const int32_t *refs, int N, bool want_used) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int words = (N + 63) / 64;
    for (int w0 = 0; w0 < words; w0 += 4 * kWavesPerGroup) {
        int r[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int page = (w0 + j * kWavesPerGroup + wave) * 64 + lane;
            r[j] = page < N ? fresh(refs + page) : 0;
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int w = w0 + j * kWavesPerGroup + wave;
            const uint64_t m = __ballot(w * 64 + lane < N && (r[j] > 0) == want_used);
            if (lane == 0 && w < words) p.bits[w] = m;
        }
    }
    __syncthreads();
    int total;
    const int mine = (int)threadIdx.x < words ? __popcll(p.bits[threadIdx.x]) : 0;
    const int upto = group_scan(mine, p.part, total);
    if ((int)threadIdx.x < words) p.base[threadIdx.x] = upto - mine;
    __syncthreads();
    return total;
}

struct SmallRequests {
    Request req[kThreads];
    int32_t prefix[kThreads];
    uint8_t valid[kThreads];
    int32_t child[kSmallRequests];
};

// Requests' prefix sums, the pages handed out, and how many were asked for.
__device__ int small_hand_out(const KvBook &b, SmallPool &p, SmallRequests &q, int n, const Request &r, int nfree,
                              int32_t *moves) {
    int asked;
    const int upto = group_scan(r.need, p.part, asked);
    q.req[threadIdx.x] = r;
    q.prefix[threadIdx.x] = upto;
    __syncthreads();
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, words = (b.N + 63) / 64;
    for (int w = wave; w < words; w += kWavesPerGroup) {
        const uint64_t m = p.bits[w];
        const int k = p.base[w] + __popcll(m & below(lane));
        if (((m >> lane) & 1) && k < asked) hand_out(b, w * 64 + lane, k, n, nfree, q.prefix, q.req, moves);
    }
    return asked;
}

__global__ __launch_bounds__(kThreads) void resize_small_kernel(KvBook b, const int32_t *new_len, int32_t *moves,
                                                                int32_t *missing) {
    __shared__ SmallPool p;
    __shared__ SmallRequests q;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, s = threadIdx.x;
    const int want = s < b.S ? new_len[s] : -1, old = s < b.S ? b.kv_len[s] : 0;
    const int tail = s < b.S ? tail_page(b, s, old) : -1;  // of use to a sequence that grows, whose row stays as it is
    const int have = pages_for(old, b.page, b.cols);
    const int keep = want < 0 ? have : pages_for(want, b.page, b.cols);
    for (uint64_t left = __ballot(keep < have); left; left &= left - 1) {  // my wave's sequences that give pages back
        const int i = __builtin_ctzll(left);
        release_row(b, wave * 64 + i, __builtin_amdgcn_readlane(keep, i), __builtin_amdgcn_readlane(have, i), lane, 64);
    }
    done_in_group();
    const int holders = tail >= 0 ? fresh(&b.refs[tail]) : 0;
    const int nfree = small_bits(p, b.refs, b.N, false);
    Request r = {0, 0, -1, -1};
    if (s < b.S) r = resize_request(b, s, want, old, tail, holders);
    const int asked = small_hand_out(b, p, q, b.S, r, nfree, moves);
    if (s == 0) *missing = asked > nfree ? asked - nfree : 0;
    if (s < b.S) resize_row(b, s, r, r.row >= 0 && (r.need == 0 || q.prefix[s] <= nfree), want, moves);
}

__global__ __launch_bounds__(kThreads) void fork_small_kernel(KvBook b, const int32_t *parent, const int32_t *child,
                                                              int n, int32_t *moves, int32_t *missing) {
    __shared__ SmallPool p;
    __shared__ SmallRequests q;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, t = threadIdx.x;
    const int to_t = t < n ? child[t] : -1, from_t = t < n ? parent[t] : -1;
    if (t < n) q.child[t] = to_t;
    __syncthreads();
    // a parent is nobody's child: its row stays as it is
    const int64_t len = slots_exist(b, from_t, to_t) ? b.kv_len[from_t] : 0;
    const int tail = tail_page(b, from_t, len);
    for (int i = wave; i < n; i += kWavesPerGroup) {
        const int from = parent[i], to = q.child[i];
        bool ok = slots_exist(b, from, to);
        for (int j = lane; j < n; j += 64) ok = ok && !((q.child[j] == to && j < i) || q.child[j] == from);
        ok = __all(ok);
        if (lane == 0) q.valid[i] = ok;
        if (ok) release_row(b, to, 0, pages_for(b.kv_len[to], b.page, b.cols), lane, 64);
    }
    done_in_group();
    const int nfree = small_bits(p, b.refs, b.N, false);
    Request r = {0, 0, -1, -1};
    if (t < n && q.valid[t]) r = fork_request(b, to_t, len, tail);
    const int asked = small_hand_out(b, p, q, n, r, nfree, moves);
    if (t == 0) *missing = asked > nfree ? asked - nfree : 0;
    for (int i = wave; i < n; i += kWavesPerGroup) {
        const Request x = q.req[i];
        fork_row(b, i, parent[i], x, x.row >= 0 && (x.need == 0 || q.prefix[i] <= nfree), moves, lane, 64);
    }
}

// ---- a launch for each step ----

__global__ __launch_bounds__(256) void resize_release_kernel(KvBook b, const int32_t *new_len) {
    const int s = blockIdx.x, want = new_len[s];
    if (want < 0) return;
    release_row(b, s, pages_for(want, b.page, b.cols), pages_for(b.kv_len[s], b.page, b.cols), threadIdx.x, 256);
}

__global__ __launch_bounds__(256) void fork_release_kernel(KvBook b, const int32_t *parent, const int32_t *child, int n,
                                                           Workspace w) {
    const int i = blockIdx.x, p = parent[i], c = child[i];
    int ok = slots_exist(b, p, c);
    if (ok)
        for (int j = threadIdx.x; j < n; j += 256) {
            const int cj = child[j];
            if ((cj == c && j < i) || cj == p) ok = 0;
        }
    ok = __syncthreads_and(ok);
    if (threadIdx.x == 0) w.valid[i] = ok;
    if (ok) release_row(b, c, 0, pages_for(b.kv_len[c], b.page, b.cols), threadIdx.x, 256);
}

// Which pages of the workgroup's chunk are free (or used), and how many.
__device__ void count_chunk(const int32_t *refs, int N, const Workspace &w, bool want_used) {
    __shared__ int part[kWavesPerGroup];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    constexpr int kEach = 64 / kWavesPerGroup;
    int r[kEach], count = 0;
#pragma unroll
    for (int j = 0; j < kEach; ++j) {
        const int64_t page = (int64_t)blockIdx.x * kChunk + (j * kWavesPerGroup + wave) * 64 + lane;
        r[j] = page < N ? refs[page] : 0;
    }
#pragma unroll
    for (int j = 0; j < kEach; ++j) {
        const int word = j * kWavesPerGroup + wave;
        const bool real = (int64_t)blockIdx.x * kChunk + word * 64 + lane < N;
        const uint64_t m = __ballot(real && (r[j] > 0) == want_used);
        if (lane == 0) w.bits[(int64_t)blockIdx.x * 64 + word] = m;
        count += __popcll(m);
    }
    if (lane == 0) part[wave] = count;
    __syncthreads();
    if (threadIdx.x == 0) {
        for (int i = 1; i < kWavesPerGroup; ++i) count += part[i];
        w.chunk_count[blockIdx.x] = count;
    }
}

// Inclusive prefix sums of the requests' needs.
template <class F>
__device__ void scan_requests(int n, const Workspace &w, F request) {
    __shared__ int part[kWavesPerGroup];
    int base = 0;
    for (int i0 = 0; i0 < n; i0 += kThreads) {
        const int i = i0 + (int)threadIdx.x;
        Request r = {0, 0, -1, -1};
        if (i < n) r = request(i);
        int total;
        const int upto = base + group_scan(r.need, part, total);
        base += total;
        if (i < n) {
            w.req[i] = r;
            w.prefix[i] = upto;
        }
    }
}

// Workgroups count a chunk each; the last one goes through the requests.
__global__ __launch_bounds__(kThreads) void resize_count_kernel(KvBook b, const int32_t *new_len, Workspace w) {
    if ((int)blockIdx.x < (int)gridDim.x - 1)
        count_chunk(b.refs, b.N, w, false);
    else
        scan_requests(b.S, w, [&](int s) {
            const int old = b.kv_len[s], tail = tail_page(b, s, old);
            return resize_request(b, s, new_len[s], old, tail, tail >= 0 ? fresh(&b.refs[tail]) : 0);
        });
}

__global__ __launch_bounds__(kThreads) void fork_count_kernel(KvBook b, const int32_t *parent, const int32_t *child,
                                                              int n, Workspace w) {
    if ((int)blockIdx.x < (int)gridDim.x - 1)
        count_chunk(b.refs, b.N, w, false);
    else
        scan_requests(n, w, [&](int i) {
            const Request none = {0, 0, -1, -1};
            if (!w.valid[i]) return none;
            const int64_t len = b.kv_len[parent[i]];
            return fork_request(b, child[i], len, tail_page(b, parent[i], len));
        });
}

// Sum of the chunk counts, and of those before chunk `upto`.
__device__ int sum_chunks(const int32_t *count, int chunks, int upto, int &before) {
    __shared__ int part[kWavesPerGroup];
    int all = 0, pre = 0;
    for (int i = threadIdx.x; i < chunks; i += kThreads) {
        const int c = count[i];
        all += c;
        if (i < upto) pre += c;
    }
    int total;
    (void)group_scan(pre, part, before);
    (void)group_scan(all, part, total);
    return total;
}

// Ranks of a chunk's words: lane i's word and the set bits before it.
__device__ __forceinline__ uint64_t chunk_word(const Workspace &w, int chunk, int lane, int before, int &base) {
    const uint64_t m = w.bits[(int64_t)chunk * 64 + lane];
    const int c = __popcll(m);
    base = before + wave_scan(c) - c;
    return m;
}

__device__ __forceinline__ uint64_t word_of(uint64_t m, int i) {
    const uint32_t lo = __builtin_amdgcn_readlane((int)(uint32_t)m, i);
    return (uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)(m >> 32), i) << 32 | lo;
}

// Hands out the free pages of one chunk.
__device__ void assign_chunk(const KvBook &b, int chunk, int chunks, int n, const Workspace &w, int32_t *moves) {
    __shared__ int32_t sums[kPrefixLds];
    int before;
    const int nfree = sum_chunks(w.chunk_count, chunks, chunk, before);
    const int asked = w.prefix[n - 1];
    if (before >= asked) return;
    if (n <= kPrefixLds) {
        for (int i = threadIdx.x; i < n; i += kThreads) sums[i] = w.prefix[i];
        __syncthreads();
    }
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    int base;
    const uint64_t words = chunk_word(w, chunk, lane, before, base);
    for (int i = wave; i < 64; i += kWavesPerGroup) {
        const uint64_t m = word_of(words, i);
        const int k = __builtin_amdgcn_readlane(base, i) + __popcll(m & below(lane));
        if (((m >> lane) & 1) && k < asked)
            hand_out(b, chunk * kChunk + i * 64 + lane, k, n, nfree, n <= kPrefixLds ? sums : w.prefix, w.req, moves);
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
    resize_row(b, s, r, r.row >= 0 && (r.need == 0 || w.prefix[s] <= nfree), new_len[s], moves);
}

// Behind the chunks a wave to each pair.
__global__ __launch_bounds__(kThreads) void fork_assign_kernel(KvBook b, const int32_t *parent, int n, Workspace w,
                                                               int32_t *moves, int32_t *missing) {
    const int chunks = chunks_of(b.N);
    if ((int)blockIdx.x < chunks) {
        assign_chunk(b, blockIdx.x, chunks, n, w, moves);
        return;
    }
    int before;
    const int nfree = sum_chunks(w.chunk_count, chunks, 0, before);
    const int i = ((int)blockIdx.x - chunks) * kWavesPerGroup + (int)(threadIdx.x >> 6), lane = threadIdx.x & 63;
    if (i == 0 && lane == 0) *missing = w.prefix[n - 1] > nfree ? w.prefix[n - 1] - nfree : 0;
    if (i >= n) return;
    const Request r = w.req[i];
    fork_row(b, i, parent[i], r, r.row >= 0 && (r.need == 0 || w.prefix[i] <= nfree), moves, lane, 64);
}

// ---- compaction ----
//
// U pages are used: the j-th used page at or behind U moves into the j-th free page before it.

__global__ __launch_bounds__(kThreads) void compact_small_kernel(KvBook b, int32_t *moves, int cap, int32_t *used) {
    __shared__ SmallPool p;
    __shared__ uint16_t hole[kSmallPages / 2];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, words = (b.N + 63) / 64;
    const int U = small_bits(p, b.refs, b.N, true);
    const int rank_u = U < b.N ? p.base[U >> 6] + __popcll(p.bits[U >> 6] & below(U & 63)) : U;
    const int made = min(U - rank_u, cap);
    if (threadIdx.x == 0) *used = U;
    for (int w = wave; w < words; w += kWavesPerGroup) {
        const uint64_t m = p.bits[w];
        const int k = p.base[w] + __popcll(m & below(lane)), page = w * 64 + lane;
        if (page >= b.N) continue;
        if (!((m >> lane) & 1)) {
            const int j = page - k;  // free pages before it
            if (page < U && j < made) {
                hole[j] = (uint16_t)page;
                moves[2 * j + 1] = page;
            }
        } else if (page >= U && k - rank_u < made) {
            moves[2 * (k - rank_u)] = page;
        }
    }
    __syncthreads();
    for (int j = made + (int)threadIdx.x; j < cap; j += kThreads) moves[2 * j] = moves[2 * j + 1] = -1;
    // tables and counts follow
    for (int s = wave; s < b.S; s += kWavesPerGroup) {
        int32_t *t = b.table + (int64_t)s * b.ld;
        const int have = pages_for(b.kv_len[s], b.page, b.cols);
        for (int c = lane; c < have; c += 64) {
            const int page = t[c];
            if (page < U || page >= b.N) continue;
            const uint64_t m = p.bits[page >> 6];
            const int j = p.base[page >> 6] + __popcll(m & below(page & 63)) - rank_u;
            if (((m >> (page & 63)) & 1) && j < made) t[c] = hole[j];
        }
    }
    for (int w = wave; w < words; w += kWavesPerGroup) {
        const uint64_t m = p.bits[w];
        const int j = p.base[w] + __popcll(m & below(lane)) - rank_u, page = w * 64 + lane;
        if (((m >> lane) & 1) && page >= U && j < made) {
            b.refs[hole[j]] = b.refs[page];
            b.refs[page] = 0;
        }
    }
}

__global__ __launch_bounds__(kThreads) void compact_count_kernel(KvBook b, Workspace w) {
    count_chunk(b.refs, b.N, w, true);
}

// Used pages in all (U), before the workgroup's chunk, and before page U.
__device__ int used_before_u(const Workspace &w, int chunks, int &U, int &before) {
    U = sum_chunks(w.chunk_count, chunks, blockIdx.x, before);
    int rank;
    const int cu = U / kChunk, in = U - cu * kChunk, lane = threadIdx.x & 63;
    (void)sum_chunks(w.chunk_count, chunks, cu, rank);
    if (cu < chunks) {
        int base;
        const uint64_t words = chunk_word(w, cu, lane, rank, base);
        rank = __builtin_amdgcn_readlane(base, __builtin_amdgcn_readfirstlane(in >> 6)) +
               __popcll(word_of(words, __builtin_amdgcn_readfirstlane(in >> 6)) & below(in & 63));
    }
    return rank;
}

__global__ __launch_bounds__(kThreads) void compact_match_kernel(KvBook b, Workspace w, int32_t *to_move,
                                                                 int32_t *moves, int cap, int32_t *used) {
    const int chunks = chunks_of(b.N);
    int U, before;
    const int rank_u = used_before_u(w, chunks, U, before);
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    if (blockIdx.x == 0 && threadIdx.x == 0) *used = U;
    int base;
    const uint64_t words = chunk_word(w, blockIdx.x, lane, before, base);
    for (int i = wave; i < 64; i += kWavesPerGroup) {
        const uint64_t m = word_of(words, i);
        const int k = __builtin_amdgcn_readlane(base, i) + __popcll(m & below(lane));
        const int page = (int)blockIdx.x * kChunk + i * 64 + lane;
        if (page >= b.N) continue;
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

// A wave to each sequence, then threads over the moves.
__global__ __launch_bounds__(kThreads) void compact_apply_kernel(KvBook b, Workspace w, const int32_t *to_move,
                                                                 const int32_t *moves, int cap, const int32_t *used) {
    const int U = *used, rows = (b.S + kWavesPerGroup - 1) / kWavesPerGroup;
    if ((int)blockIdx.x < rows) {
        const int s = blockIdx.x * kWavesPerGroup + (threadIdx.x >> 6);
        if (s >= b.S) return;
        const int have = pages_for(b.kv_len[s], b.page, b.cols);
        int32_t *t = b.table + (int64_t)s * b.ld;
        for (int c = threadIdx.x & 63; c < have; c += 64) {
            const int page = t[c];
            if (page < U || page >= b.N || !((w.bits[page >> 6] >> (page & 63)) & 1)) continue;
            const int j = to_move[page];
            if (j < cap) t[c] = moves[2 * j + 1];
        }
        return;
    }
    for (int64_t j = (int64_t)((int)blockIdx.x - rows) * kThreads + threadIdx.x; j < cap;
         j += (int64_t)((int)gridDim.x - rows) * kThreads) {
        const int of = moves[2 * j], to = moves[2 * j + 1];
        if (of < 0) break;
        b.refs[to] = b.refs[of];
        b.refs[of] = 0;
    }
}

// ---- page bytes ----

// Page bytes: each workgroup takes pieces of 16 KiB, four 16-byte loads in flight per
// thread.  Moves whose pages are not in the pool are left out.
constexpr int kPiece = 16384;

constexpr int kCopyThreads = 256;

__global__ __launch_bounds__(kCopyThreads) void copy_pages_kernel(uint8_t *cache, int64_t num_pages, int64_t page_bytes,
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
            if ((int)threadIdx.x + k * kCopyThreads < words) x[k] = __builtin_nontemporal_load(from + threadIdx.x + k * kCopyThreads);
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if ((int)threadIdx.x + k * kCopyThreads < words) __builtin_nontemporal_store(x[k], to + threadIdx.x + k * kCopyThreads);
    }
}

// Whether one workgroup takes an operator; n: pairs of a fork.
bool small(int64_t N, int64_t S, int64_t n, int64_t cols) {
    return N <= kSmallPages && S <= kSmallRows && n <= kSmallRequests && (S > n ? S : n) * cols <= kSmallEntries;
}

size_t compact_base(int64_t N) {
    const int64_t chunks = chunks_of(N);
    return (size_t)(chunks * 64 * 8 + ((chunks * 4 + 15) & ~(int64_t)15));
}

}  // namespace

size_t kv_pages_workspace(int64_t S, int64_t n_pairs, int64_t num_pages, int64_t cols) {
    if (small(num_pages, S, n_pairs, cols)) return 0;
    const int64_t requests = n_pairs > S ? n_pairs : S;
    const size_t chunks = (size_t)chunks_of(num_pages);
    const size_t ask = chunks * 64 * 8 + (size_t)requests * sizeof(Request) + chunks * 4 + (size_t)requests * 8;
    const size_t compact = compact_base(num_pages) + (size_t)num_pages * 4;
    return ask > compact ? ask : compact;
}

hipError_t launch_kv_fork(const KvBook &b, const int32_t *parent, const int32_t *child, int n, int32_t *moves,
                          int32_t *missing, void *ws, hipStream_t st) {
    if (small(b.N, b.S, n, b.cols)) {
        fork_small_kernel<<<1, kThreads, 0, st>>>(b, parent, child, n, moves, missing);
        return hipGetLastError();
    }
    const Workspace w = split_ws(ws, n, b.N);
    const int chunks = chunks_of(b.N);
    fork_release_kernel<<<n, 256, 0, st>>>(b, parent, child, n, w);
    fork_count_kernel<<<chunks + 1, kThreads, 0, st>>>(b, parent, child, n, w);
    fork_assign_kernel<<<chunks + (n + kWavesPerGroup - 1) / kWavesPerGroup, kThreads, 0, st>>>(b, parent, n, w, moves,
                                                                                             missing);
    return hipGetLastError();
}

hipError_t launch_kv_resize(const KvBook &b, const int32_t *new_len, int32_t *moves, int32_t *missing, void *ws,
                            hipStream_t st) {
    if (small(b.N, b.S, 0, b.cols)) {
        resize_small_kernel<<<1, kThreads, 0, st>>>(b, new_len, moves, missing);
        return hipGetLastError();
    }
    const Workspace w = split_ws(ws, b.S, b.N);
    const int chunks = chunks_of(b.N);
    resize_release_kernel<<<b.S, 256, 0, st>>>(b, new_len);
    resize_count_kernel<<<chunks + 1, kThreads, 0, st>>>(b, new_len, w);
    resize_assign_kernel<<<chunks + (b.S + kThreads - 1) / kThreads, kThreads, 0, st>>>(b, new_len, w, moves, missing);
    return hipGetLastError();
}

hipError_t launch_kv_compact(const KvBook &b, int32_t *moves, int cap, int32_t *used, void *ws, hipStream_t st) {
    if (small(b.N, b.S, 0, b.cols)) {
        compact_small_kernel<<<1, kThreads, 0, st>>>(b, moves, cap, used);
        return hipGetLastError();
    }
    const Workspace w = split_ws(ws, 0, b.N);
    int32_t *to_move = (int32_t *)((char *)ws + compact_base(b.N));
    const int chunks = chunks_of(b.N);
    compact_count_kernel<<<chunks, kThreads, 0, st>>>(b, w);
    compact_match_kernel<<<chunks, kThreads, 0, st>>>(b, w, to_move, moves, cap, used);
    const int64_t more = ((int64_t)cap + kThreads - 1) / kThreads;
    const int rows = (b.S + kWavesPerGroup - 1) / kWavesPerGroup;
    compact_apply_kernel<<<rows + (int)(more < 64 ? more : 64), kThreads, 0, st>>>(b, w, to_move, moves, cap, used);
    return hipGetLastError();
}

hipError_t launch_kv_copy_pages(uint8_t *cache, int64_t num_pages, int64_t page_bytes, int64_t layers,
                                int64_t layer_stride, const int32_t *moves, int n, hipStream_t st) {
    const int64_t units = (int64_t)n * layers * ((page_bytes + kPiece - 1) / kPiece);
    copy_pages_kernel<<<(unsigned)(units < 4096 ? units : 4096), kCopyThreads, 0, st>>>(cache, num_pages, page_bytes, layers,
                                                                                  layer_stride, moves, n);
    return hipGetLastError();
}

}  // namespace nmk

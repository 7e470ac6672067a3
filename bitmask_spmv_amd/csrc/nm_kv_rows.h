// nm_kv_rows.h -- which sequence a row of a ragged batch belongs to and where the cache keeps it.
#pragma once

#include "nm_device.h"
#include "nm_kv.h"

namespace nmk {
namespace {

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

// Workgroups go to the XCDs in turn: a number for each by which those of an XCD, which share its L2, are neighbours.
constexpr int kXcds = 8;
__device__ __forceinline__ int by_xcd(int block, int blocks) {
    const int per = blocks / kXcds, rest = blocks % kXcds, xcd = block % kXcds;
    return xcd * per + min(xcd, rest) + block / kXcds;
}

// Row t's sequence, called by a whole wave with one t: up to 64 sequences are read at once, with what is wanted of them.
struct RowSeq {
    int s, q0, q1, len;
    template <class B>
    __device__ __forceinline__ RowSeq(const B &b, int t, int lane) {
        if (b.S <= kWave) {
            const int i = min(lane, b.S - 1);
            const int from = b.q_start[i], to = b.q_start[i + 1], n = b.kv_len[i];
            const uint64_t m = __ballot(lane < b.S && from <= t);
            s = m ? 63 - __clzll((long long)m) : 0;
            q0 = __builtin_amdgcn_readlane(from, s);
            q1 = __builtin_amdgcn_readlane(to, s);
            len = __builtin_amdgcn_readlane(n, s);
        } else {
            s = __builtin_amdgcn_readfirstlane(find_seq(b.q_start, b.S, t, lane));
            q0 = b.q_start[s];
            q1 = b.q_start[s + 1];
            len = b.kv_len[s];
        }
    }
};

// Where row t is kept: the head-0 block of its page and its token within the page; null
// where the sequence has no place or no valid page for it.
template <class B>
__device__ __forceinline__ uint8_t *place_of(const B &b, int s, int t, int &tok) {
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

}  // namespace
}  // namespace nmk

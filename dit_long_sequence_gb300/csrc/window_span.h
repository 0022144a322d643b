// window_span.h -- a sliding window of frames with sinks: what a query sees, the key
// tiles of a block of queries, the mask words of a tile.
#pragma once

#include <cstdint>

#include "fast_div.h"

namespace dit {

// A query at position p, in the frame that starts at s = floor(p / frame) * frame,
// sees the keys [0, min(sinks, hi)) and [lo, hi) with lo = s - back and
// hi = s + ahead, both within the sequence.
struct Window {
    int frame;              // tokens of a frame, >= 1
    FastDiv by_frame;
    int64_t back, ahead;    // kUnbounded: no bound on that side
    int sinks;
};
constexpr int64_t kUnbounded = int64_t(1) << 40;

struct Span {
    int lo, hi;             // 0 <= lo <= hi <= kv_len
};
DIT_HD Span span_of(const Window& w, int pos, int kv_len) {
    const uint32_t up = static_cast<uint32_t>(pos < 0 ? -(pos + 1) : pos);   // (a negative position's frame is the one below)
    const int64_t q = w.by_frame.div(up);
    const int64_t s = (pos < 0 ? -q - 1 : q) * w.frame;
    const int64_t lo = s - w.back, hi = s + w.ahead;
    Span r;
    r.hi = static_cast<int>(hi < 0 ? 0 : (hi > kv_len ? kv_len : hi));
    r.lo = static_cast<int>(lo < 0 ? 0 : (lo > r.hi ? r.hi : lo));
    return r;
}

// The queries 0 <= i < n, query i at position offset + i, that see a key of [k0, k1),
// 0 <= k0 < k1, and those that see all of them.  Both are ranges: hi grows with the
// position and so does lo (but for the sinks).
struct QueryRange {
    int64_t first, end;             // that see a key, none where first >= end
    int64_t full, full_end;         // that see all (at least these: sinks and window together may show all, too)
};
DIT_HD QueryRange query_range(const Window& w, int64_t k0, int64_t k1, int sinks, int n, int offset) {
    auto from = [&](int64_t s) {        // first query whose frame starts at s or later
        const int64_t f = (s >= 0 ? s + w.frame - 1 : s) / w.frame;      // (rounds up)
        const int64_t i = f * w.frame - offset;
        return i < 0 ? int64_t(0) : (i > n ? static_cast<int64_t>(n) : i);
    };
    const bool all = w.ahead >= kUnbounded, ever = w.back >= kUnbounded;
    QueryRange r;
    r.first = all ? 0 : from(k0 - w.ahead + 1);
    r.full = all ? 0 : from(k1 - w.ahead);
    r.end = ever || k0 < sinks ? n : from(k1 + w.back);
    r.full_end = ever || k1 <= sinks ? n : from(k0 + w.back + 1);
    return r;
}

// The 128-key tiles that queries at positions [first, last] see, in order: the
// sinks' tiles [0, ns), then those of the window from w0 on (both bounds of a
// span only grow with the position).
struct KeyTiles {
    int n;                  // tiles in all
    int ns, w0;
    int lo, hi, sinks;      // keys that some query sees: [0, sinks) and [lo, hi)
    DIT_HD int at(int i) const { return i < ns ? i : w0 + (i - ns); }
};
DIT_HD KeyTiles key_tiles(const Window& w, int first, int last, int kv_len) {
    KeyTiles t;
    t.lo = span_of(w, first, kv_len).lo;
    t.hi = span_of(w, last, kv_len).hi;
    t.sinks = w.sinks < t.hi ? w.sinks : t.hi;
    t.w0 = t.lo >> 7;
    const int end = t.lo < t.hi ? (t.hi + 127) >> 7 : t.w0;
    t.ns = (t.sinks + 127) >> 7;
    if (end > t.w0 && t.ns > t.w0) t.ns = t.w0;         // (an empty window: the sinks alone)
    t.n = t.ns + end - t.w0;
    return t;
}

#ifdef __CUDACC__
// Bits [0, n) of a word.
__device__ __forceinline__ uint32_t bits_below(int n) { return n <= 0 ? 0u : (n >= 32 ? ~0u : (1u << n) - 1u); }
// Which of the 32 keys from c on a row sees: [0, sinks) and [lo, hi).
__device__ __forceinline__ uint32_t seen_word(int lo, int hi, int sinks, int c) {
    return bits_below(hi - c) & (~bits_below(lo - c) | bits_below(sinks - c));
}
// Does a row see all keys of the tile from k0 on?
__device__ __forceinline__ bool sees_all(int lo, int hi, int sinks, int k0) {
    return hi - k0 >= 128 && (lo <= k0 || sinks - k0 >= 128);
}
#endif

}  // namespace dit

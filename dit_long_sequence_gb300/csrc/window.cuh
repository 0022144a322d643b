// window.cuh -- device code that the windowed attention kernels share: paged copies,
// the online softmax of one tile, the store of a row.
#pragma once

#include "debug.cuh"
#include "internal.h"
#include "ptx.cuh"
#include "window.h"

namespace dit {

enum WindowSite : uint32_t {
    SITE_Q_EMPTY = 31, SITE_ITEM_FULL = 32, SITE_ITEM_EMPTY = 33, SITE_CLAIM = 34,
    SITE_O_SETTLED = 35
};
constexpr int kWinTile = 128;      // rows of a query tile, keys of a key tile
constexpr float kWinLn2 = 0.6931471805599453f;
constexpr float kWinSumLimit = 549755813888.0f;  // 2^39: largest row sum of a tile kept without a rescale
constexpr int kNoBound = 0x7fffffff;

// 5-D tiled load (coordinates innermost first) completing on `bar` (tx bytes).
__device__ __forceinline__ void tma_load_5d(uint32_t dst, const void* tmap, uint32_t bar, int c0, int c1, int c2, int c3, int c4) {
    asm volatile(
        "cp.async.bulk.tensor.5d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4, %5, %6, %7}], [%2];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(tmap)), "r"(bar), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(c4)
        : "memory");
}
// Orders this thread's shared-memory accesses before later asynchronous ones.
__device__ __forceinline__ void fence_async() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

// ------------------------------------------------------------------ pages

// The page that holds chunk `lane` of a key tile, -1 in lanes without a chunk or
// whose keys are not there.  A whole warp; loaded a tile ahead of its use.
__device__ __forceinline__ int page_entry(const WindowArgs& a, const int32_t* row, int tile, int kv_len) {
    const int lane = static_cast<int>(lane_id());
    // (unsigned: a lane without a chunk may be past 2^31 at the far end of a table)
    const uint32_t key = static_cast<uint32_t>(tile) * kWinTile + static_cast<uint32_t>(lane * a.chunk);
    const bool mine = lane * a.chunk < kWinTile && key < static_cast<uint32_t>(kv_len);
    return mine ? __ldg(row + a.div_page.div(key)) : -1;
}
__device__ __forceinline__ bool page_there(const WindowArgs& a, int entry) { return entry >= 0 && entry < a.n_pages; }
// Bit c: chunk c has a page, or no key below kv_len (those are hidden by a row's hi).
// All ones in the usual case.
__device__ __forceinline__ uint32_t pages_there(const WindowArgs& a, int entry, int tile, int kv_len) {
    const int lane = static_cast<int>(lane_id());
    const uint32_t key = static_cast<uint32_t>(tile) * kWinTile + static_cast<uint32_t>(lane * a.chunk);
    const bool past = lane * a.chunk >= kWinTile || key >= static_cast<uint32_t>(kv_len);
    return __ballot_sync(0xffffffffu, past || page_there(a, entry));
}
// The keys of word w of a tile whose pages are there.
__device__ __forceinline__ uint32_t paged_word(uint32_t there, int chunk, int w) {
    uint32_t r = 0;
    for (int k = 0; k < 32; k += chunk)
        if ((there >> ((32 * w + k) / chunk)) & 1u) r |= bits_below(chunk) << k;
    return r;
}
// Copies a paged tile of D channels to `dst`, every lane its own chunk; keys without
// a page arrive as zeros (a page past the last is outside the map).
template <int D>
__device__ __forceinline__ void copy_paged(const WindowArgs& a, const CUtensorMap* tm, uint32_t dst, uint32_t bar, int entry,
                                           int tile, int head) {
    const int lane = static_cast<int>(lane_id());
    if (lane * a.chunk >= kWinTile) return;
    const uint32_t key = static_cast<uint32_t>(tile) * kWinTile + lane * a.chunk;
    uint32_t row;
    a.div_page.divmod(key, row);
    const int page = page_there(a, entry) ? entry : a.n_pages;
#pragma unroll
    for (int c = 0; c < D / 64; ++c)
        tma_load_4d(dst + c * kWinTile * 128 + lane * a.chunk * 128, tm, bar, c * 64, static_cast<int>(row), head, page);
}

// Zeroes the V rows of the key tile from k0 on that no query of the item sees, so
// that what lies there (a page's stale rows may hold NaN) never meets a product's
// zero probability.  A whole warp, before it issues the product.
template <int D>
__device__ __forceinline__ void clear_unseen(uint8_t* v, const KeyTiles& t, int k0) {
    const int s = t.sinks - k0, lo = t.lo - k0, hi = t.hi - k0;
    // (8 or 16 lanes a row, 16 bytes each)
    constexpr int kLanes = D / 8;
    const int part = static_cast<int>(lane_id()) % kLanes;
    uint8_t* const at = v + (part >> 3) * kWinTile * 128 + (part & 7) * 16;
    auto clear = [&](int begin, int end) {
        for (int row = begin + static_cast<int>(lane_id()) / kLanes; row < end; row += 32 / kLanes)
            *reinterpret_cast<uint4*>(at + row * 128) = make_uint4(0u, 0u, 0u, 0u);
    };
    const int after_sinks = max(s, 0), after = max(hi, after_sinks);
    if (after_sinks >= kWinTile || (lo <= after_sinks && after >= kWinTile)) return;
    clear(after_sinks, min(lo, kWinTile));
    clear(after, kWinTile);
    fence_async();
    __syncwarp();
}

// ------------------------------------------------------------------ softmax

// 32 lanes x 8 columns (one row a thread), there and back.
__device__ __forceinline__ void tmem_ld8(uint32_t taddr, uint32_t (&r)[8]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
        : "r"(taddr)
        : "memory");
}
__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t (&r)[8]) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(taddr), "r"(r[0]), "r"(r[1]),
                 "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
                 : "memory");
}

// Max over 64 scores: eight 3-input max chains, then a small tree.
__device__ __forceinline__ float max_of_64(const float* v) {
    float t[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) t[k] = max3f(v[k], v[8 + k], v[16 + k]);
#pragma unroll
    for (int i = 24; i < 56; i += 16)
#pragma unroll
        for (int k = 0; k < 8; ++k) t[k] = max3f(t[k], v[i + k], v[i + 8 + k]);
#pragma unroll
    for (int k = 0; k < 8; ++k) t[k] = fmaxf(t[k], v[56 + k]);
    return max3f(max3f(t[0], t[1], t[2]), max3f(t[3], t[4], t[5]), fmaxf(t[6], t[7]));
}
// P = 2^(s * sl2 - m) of 64 scores, as bf16 pairs to 32 TMEM columns; returns the
// sum of the fp32 P.  The rounding of P to bf16 is the product's operand type.
__device__ __forceinline__ float exp_to_p(const float* v, uint32_t tP, float sl2, float m) {
    float a0 = 0.f, a1 = 0.f, b0 = 0.f, b1 = 0.f;
#pragma unroll
    for (int cc = 0; cc < 2; ++cc) {
        uint32_t pk[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            float x0, x1;
            ffma2_bc(x0, x1, v[32 * cc + 2 * i], v[32 * cc + 2 * i + 1], sl2, -m);
            const float p0 = ex2_approx(x0), p1 = ex2_approx(x1);
            if (i & 1) fadd2_acc(b0, b1, p0, p1);
            else fadd2_acc(a0, a1, p0, p1);
            pk[i] = pack_bf16x2(p0, p1);
        }
        tmem_st16(tP + cc * 16, pk);
    }
    return (a0 + a1) + (b0 + b1);
}

// One key tile of a thread's row: S from tensor memory, P back over its first
// half, the running offset m (log2 units) and sum l.  m is the row's maximum when
// its first key is seen and moves only when a tile's row sum passes 2^39 (O and l
// are then scaled by 2^(m_old - m_new)): every P is at most 2^39, which bf16 and
// the fp32 sums carry with the precision they have at 1.  `first`: the item's
// first tile, O holds nothing yet.  `masked` (warp-uniform): apply the words.
// settled() returns when the products before this tile's P are done with O.
template <int D, typename F>
__device__ __forceinline__ void soften_tile(uint32_t tS, uint32_t tO, float sl2, bool first, bool masked,
                                            const uint32_t (&words)[4], float& m, float& l, F&& settled) {
    uint32_t sr[4][32];
    tmem_ld32(tS, sr[0]);
    tmem_ld32(tS + 32, sr[1]);
    tmem_ld_wait_dep(sr[0]);
    reg_dep(sr[1]);
    tmem_ld32(tS + 64, sr[2]);
    tmem_ld32(tS + 96, sr[3]);
    float s[128];
    auto take = [&](int half) {
#pragma unroll
        for (int c = 0; c < 64; ++c) s[64 * half + c] = __uint_as_float(sr[2 * half + (c >> 5)][c & 31]);
        if (masked) {
#pragma unroll
            for (int c = 0; c < 64; ++c)
                if (!((words[2 * half + (c >> 5)] >> (c & 31)) & 1u)) s[64 * half + c] = -INFINITY;
        }
    };
    auto off = [](float mm) { return mm == -INFINITY ? 0.f : mm; };     // no key seen: every P is 0
    take(0);
    if (first) {
        const float mx = max_of_64(s);
        tmem_ld_wait_dep(sr[2]);
        reg_dep(sr[3]);
        take(1);
        m = fmaxf(mx, max_of_64(s + 64)) * sl2;
        l = exp_to_p(s, tS, sl2, off(m));
        l += exp_to_p(s + 64, tS + 32, sl2, off(m));
        return;
    }
    float la = exp_to_p(s, tS, sl2, off(m));
    tmem_ld_wait_dep(sr[2]);
    reg_dep(sr[3]);
    take(1);
    float lb = exp_to_p(s + 64, tS + 32, sl2, off(m));
    // (also true of inf and NaN)
    const bool need = !(la + lb <= kWinSumLimit) || m == -INFINITY;
    if (__any_sync(0xffffffffu, need)) {
        const float mt = fmaxf(max_of_64(s), max_of_64(s + 64)) * sl2;
        const float m_new = need ? fmaxf(mt, m) : m;
        // (when no row's offset moves, O and P stand as they are)
        if (__any_sync(0xffffffffu, m_new != m)) {
            // (8 columns at a time: with 32 the loads' registers beside the scores spill in
            // every tile, 1,954 us against 1,607 of the LTX-2-shaped frames without this path)
            tmem_st_wait();
            settled();
            const float alpha = m_new == -INFINITY ? 1.f : ex2_approx(m - m_new);
            l *= alpha;
#pragma unroll 1
            for (int cc = 0; cc < D / 8; ++cc) {
                uint32_t o[8];
                tmem_ld8(tO + cc * 8, o);
#pragma unroll
                for (int i = 0; i < 8; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * alpha);
                tmem_st8(tO + cc * 8, o);
            }
            m = m_new;
            la = exp_to_p(s, tS, sl2, off(m));
            lb = exp_to_p(s + 64, tS + 32, sl2, off(m));
        }
    }
    l += la + lb;
}

// ------------------------------------------------------------------ results

// 8 consecutive 32-bit words (32-byte aligned, or as two 16-byte halves).
__device__ __forceinline__ void store_words(void* p, const uint32_t (&v)[8], bool wide) {
    if (wide)
        asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(v[0]), "r"(v[1]), "r"(v[2]),
                     "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
                     : "memory");
    else {
        reinterpret_cast<uint4*>(p)[0] = make_uint4(v[0], v[1], v[2], v[3]);
        reinterpret_cast<uint4*>(p)[1] = make_uint4(v[4], v[5], v[6], v[7]);
    }
}
// 32 channels of a row, rounded once, to element `off` of out; or as fp32 to a partial.
__device__ __forceinline__ void store_32(const WindowArgs& a, float* partial, int64_t off, const uint32_t (&o)[32]) {
    if (partial != nullptr || !a.out_bf16) {
        float* const dst = partial != nullptr ? partial : static_cast<float*>(a.out) + off;
        const bool wide = partial == nullptr && a.wide;
#pragma unroll
        for (int i = 0; i < 32; i += 8) {
            const uint32_t v[8] = {o[i], o[i + 1], o[i + 2], o[i + 3], o[i + 4], o[i + 5], o[i + 6], o[i + 7]};
            store_words(dst + i, v, wide);
        }
    } else {
        uint16_t* const dst = static_cast<uint16_t*>(a.out) + off;
#pragma unroll
        for (int i = 0; i < 32; i += 16) {
            uint32_t v[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) v[k] = pack_bf16x2(__uint_as_float(o[i + 2 * k]), __uint_as_float(o[i + 2 * k + 1]));
            store_words(dst + i, v, a.wide);
        }
    }
}

}  // namespace dit

// window.h -- windowed attention and the paged cache: the launch-side declarations
// shared by the kernels and the C-ABI layer (api_window.cu).  Not part of the public
// interface.
#pragma once

#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>

#include "dit_attn.h"
#include "train.h"
#include "window_span.h"

namespace dit {

constexpr int kMaxPiecesFwd = 64;   // key ranges an item is cut into at most

// Attention over a window.  A work item is a block of query rows of one batch
// entry and one K/V head; its rows are (token, query head of the group), the
// heads fastest, so that the heads that share K and V share their tiles.  A
// 128-row tile holds `tokens` whole tokens, `tokens` * `group` rows.
struct WindowArgs {
    int B, T, H, Hkv, group, tokens;
    int kv_len, offset;         // contiguous: keys, position of query 0
    Window win;
    float scale_log2;
    void* out;                  // element (b, n, h, d); fp32 or bf16
    bool out_bf16, wide;        // wide: rows may be stored 32 bytes at a time
    int64_t o_sb, o_sn, o_sh;
    float* lse;                 // [B, H, T]
    // Grid: items (b, K/V head, block of two tiles), blocks fastest and the last
    // first, each in f key ranges whose partials (O normalised, LSE) go to ws_o
    // [item][f][part_rows][D] and ws_lse [item][f][part_rows].
    // The first `late` blocks of every head, which see the fewest keys of a causal
    // mask, come behind all others, heads fastest: the end of the grid is made of them.
    int n_blk, late, n_main, f, n_items;    // n_main: items before those; n_items: pieces counted
    FastDiv div_bhk;
    int part_rows;              // 256, or the rows of the one tile
    FastDiv div_f, div_blk, div_hkv, div_group;
    float *ws_o, *ws_lse;
    // Paged: position x of sequence b is row x mod page of page
    // table[b * table_sb + x / page]; `chunk` rows of a page are copied at a time.
    const int32_t *table, *kv_lens, *q_lens;
    int64_t table_sb;
    int n_pages, page, chunk, capacity;     // capacity: keys that a table row has pages for
    FastDiv div_page;
    unsigned int* status;
    unsigned long long timeout_ns;
    int64_t dbg_o_elems;        // debug library: O elements reachable through its strides
    int dbg_keys_short;         // debug library: keys off the end that the bounds check of a tile allows
};

// Batch entry, K/V head and block of an item's number.
DIT_HD void place(const WindowArgs& a, uint32_t item, int& b, int& hk, int& blk) {
    uint32_t inner, head, bhk;
    if (item < static_cast<uint32_t>(a.n_main)) {
        bhk = a.div_blk.divmod(item, inner);
        blk = a.n_blk - 1 - static_cast<int>(inner);
    } else {
        blk = a.late - 1 - static_cast<int>(a.div_bhk.divmod(item - static_cast<uint32_t>(a.n_main), bhk));
    }
    b = static_cast<int>(a.div_hkv.divmod(bhk, head));
    hk = static_cast<int>(head);
}

// All rows of a sequence and K/V head fit one query tile.
inline bool one_tile(const WindowArgs& a) { return a.T <= a.tokens; }
cudaError_t launch_attn_window(const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv, const WindowArgs& a,
                               int D, bool paged, cudaStream_t s);

// Copy of new tokens into the pages; thread units of 8 channels, K then V of a token.
struct AppendArgs {
    const uint16_t *k, *v;
    uint16_t *k_cache, *v_cache;
    dit_strides4_t sk, sv, dk, dv;      // of the new tokens (b, t, h) and of the cache (page, row, h)
    const int32_t *table, *kv_lens, *new_lens;
    int64_t table_sb, capacity;
    int T, pages;
    uint32_t n, half;                   // units in all, of a token's K
    FastDiv div_parts, div_t, div_d8, div_page;
};
cudaError_t launch_paged_append(const AppendArgs& a, bool vec, cudaStream_t s);

}  // namespace dit

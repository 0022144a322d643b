// bwd_plan.h -- host-only plan of the attention backward grid: into how many
// pieces each key item and each query item is cut, and the workspace that
// takes.  Used by api_train.cu.
#pragma once

#include <cstdint>
#include <initializer_list>

namespace dit {

// A tile pair costs a key item four products and a query item three.  With the
// whole grid's cost spread evenly over the SMs, an item longer than that even
// share is cut into pieces of about that length (at least kMinPieceTiles
// streamed tiles, at most kMaxPieces).  In a grid of more items only the last
// query items may be cut, where that fills the end of the grid: 6,144 x 6,144
// with 8 heads of 128 has 768 items for 152 SMs, and whole ones leave the SMs
// idle for an eighth of the time (353 us; with the last 38 in four pieces 340;
// 12,660 rows of 2 heads of 64: 288 and 253).  With seven items an SM and more the
// prediction fails as often as not (8,192 rows of 8 heads of 64: 416 and 428).
struct BwdPlan {
    int q_tiles, kv_tiles, kv_out_tiles;
    int64_t key_items, query_items;
    int f_kv, f_q;              // pieces of a key item, of a cut query item
    int64_t q_whole;            // query items that are not cut, the first of the grid's order
    int64_t stat_bytes, part_kv_bytes, part_q_bytes;
};
constexpr int kMinPieceTiles = 2;
constexpr int kMaxPieces = 64;

// SMs that have been given work until time t.
struct BwdLevel {
    int64_t t, sms;
};
// Deals n items of one cost, each to an SM that is free first, as the grid's
// counter does.
inline void deal(BwdLevel (&g)[8], int& levels, int64_t n, int64_t cost) {
    while (n > 0) {
        int lo = 0;
        for (int i = 1; i < levels; ++i)
            if (g[i].t < g[lo].t) lo = i;
        const int64_t t = g[lo].t + cost, take = n < g[lo].sms ? n : g[lo].sms;
        n -= take;
        g[lo].sms -= take;
        if (g[lo].sms == 0) g[lo] = g[--levels];    // (at most one level more a call)
        int to = 0;
        while (to < levels && g[to].t != t) ++to;
        if (to == levels) g[levels++] = BwdLevel{t, 0};
        g[to].sms += take;
    }
}
// When the grid ends, in sixths of a product, with the last `cut` query items in
// f pieces.  An item costs about six products beside its own (first copies, the
// gradient's way out), whether whole or a piece.
inline int64_t grid_end(const BwdPlan& p, int sms, int64_t cut, int f) {
    BwdLevel g[8] = {{0, sms}};
    int levels = 1;
    deal(g, levels, p.key_items, 24LL * p.q_tiles + 36);
    deal(g, levels, p.query_items - cut, 18LL * p.kv_tiles + 36);
    deal(g, levels, cut * f, 18LL * p.kv_tiles / f + 36);
    int64_t end = 0;
    for (int i = 0; i < levels; ++i) end = g[i].t > end ? g[i].t : end;
    return end;
}
constexpr int kMaxRounds = 6;       // items an SM beyond which the items' own variation hides the end of the grid
constexpr int kSumCost = 66;        // of the sum kernel, some 4 us, in sixths of a product

inline BwdPlan plan_attn_bwd(int B, int Nq, int Nkv, int H, int D, int key_valid_len, int sms) {
    BwdPlan p{};
    const int64_t bh = static_cast<int64_t>(B) * H;
    p.q_tiles = static_cast<int>((static_cast<int64_t>(Nq) + 127) / 128);
    p.kv_tiles = static_cast<int>((static_cast<int64_t>(key_valid_len) + 127) / 128);
    p.kv_out_tiles = static_cast<int>((static_cast<int64_t>(Nkv) + 127) / 128);
    p.key_items = bh * p.kv_out_tiles;
    p.query_items = bh * p.q_tiles;
    p.f_kv = p.f_q = 1;
    if (sms > 0 && p.kv_tiles > 0 && bh > 0) {
        const double share = 7.0 * static_cast<double>(bh) * p.q_tiles * p.kv_tiles / sms;   // per SM, in products
        auto pieces = [&](double cost, int tiles) {
            int f = static_cast<int>(cost / share + 0.999);
            if (f > tiles / kMinPieceTiles) f = tiles / kMinPieceTiles;
            if (f > kMaxPieces) f = kMaxPieces;
            return f < 1 ? 1 : f;
        };
        p.f_kv = pieces(4.0 * p.q_tiles, p.q_tiles);
        p.f_q = pieces(3.0 * p.kv_tiles, p.kv_tiles);
    }
    p.q_whole = p.f_q > 1 ? 0 : p.query_items;
    if (sms > 0 && p.kv_tiles > 0 && p.f_kv == 1 && p.f_q == 1 && p.key_items + p.query_items <= static_cast<int64_t>(kMaxRounds) * sms) {
        const int64_t whole = grid_end(p, sms, 0, 1);
        int64_t best = whole - whole / 50 - kSumCost;      // worth 2% at least
        for (int f = 2; f <= 4; ++f)
            for (int64_t cut : {sms / 4, sms / 2, 3 * sms / 4, sms}) {
                if (cut < 1 || cut > p.query_items || p.kv_tiles < f * kMinPieceTiles) continue;
                const int64_t end = grid_end(p, sms, cut, f);
                if (end >= best) continue;
                best = end;
                p.f_q = f;
                p.q_whole = p.query_items - cut;
            }
    }
    auto up = [](int64_t n) { return (n + 255) / 256 * 256; };
    p.stat_bytes = up(bh * 2 * p.q_tiles * 128 * 4) + 256;     // and the item counter
    p.part_kv_bytes = p.f_kv > 1 ? up(p.key_items * p.f_kv * 2 * 128 * D * 4) : 0;
    p.part_q_bytes = p.f_q > 1 ? up((p.query_items - p.q_whole) * p.f_q * 128 * D * 4) : 0;
    return p;
}

}  // namespace dit

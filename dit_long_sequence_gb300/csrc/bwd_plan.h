// bwd_plan.h -- host-only plan of the attention backward grid: into how many
// pieces each key item and each query item is cut, and the workspace that
// takes.  Used by api_train.cu.
#pragma once

#include <cstdint>

namespace dit {

// A tile pair costs a key item four products and a query item three.  With the
// whole grid's cost spread evenly over the SMs, an item longer than that even
// share is cut into pieces of about that length (at least kMinPieceTiles
// streamed tiles, at most kMaxPieces); a grid of many items is not cut.
struct BwdPlan {
    int q_tiles, kv_tiles, kv_out_tiles;
    int64_t key_items, query_items;
    int f_kv, f_q;
    int64_t stat_bytes, part_kv_bytes, part_q_bytes;
};
constexpr int kMinPieceTiles = 2;
constexpr int kMaxPieces = 64;

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
    auto up = [](int64_t n) { return (n + 255) / 256 * 256; };
    p.stat_bytes = up(bh * 2 * p.q_tiles * 128 * 4) + 256;     // and the item counter
    p.part_kv_bytes = p.f_kv > 1 ? up(p.key_items * p.f_kv * 2 * 128 * D * 4) : 0;
    p.part_q_bytes = p.f_q > 1 ? up(p.query_items * p.f_q * 128 * D * 4) : 0;
    return p;
}

}  // namespace dit

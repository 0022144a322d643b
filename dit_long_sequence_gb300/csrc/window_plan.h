// window_plan.h -- host-only plan of the windowed attention's grid: into how many
// key ranges an item is cut, and the workspace that takes.  Used by api_window.cu
// and, for the backward grid, by bwd_plan.h.
#pragma once

#include <cstdint>

#include "window.h"

namespace dit {

inline bool sound_window(const dit_window_t* w) { return w != nullptr && w->frame >= 1 && w->frame <= (1 << 30) && w->sinks >= 0; }

inline Window make_window(const dit_window_t& w) {
    Window r;
    r.frame = w.frame;
    r.by_frame = FastDiv(static_cast<uint32_t>(w.frame));
    // (positions and frames are below 2^31: from 2^32 on a bound is none)
    auto tokens = [&](int64_t frames) { return frames * w.frame < (int64_t(1) << 32) ? frames * w.frame : kUnbounded; };
    r.back = w.left < 0 ? kUnbounded : tokens(w.left);
    r.ahead = w.right < 0 ? kUnbounded : tokens(static_cast<int64_t>(w.right) + 1);
    r.sinks = w.sinks;
    return r;
}

// Key tiles an item (`rows` query tokens of a sequence of T from position `offset`)
// walks on the average, from at most 64 of them.
inline double mean_key_tiles(const Window& w, int T, int rows, int offset, int kv_len) {
    const int64_t blocks = (static_cast<int64_t>(T) + rows - 1) / rows;
    const int64_t step = blocks > 32 ? blocks / 32 : 1;
    double sum = 0;
    int64_t n = 0;
    for (int64_t i = 0; i < blocks; i += step, ++n) {
        const int64_t first = i * rows, last = first + rows < T ? first + rows - 1 : T - 1;
        sum += key_tiles(w, static_cast<int>(offset + first), static_cast<int>(offset + last), kv_len).n;
    }
    return n > 0 ? sum / static_cast<double>(n) : 0;
}

// Items of `tiles` key tiles each go to the SMs in turns, so the grid takes the
// turns of its last SM; cut into f ranges, an item has f turns of a part of its
// tiles.  A turn costs about kTurnTiles tiles beside its own (first copies, the
// result's way out) and the join of the pieces kJoinTiles; a cut that does not
// save a twentieth is not made.  From two turns on the claims even the grid out and
// the partials' 132 KB a piece cost more than they give (480 items of 6 ragged chunks,
// both on the same lengths: 324 us in three pieces, 242 whole); the last, partial turn
// is not evened out (384 equal items end 1.19 times the even share).
constexpr double kTurnTiles = 3, kJoinTiles = 4;
inline int plan_pieces(int64_t items, double tiles, int sms) {
    if (items <= 0 || sms <= 0 || items >= 2LL * sms) return 1;
    double best = 0;
    int f_best = 1;
    for (int f = 1; f <= 16 && (f == 1 || tiles / f >= 2); ++f) {
        const double turns = static_cast<double>((items * f + sms - 1) / sms);
        double cost = turns * (tiles / f + kTurnTiles);
        if (f > 1) cost = (cost + kJoinTiles) / 0.95;
        if (f == 1 || cost < best) {
            best = cost;
            f_best = f;
        }
    }
    return f_best;
}

// Blocks of every head that come last: about two turns of the SMs, where a sequence's
// first rows see half the keys of the others or less (LTX-2-shaped frames, single passes
// timed in turn: 1,661 us, one turn 1,674, none 1,695).  A chunk behind a long past has
// no such rows, and its longest sequence's items would come last (another draw of ragged
// chunks: 324 us, without 315).
inline int late_blocks(double first_tiles, double mean_tiles, int64_t heads, int64_t n_blk, int sms) {
    if (2 * first_tiles > mean_tiles || heads <= 0) return 0;
    const int64_t n = (2LL * sms + heads - 1) / heads;
    return static_cast<int>(n < n_blk / 2 ? n : n_blk / 2);
}

// Settles the items' order (place()) for a's sizes, blocks and heads.
inline void order_items(WindowArgs& a, int late) {
    const int64_t heads = static_cast<int64_t>(a.B) * a.Hkv, main = heads * (a.n_blk - late);
    a.late = late;
    a.n_main = static_cast<int>(main < 0x7fffffff ? main : 0x7fffffff);
    a.div_blk = FastDiv(static_cast<uint32_t>(a.n_blk > late ? a.n_blk - late : 1));
    a.div_bhk = FastDiv(static_cast<uint32_t>(heads));
    a.div_hkv = FastDiv(static_cast<uint32_t>(a.Hkv));
}

// A few new tokens over a cache (one tile an item, HBM-bound): sequences' lengths
// differ and only the device knows them, so the pieces are made for about
// kPiecesPerSm turns of every SM, of two key tiles at least, which the claims deal
// out evenly (a token for 48 ragged sequences, 32 heads on 8: 250 us; 4 turns 260, 16
// 275).  The number of rows is not looked at: partials are group * T rows a piece (16
// tokens of eight heads a K/V head for those sequences: 101 MB, 322 us against 270 for
// one token), and one sequence is cut finer than it needs (16,384 keys, eight K/V heads
// of eight heads each: 48 us for one token, 60 for 16, and 32 for 17, which is
// plan_pieces()).
constexpr int kPiecesPerSm = 8;
inline int plan_pieces_few(int64_t items, double tiles, int sms) {
    if (items <= 0 || sms <= 0) return 1;
    int64_t f = (static_cast<int64_t>(kPiecesPerSm) * sms + items - 1) / items;
    if (f > kMaxPiecesFwd) f = kMaxPiecesFwd;
    if (static_cast<double>(f) > tiles / 2) f = static_cast<int64_t>(tiles / 2);
    return f < 1 ? 1 : static_cast<int>(f);
}

// Rows of a piece's partial, and the partials' bytes: O in fp32, then its LSE.
inline int part_rows_of(int T, int group) { return T <= 128 / group ? T * group : 256; }
inline int64_t pieces_bytes(int64_t items, int f, int rows, int D) { return f > 1 ? items * f * rows * (D + 1) * 4 : 0; }

}  // namespace dit

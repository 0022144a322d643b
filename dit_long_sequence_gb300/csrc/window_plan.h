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
// walks on the average, from at most 128 of them.
inline double mean_key_tiles(const Window& w, int T, int rows, int offset, int kv_len) {
    const int64_t blocks = (static_cast<int64_t>(T) + rows - 1) / rows;
    const int64_t step = blocks > 64 ? blocks / 64 : 1;
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
// save a twentieth is not made.
constexpr double kTurnTiles = 3, kJoinTiles = 4;
inline int plan_pieces(int64_t items, double tiles, int sms) {
    if (items <= 0 || sms <= 0 || items >= 4LL * sms) return 1;
    double best = 0;
    int f_best = 1;
    for (int f = 1; f <= kMaxPiecesFwd && (f == 1 || tiles / f >= 2); ++f) {
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

// Partials of n pieces: 256 rows of O in fp32, then their LSE.
inline int64_t pieces_bytes(int64_t items, int f, int D) { return f > 1 ? items * f * 256 * (D + 1) * 4 : 0; }

}  // namespace dit

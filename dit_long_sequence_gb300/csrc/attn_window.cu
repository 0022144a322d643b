// attn_window.cu -- attention over a sliding window of frames with sinks, forward,
// sm_103a: TMA-fed tiles, tcgen05 products with TMEM accumulators, warp-specialised
// roles that run on through a CTA's work items.
//
//     O_i = sum_j softmax_j(scale q_i . k_j) v_j,  LSE_i = ln sum_j exp(scale q_i . k_j)
// over the keys [0, min(sinks, hi_i)) and [lo_i, hi_i) of row i (window_span.h).  K
// and V are strided tensors, or the pages of a cache (PAGED).
//
// A work item is 256 query rows, two 128-row tiles, of one (batch entry, K/V head);
// where all rows of a sequence fit one tile (ONE: a few new tokens) it is that tile.
// Rows are (token, query head of the group): heads that share K and V share their
// tiles too.  The item walks the key tiles that some row of it sees, the sinks'
// first; a tile that every row of a warp sees whole passes without a mask, others
// through four mask words a row, computed from the row's bounds.
//
// 12 warps:
//   warps 0-3, 4-7  softmax of query tile 0, 1 (one TMEM lane = one row per thread)
//   warp 8          tcgen05.mma issuer (warp-wide); owns the TMEM allocation
//   warp 9          TMA producer: Q, then K_0, V_0, K_1, V_1, ... through a ring
//   warps 10, 11    idle (they complete the third warpgroup)
// Registers: 168 at launch; softmax 208, the rest 88: 256*208 + 128*88 = 384*168.
// TMEM (512 columns): S0 [0,128) S1 [128,256) O0 [256,256+D) O1 [256+D,256+2D); P_t
// (bf16) lies over the first half of S_t and is the PV product's TMEM operand.
//
// The grid has one CTA per item; a CTA that is done claims the next one that has not
// begun (cluster launch control), so that its roles go on: while the softmax warps
// write one item's result, the next one's first tiles are on their way and its
// first products run.  The last blocks of a sequence, which see the most keys of a
// causal mask, come first.
//
// ONE: S of consecutive tiles alternates between the two buffers, Q_1's shared memory
// goes to the ring (192 KB of K and V on their way), warps 4-7 leave at once.
//
// Few items are cut into key ranges (f pieces), whose normalised partials
// window_merge_kernel joins.
//
// Bound by the tensor pipe and each tile's chain of scores, softmax and product (12,288
// tokens in frames of 1,536, 8 heads: pipe 66% active); ONE by HBM.  Measured over the
// Python call: 24,576 tokens in frames of 1,536, three back and the first always, 32
// heads of 128: 1,760 to 1,800 us (1,500 to 1,530 TFLOP/s); 44,160 tokens, window of
// 2,048, 16 heads on 4: 590 us (1,240 TFLOP/s).  ONE: a token for 48 sequences of up to
// 16,384, 32 heads on 8: 252 and 278 us for two draws of lengths, 6.1 TB/s.
#include <cuda.h>
#include <cuda_runtime.h>

#include "window.cuh"

namespace dit {
namespace {

constexpr int kT = kWinTile;
constexpr int kThreads = 384;
constexpr uint32_t kSoftmaxRegs = 208;
constexpr uint32_t kOtherRegs = 88;
static_assert(256 * kSoftmaxRegs + 128 * kOtherRegs <= kThreads * 168, "register split");

// ONE: all rows of an item fit one query tile; its Q takes one tile of shared memory
// and the ring the rest.
template <int D, bool ONE>
struct Cfg {
    static constexpr int kTile = kT * D * 2;
    static constexpr int kQTiles = ONE ? 1 : 2;
    static constexpr int kStages = (D == 128 ? 6 : 12) - (ONE ? 0 : (D == 128 ? 2 : 4));     // K/V ring slots
    static constexpr int kBlock = kT * 128;              // 128 rows x 64 bf16 (one swizzle column)
    static constexpr int kQueue = 4;                     // items published ahead at most
    // barriers
    static constexpr int kQFull = 0, kQEmpty = 1;
    static constexpr int kKVFull = 2;
    static constexpr int kKVEmpty = kKVFull + kStages;
    static constexpr int kSFull = kKVEmpty + kStages;    // two
    static constexpr int kPFull = kSFull + 2;            // two
    static constexpr int kOFinal = kPFull + 2;           // two
    static constexpr int kOSettled = kOFinal + 1;        // ONE: every PV
    static constexpr int kDrain = kOFinal + 2;
    static constexpr int kItemFull = kDrain + 1, kItemEmpty = kItemFull + kQueue;
    static constexpr int kClaim = kItemEmpty + kQueue;
    static constexpr int kNumBars = kClaim + 1;
    static constexpr int kClaimOffset = (kQTiles + kStages) * kTile;           // 16 bytes
    static constexpr int kBarOffset = kClaimOffset + 16;
    static constexpr int kItemOffset = kBarOffset + kNumBars * 8;
    static constexpr int kSmemBytes = 1024 /*alignment slack*/ + kItemOffset + kQueue * 4 + 16;
    static_assert(kSmemBytes <= 232448, "shared memory");
};

// Claims a CTA of the grid that has not begun: the answer arrives at `dst` (16
// bytes) and counts on `bar`.
__device__ __forceinline__ void claim_ask(uint32_t dst, uint32_t bar) {
    asm volatile("clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];" ::"r"(dst), "r"(bar)
                 : "memory");
}
// The claimed CTA's index, or -1 when none was left.
__device__ __forceinline__ int claim_answer(uint32_t src) {
    int x;
    asm volatile(
        "{\n\t.reg .b128 h;\n\t.reg .pred p;\n\t.reg .b32 y, z, w;\n\t"
        "ld.shared.b128 h, [%1];\n\t"
        "clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, h;\n\t"
        "mov.b32 %0, -1;\n\t"
        "@p clusterlaunchcontrol.query_cancel.get_first_ctaid.v4.b32.b128 {%0, y, z, w}, h;\n\t}"
        : "=r"(x)
        : "r"(src)
        : "memory");
    return x;
}

// One item, the same for every role.
struct Item {
    int b, hk, blk, id;         // id: with its piece
    int first;                  // first token of the item
    int tokens;                 // tokens of the sequence that are queries
    int pos;                    // position of query 0
    int kv_len;                 // keys
    KeyTiles tiles;
    int begin, end;             // the piece's tiles
};
template <bool PAGED>
__device__ __forceinline__ Item decode(const WindowArgs& a, int id) {
    Item it;
    it.id = id;
    uint32_t piece = 0, rest = static_cast<uint32_t>(id);
    if (a.f > 1) rest = a.div_f.divmod(rest, piece);
    place(a, rest, it.b, it.hk, it.blk);
    it.first = it.blk * 2 * a.tokens;
    if constexpr (PAGED) {
        const int len = max(__ldg(a.kv_lens + it.b), 0);
        it.tokens = a.q_lens != nullptr ? min(max(__ldg(a.q_lens + it.b), 0), a.T) : a.T;
        it.pos = len - it.tokens;
        it.kv_len = min(len, a.capacity);
    } else {
        it.tokens = a.T;
        it.pos = a.offset;
        it.kv_len = a.kv_len;
    }
    it.begin = it.end = 0;
    it.tiles.n = 0;
    if (it.first < it.tokens) {
        const int last = min(it.first + 2 * a.tokens, it.tokens) - 1;
        it.tiles = key_tiles(a.win, it.pos + it.first, it.pos + last, it.kv_len);
        it.end = it.tiles.n;
        if (a.f > 1) {
            it.begin = static_cast<int>(a.div_f.div(piece * static_cast<uint32_t>(it.tiles.n)));
            it.end = static_cast<int>(a.div_f.div((piece + 1) * static_cast<uint32_t>(it.tiles.n)));
        }
    }
    return it;
}

// What the roles of a CTA share.
template <int D, bool ONE>
struct Cta {
    using C = Cfg<D, ONE>;
    uint8_t* smem;
    uint32_t base, bars, tmem;
    Watchdog wd, wd_drain;      // wd_drain ignores the abort flag: it waits for work already in flight
    __device__ __forceinline__ uint32_t bar(int i) const { return bars + i * 8; }
    __device__ __forceinline__ uint32_t q(int t) const { return base + t * C::kTile; }
    __device__ __forceinline__ uint32_t slot_offset(int i) const { return (C::kQTiles + static_cast<uint32_t>(i) % C::kStages) * C::kTile; }
};
__device__ __forceinline__ uint32_t turn(int n, int r) { return static_cast<uint32_t>(n / r) & 1u; }

// The CTA's items, in order: the producer publishes them, the other roles' warps
// take them.  a.n_items is the end.
template <int D, bool ONE>
__device__ __forceinline__ bool publish(const Cta<D, ONE>& s, int n, int id) {
    using C = Cfg<D, ONE>;
    const int slot = n % C::kQueue;
    const bool ok = wait_bounded_warp(s.bar(C::kItemEmpty + slot), turn(n, C::kQueue) ^ 1u, s.wd, ROLE_LOAD, SITE_ITEM_EMPTY);
    if (ok && lane_id() == 0) {
        *reinterpret_cast<volatile int*>(s.smem + C::kItemOffset + slot * 4) = id;
        mbar_arrive(s.bar(C::kItemFull + slot));
    }
    return ok;
}
template <int D, bool ONE>
__device__ __forceinline__ int take(const Cta<D, ONE>& s, const WindowArgs& a, int n, uint32_t role) {
    using C = Cfg<D, ONE>;
    const int slot = n % C::kQueue;
    const bool ok = wait_bounded_warp(s.bar(C::kItemFull + slot), turn(n, C::kQueue), s.wd, role, SITE_ITEM_FULL);
    const int id = ok ? *reinterpret_cast<volatile int*>(s.smem + C::kItemOffset + slot * 4) : a.n_items;
    __syncwarp();
    if (ok && lane_id() == 0) mbar_arrive(s.bar(C::kItemEmpty + slot));
    return id;
}

// ------------------------------------------------------------ TMA producer (a warp)
template <int D, bool PAGED, bool ONE>
__device__ __forceinline__ void produce(const Cta<D, ONE>& s, const CUtensorMap& tm_q, const CUtensorMap& tm_k, const CUtensorMap& tm_v,
                                        const WindowArgs& a) {
    using C = Cfg<D, ONE>;
    constexpr int S = C::kStages;
    const bool leader = lane_id() == 0;
    auto wait = [&](int i, uint32_t parity, uint32_t site) { return wait_bounded_warp(s.bar(i), parity, s.wd, ROLE_LOAD, site); };
    int I = 0, J = 0;                   // items with tiles, copies
    int asked = 0, claims = 0;          // claims made and answered
    bool ok = true;
    int id = static_cast<int>(blockIdx.x);
    for (int n = 0; ok; ++n) {
        ok = publish(s, n, id);
        if (!ok || id >= a.n_items) break;
        const Item it = decode<PAGED>(a, id);
        const int32_t* const row = PAGED ? a.table + it.b * a.table_sb : nullptr;
        if (it.begin < it.end) {
            ok = wait(C::kQEmpty, (I & 1) ^ 1u, SITE_Q_EMPTY);
            if (!ok) break;
            if (leader) {
                mbar_arrive_expect_tx(s.bar(C::kQFull), C::kQTiles * a.tokens * a.group * D * 2);
                for (int t = 0; t < C::kQTiles; ++t)
                    for (int c = 0; c < D / 64; ++c)
                        tma_load_5d(s.q(t) + c * C::kBlock, &tm_q, s.bar(C::kQFull), c * 64, 0, it.first + t * a.tokens, it.hk, it.b);
            }
            ++I;
        }
        const int ask_at = max(it.begin, it.end - 2);      // claim late: another CTA may be free earlier
        int entry = PAGED && it.begin < it.end ? page_entry(a, row, it.tiles.at(it.begin), it.kv_len) : 0;
        for (int i = it.begin; i <= it.end; ++i) {
            if (i == ask_at) {
                if (leader) {
                    fence_async();      // (the previous answer has been read)
                    mbar_arrive_expect_tx(s.bar(C::kClaim), 16);
                    claim_ask(s.base + C::kClaimOffset, s.bar(C::kClaim));
                }
                ++asked;
            }
            if (i == it.end) break;
            const int tile = it.tiles.at(i);
            if (!in_bounds(tile >= 0 && tile * kT < it.kv_len - a.dbg_keys_short, a.status, ROLE_LOAD, BND_KEY)) {
                *s.wd.abort_flag = 1;
                ok = false;
                break;
            }
            const int entry_next = PAGED && i + 1 < it.end ? page_entry(a, row, it.tiles.at(i + 1), it.kv_len) : 0;
            for (int kv = 0; kv < 2; ++kv, ++J) {
                ok = wait(C::kKVEmpty + J % S, turn(J, S) ^ 1u, SITE_KV_EMPTY);
                if (!ok) break;
                const uint32_t full = s.bar(C::kKVFull + J % S), dst = s.base + s.slot_offset(J);
                const CUtensorMap* const tm = kv ? &tm_v : &tm_k;
                if (leader) mbar_arrive_expect_tx(full, C::kTile);
                if constexpr (PAGED) {
                    __syncwarp();
                    copy_paged<D>(a, tm, dst, full, entry, tile, it.hk);
                } else if (leader) {
                    for (int c = 0; c < D / 64; ++c) tma_load_4d(dst + c * C::kBlock, tm, full, c * 64, tile * kT, it.hk, it.b);
                }
            }
            if (!ok) break;
            entry = entry_next;
        }
        if (!ok) break;
        ok = wait(C::kClaim, claims & 1, SITE_CLAIM);
        if (!ok) break;
        ++claims;
        const int got = claim_answer(s.base + C::kClaimOffset);
        id = got >= 0 ? got : a.n_items;
        __syncwarp();
    }
    if (!ok) {
        // Winding down: wait (bounded) until every copy issued has landed.
        auto land = [&](int i, uint32_t parity) { wait_bounded_warp(s.bar(i), parity, s.wd_drain, ROLE_LOAD, SITE_LOAD_DRAIN); };
        for (int j = J > S ? J - S : 0; j < J; ++j) land(C::kKVFull + j % S, turn(j, S));
        if (I > 0) land(C::kQFull, (I - 1) & 1);
        if (asked > claims) land(C::kClaim, claims & 1);
    }
}

// ------------------------------------------------------------ MMA issuer (a warp)
template <int D, bool PAGED, bool ONE>
__device__ __forceinline__ void multiply(const Cta<D, ONE>& s, const WindowArgs& a) {
    using C = Cfg<D, ONE>;
    constexpr int S = C::kStages;
    constexpr uint32_t kIdescQK = idesc_bf16_f32(kT, kT, false);
    constexpr uint32_t kIdescPV = idesc_bf16_f32(kT, D, true);
    auto wait = [&](int i, uint32_t parity, uint32_t site) { return wait_bounded_warp(s.bar(i), parity, s.wd, ROLE_MMA, site); };
    auto commit = [&](int i) { umma_commit_warp(s.bar(i)); };
    // S = Q_t K^T in buffer b: both K-major, K = D channels
    auto issue_qk = [&](int t, int b, uint32_t k_addr) {
        const uint64_t dq = sdesc_sw128(s.q(t), 16, 1024), dk = sdesc_sw128(k_addr, 16, 1024);
        static_for<D / 16>([&](auto kk) {
            constexpr uint32_t off = (kk.value >> 2) * C::kBlock + (kk.value & 3) * 32;
            umma_ss_warp<off>(s.tmem + b * 128, dq, dk, kIdescQK, kk.value > 0 ? 1u : 0u);
        });
    };
    // O_t (+)= P V: P from TMEM, V MN-major, K = 128 keys
    auto issue_pv = [&](int t, int b, uint32_t v_addr, bool accumulate) {
        const uint64_t dv = sdesc_sw128(v_addr, C::kBlock, 1024);
        static_for<kT / 16>([&](auto kk) {
            umma_ts_warp<kk.value * 16 * 128>(s.tmem + 256 + t * D, s.tmem + b * 128 + kk.value * 8, dv, kIdescPV,
                                              (accumulate || kk.value > 0) ? 1u : 0u);
        });
    };
    int I = 0, R = 0;           // items with tiles, ring slots taken
    int J = 0;                  // key tiles
    bool ok = true;
    if constexpr (ONE) {
        // One query tile: S takes the two buffers in turns, so that the next tile's
        // scores are there when the softmax warps are done with this one's.
        for (int n = 0; ok; ++n) {
            const int id = take(s, a, n, ROLE_MMA);
            if (id >= a.n_items) break;
            const Item it = decode<PAGED>(a, id);
            if (it.begin >= it.end) continue;
            ok = wait(C::kQFull, I & 1, SITE_Q_FULL);
            auto next_s = [&](int slot, int j) {
                ok = ok && wait(C::kKVFull + slot % S, turn(slot, S), SITE_KV_FULL);
                if (!ok) return;
                tc_fence_after();
                issue_qk(0, j & 1, s.base + s.slot_offset(slot));
                commit(C::kSFull + (j & 1));
                commit(C::kKVEmpty + slot % S);
            };
            next_s(R, J);
            if (!ok) break;
            if (it.begin + 1 == it.end) commit(C::kQEmpty);
            for (int i = it.begin; i < it.end; ++i, ++J, R += 2) {
                const bool more = i + 1 < it.end;
                if (more) next_s(R + 2, J + 1);
                if (ok && i + 2 == it.end) commit(C::kQEmpty);
                const int rv = R + 1;
                ok = ok && wait(C::kKVFull + rv % S, turn(rv, S), SITE_KV_FULL);
                if (!ok) break;
                clear_unseen<D>(s.smem + s.slot_offset(rv), it.tiles, it.tiles.at(i) * kT);
                ok = wait(C::kPFull + (J & 1), turn(J, 2), SITE_P_FULL);
                if (!ok) break;
                tc_fence_after();
                issue_pv(0, J & 1, s.base + s.slot_offset(rv), i > it.begin);
                commit(C::kKVEmpty + rv % S);
                commit(C::kOSettled);
                if (!more) commit(C::kOFinal + 0);
            }
            ++I;
        }
    }
    for (int n = 0; !ONE && ok; ++n) {
        const int id = take(s, a, n, ROLE_MMA);
        if (id >= a.n_items) break;
        const Item it = decode<PAGED>(a, id);
        if (it.begin >= it.end) continue;
        ok = wait(C::kQFull, I & 1, SITE_Q_FULL) && wait(C::kKVFull + R % S, turn(R, S), SITE_KV_FULL);
        if (!ok) break;
        tc_fence_after();
        issue_qk(0, 0, s.base + s.slot_offset(R));
        commit(C::kSFull + 0);
        issue_qk(1, 1, s.base + s.slot_offset(R));
        commit(C::kSFull + 1);
        commit(C::kKVEmpty + R % S);
        if (it.begin + 1 == it.end) commit(C::kQEmpty);
        ++R;
        for (int i = it.begin; i < it.end; ++i, ++J) {
            const bool more = i + 1 < it.end;
            const int rv = R, rk = R + 1;
            const uint32_t v_addr = s.base + s.slot_offset(rv), k_addr = s.base + s.slot_offset(rk);
            ok = wait(C::kKVFull + rv % S, turn(rv, S), SITE_KV_FULL);
            if (!ok) break;
            clear_unseen<D>(s.smem + s.slot_offset(rv), it.tiles, it.tiles.at(i) * kT);
            ok = wait(C::kPFull + 0, J & 1, SITE_P_FULL);
            if (!ok) break;
            tc_fence_after();
            issue_pv(0, 0, v_addr, i > it.begin);
            if (more) {
                ok = wait(C::kKVFull + rk % S, turn(rk, S), SITE_KV_FULL);
                if (!ok) break;
                tc_fence_after();
                issue_qk(0, 0, k_addr);
                commit(C::kSFull + 0);
            } else {
                commit(C::kOFinal + 0);
            }
            ok = wait(C::kPFull + 1, J & 1, SITE_P_FULL);
            if (!ok) break;
            tc_fence_after();
            issue_pv(1, 1, v_addr, i > it.begin);
            commit(C::kKVEmpty + rv % S);
            if (more) {
                issue_qk(1, 1, k_addr);
                commit(C::kSFull + 1);
                commit(C::kKVEmpty + rk % S);
                if (i + 2 == it.end) commit(C::kQEmpty);
                R += 2;
            } else {
                commit(C::kOFinal + 1);
                R += 1;
            }
        }
        ++I;
    }
    // Every product issued must finish before TMEM is released.
    commit(C::kDrain);
    wait_bounded_warp(s.bar(C::kDrain), 0, s.wd_drain, ROLE_MMA, SITE_DRAIN);
}

// ------------------------------------------------------------ softmax warps (0-7)
// This thread's query row of an item.  Worked out where it is used, not held: the
// softmax loop's scores leave few registers.
struct Row {
    int tile_row;               // of the item's 256
    int head, q_at;             // head of the group, token of the sequence
    bool mine;
    __device__ __forceinline__ Row(const WindowArgs& a, const Item& it) {
        int tid;
        asm volatile("mov.u32 %0, %%tid.x;" : "=r"(tid));
        tile_row = tid;
        uint32_t g;
        const int token = static_cast<int>(a.div_group.divmod(static_cast<uint32_t>(tid % kT), g));
        head = static_cast<int>(g);
        q_at = it.first + tid / kT * a.tokens + token;
        mine = token < a.tokens && q_at < it.tokens;
    }
};
// Which chunks of the next tile have a page, asked for a tile ahead.
template <bool PAGED>
struct PagedRow {
    __device__ PagedRow(const WindowArgs&, int) {}
    __device__ __forceinline__ void ask(const WindowArgs&, int, bool) {}
    __device__ __forceinline__ uint32_t there(const WindowArgs&, int) const { return ~0u; }
};
template <>
struct PagedRow<true> {
    const int32_t* row;
    int kv_len, entry;
    __device__ PagedRow(const WindowArgs& a, int id) : entry(-1) {
        const Item it = decode<true>(a, id);
        row = a.table + it.b * a.table_sb;
        kv_len = it.kv_len;
    }
    __device__ __forceinline__ void ask(const WindowArgs& a, int tile, bool any) {
        if (any) entry = page_entry(a, row, tile, kv_len);
    }
    __device__ __forceinline__ uint32_t there(const WindowArgs& a, int tile) const { return pages_there(a, entry, tile, kv_len); }
};
template <int D, bool PAGED, bool ONE>
__device__ __forceinline__ void soften(const Cta<D, ONE>& s, const WindowArgs& a) {
    using C = Cfg<D, ONE>;
    const int warp = threadIdx.x >> 5;
    const int t = warp >> 2;    // query tile
    const int wq = warp & 3;    // TMEM lane quadrant
    const uint32_t lane_off = static_cast<uint32_t>(wq * 32) << 16;
    const uint32_t tS = s.tmem + lane_off + t * 128, tO = s.tmem + lane_off + 256 + t * D;
    if (ONE && t > 0) return;   // (nothing of theirs is waited for)
    int I = 0, J = 0;
    bool ok = true;
    for (int n = 0; ok; ++n) {
        const int id = take(s, a, n, ROLE_SOFTMAX);
        if (id >= a.n_items) break;
        // Held across the tiles: the row's bounds and the tiles' order.
        int lo = 0, hi = kNoBound, i, end, ns, shift;
        bool any_tile, any_row = true;
        {
            const Item it = decode<PAGED>(a, id);
            const Row row(a, it);
            // rows that are not there see everything, so that they mask no tile
            if (row.mine) {
                const Span sp = span_of(a.win, it.pos + row.q_at, it.kv_len);
                lo = sp.lo;
                hi = sp.hi;
            }
            if (ONE) any_row = __any_sync(0xffffffffu, row.mine);
            i = it.begin;
            end = it.end;
            ns = it.tiles.ns;
            shift = it.tiles.w0 - ns;
            any_tile = i < end;
        }
        PagedRow<PAGED> pages(a, id);
        pages.ask(a, i < ns ? i : i + shift, any_tile);
        float m = -INFINITY, l = 0.f;
        for (bool first = true; i < end; ++J, first = false) {
            const int tile = i < ns ? i : i + shift, k0 = tile * kT;
            ++i;
            const uint32_t there = pages.there(a, tile);
            pages.ask(a, i < ns ? i : i + shift, i < end);
            const bool masked = !__all_sync(0xffffffffu, sees_all(lo, hi, a.win.sinks, k0)) || there != ~0u;
            uint32_t words[4] = {~0u, ~0u, ~0u, ~0u};
            if (masked) {
#pragma unroll
                for (int w = 0; w < 4; ++w) {
                    words[w] = seen_word(lo, hi, a.win.sinks, k0 + 32 * w);
                    if (PAGED && there != ~0u) words[w] &= paged_word(there, a.chunk, w);
                }
            }
            const int b = ONE ? J & 1 : t;      // S's buffer, and its barriers
            ok = wait_bounded(s.bar(C::kSFull + b), ONE ? turn(J, 2) : J & 1, s.wd, ROLE_SOFTMAX, SITE_S_FULL);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            tc_fence_after();
            if (any_row) {      // (a warp without a row leaves its lanes' P as they are: no other row reads them)
                // (two tiles: S(j) was committed behind PV(j - 1); one: its own barrier)
                soften_tile<D>(ONE ? tS + b * 128 : tS, tO, a.scale_log2, first, masked, words, m, l, [&]() {
                    if (ONE && wait_bounded_warp(s.bar(C::kOSettled), (J - 1) & 1, s.wd, ROLE_SOFTMAX, SITE_O_SETTLED)) tc_fence_after();
                });
                tmem_st_wait();
            }
            tc_fence_before();
            mbar_arrive(s.bar(C::kPFull + b));
        }
        if (!ok) break;
        if (any_tile) {
            ok = wait_bounded(s.bar(C::kOFinal + t), I & 1, s.wd, ROLE_SOFTMAX, SITE_O_FINAL);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            tc_fence_after();
            ++I;
        }
        // The result, from this thread's row: whole 32-byte sectors.  (PV of the
        // next item's first tile overwrites O only after this thread's next P.)
        int again = id;         // decoded anew: only its number is held across the tiles
        asm volatile("" : "+r"(again));
        const Item it = decode<PAGED>(a, again);
        const Row row(a, it);
        const bool any_key = l > 0.f || l != l;
        const float inv = any_key ? 1.f / l : 0.f;
        const float lse = any_key ? (m + log2f(l)) * kWinLn2 : -INFINITY;
        const int h = it.hk * a.group + row.head;
        const int64_t off = it.b * a.o_sb + static_cast<int64_t>(row.q_at) * a.o_sn + h * a.o_sh;
        const int64_t part = static_cast<int64_t>(it.id) * a.part_rows + row.tile_row;
        const bool stored = row.mine && in_bounds(a.f > 1 || (off >= 0 && off + D <= a.dbg_o_elems), a.status, ROLE_SOFTMAX, BND_OUT);
#pragma unroll 1
        for (int cc = 0; cc < D / 32; ++cc) {
            uint32_t o[32];
            if (any_tile) {
                tmem_ld32(tO + cc * 32, o);
                tmem_ld_wait_dep(o);
            }
#pragma unroll
            for (int k = 0; k < 32; ++k) o[k] = any_key ? __float_as_uint(__uint_as_float(o[k]) * inv) : 0u;
            if (stored) store_32(a, a.f > 1 ? a.ws_o + part * D + cc * 32 : nullptr, off + cc * 32, o);
            __syncwarp();
        }
        if (stored) {
            if (a.f > 1) a.ws_lse[part] = lse;
            else a.lse[(static_cast<int64_t>(it.b) * a.H + h) * a.T + row.q_at] = lse;
        }
        tc_fence_before();
    }
}

template <int D, bool PAGED, bool ONE>
__global__ void __launch_bounds__(kThreads, 1)
    attn_window_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                       const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ WindowArgs a) {
    using C = Cfg<D, ONE>;
    extern __shared__ uint8_t smem_raw[];
    Cta<D, ONE> s;
    s.smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    s.base = smem_u32(s.smem);
    s.bars = s.base + C::kBarOffset;
    uint32_t* const tmem_slot = reinterpret_cast<uint32_t*>(s.smem + C::kItemOffset + C::kQueue * 4);
    volatile int* const abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
    volatile int* const never_flag = reinterpret_cast<volatile int*>(tmem_slot + 2);
    s.wd = Watchdog{a.status, a.timeout_ns, abort_flag};
    s.wd_drain = Watchdog{a.status, a.timeout_ns, never_flag};
    const int warp = threadIdx.x >> 5;

    if (threadIdx.x == 0) {
        for (int i = 0; i < C::kNumBars; ++i) {
            const bool all = i == C::kPFull || i == C::kPFull + 1;
            const bool takers = i >= C::kItemEmpty && i < C::kItemEmpty + C::kQueue;     // the MMA and softmax warps
            mbar_init(s.bar(i), all ? 128 : (takers ? (ONE ? 5 : 9) : 1));
        }
        *abort_flag = 0;
        *never_flag = 0;
        fence_mbar_init();
        if (a.f > 1) let_next();
    }
    // Rows of a query tile past its last whole token hold nothing that is copied:
    // zeros, so that they make no NaN and no rescale.
    const int spare = kT - a.tokens * a.group;
    for (int u = threadIdx.x; u < C::kQTiles * (D / 64) * spare * 8; u += kThreads) {
        const int block = u / (spare * 8), rest = u % (spare * 8);
        *reinterpret_cast<uint4*>(s.smem + block * C::kBlock + (kT - spare + rest / 8) * 128 + (rest & 7) * 16) = make_uint4(0u, 0u, 0u, 0u);
    }
    fence_async();
    if (warp == 8) {
        tmem_alloc(smem_u32(tmem_slot), 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    s.tmem = *tmem_slot;

    if (warp >= 8) {
        regs_decrease<kOtherRegs>();
        if (warp == 8) {
            multiply<D, PAGED, ONE>(s, a);
        } else if (warp == 9) {
            if (lane_id() == 0 && (PAGED ? a.capacity : a.kv_len) > 0) {      // (no keys, no maps)
                tma_prefetch_desc(&tm_q);
                tma_prefetch_desc(&tm_k);
                tma_prefetch_desc(&tm_v);
            }
            produce<D, PAGED, ONE>(s, tm_q, tm_k, tm_v, a);
        }
        __syncwarp();
    } else {
        regs_increase<kSoftmaxRegs>();
        soften<D, PAGED, ONE>(s, a);
    }

    tc_fence_before();
    __syncthreads();
    if (warp == 8) {
        tc_fence_after();
        tmem_dealloc(s.tmem, 512);
    }
}

// Joins the f pieces of every item: with M = max_p LSE_p and w_p = e^(LSE_p - M),
// O = sum_p w_p O_p / sum_p w_p and LSE = M + ln sum_p w_p.  A piece without a key
// of the row has LSE_p = -inf and weight 0.  D / 4 lanes a row.  (The partials are
// written while this kernel may already be set up: no read-only loads of them.)
template <int D, bool PAGED>
__global__ void __launch_bounds__(256) window_merge_kernel(const __grid_constant__ WindowArgs a) {
    constexpr int LPR = D / 4;
    after_previous();
    const int64_t unit = (static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x) / LPR;
    const int c4 = static_cast<int>(threadIdx.x % LPR);
    const int item = static_cast<int>(unit / a.part_rows), rr = static_cast<int>(unit % a.part_rows);
    if (item >= a.n_items / a.f) return;
    uint32_t g;
    int b, hk, blk;
    place(a, static_cast<uint32_t>(item), b, hk, blk);
    const int t = rr / kT;
    const int token = static_cast<int>(a.div_group.divmod(static_cast<uint32_t>(rr % kT), g));
    const int q_at = blk * 2 * a.tokens + t * a.tokens + token;
    const int tokens = PAGED && a.q_lens != nullptr ? min(__ldg(a.q_lens + b), a.T) : a.T;
    if (token >= a.tokens || q_at >= tokens) return;
    const int64_t p0 = static_cast<int64_t>(item) * a.f * a.part_rows + rr;
    float mx = -INFINITY;
    for (int p = 0; p < a.f; ++p) mx = fmaxf(mx, __ldcg(a.ws_lse + p0 + static_cast<int64_t>(p) * a.part_rows));
    float sum = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    bool bad = false;           // (a NaN must stay one)
    for (int p = 0; p < a.f; ++p) {
        const float lp = __ldcg(a.ws_lse + p0 + static_cast<int64_t>(p) * a.part_rows);
        bad = bad || lp != lp;
        if (lp == -INFINITY) continue;
        const float w = expf(lp - mx);
        const float4 o = __ldcg(reinterpret_cast<const float4*>(a.ws_o + (p0 + static_cast<int64_t>(p) * a.part_rows) * D) + c4);
        sum += w;
        acc.x = fmaf(w, o.x, acc.x);
        acc.y = fmaf(w, o.y, acc.y);
        acc.z = fmaf(w, o.z, acc.z);
        acc.w = fmaf(w, o.w, acc.w);
    }
    const float inv = bad ? NAN : (sum > 0.f ? 1.f / sum : 0.f);
    const int h = hk * a.group + static_cast<int>(g);
    const int64_t off = b * a.o_sb + static_cast<int64_t>(q_at) * a.o_sn + h * a.o_sh + 4 * c4;
    if (!in_bounds(off >= 0 && off + 4 <= a.dbg_o_elems, a.status, 0, BND_OUT)) return;
    if (a.out_bf16)
        *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.out) + off) =
            make_uint2(pack_bf16x2(acc.x * inv, acc.y * inv), pack_bf16x2(acc.z * inv, acc.w * inv));
    else
        *reinterpret_cast<float4*>(static_cast<float*>(a.out) + off) = make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv);
    if (c4 == 0)
        a.lse[(static_cast<int64_t>(b) * a.H + h) * a.T + q_at] = bad ? NAN : (sum > 0.f ? mx + logf(sum) : -INFINITY);
}

template <int D, bool PAGED, bool ONE>
cudaError_t launch_impl(const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv, const WindowArgs& a, cudaStream_t s) {
    auto kern = attn_window_kernel<D, PAGED, ONE>;
    constexpr int kSmem = Cfg<D, ONE>::kSmemBytes;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
    if (e != cudaSuccess) return e;
    kern<<<static_cast<unsigned>(a.n_items), kThreads, kSmem, s>>>(tq, tk, tv, a);
    if ((e = cudaGetLastError()) != cudaSuccess || a.f == 1) return e;
    const int64_t threads = static_cast<int64_t>(a.n_items / a.f) * a.part_rows * (D / 4);
    return launch_behind(window_merge_kernel<D, PAGED>, static_cast<unsigned>((threads + 255) / 256), 256, 0, s, a);
}

}  // namespace

cudaError_t launch_attn_window(const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv, const WindowArgs& a,
                               int D, bool paged, cudaStream_t s) {
    const bool one = one_tile(a);
    if (D == 128) {
        if (paged) return one ? launch_impl<128, true, true>(tq, tk, tv, a, s) : launch_impl<128, true, false>(tq, tk, tv, a, s);
        return one ? launch_impl<128, false, true>(tq, tk, tv, a, s) : launch_impl<128, false, false>(tq, tk, tv, a, s);
    }
    if (paged) return one ? launch_impl<64, true, true>(tq, tk, tv, a, s) : launch_impl<64, true, false>(tq, tk, tv, a, s);
    return one ? launch_impl<64, false, true>(tq, tk, tv, a, s) : launch_impl<64, false, false>(tq, tk, tv, a, s);
}

}  // namespace dit

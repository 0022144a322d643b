// attn_bwd.cu -- attention backward, sm_103a, TMA + tcgen05 (TMEM
// accumulators), warp-specialised like the forward kernel.
//
// With S = scale * Q K^T over the keys a row may attend and the forward pass'
// LSE,
//     P = exp(S - LSE),  dV = P^T dO,  delta_i = sum_d dO_id O_id - dLSE_i,
//     dS = P o (dO V^T - delta),  dQ = scale dS K,  dK = scale dS^T Q:
// the probabilities are recomputed tile by tile, never stored.
//
// Two kinds of work item, so that no gradient is summed through memory and
// every result repeats bit for bit (no atomics):
//   key item    one 128-key tile of a (b, h); streams the 128-row query tiles,
//               S^T = K Q^T and dP^T = V dO^T (rows are keys), then
//               dV += P^T dO and dK += dS^T Q;
//   query item  one 128-row query tile; streams the key tiles,
//               S = Q K^T and dP = dO V^T, then dQ += dS K.
// Seven products a tile pair instead of five: the two recomputed ones cost
// 40% more tensor work, against fp32 atomics of 64 KB a tile pair into L2 (or a
// serial order of CTAs) for one kind of item that also adds into dQ.
//
// One CTA per SM takes items from a common counter, the key items first, until
// none is left (which CTA works on an item changes nothing in its result).  Its
// roles run on through the items without meeting: while the softmax warps write
// one item's gradient, the next one's fixed tiles are on their way and its first
// products run.
//
// In both, the streamed tiles come in pairs (X0, X1) = (Q, dO) or (K, V), the
// fixed ones are (F0, F1) = (K, V) or (Q, dO), and
//   T0 = F0 X0^T, T1 = F1 X1^T, ACC1 += P X1 (key item), ACC0 += dS X0,
// with P and dS the TMEM A operands, written by the softmax warps in bf16 over
// their own half of T0 / T1.
//
// 12 warps:
//   warps 0-3, 4-7  softmax warpgroups: columns [0, 64) and [64, 128) of every
//                   tile, one TMEM lane = one row per thread
//   warp 8          tcgen05.mma issuer (warp-wide, one elected lane issues);
//                   owns the TMEM allocation
//   warp 9          TMA producer (one lane issues)
//   warps 10, 11    idle (they complete the third warpgroup)
// Registers: 168 at launch; softmax 208, the rest 88 (as the forward kernel).
// TMEM (512 columns): T0 [0,128) T1 [128,256) ACC0 [256,256+D)
// ACC1 [256+D,256+2D) (key items), a second T0 [384,512) (query items; D = 64).
//
// Order of products.  An issue that finds the tensor pipe busy waits for it, so
// every wait of the MMA warp on a barrier (some 100 cycles when it is met) is
// idle time of the pipe, and the loop makes as few as it can.
//   query items: T0 one tile ahead of T1; once dS(j) is ready (so dP(j) has been
//     read) dP(j+1), dQ(j), S(j+2): one wait a tile for dS(j) and X(j+2) together.
//   key items, D = 64: the same with P: dV(j), S(j+2) behind P(j); dK(j), dP(j+1)
//     behind dS(j).
//   key items, D = 128 (one T0): dV(j), S(j+1) behind P(j); dK(j), dP(j+1) behind
//     dS(j).  (P handed over in two halves, so that dV(j) begins with the first,
//     measured 1.5% on the key items: another wait eats most of it.)
//
// Measured, 16,384 x 16,384, 8 heads: D = 128 2.21 to 2.35 ms (the power cap
// decides), 1.7 PFLOP/s executed, tensor pipe 73% active; D = 64 1.58 ms, 51%: products with
// N = 64 cost as much as with N = 128, and the softmax warps' chain is longer than
// what is left to hide it behind (issue 45%, exponential unit 29%, tensor memory 64%).
// 16 softmax warps of half as many columns were 5 to 10% slower.
//
// Rows without an allowed key have LSE = -inf; they, and the rows past Nq, get
// P = 0 through a stored -LSE of -inf (and a stored delta of 0).  Keys past kv_len are zero-filled by the
// tensor maps and masked (query item) or not stored (key item: their gradients
// are written as zeros).
#include <cuda.h>
#include <cuda_runtime.h>

#include "debug.cuh"
#include "internal.h"
#include "ptx.cuh"
#include "train.h"

namespace dit {
namespace {

constexpr int kT = 128;            // rows of a tile
constexpr int kThreads = 384;
constexpr uint32_t kSoftmaxRegs = 208;
constexpr uint32_t kOtherRegs = 88;
static_assert(256 * kSoftmaxRegs + 128 * kOtherRegs <= kThreads * 168, "register split");
constexpr float kLog2e = 1.4426950408889634f;

enum BwdSite : uint32_t {
    SITE_FIX_FULL = 11, SITE_X_FULL = 12, SITE_X_EMPTY = 13, SITE_T0_FULL = 14, SITE_T1_FULL = 15, SITE_P_READY = 16,
    SITE_DS_READY = 17, SITE_ACC_FINAL = 19, SITE_BWD_DRAIN = 21,
    SITE_NO_ROOM = 22, SITE_FIX_EMPTY = 23, SITE_ACC_FREE = 24,
    SITE_ITEM = 25
};

// Untiled bulk copy global -> shared (16-byte aligned, a multiple of 16 bytes).
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
                 "l"(reinterpret_cast<uint64_t>(src)), "r"(bytes), "r"(bar)
                 : "memory");
}

// 32 lanes x 32 32-bit columns: r[16 u + 4k + i] is lane 16 u + t / 4 + 8 (i / 2),
// column 8k + 2 (t mod 4) + (i mod 2) for thread t of the warp.
__device__ __forceinline__ void tmem_ld_16x256b_x4x2(uint32_t taddr, uint32_t (&r)[32]) {
#pragma unroll
    for (int u = 0; u < 2; ++u)
        asm volatile(
            "tcgen05.ld.sync.aligned.16x256b.x4.b32 "
            "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
            : "=r"(r[16 * u]), "=r"(r[16 * u + 1]), "=r"(r[16 * u + 2]), "=r"(r[16 * u + 3]), "=r"(r[16 * u + 4]),
              "=r"(r[16 * u + 5]), "=r"(r[16 * u + 6]), "=r"(r[16 * u + 7]), "=r"(r[16 * u + 8]), "=r"(r[16 * u + 9]),
              "=r"(r[16 * u + 10]), "=r"(r[16 * u + 11]), "=r"(r[16 * u + 12]), "=r"(r[16 * u + 13]),
              "=r"(r[16 * u + 14]), "=r"(r[16 * u + 15])
            : "r"(taddr + (static_cast<uint32_t>(16 * u) << 16)));
}
// 32 lanes x 16 32-bit columns: r[8 u + 2k + i] goes to lane 16 u + t / 4 + 8 i,
// column 4k + t mod 4.  Two neighbouring values of the load above, packed, land
// on the columns of their pair.
__device__ __forceinline__ void tmem_st_16x128b_x4x2(uint32_t taddr, const uint32_t (&r)[16]) {
#pragma unroll
    for (int u = 0; u < 2; ++u)
        asm volatile("tcgen05.st.sync.aligned.16x128b.x4.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(
                         taddr + (static_cast<uint32_t>(16 * u) << 16)),
                     "r"(r[8 * u]), "r"(r[8 * u + 1]), "r"(r[8 * u + 2]), "r"(r[8 * u + 3]), "r"(r[8 * u + 4]),
                     "r"(r[8 * u + 5]), "r"(r[8 * u + 6]), "r"(r[8 * u + 7])
                     : "memory");
}

// (d0, d1) = (a0*b + c0, a1*b + c1), one packed FMA.
__device__ __forceinline__ void ffma2(float& d0, float& d1, float a0, float a1, float b, float c0, float c1) {
    asm("{\n\t.reg .b64 ra, rb, rc, rd;\n\t"
        "mov.b64 ra, {%2, %3};\n\t"
        "mov.b64 rb, {%4, %4};\n\t"
        "mov.b64 rc, {%5, %6};\n\t"
        "fma.rn.f32x2 rd, ra, rb, rc;\n\t"
        "mov.b64 {%0, %1}, rd;\n\t}"
        : "=f"(d0), "=f"(d1)
        : "f"(a0), "f"(a1), "f"(b), "f"(c0), "f"(c1));
}
// (d0, d1) = ((a0 + c0) * b0, (a1 + c1) * b1), packed.
__device__ __forceinline__ void fadd2_mul2(float& d0, float& d1, float a0, float a1, float c0, float c1, float b0, float b1) {
    asm("{\n\t.reg .b64 ra, rb, rc;\n\t"
        "mov.b64 ra, {%2, %3};\n\t"
        "mov.b64 rc, {%4, %5};\n\t"
        "mov.b64 rb, {%6, %7};\n\t"
        "add.rn.f32x2 ra, ra, rc;\n\t"
        "mul.rn.f32x2 ra, ra, rb;\n\t"
        "mov.b64 {%0, %1}, ra;\n\t}"
        : "=f"(d0), "=f"(d1)
        : "f"(a0), "f"(a1), "f"(c0), "f"(c1), "f"(b0), "f"(b1));
}

template <int D>
struct Cfg {
    static constexpr int kTile = kT * D * 2;
    // Ring slots of X0 and of X1.  X0(j) is held until the last product of tile j,
    // so three of it keep the next copy three products ahead of its use; with
    // two and two, both kinds of item ran at 1.6 us a tile pair whatever their
    // products, waiting for copies.
    static constexpr int kR0 = D == 128 ? 3 : 4;
    static constexpr int kR1 = D == 128 ? 2 : 4;
    static constexpr int kStats = kR1;                   // statistics of this many tiles
    static constexpr int kBlock = kT * 128;              // 128 rows x 64 bf16 (one swizzle column)
    static constexpr int kStatBytes = 2 * kT * 4;        // -lse2[128], -delta[128]
    // barriers
    static constexpr int kFixFull = 0;
    static constexpr int kXFull = 1;                     // X0 and X1 of a tile (by X0's slot)
    static constexpr int kX0Empty = kXFull + kR0;
    static constexpr int kX1Empty = kX0Empty + kR0;
    static constexpr int kT0Full = kX1Empty + kR1;       // two (two T0)
    static constexpr int kT1Full = kT0Full + 2;
    // P ready; two by the tile's parity where key items have two T0 (D = 64): with
    // S issued ahead the softmax warps may finish P(j+1) before the MMA warp has
    // looked for P(j), and one barrier would be a phase past the one it waits for.
    // (dS(j+1) needs dP(j+1), issued after the wait for dS(j): one barrier.)
    static constexpr int kP = kT1Full + 1;
    static constexpr int kDS = kP + 2;
    static constexpr int kAccFinal = kDS + 1;
    static constexpr int kAccFree = kAccFinal + 1;       // the accumulators have been read
    static constexpr int kFixEmpty = kAccFree + 1;       // the last T0, T1 of an item are done
    static constexpr int kDrain = kFixEmpty + 1;
    static constexpr int kNumBars = kDrain + 1;
    static constexpr int kStatOffset = (2 + kR0 + kR1) * kTile;
    static constexpr int kBarOffset = kStatOffset + kStats * kStatBytes;
    // two sets of barriers: key items', query items'; then the item queue's
    static constexpr int kQueue = 4;                     // items published ahead at most
    static constexpr int kItemFull = 2 * kNumBars, kItemEmpty = kItemFull + kQueue;
    static constexpr int kItemOffset = kBarOffset + (kItemEmpty + kQueue) * 8;
    static constexpr int kUsedBytes = kItemOffset + kQueue * 4 + 16;
    // with room to start on a 1,024-byte boundary where the buffer does not
    static constexpr int kSmemBytes = kUsedBytes + 1024 <= 232448 ? kUsedBytes + 1024 : 232448;
    static_assert(kUsedBytes <= kSmemBytes, "shared memory");
    // TMEM columns
    static constexpr int kColT0 = 0, kColT1 = 128, kColAcc0 = 256, kColAcc1 = 256 + D, kColT0b = 384;
    static constexpr bool kKeyDouble = kColAcc1 + D <= kColT0b;     // key items have a second T0
    // with two T0, S(j+2) is issued while X0(j) is still held: three slots
    static_assert(kR0 >= 3, "ring");
};

// One item: its fixed tile, and the streamed tiles [begin, end) of its piece.
template <bool KEY>
struct Item {
    int b, h, fixed, begin, end;
    bool cut;                   // a piece: its result goes to the partials
    int64_t part_tile;          // its place among them
};

// Items count pieces fastest, then tiles, then heads, so that the CTAs at work
// share a few heads' tiles in L2; with a mask heads before tiles, since masks
// tend to load some tiles of every head more than others, and those then begin
// together: key items from the first (the keys that all rows attend), query
// items from the last (rows behind the masked ones, late rows of a causal mask).
template <bool KEY, bool MASK>
__device__ __forceinline__ Item<KEY> decode(const AttnBwdArgs& a, int id) {
    Item<KEY> it;
    const int slot = KEY ? id : id - a.n_kv_items;
    const uint32_t f = static_cast<uint32_t>(KEY ? a.f_kv : a.f_q);
    const int tiles = KEY ? a.kv_out_tiles : a.q_tiles;
    uint32_t piece = 0, inner, h, item = static_cast<uint32_t>(slot);
    it.cut = KEY ? f > 1 : slot >= a.q_whole;
    if (it.cut) {
        const uint32_t first = static_cast<uint32_t>(KEY ? 0 : a.q_whole);
        item = first + (KEY ? a.div_f_kv : a.div_f_q).divmod(static_cast<uint32_t>(slot) - first, piece);
    }
    const uint32_t outer = (MASK ? a.div_bh : (KEY ? a.div_kv_tiles : a.div_q_tiles)).divmod(item, inner);
    const uint32_t bh = MASK ? inner : outer;
    it.fixed = static_cast<int>(!MASK ? inner : KEY ? outer : tiles - 1 - outer);
    it.b = static_cast<int>(a.div_h.divmod(bh, h));
    it.h = static_cast<int>(h);
    it.part_tile = (static_cast<int64_t>(bh) * tiles + it.fixed - (KEY ? 0 : a.q_whole)) * f + piece;
    // a key tile wholly past kv_len has nothing to stream: its gradient is zero
    const uint32_t x_tiles = static_cast<uint32_t>(KEY ? (it.fixed < a.kv_tiles ? a.q_tiles : 0) : a.kv_tiles);
    it.begin = 0;
    it.end = static_cast<int>(x_tiles);
    if (it.cut) {
        it.begin = static_cast<int>((KEY ? a.div_f_kv : a.div_f_q).div(piece * x_tiles));
        it.end = static_cast<int>((KEY ? a.div_f_kv : a.div_f_q).div((piece + 1) * x_tiles));
    }
    return it;
}

// The streamed tiles of an item in order: all of [begin, end), or with an
// occupancy map those whose bit is set -- a key item's the bit of its key tile
// in each 256-row query block's words, a query item's the bits of its block's
// words.  A warp holds the bits in its lanes (lane w: bits 32 w ..), 1,024 of
// them; items beyond that many blocks (key) or key tiles (query) are streamed
// whole.  Every call is made by a whole, converged warp.
template <bool KEY, bool MASK>
struct Stream {
    int t, end;
    uint32_t bits;
    bool whole;
    __device__ Stream(const AttnBwdArgs& a, const Item<KEY>& it) : t(it.begin), end(it.end), bits(0u), whole(true) {
        if constexpr (MASK) {
            const int n = KEY ? (a.q_tiles + 1) >> 1 : a.kv_tiles;
            if (a.occ == nullptr || n > 1024 || t >= end) return;
            whole = false;
            const int lane = static_cast<int>(lane_id());
            const uint32_t* occ = a.occ + static_cast<int64_t>(it.b) * a.occ_blocks * a.occ_words;
            if constexpr (KEY) {
                for (int w = 0; w * 32 < n; ++w) {
                    const int blk = w * 32 + lane;
                    const bool on = blk < n && ((occ[static_cast<int64_t>(blk) * a.occ_words + (it.fixed >> 5)] >> (it.fixed & 31)) & 1u);
                    const uint32_t all = __ballot_sync(0xffffffffu, on);
                    if (lane == w) bits = all;
                }
            } else {
                if (lane < a.occ_words) bits = occ[static_cast<int64_t>(it.fixed >> 1) * a.occ_words + lane];
            }
        }
    }
    // the next tile, or -1
    __device__ __forceinline__ int next() {
        if constexpr (MASK) {
            while (!whole && t < end) {
                const int i = KEY ? t >> 1 : t;
                const uint32_t w = __shfl_sync(0xffffffffu, bits, i >> 5) >> (i & 31);
                if (w & 1u) break;
                const int skip = w != 0u ? __ffs(static_cast<int>(w)) - 1 : 32 - (i & 31);
                t = KEY ? (i + skip) * 2 : i + skip;
            }
        }
        return t < end ? t++ : -1;
    }
    __device__ __forceinline__ int count() const {
        if constexpr (MASK) {
            if (!whole) {
                Stream c = *this;
                int n = 0;
                while (c.next() >= 0) ++n;
                return n;
            }
        }
        return end - t;
    }
};

// What the roles of a CTA share.
template <int D>
struct Cta {
    using C = Cfg<D>;
    uint8_t* smem;
    uint32_t base, bars, tmem;
    Watchdog wd, wd_drain;      // wd_drain ignores the abort flag: it waits for work already in flight
    template <bool KEY>
    __device__ __forceinline__ uint32_t bar(int i) const { return bars + ((KEY ? 0 : C::kNumBars) + i) * 8; }
    __device__ __forceinline__ uint32_t f0() const { return base; }
    __device__ __forceinline__ uint32_t f1() const { return base + C::kTile; }
    __device__ __forceinline__ uint32_t x0(int j) const { return base + (2 + j % C::kR0) * C::kTile; }
    __device__ __forceinline__ uint32_t x1(int j) const { return base + (2 + C::kR0 + j % C::kR1) * C::kTile; }
};
// The items a CTA works on, in order: its producer takes them from the counter
// and publishes them one ahead; every other role's warps take them from there.
// Ids from n_kv_items on are query items, n_kv_items + n_q_items is the end.
struct Queue {
    uint32_t n = 0;
};
template <int D>
__device__ __forceinline__ bool publish(const Cta<D>& s, Queue& q, int id) {
    using C = Cfg<D>;
    const uint32_t slot = q.n % C::kQueue;
    const bool ok = wait_bounded_warp(s.bars + (C::kItemEmpty + slot) * 8, ((q.n / C::kQueue) & 1u) ^ 1u, s.wd, ROLE_LOAD, SITE_ITEM);
    if (ok && lane_id() == 0) {
        *reinterpret_cast<volatile int*>(s.smem + C::kItemOffset + slot * 4) = id;
        mbar_arrive(s.bars + (C::kItemFull + slot) * 8);
    }
    ++q.n;
    return ok;
}
template <int D>
__device__ __forceinline__ int take(const Cta<D>& s, const AttnBwdArgs& a, Queue& q, uint32_t role) {
    using C = Cfg<D>;
    const uint32_t slot = q.n % C::kQueue;
    const bool ok = wait_bounded_warp(s.bars + (C::kItemFull + slot) * 8, (q.n / C::kQueue) & 1u, s.wd, role, SITE_ITEM);
    const int id = ok ? *reinterpret_cast<volatile int*>(s.smem + C::kItemOffset + slot * 4) : a.n_kv_items + a.n_q_items;
    __syncwarp();
    if (ok && lane_id() == 0) mbar_arrive(s.bars + (C::kItemEmpty + slot) * 8);
    ++q.n;
    return id;
}
// The producer's next item: the first is the CTA's own number.
__device__ __forceinline__ int next_item(const AttnBwdArgs& a, int last) {
    if (a.counter == nullptr) return min(last + static_cast<int>(gridDim.x), a.n_kv_items + a.n_q_items);
    int id = 0;
    if (lane_id() == 0) id = static_cast<int>(gridDim.x) + static_cast<int>(atomicAdd(a.counter, 1u));
    return min(__shfl_sync(0xffffffffu, id, 0), a.n_kv_items + a.n_q_items);
}
// The parity of use n of a slot of r.
__device__ __forceinline__ uint32_t turn(int n, int r) { return static_cast<uint32_t>(n / r) & 1u; }

// ------------------------------------------------------------ TMA producer (a warp; lane 0 issues)
template <int D, bool KEY, bool MASK>
__device__ __forceinline__ void produce(const Cta<D>& s, const CUtensorMap& tm_f0, const CUtensorMap& tm_f1,
                                        const CUtensorMap& tm_x0, const CUtensorMap& tm_x1, const AttnBwdArgs& a,
                                        Queue& queue, int& id) {
    using C = Cfg<D>;
    constexpr int R0 = C::kR0, R1 = C::kR1;
    const bool leader = lane_id() == 0;
    auto bar = [&](int i) { return s.template bar<KEY>(i); };
    auto wait = [&](int i, uint32_t parity, uint32_t site) { return wait_bounded_warp(bar(i), parity, s.wd, ROLE_LOAD, site); };
    auto copy = [&](const CUtensorMap* tm, uint32_t dst, int full, int row, int h, int b) {
        for (int c = 0; c < D / 64; ++c) tma_load_4d(dst + c * C::kBlock, tm, bar(full), c * 64, row, h, b);
    };
    int J = 0, I = 0;                   // tiles and items so far
    int done = 0;                       // tiles copied
    int half = -1;                      // a tile whose X0 alone was copied
    bool ok = true;
    const int last = KEY ? a.n_kv_items : a.n_kv_items + a.n_q_items;
    for (int next; ok && id < last; id = next) {
        const Item<KEY> it = decode<KEY, MASK>(a, id);
        Stream<KEY, MASK> stream(a, it);
        const int n = stream.count();
        if (n > 0) {
            ok = wait(C::kFixEmpty, (I & 1) ^ 1u, SITE_FIX_EMPTY);
            if (!ok) break;
            if (leader) {
                mbar_arrive_expect_tx(bar(C::kFixFull), 2 * C::kTile);
                copy(&tm_f0, s.f0(), C::kFixFull, it.fixed * kT, it.h, it.b);
                copy(&tm_f1, s.f1(), C::kFixFull, it.fixed * kT, it.h, it.b);
            }
            ++I;
        }
        next = next_item(a, id);        // (its latency behind the copies)
        ok = publish(s, queue, next);
        if (!ok) break;
        const float* const stat = a.stat + (static_cast<int64_t>(it.b) * a.H + it.h) * 2 * (static_cast<int64_t>(a.q_tiles) * kT);
        for (int j = 0; j < n; ++j, ++J) {
            const int x_row = stream.next() * kT;
            // A tile that is not there ends the CTA's work, as a wait that ran out
            // does: the flag tells every role, this one's query items among them.
            if (!in_bounds(x_row >= 0 && x_row < (KEY ? a.Nq : a.kv_len) - a.dbg_rows_short, a.status, ROLE_LOAD, BND_KEY)) {
                *s.wd.abort_flag = 1;
                ok = false;
                break;
            }
            ok = wait(C::kX0Empty + J % R0, turn(J, R0) ^ 1u, SITE_X_EMPTY);
            if (!ok) break;
            const int full = C::kXFull + J % R0;
            if (leader) {
                mbar_arrive_expect_tx(bar(full), 2 * C::kTile + (KEY ? C::kStatBytes : 0));
                copy(&tm_x0, s.x0(J), full, x_row, it.h, it.b);
            }
            half = J;
            ok = wait(C::kX1Empty + J % R1, turn(J, R1) ^ 1u, SITE_X_EMPTY);
            if constexpr (KEY && R0 > C::kStats) {
                // The rows' statistics come with X1; their stage is free when X0 of
                // kStats tiles ago has been released.
                const int o = J - C::kStats;
                if (o >= 0) ok = ok && wait(C::kX0Empty + o % R0, turn(o, R0), SITE_X_EMPTY);
            }
            if (!ok) break;
            if (leader) {
                copy(&tm_x1, s.x1(J), full, x_row, it.h, it.b);
                if constexpr (KEY) {
                    const uint32_t sd = s.base + C::kStatOffset + J % C::kStats * C::kStatBytes;
                    bulk_load(sd, stat + x_row, kT * 4, bar(full));
                    bulk_load(sd + kT * 4, stat + static_cast<int64_t>(a.q_tiles) * kT + x_row, kT * 4, bar(full));
                }
            }
            done = J + 1;
            half = -1;
        }
    }
    // Every slot released: the query items' copies may follow the key items'.
    for (int j = J > R0 ? J - R0 : 0; ok && j < J; ++j) ok = wait(C::kX0Empty + j % R0, turn(j, R0), SITE_X_EMPTY);
    for (int j = J > R1 ? J - R1 : 0; ok && j < J; ++j) ok = wait(C::kX1Empty + j % R1, turn(j, R1), SITE_X_EMPTY);
    if (ok && I > 0) ok = wait(C::kFixEmpty, (I - 1) & 1, SITE_FIX_EMPTY);
    if (!ok) {
        // Winding down: wait (bounded) until every copy issued has landed.
        auto land = [&](int i, uint32_t parity) { wait_bounded_warp(bar(i), parity, s.wd_drain, ROLE_LOAD, SITE_LOAD_DRAIN); };
        // (an X0 copied alone: account for its X1 and statistics, so that its barrier completes)
        if (half >= 0 && leader)
            asm volatile("mbarrier.complete_tx.relaxed.cta.shared::cta.b64 [%0], %1;" ::"r"(bar(C::kXFull + half % R0)),
                         "r"(C::kTile + (KEY ? C::kStatBytes : 0)) : "memory");
        if (half >= 0) done = half + 1;
        for (int j = done > R0 ? done - R0 : 0; j < done; ++j) land(C::kXFull + j % R0, turn(j, R0));
        if (I > 0) land(C::kFixFull, (I - 1) & 1);
    }
}

// ------------------------------------------------------------ MMA issuer (a warp)
// A position in a ring: slot, the parity of its use, and the low word of its
// tile's matrix descriptor (the start address field).  Stepped, not computed from
// the tile's number: the issue loop is on the products' critical path.
template <int R, int STEP>
struct RingPos {
    uint32_t slot = 0, parity = 0, addr;
    __device__ explicit RingPos(uint32_t a) : addr(a) {}
    __device__ __forceinline__ void step() {
        if (slot == R - 1) {
            slot = 0;
            parity ^= 1u;
            addr -= (R - 1) * STEP;
        } else {
            ++slot;
            addr += STEP;
        }
    }
};

// Returns the items worked on; `before`: the key items this CTA worked on, whose
// accumulators must have been read before the query items' products overwrite them.
template <int D, bool KEY, bool MASK>
__device__ __forceinline__ int multiply(const Cta<D>& s, const AttnBwdArgs& a, Queue& queue, int& id, int before) {
    using C = Cfg<D>;
    constexpr uint32_t kIdescT = idesc_bf16_f32(kT, kT, false);
    constexpr uint32_t kIdescAcc = idesc_bf16_f32(kT, D, true);
    constexpr bool kDouble = !KEY || C::kKeyDouble;              // two T0: S(j+2) issued at tile j
    const uint32_t tT0 = s.tmem + C::kColT0, tT1 = s.tmem + C::kColT1, tT0b = s.tmem + C::kColT0b;
    const uint32_t tA0 = s.tmem + C::kColAcc0, tA1 = s.tmem + C::kColAcc1;
    const uint32_t bars = s.template bar<KEY>(0);
    auto wait = [&](uint32_t i, uint32_t parity, uint32_t site) { return wait_bounded_warp(bars + 8 * i, parity, s.wd, ROLE_MMA, site); };
    // two barriers at once: one vote when both are met
    auto wait2 = [&](uint32_t i, uint32_t pi, uint32_t site_i, uint32_t k, uint32_t pk, uint32_t site_k) {
        const bool a0 = mbar_try_wait(bars + 8 * i, pi), b0 = mbar_try_wait(bars + 8 * k, pk);
        if (__all_sync(0xffffffffu, a0 && b0)) return true;
        return wait(i, pi, site_i) && wait(k, pk, site_k);
    };
    auto commit = [&](uint32_t i) { umma_commit_warp(bars + 8 * i); };

    // Descriptors: K-major operands of T, MN-major ones of ACC; only the start
    // address (in the low word) differs between tiles.
    const uint64_t dT = sdesc_sw128(0, 16, 1024), dAcc = sdesc_sw128(0, C::kBlock, 1024);
    const uint64_t f0 = dT + (s.f0() >> 4), f1 = dT + (s.f1() >> 4);
    constexpr uint32_t kStep = C::kTile >> 4;
    // T = F X^T, both K-major, K = D channels.
    auto issue_t = [&](uint32_t tT, uint64_t df, uint32_t x_addr) {
        tc_fence_after();
        const uint64_t dx = dT + x_addr;
        static_for<D / 16>([&](auto kk) {
            constexpr uint32_t off = (kk.value >> 2) * C::kBlock + (kk.value & 3) * 32;
            umma_ss_warp<off>(tT, df, dx, kIdescT, kk.value > 0 ? 1u : 0u);
        });
    };
    // ACC (+)= A X, A = bf16 pairs in TMEM (K columns 0-63 in the first 32
    // columns of T's first half, 64-127 in those of its second), X MN-major.
    auto issue_acc = [&](uint32_t tA, uint32_t tOp, uint32_t x_addr, bool accumulate) {
        tc_fence_after();
        const uint64_t dx = dAcc + x_addr;
        static_for<kT / 16>([&](auto kk) {
            umma_ts_warp<kk.value * 16 * 128>(tA, tOp + (kk.value >> 2) * 64 + (kk.value & 3) * 8, dx, kIdescAcc,
                                              (accumulate || kk.value > 0) ? 1u : 0u);
        });
    };
    // The next tile of T0, the next of T1 and the tile whose P, dS are due; with
    // the parity of T0's next tile.
    RingPos<C::kR0, kStep> n0(s.x0(0) >> 4), c0(s.x0(0) >> 4);
    RingPos<C::kR1, kStep> n1(s.x1(0) >> 4), c1(s.x1(0) >> 4);
    uint32_t odd = 0;
    auto next_t0 = [&]() {
        issue_t(kDouble && odd ? tT0b : tT0, f0, n0.addr);
        commit(C::kT0Full + (kDouble ? odd : 0));
        if (kDouble) odd ^= 1u;
        n0.step();
    };
    auto next_t1 = [&](bool last) {
        issue_t(tT1, f1, n1.addr);
        commit(C::kT1Full);
        if (!KEY) commit(C::kX1Empty + n1.slot);
        if (last) commit(C::kFixEmpty);      // the item's last T0 has been issued before
        n1.step();
    };

    bool ok = true;
    if (!KEY && before > 0)
        ok = wait_bounded_warp(s.template bar<true>(C::kAccFree), (before - 1) & 1, s.wd, ROLE_MMA, SITE_ACC_FREE);
    uint32_t J = 0;
    int I = 0;
    for (; ok && id < (KEY ? a.n_kv_items : a.n_kv_items + a.n_q_items); id = take(s, a, queue, ROLE_MMA)) {
        const int n = Stream<KEY, MASK>(a, decode<KEY, MASK>(a, id)).count();
        if (n == 0) continue;
        // the item's first T0, T1 (the previous item's last products are done with
        // T0, and its dS(last) was written after dP(last) had been read: in order)
        ok = wait(C::kFixFull, I & 1, SITE_FIX_FULL) && wait(C::kXFull + n0.slot, n0.parity, SITE_X_FULL);
        if (!ok) break;
        next_t0();
        next_t1(n == 1);
        if (kDouble && n > 1) {
            ok = wait(C::kXFull + n0.slot, n0.parity, SITE_X_FULL);
            if (!ok) break;
            next_t0();
        }
        for (int j = 0; j < n; ++j, ++J) {
            const bool more = j + 1 < n;
            const bool t0_due = j + (kDouble ? 2 : 1) < n;     // T0 has a tile to issue at this one
            const bool first = j == 0 && I > 0;                  // the accumulators must have been read
            // With four slots X(j+2) has long been on its way and is awaited together
            // with P or dS; with three it is needed two products later, and awaited
            // then (together: query items of D = 128 1.31 ms against 0.95).
            constexpr bool kTogether = kDouble && C::kR0 >= 4;
            auto x_due = [&]() { return wait(C::kXFull + n0.slot, n0.parity, SITE_X_FULL); };
            if constexpr (KEY) {
                const uint32_t p = C::kP + (kDouble ? (J & 1) : 0), pp = kDouble ? (J >> 1) & 1 : J & 1;
                ok = kTogether && t0_due ? wait2(p, pp, SITE_P_READY, C::kXFull + n0.slot, n0.parity, SITE_X_FULL)
                                         : wait(p, pp, SITE_P_READY);
                if (ok && first) ok = wait(C::kAccFree, (I - 1) & 1, SITE_ACC_FREE);
                if (!ok) break;
                issue_acc(tA1, kDouble && (J & 1) ? tT0b : tT0, c1.addr, j > 0);
                commit(C::kX1Empty + c1.slot);
                if (t0_due) {
                    if (!kTogether) ok = x_due();
                    if (!ok) break;
                    next_t0();
                }
                ok = wait(C::kDS, J & 1, SITE_DS_READY);
                if (!ok) break;
                issue_acc(tA0, tT1, c0.addr, j > 0);
                commit(C::kX0Empty + c0.slot);
                if (more) next_t1(j + 2 == n);
            } else {
                ok = kTogether && t0_due ? wait2(C::kDS, J & 1, SITE_DS_READY, C::kXFull + n0.slot, n0.parity, SITE_X_FULL)
                                         : wait(C::kDS, J & 1, SITE_DS_READY);
                if (!ok) break;
                if (more) next_t1(j + 2 == n);
                if (first) ok = wait(C::kAccFree, (I - 1) & 1, SITE_ACC_FREE);
                if (!ok) break;
                issue_acc(tA0, (J & 1) ? tT0b : tT0, c0.addr, j > 0);
                commit(C::kX0Empty + c0.slot);
                if (kDouble && t0_due) {
                    if (!kTogether) ok = x_due();
                    if (!ok) break;
                    next_t0();
                }
            }
            c0.step();
            c1.step();
        }
        if (!ok) break;
        commit(C::kAccFinal);
        ++I;
    }
    // Every product issued must finish before TMEM is released.
    commit(C::kDrain);
    wait_bounded_warp(bars + 8 * C::kDrain, 0, s.wd_drain, ROLE_MMA, SITE_BWD_DRAIN);
    return I;
}

// ------------------------------------------------------- softmax warps (0-7)
// 8 consecutive 32-bit words (32-byte aligned, or as two 16-byte halves).
__device__ __forceinline__ void store8(void* p, const uint32_t (&v)[8], bool wide) {
    if (wide)
        asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(v[0]), "r"(v[1]), "r"(v[2]),
                     "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
                     : "memory");
    else {
        reinterpret_cast<uint4*>(p)[0] = make_uint4(v[0], v[1], v[2], v[3]);
        reinterpret_cast<uint4*>(p)[1] = make_uint4(v[4], v[5], v[6], v[7]);
    }
}

template <int D, bool KEY, bool OUT_BF16, bool MASK>
__device__ __forceinline__ void soften(const Cta<D>& s, const AttnBwdArgs& a, Queue& queue, int& id) {
    using C = Cfg<D>;
    constexpr int R0 = C::kR0;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int g = warp >> 2;    // column half
    const int wq = warp & 3;    // TMEM lane quadrant
    const uint32_t lane_off = static_cast<uint32_t>(wq * 32) << 16;
    const uint32_t tT0 = s.tmem + lane_off + C::kColT0 + 64 * g;
    const uint32_t tT0b = s.tmem + lane_off + C::kColT0b + 64 * g;
    const uint32_t tT1 = s.tmem + lane_off + C::kColT1 + 64 * g;
    constexpr bool kDouble = !KEY || C::kKeyDouble;
    const float sl2 = a.scale_log2;
    auto bar = [&](int i) { return s.template bar<KEY>(i); };
    auto wait = [&](int i, uint32_t parity, uint32_t site) { return wait_bounded(bar(i), parity, s.wd, ROLE_SOFTMAX, site); };
    // 32 columns of T (half `hf` of this warp's 64) to 32 registers and, packed to
    // bf16 pairs, back to 16 columns.  Query item: a row a thread.  Key item: four
    // rows, lane / 4 + 8 i, and of every 8 columns the pair 2 (lane mod 4).
    auto load = [&](uint32_t t, int hf, uint32_t (&r)[32]) {
        if constexpr (KEY) tmem_ld_16x256b_x4x2(t + 32 * hf, r);
        else tmem_ld32(t + 32 * hf, r);
    };
    auto store = [&](uint32_t t, int hf, const float* v) {
        uint32_t pk[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) pk[i] = pack_bf16x2(v[2 * i], v[2 * i + 1]);
        if constexpr (KEY) tmem_st_16x128b_x4x2(t + 16 * hf, pk);
        else tmem_st16(t + 16 * hf, pk);
    };
    // A query item's row statistics, asked for one item ahead.
    float next_nlse = 0.f, next_ndelta = 0.f;
    const int last = KEY ? a.n_kv_items : a.n_kv_items + a.n_q_items;
    auto ask = [&](int which) {
        if (KEY || which >= last || a.stat == nullptr) return;    // (without keys there are no statistics)
        const Item<KEY> it = decode<KEY, MASK>(a, which);
        const float* p = a.stat + (static_cast<int64_t>(it.b) * a.H + it.h) * 2 * (static_cast<int64_t>(a.q_tiles) * kT) + it.fixed * kT + wq * 32 + lane;
        next_nlse = __ldg(p);
        next_ndelta = __ldg(p + static_cast<int64_t>(a.q_tiles) * kT);
    };

    int J = 0, I = 0;
    bool ok = true;
    ask(id);
    for (int next; ok && id < last; id = next) {
        next = take(s, a, queue, ROLE_SOFTMAX);
        const Item<KEY> it = decode<KEY, MASK>(a, id);
        const int row0 = it.fixed * kT;
        const int row = row0 + wq * 32 + lane;      // this thread's row of the fixed tile
        Stream<KEY, MASK> stream(a, it);
        const int n_tiles = stream.count();
        const float nlse = next_nlse, ndelta = next_ndelta;
        ask(next);
        // Mask words, asked for one tile ahead.  Query item: this row's two words of
        // the tile's half.  Key item: the word of this warp's 32 keys in query rows
        // `lane` and 32 + `lane` of the half; the others' come by shuffles.
        const uint32_t* const words = MASK ? a.mask + it.b * a.mask_sb : nullptr;
        auto word_of = [&](int tile) {
            uint2 w = make_uint2(~0u, ~0u);
            if constexpr (MASK) {
                if (tile < 0) return w;
                if constexpr (KEY) {
                    const int i = tile * kT + 64 * g + lane;
                    const uint32_t* p = words + i * a.mask_si + 4 * it.fixed + wq;
                    if (i < a.mask_rows) w.x = __ldg(p);
                    if (i + 32 < a.mask_rows) w.y = __ldg(p + 32 * a.mask_si);
                } else {
                    if (row < a.mask_rows) w = __ldg(reinterpret_cast<const uint2*>(words + row * a.mask_si + 4 * tile) + g);
                }
            }
            return w;
        };
        int tile_next = stream.next();
        uint2 mw_next = word_of(tile_next);

        for (int j = 0; j < n_tiles; ++j, ++J) {
            const int tile = tile_next;
            const int st = J % C::kStats;
            const uint2 mw = mw_next;
            // Most tiles of a mask that is made of blocks forbid nothing: those pass
            // without the tests of single bits.
            const bool some = MASK && !__all_sync(0xffffffffu, (mw.x & mw.y) == ~0u);
            tile_next = stream.next();
            mw_next = word_of(tile_next);
            ok = kDouble ? wait(C::kT0Full + (J & 1), turn(J, 2), SITE_T0_FULL) : wait(C::kT0Full, J & 1, SITE_T0_FULL);
            // the statistics of this stage have landed
            if (KEY) ok = ok && wait(C::kXFull + J % R0, turn(J, R0), SITE_X_FULL);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            tc_fence_after();
            const uint32_t tS = (kDouble && (J & 1)) ? tT0b : tT0;
            // P, then dS: 64 values a thread, half by half, the second half's load
            // behind the first half's arithmetic.  A query item's statistics are its
            // row's, in registers.  A key item's go by column: a thread reads those of
            // a quarter of them -- with a row a thread, broadcasting them from shared
            // memory took half of its bandwidth from the products (1.50 ms of key
            // items against 1.20).
            float p[64];
            const float2* nl = reinterpret_cast<const float2*>(s.smem + C::kStatOffset + st * C::kStatBytes) + 32 * g + (lane & 3);
            uint32_t r0[32], r1[32];
            // x = S scale log2(e) - LSE log2(e) of one half, then its power of two
            auto power = [&](int hf, const uint32_t (&r)[32]) {
                float* q = p + 32 * hf;
#pragma unroll
                for (int c = 0; c < 16; c += 4) {
                    const float2 n = KEY ? nl[16 * hf + c] : make_float2(nlse, nlse);
#pragma unroll
                    for (int i = 0; i < 4; i += 2) {
                        ffma2(q[c + i], q[c + i + 1], __uint_as_float(r[c + i]), __uint_as_float(r[c + i + 1]), sl2, n.x, n.y);
                        ffma2(q[16 + c + i], q[16 + c + i + 1], __uint_as_float(r[16 + c + i]), __uint_as_float(r[16 + c + i + 1]), sl2, n.x, n.y);
                    }
                }
#pragma unroll
                for (int c = 0; c < 32; ++c) q[c] = ex2_approx(q[c]);
                if (MASK && KEY && some) {
                    const uint32_t held = hf ? mw.y : mw.x;
                    const int row4 = lane >> 2, col = 2 * (lane & 3);
#pragma unroll
                    for (int c = 0; c < 16; c += 4) {       // columns 2c + col, 2c + col + 1
                        const uint32_t w0 = __shfl_sync(0xffffffffu, held, 2 * c + col), w1 = __shfl_sync(0xffffffffu, held, 2 * c + col + 1);
#pragma unroll
                        for (int i = 0; i < 4; ++i) {       // rows lane / 4 + 8 i: values 16 (i / 2) + c + 2 (i mod 2)
                            const int at = 16 * (i >> 1) + c + 2 * (i & 1);
                            if (!((w0 >> (row4 + 8 * i)) & 1u)) q[at] = 0.f;
                            if (!((w1 >> (row4 + 8 * i)) & 1u)) q[at + 1] = 0.f;
                        }
                    }
                }
                if (MASK && !KEY && some) {
                    const uint32_t w = hf ? mw.y : mw.x;
#pragma unroll
                    for (int c = 0; c < 32; ++c)
                        if (!((w >> c) & 1u)) q[c] = 0.f;
                }
                if constexpr (!KEY) {
                    const int valid = a.kv_len - tile * kT - 64 * g - 32 * hf;   // keys left in this half
                    if (valid < 32) {
#pragma unroll
                        for (int c = 0; c < 32; ++c)
                            if (c >= valid) q[c] = 0.f;
                    }
                }
            };
            load(tS, 0, r0);
            tmem_ld_wait_dep(r0);
            load(tS, 1, r1);
            power(0, r0);
            if constexpr (KEY) {
                store(tS, 0, p);
            }
            tmem_ld_wait_dep(r1);
            power(1, r1);
            if constexpr (KEY) {
                store(tS, 1, p + 32);
                tmem_st_wait();
                tc_fence_before();
                mbar_arrive(bar(C::kP + (kDouble ? (J & 1) : 0)));
            }
            // dS = P o (dP - delta), from the fp32 P
            ok = wait(C::kT1Full, J & 1, SITE_T1_FULL);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            tc_fence_after();
            auto differ = [&](int hf, const uint32_t (&r)[32]) {
                float* q = p + 32 * hf;
#pragma unroll
                for (int c = 0; c < 16; c += 4) {
                    const float2 n = KEY ? nl[kT / 2 + 16 * hf + c] : make_float2(ndelta, ndelta);
#pragma unroll
                    for (int i = 0; i < 4; i += 2) {
                        fadd2_mul2(q[c + i], q[c + i + 1], __uint_as_float(r[c + i]), __uint_as_float(r[c + i + 1]), n.x, n.y, q[c + i], q[c + i + 1]);
                        fadd2_mul2(q[16 + c + i], q[16 + c + i + 1], __uint_as_float(r[16 + c + i]), __uint_as_float(r[16 + c + i + 1]), n.x, n.y, q[16 + c + i], q[16 + c + i + 1]);
                    }
                }
            };
            const uint32_t tD = KEY ? tT1 : tS;
            load(tT1, 0, r0);
            tmem_ld_wait_dep(r0);
            load(tT1, 1, r1);
            differ(0, r0);
            store(tD, 0, p);
            tmem_ld_wait_dep(r1);
            differ(1, r1);
            store(tD, 1, p + 32);
            tmem_st_wait();
            tc_fence_before();
            mbar_arrive(bar(C::kDS));
        }

        // The gradient: key item, warps 0-3 write dV and warps 4-7 dK, all D
        // channels; query item, each half of the warps half of dQ's channels.  A
        // thread writes its row, 32 bytes (a sector) at a time.
        if (ok && n_tiles > 0) {
            ok = wait(C::kAccFinal, I & 1, SITE_ACC_FINAL);
            ok = __all_sync(0xffffffffu, ok);
        }
        if (!ok) break;
        {
            tc_fence_after();
            // the item decoded anew: nothing of it is held across the tiles but its number
            int again = id;
            asm volatile("" : "+r"(again));
            const Item<KEY> it = decode<KEY, MASK>(a, again);
            const int row0 = it.fixed * kT;
            const int row = row0 + wq * 32 + lane;
            constexpr int kChunks = KEY ? D / 32 : D / 64;
            const int c0 = KEY ? 0 : g * kChunks;
            const uint32_t tA = s.tmem + lane_off + (KEY && g == 0 ? C::kColAcc1 : C::kColAcc0);
            const bool split = it.cut;
            const float mult = split ? 1.f : (KEY && g == 0 ? 1.f : a.scale);
            const bool zero_row = n_tiles == 0 || row >= (KEY ? a.kv_len : a.Nq);    // (key item: rows past kv_len are zeros)
            const bool inside = split || row < (KEY ? a.Nkv : a.Nq);
            const dit_strides4_t& so = KEY ? (g == 0 ? a.sdv : a.sdk) : a.sdq;
            void* const out = KEY ? (g == 0 ? a.dv : a.dk) : a.dq;
            const int64_t off = it.b * so.b + static_cast<int64_t>(row) * so.n + it.h * so.h;
            float* const part = (KEY ? a.part_kv + (it.part_tile * 2 + g) * kT * D : a.part_q + it.part_tile * kT * D) + (row - row0) * D;
#pragma unroll 1
            for (int cc = c0; cc < c0 + kChunks; ++cc) {
                uint32_t o[32];
                if (n_tiles > 0) {
                    tmem_ld32(tA + cc * 32, o);
                    tmem_ld_wait_dep(o);
                }
#pragma unroll
                for (int i = 0; i < 32; ++i) o[i] = zero_row ? 0u : __float_as_uint(__uint_as_float(o[i]) * mult);
                if (!inside) {
                    // nothing to store: past the last row
                } else if (!OUT_BF16 || split) {
                    float* dst = (split ? part : static_cast<float*>(out) + off) + cc * 32;
#pragma unroll
                    for (int i = 0; i < 32; i += 8) {
                        const uint32_t v[8] = {o[i], o[i + 1], o[i + 2], o[i + 3], o[i + 4], o[i + 5], o[i + 6], o[i + 7]};
                        store8(dst + i, v, split || a.wide);
                    }
                } else {
                    uint16_t* dst = static_cast<uint16_t*>(out) + off + cc * 32;
#pragma unroll
                    for (int i = 0; i < 32; i += 16) {
                        uint32_t v[8];
#pragma unroll
                        for (int k = 0; k < 8; ++k)
                            v[k] = pack_bf16x2(__uint_as_float(o[i + 2 * k]), __uint_as_float(o[i + 2 * k + 1]));
                        store8(dst + i, v, a.wide);
                    }
                }
                __syncwarp();       // the next load is the whole warp's
            }
        }
        if (n_tiles > 0) {
            tc_fence_before();
            mbar_arrive(bar(C::kAccFree));
            ++I;
        }
    }
}

template <int D, bool OUT_BF16, bool MASK>
__global__ void __launch_bounds__(kThreads, 1)
    attn_bwd_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                    const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ CUtensorMap tm_do,
                    const __grid_constant__ AttnBwdArgs a) {
    using C = Cfg<D>;
    extern __shared__ uint8_t smem_raw[];
    Cta<D> s;
    s.smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    s.base = smem_u32(s.smem);
    // Dynamic shared memory starts on a 1,024-byte boundary when a kernel has no
    // other; the whole grid would give up alike if it ever did not fit.
    if (s.base + C::kUsedBytes > smem_u32(smem_raw) + C::kSmemBytes) {
        if (threadIdx.x == 0 && atomicCAS(a.status, 0u, 5u) == 0u) atomicExch(a.status + 3, static_cast<unsigned>(SITE_NO_ROOM));
        return;
    }
    s.bars = s.base + C::kBarOffset;
    uint32_t* const tmem_slot = reinterpret_cast<uint32_t*>(s.smem + C::kItemOffset + C::kQueue * 4);
    volatile int* const abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
    volatile int* const never_flag = reinterpret_cast<volatile int*>(tmem_slot + 2);
    s.wd = Watchdog{a.status, a.timeout_ns, abort_flag};
    s.wd_drain = Watchdog{a.status, a.timeout_ns, never_flag};
    const int warp = threadIdx.x >> 5;

    if (threadIdx.x == 0) {
        for (int i = 0; i < 2 * C::kNumBars; ++i) {
            const int k = i % C::kNumBars;
            const bool all = (k >= C::kP && k <= C::kDS) || k == C::kAccFree;
            mbar_init(s.bars + i * 8, all ? 256 : 1);
        }
        for (int i = 0; i < C::kQueue; ++i) {
            mbar_init(s.bars + (C::kItemFull + i) * 8, 1);
            mbar_init(s.bars + (C::kItemEmpty + i) * 8, 9);    // the MMA and softmax warps
        }
        *abort_flag = 0;
        *never_flag = 0;
        fence_mbar_init();
    }
    if (warp == 8) {
        tmem_alloc(smem_u32(tmem_slot), 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    s.tmem = *tmem_slot;
    if (threadIdx.x == 0) let_next();
    after_previous();      // the statistics, and the counter's zero

    // Each role runs through the key items, then the query items.  Nothing but
    // its barriers holds one back; a role that gave up leaves the others to.
    Queue queue;
    if (warp >= 8) {
        regs_decrease<kOtherRegs>();
        if (warp == 8) {
            int id = take(s, a, queue, ROLE_MMA);
            const int worked = multiply<D, true, MASK>(s, a, queue, id, 0);
            __syncwarp();
            if (!__any_sync(0xffffffffu, *abort_flag)) multiply<D, false, MASK>(s, a, queue, id, worked);
        } else if (warp == 9) {
            if (lane_id() == 0) {
                tma_prefetch_desc(&tm_q);
                tma_prefetch_desc(&tm_k);
                tma_prefetch_desc(&tm_v);
                tma_prefetch_desc(&tm_do);
            }
            int id = static_cast<int>(blockIdx.x);       // (the grid is no larger than the items)
            publish(s, queue, id);
            produce<D, true, MASK>(s, tm_k, tm_v, tm_q, tm_do, a, queue, id);
            __syncwarp();
            if (!__any_sync(0xffffffffu, *abort_flag)) produce<D, false, MASK>(s, tm_q, tm_do, tm_k, tm_v, a, queue, id);
        }
        __syncwarp();
    } else {
        regs_increase<kSoftmaxRegs>();
        int id = take(s, a, queue, ROLE_SOFTMAX);
        soften<D, true, OUT_BF16, MASK>(s, a, queue, id);
        __syncwarp();
        if (!__any_sync(0xffffffffu, *abort_flag)) soften<D, false, OUT_BF16, MASK>(s, a, queue, id);
    }

    tc_fence_before();
    __syncthreads();
    if (warp == 8) {
        tc_fence_after();
        tmem_dealloc(s.tmem, 512);
    }
}

// stat[b*H + h][0][i] = -lse * log2(e) (-inf for rows without a key and rows
// past Nq, so that their P is 0), [1][i] = dlse - sum_d dO O (0 for those rows,
// whose O and dlse may be anything: 0 * NaN would reach every key).  One row per
// D / 8 lanes, 16 bytes of dO each; a block's 2,048 / D rows are of one (b, h),
// which divides a head's padded rows.  HBM-bound (reads dO and O once).
template <int D, bool OUT_BF16>
__global__ void __launch_bounds__(256) attn_bwd_stat_kernel(const AttnBwdStatArgs a) {
    constexpr int LPR = D / 8, kRows = 256 / LPR;
    static_assert(kT % kRows == 0, "rows of a block");
    if (threadIdx.x == 0) let_next();
    if (blockIdx.x == 0 && threadIdx.x == 0) *a.counter = 0u;      // of the main kernel's items
    const int per_bh = a.rows_pad / kRows;
    const unsigned unit = blockIdx.x / static_cast<unsigned>(per_bh);
    const int64_t bh = unit;
    const int c = static_cast<int>(threadIdx.x % LPR);
    const int i = static_cast<int>(blockIdx.x - unit * per_bh) * kRows + static_cast<int>(threadIdx.x / LPR);
    const int b = static_cast<int>(unit / static_cast<unsigned>(a.H)), h = static_cast<int>(unit - b * static_cast<unsigned>(a.H));
    float s = 0.f, nl = -INFINITY;
    if (i < a.Nq) {
        const int64_t od = b * a.sdo.b + static_cast<int64_t>(i) * a.sdo.n + h * a.sdo.h + 8 * c;
        const int64_t oo = b * a.so.b + static_cast<int64_t>(i) * a.so.n + h * a.so.h + 8 * c;
        const uint4 d = __ldg(reinterpret_cast<const uint4*>(a.dout + od));
        float o[8];
        if constexpr (OUT_BF16) {
            const uint4 v = __ldg(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.out) + oo));
            const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                o[2 * k] = __uint_as_float(w[k] << 16);
                o[2 * k + 1] = __uint_as_float(w[k] & 0xFFFF0000u);
            }
        } else {
            const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(a.out) + oo);
            const float4 lo = __ldg(p), hi = __ldg(p + 1);
            o[0] = lo.x; o[1] = lo.y; o[2] = lo.z; o[3] = lo.w;
            o[4] = hi.x; o[5] = hi.y; o[6] = hi.z; o[7] = hi.w;
        }
        const uint32_t w[4] = {d.x, d.y, d.z, d.w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            s = fmaf(__uint_as_float(w[k] << 16), o[2 * k], s);
            s = fmaf(__uint_as_float(w[k] & 0xFFFF0000u), o[2 * k + 1], s);
        }
        const float l = __ldg(a.lse + bh * a.Nq + i);
        nl = l == -INFINITY ? -INFINITY : -l * kLog2e;
    }
#pragma unroll
    for (int o = LPR / 2; o >= 1; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    if (c == 0) {
        float* const dst = a.stat + bh * 2 * a.rows_pad + i;
        if (a.dlse != nullptr && i < a.Nq) s -= __ldg(a.dlse + bh * a.Nq + i);
        dst[0] = nl;
        dst[a.rows_pad] = nl == -INFINITY ? 0.f : -s;
    }
}

// Sums the pieces' partials of one item in slot order and writes the gradient.
// blockIdx.y: 0 dv, 1 dk, 2 dq (those that were split).
template <int D, bool OUT_BF16>
__global__ void __launch_bounds__(256) attn_bwd_sum_kernel(const AttnBwdArgs a, int first) {
    after_previous();
    const int which = static_cast<int>(blockIdx.y) + first;
    const bool key = which < 2;
    const int f = key ? a.f_kv : a.f_q;
    const int tiles = key ? a.kv_out_tiles : a.q_tiles;
    const int64_t g = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
    const int64_t unit = g / (D / 4);
    const int c4 = static_cast<int>(g % (D / 4));
    const int nth = static_cast<int>(unit / kT), r = static_cast<int>(unit % kT);
    const int item = nth + (key ? 0 : a.q_whole);
    if (unit >= (static_cast<int64_t>(a.B) * a.H * tiles - (key ? 0 : a.q_whole)) * kT) return;
    const int row = (item % tiles) * kT + r;
    const int h = (item / tiles) % a.H, b = item / tiles / a.H;
    if (row >= (key ? a.Nkv : a.Nq)) return;
    const int64_t stride = static_cast<int64_t>(key ? 2 : 1) * kT * D;
    const float* p = (key ? a.part_kv + (static_cast<int64_t>(nth) * f * 2 + which) * kT * D
                          : a.part_q + static_cast<int64_t>(nth) * f * kT * D) + r * D + 4 * c4;
    float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int k = 0; k < f; ++k) {
        const float4 v = __ldcs(reinterpret_cast<const float4*>(p + k * stride));
        s.x += v.x; s.y += v.y; s.z += v.z; s.w += v.w;
    }
    if (which != 0) { s.x *= a.scale; s.y *= a.scale; s.z *= a.scale; s.w *= a.scale; }
    const dit_strides4_t so = which == 0 ? a.sdv : (which == 1 ? a.sdk : a.sdq);
    void* const out = which == 0 ? a.dv : (which == 1 ? a.dk : a.dq);
    const int64_t off = b * so.b + static_cast<int64_t>(row) * so.n + h * so.h + 4 * c4;
    if constexpr (OUT_BF16)
        *reinterpret_cast<uint2*>(static_cast<uint16_t*>(out) + off) = make_uint2(pack_bf16x2(s.x, s.y), pack_bf16x2(s.z, s.w));
    else
        *reinterpret_cast<float4*>(static_cast<float*>(out) + off) = s;
}

template <int D, bool OUT_BF16, bool MASK>
cudaError_t launch_impl(const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv, const CUtensorMap& tdo,
                        const AttnBwdArgs& a, cudaStream_t s) {
    auto kern = attn_bwd_kernel<D, OUT_BF16, MASK>;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg<D>::kSmemBytes);
    if (e != cudaSuccess) return e;
    return launch_behind(kern, a.grid, kThreads, Cfg<D>::kSmemBytes, s, tq, tk, tv, tdo, a);
}

}  // namespace

cudaError_t launch_attn_bwd_stat(const AttnBwdStatArgs& a, int D, bool out_bf16, cudaStream_t s) {
    const unsigned blocks = static_cast<unsigned>(static_cast<int64_t>(a.B) * a.H * (a.rows_pad / (2048 / D)));
    if (D == 128) {
        if (out_bf16) attn_bwd_stat_kernel<128, true><<<blocks, 256, 0, s>>>(a);
        else attn_bwd_stat_kernel<128, false><<<blocks, 256, 0, s>>>(a);
    } else {
        if (out_bf16) attn_bwd_stat_kernel<64, true><<<blocks, 256, 0, s>>>(a);
        else attn_bwd_stat_kernel<64, false><<<blocks, 256, 0, s>>>(a);
    }
    return cudaGetLastError();
}

cudaError_t launch_attn_bwd(const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv, const CUtensorMap& tdo,
                            const AttnBwdArgs& a, int D, bool grad_bf16, cudaStream_t s) {
    if (a.mask != nullptr) {
        if (D == 128) return grad_bf16 ? launch_impl<128, true, true>(tq, tk, tv, tdo, a, s)
                                       : launch_impl<128, false, true>(tq, tk, tv, tdo, a, s);
        return grad_bf16 ? launch_impl<64, true, true>(tq, tk, tv, tdo, a, s)
                         : launch_impl<64, false, true>(tq, tk, tv, tdo, a, s);
    }
    if (D == 128) return grad_bf16 ? launch_impl<128, true, false>(tq, tk, tv, tdo, a, s)
                                   : launch_impl<128, false, false>(tq, tk, tv, tdo, a, s);
    return grad_bf16 ? launch_impl<64, true, false>(tq, tk, tv, tdo, a, s)
                     : launch_impl<64, false, false>(tq, tk, tv, tdo, a, s);
}

cudaError_t launch_attn_bwd_sum(const AttnBwdArgs& a, int D, bool grad_bf16, cudaStream_t s) {
    const bool kv = a.f_kv > 1, q = a.f_q > 1;
    if (!kv && !q) return cudaSuccess;
    const int64_t bh = static_cast<int64_t>(a.B) * a.H;
    const int64_t kv_items = kv ? bh * a.kv_out_tiles : 0, q_items = q ? bh * a.q_tiles - a.q_whole : 0;
    const int64_t threads = (kv_items > q_items ? kv_items : q_items) * kT * (D / 4);
    const dim3 grid(static_cast<unsigned>((threads + 255) / 256), (kv ? 2 : 0) + (q ? 1 : 0));
    const int first = kv ? 0 : 2;
    if (D == 128) {
        if (grad_bf16) return launch_behind(attn_bwd_sum_kernel<128, true>, grid, 256, 0, s, a, first);
        else return launch_behind(attn_bwd_sum_kernel<128, false>, grid, 256, 0, s, a, first);
    } else {
        if (grad_bf16) return launch_behind(attn_bwd_sum_kernel<64, true>, grid, 256, 0, s, a, first);
        else return launch_behind(attn_bwd_sum_kernel<64, false>, grid, 256, 0, s, a, first);
    }
}

}  // namespace dit

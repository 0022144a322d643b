// attn_bwd.cu -- attention backward, sm_103a, TMA + tcgen05 (TMEM
// accumulators), warp-specialised like the forward kernel.
//
// With S = scale * Q K^T over the keys a row may attend and the forward pass'
// LSE,
//     P = exp(S - LSE),  dV = P^T dO,  delta_i = sum_d dO_id O_id - dLSE_i,
//     dS = P o (dO V^T - delta),  dQ = scale dS K,  dK = scale dS^T Q:
// the probabilities are recomputed tile by tile, never stored.
//
// Two kinds of CTA in one grid, so that no gradient is summed through memory
// and every result repeats bit for bit (no atomics):
//   key CTA    one 128-key tile of a (b, h); streams the 128-row query tiles,
//              S^T = K Q^T and dP^T = V dO^T (rows are keys), then
//              dV += P^T dO and dK += dS^T Q;
//   query CTA  one 128-row query tile; streams the key tiles,
//              S = Q K^T and dP = dO V^T, then dQ += dS K.
// Seven products a tile pair instead of five: the two recomputed ones cost
// 40% more tensor work, against fp32 atomics of 64 KB a tile pair into L2 (or a
// serial order of CTAs) for one kind of CTA that also adds into dQ.
//
// In both, the streamed tiles come in pairs (X0, X1) = (Q, dO) or (K, V), the
// fixed ones are (F0, F1) = (K, V) or (Q, dO), and
//   T0 = F0 X0^T, T1 = F1 X1^T, ACC1 += P X1 (key CTA), ACC0 += dS X0,
// with P and dS the TMEM A operands, written by the softmax warps in bf16 over
// their own half of T0 / T1.
//
// 12 warps:
//   warps 0-3, 4-7  softmax warpgroups: columns [0, 64) and [64, 128) of every
//                   tile, one TMEM lane = one row per thread
//   warp 8          tcgen05.mma issuer (warp-wide, one elected lane issues);
//                   owns the TMEM allocation
//   warp 9          TMA producer (one thread)
//   warp 10         stages mask words (key CTAs with a mask)
// Registers: 168 at launch; softmax 208, the rest 88 (as the forward kernel).
// TMEM (512 columns): T0 [0,128) T1 [128,256) ACC0 [256,256+D)
// ACC1 or the second T0 [256+D, ...).
//
// Order of products.  Key CTA, per tile j: dV(j) when P(j) is ready, S(j+1),
// dK(j) when dS(j) is ready, dP(j+1); the softmax warps form P(j+1) while dK(j)
// and dP(j+1) run and dS(j) while dV(j) and S(j+1) run.  Query CTA: S(j+1) into
// the other T0, dP(j+1) once dP(j) is in registers, dQ(j) when dS(j) (written
// over S(j)) is ready.
//
// Rows without an allowed key have LSE = -inf; they, and the rows past Nq, get
// P = 0 through a stored -LSE of -inf.  Keys past kv_len are zero-filled by the
// tensor maps and masked (query CTA) or not stored (key CTA: their gradients
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
    SITE_DS_READY = 17, SITE_T1_READ = 18, SITE_ACC_FINAL = 19, SITE_MASK_FULL = 20, SITE_BWD_DRAIN = 21,
    SITE_NO_ROOM = 22
};
constexpr uint32_t ROLE_MASK = 4;

// Untiled bulk copy global -> shared (16-byte aligned, a multiple of 16 bytes).
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
                 "l"(reinterpret_cast<uint64_t>(src)), "r"(bytes), "r"(bar)
                 : "memory");
}

// 16 lanes x 64 32-bit columns: r[4k + i] is lane t / 4 + 8 (i / 2), column
// 8k + 2 (t mod 4) + (i mod 2) for thread t of the warp.
__device__ __forceinline__ void tmem_ld_16x256b_x8(uint32_t taddr, uint32_t (&r)[32]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.16x256b.x8.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
          "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
          "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(taddr));
}
// 16 lanes x 32 32-bit columns: r[2k + i] goes to lane t / 4 + 8 i, column
// 4k + t mod 4.  Two neighbouring values of the load above, packed, land on the
// columns of their pair.
__device__ __forceinline__ void tmem_st_16x128b_x8(uint32_t taddr, const uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.16x128b.x8.b32 [%0], "
        "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
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

// MASK: a key CTA also stages mask words, which leaves D = 128 one slot less.
template <int D, bool MASK>
struct Cfg {
    static constexpr int kTile = kT * D * 2;
    // Ring slots of X0 and of X1.  X0(j) is held until the last product of tile j,
    // so three of it keep the next copy three products ahead of its use; with
    // two and two, both kinds of CTA ran at 1.6 us a tile pair whatever their
    // products, waiting for copies.
    static constexpr int kR0 = D == 128 ? (MASK ? 2 : 3) : 4;
    static constexpr int kR1 = D == 128 ? 2 : 4;
    static constexpr int kStats = kR1;                   // statistics (and mask words) of this many tiles
    static constexpr int kBlock = kT * 128;              // 128 rows x 64 bf16 (one swizzle column)
    static constexpr int kStatBytes = 2 * kT * 4;        // -lse2[128], -delta[128]
    static constexpr int kMaskBytes = MASK ? kT * 16 : 0;   // 4 words x 128 rows
    // barriers
    static constexpr int kFixFull = 0;
    static constexpr int kX0Full = 1;
    static constexpr int kX0Empty = kX0Full + kR0;
    static constexpr int kX1Full = kX0Empty + kR0;
    static constexpr int kX1Empty = kX1Full + kR1;
    static constexpr int kT0Full = kX1Empty + kR1;       // two (query CTA's two T0)
    static constexpr int kT1Full = kT0Full + 2;
    static constexpr int kP = kT1Full + 1;
    // Two, by the tile's parity: a query CTA's softmax warps may finish dS(j+1)
    // before the MMA warp has looked for dS(j), and one barrier would then be a
    // phase past the one it waits for.  (dS(j+2) needs T1(j+2), issued after that.)
    static constexpr int kDS = kP + 1;
    static constexpr int kT1Read = kDS + 2;
    static constexpr int kAccFinal = kT1Read + 1;
    static constexpr int kMaskFull = kAccFinal + 1;
    static constexpr int kDrain = kMaskFull + kStats;
    static constexpr int kNumBars = kDrain + 1;
    static constexpr int kStatOffset = (2 + kR0 + kR1) * kTile;
    static constexpr int kMaskOffset = kStatOffset + kStats * kStatBytes;
    static constexpr int kBarOffset = kMaskOffset + kStats * kMaskBytes;
    static constexpr int kUsedBytes = kBarOffset + kNumBars * 8 + 16;
    // with room to start on a 1,024-byte boundary where the buffer does not
    static constexpr int kSmemBytes = kUsedBytes + 1024 <= 232448 ? kUsedBytes + 1024 : 232448;
    static_assert(kUsedBytes <= kSmemBytes && (!MASK || kStats == kR0), "shared memory");
    // TMEM columns
    static constexpr int kColT0 = 0, kColT1 = 128, kColAcc0 = 256, kColAcc1 = 256 + D;
    static_assert(kColAcc1 + 128 <= 512, "TMEM");
};

// The streamed tiles of a CTA in order: all of [begin, end), or those whose
// occupancy bit is set -- for a key CTA the bit of its key tile in each query
// block's words, for a query CTA the set bits of its block's words.
template <bool KEY>
struct Stream {
    const uint32_t* occ;      // nullptr: all.  KEY: batch's words; else: this block's words
    int words, fixed, t, end;
    __device__ Stream(const uint32_t* o, int w, int f, int begin, int e) : occ(o), words(w), fixed(f), t(begin), end(e) {}
    __device__ bool hit(int i) const {
        if (occ == nullptr) return true;
        if (KEY) return (occ[static_cast<int64_t>(i >> 1) * words + (fixed >> 5)] >> (fixed & 31)) & 1u;
        return (occ[i >> 5] >> (i & 31)) & 1u;
    }
    __device__ int next() {
        while (t < end) {
            const int i = t++;
            if (hit(i)) return i;
        }
        return -1;
    }
    __device__ int count() const {
        if (occ == nullptr) return end - t;
        int c = 0;
        for (int i = t; i < end; ++i) c += hit(i) ? 1 : 0;
        return c;
    }
};

template <int D, bool KEY, bool OUT_BF16, bool MASK>
__device__ __forceinline__ void bwd_body(const CUtensorMap& tm_f0, const CUtensorMap& tm_f1, const CUtensorMap& tm_x0,
                                         const CUtensorMap& tm_x1, const AttnBwdArgs& a, int slot) {
    using C = Cfg<D, MASK>;
    constexpr int R0 = C::kR0, R1 = C::kR1;
    constexpr int TILE = C::kTile;

    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const uint32_t s_base = smem_u32(smem);
    // Dynamic shared memory starts on a 1,024-byte boundary when a kernel has no
    // other; the whole grid would give up alike if it ever did not fit.
    if (s_base + C::kUsedBytes > smem_u32(smem_raw) + C::kSmemBytes) {
        if (threadIdx.x == 0 && atomicCAS(a.status, 0u, 5u) == 0u) atomicExch(a.status + 3, static_cast<unsigned>(SITE_NO_ROOM));
        return;
    }
    const uint32_t sF0 = s_base, sF1 = s_base + TILE;
    const uint32_t sX0 = s_base + 2 * TILE, sX1 = sX0 + R0 * TILE;
    const uint32_t sStat = s_base + C::kStatOffset;
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::kBarOffset);
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + C::kNumBars);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
    volatile int* never_flag = reinterpret_cast<volatile int*>(tmem_slot + 2);
    auto bar = [&](int i) -> uint32_t { return smem_u32(bars + i); };

    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;

    // The item (b, h, fixed tile) and its range of streamed tiles.
    const int f = KEY ? a.f_kv : a.f_q;
    const int tiles = KEY ? a.kv_out_tiles : a.q_tiles;
    const int piece = slot % f;
    const int item = slot / f;
    const int fixed = item % tiles;
    const int h = (item / tiles) % a.H;
    const int b = item / tiles / a.H;
    const int row0 = fixed * kT;
    // a key tile wholly past kv_len has nothing to stream: its gradient is zero
    const int x_tiles = KEY ? (fixed < a.kv_tiles ? a.q_tiles : 0) : a.kv_tiles;
    const int begin = static_cast<int>(static_cast<int64_t>(piece) * x_tiles / f);
    const int end = static_cast<int>(static_cast<int64_t>(piece + 1) * x_tiles / f);
    if (!in_bounds(b < a.B && fixed < tiles && begin >= 0 && end <= x_tiles, a.status, 0, BND_ITEM)) return;
    const uint32_t* occ = nullptr;
    if (MASK && a.occ != nullptr)
        occ = a.occ + (static_cast<int64_t>(b) * a.occ_blocks + (KEY ? 0 : fixed >> 1)) * a.occ_words;
    const Stream<KEY> stream(occ, a.occ_words, fixed, begin, end);
    const int n_tiles = stream.count();
    const float* const stat = a.stat + (static_cast<int64_t>(b) * a.H + h) * 2 * (static_cast<int64_t>(a.q_tiles) * kT);

    if (threadIdx.x == 0) {
        mbar_init(bar(C::kFixFull), 1);
        for (int s = 0; s < R0; ++s) {
            mbar_init(bar(C::kX0Full + s), 1);
            mbar_init(bar(C::kX0Empty + s), 1);
        }
        for (int s = 0; s < R1; ++s) {
            mbar_init(bar(C::kX1Full + s), 1);
            mbar_init(bar(C::kX1Empty + s), 1);
        }
        mbar_init(bar(C::kT0Full), 1);
        mbar_init(bar(C::kT0Full + 1), 1);
        mbar_init(bar(C::kT1Full), 1);
        mbar_init(bar(C::kP), 256);
        mbar_init(bar(C::kDS), 256);
        mbar_init(bar(C::kDS + 1), 256);
        mbar_init(bar(C::kT1Read), 256);
        mbar_init(bar(C::kAccFinal), 1);
        for (int s = 0; s < C::kStats; ++s) mbar_init(bar(C::kMaskFull + s), 32);
        mbar_init(bar(C::kDrain), 1);
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
    const uint32_t tmem = *tmem_slot;
    const Watchdog wd{a.status, a.timeout_ns, abort_flag};
    const Watchdog wd_drain{a.status, a.timeout_ns, never_flag};   // ignores the abort flag: work already in flight

    if (warp == 11) {
        regs_decrease<kOtherRegs>();
    } else if (warp == 10) {
        regs_decrease<kOtherRegs>();
        // ------------------------------------- mask words of the streamed query rows
        // Stage j holds word w (keys 32w .. of the fixed tile) of row r at [w][r];
        // a stage is free again when its X0 slot is (dK of that tile is done).
        if (KEY && MASK) {
            Stream<KEY> cur = stream;
            for (int j = 0; j < n_tiles; ++j) {
                const int tile = cur.next();
                const int st = j % C::kStats;
                const uint32_t ph = static_cast<uint32_t>(j / C::kStats) & 1u;
                if (!wait_bounded_warp(bar(C::kX0Empty + st), ph ^ 1u, wd, ROLE_MASK, SITE_X_EMPTY)) break;
                uint32_t* dst = reinterpret_cast<uint32_t*>(smem + C::kMaskOffset + st * C::kMaskBytes);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int r = i * 32 + lane, row = tile * kT + r;
                    uint4 w = make_uint4(~0u, ~0u, ~0u, ~0u);
                    if (row < a.mask_rows)
                        w = __ldg(reinterpret_cast<const uint4*>(a.mask + b * a.mask_sb + row * a.mask_si) + fixed);
                    dst[r] = w.x;
                    dst[kT + r] = w.y;
                    dst[2 * kT + r] = w.z;
                    dst[3 * kT + r] = w.w;
                }
                mbar_arrive(bar(C::kMaskFull + st));
            }
        }
        __syncwarp();
    } else if (warp == 9) {
        regs_decrease<kOtherRegs>();
        // ------------------------------------------------------------ TMA producer
        if (lane == 0 && n_tiles > 0) {
            tma_prefetch_desc(&tm_f0);
            tma_prefetch_desc(&tm_f1);
            tma_prefetch_desc(&tm_x0);
            tma_prefetch_desc(&tm_x1);
            mbar_arrive_expect_tx(bar(C::kFixFull), 2 * TILE);
            for (int c = 0; c < D / 64; ++c) {
                tma_load_4d(sF0 + c * C::kBlock, &tm_f0, bar(C::kFixFull), c * 64, row0, h, b);
                tma_load_4d(sF1 + c * C::kBlock, &tm_f1, bar(C::kFixFull), c * 64, row0, h, b);
            }
            int issued0 = 0, issued1 = 0;
            Stream<KEY> cur = stream;
            auto copy = [&](const CUtensorMap* tm, uint32_t dst, int full, int x_row) {
                for (int c = 0; c < D / 64; ++c)
                    tma_load_4d(dst + c * C::kBlock, tm, bar(full), c * 64, x_row, h, b);
            };
            for (int j = 0; j < n_tiles; ++j) {
                const int x_row = cur.next() * kT;
                if (!in_bounds(x_row >= 0 && x_row < (KEY ? a.Nq : a.kv_len), a.status, ROLE_LOAD, BND_KEY)) break;
                if (!wait_bounded(bar(C::kX0Empty + j % R0), (static_cast<uint32_t>(j / R0) & 1u) ^ 1u, wd, ROLE_LOAD, SITE_X_EMPTY)) break;
                mbar_arrive_expect_tx(bar(C::kX0Full + j % R0), TILE);
                copy(&tm_x0, sX0 + j % R0 * TILE, C::kX0Full + j % R0, x_row);
                issued0 = j + 1;
                if (!wait_bounded(bar(C::kX1Empty + j % R1), (static_cast<uint32_t>(j / R1) & 1u) ^ 1u, wd, ROLE_LOAD, SITE_X_EMPTY)) break;
                if constexpr (KEY) {
                    // The rows' statistics come with X1; their stage is free when X0
                    // of kStats tiles ago has been released.
                    const int o = j - C::kStats;
                    if (R0 > C::kStats && o >= 0 &&
                        !wait_bounded(bar(C::kX0Empty + o % R0), static_cast<uint32_t>(o / R0) & 1u, wd, ROLE_LOAD, SITE_X_EMPTY)) break;
                }
                mbar_arrive_expect_tx(bar(C::kX1Full + j % R1), TILE + (KEY ? C::kStatBytes : 0));
                copy(&tm_x1, sX1 + j % R1 * TILE, C::kX1Full + j % R1, x_row);
                if constexpr (KEY) {
                    const uint32_t sd = sStat + j % C::kStats * C::kStatBytes;
                    bulk_load(sd, stat + x_row, kT * 4, bar(C::kX1Full + j % R1));
                    bulk_load(sd + kT * 4, stat + static_cast<int64_t>(a.q_tiles) * kT + x_row, kT * 4, bar(C::kX1Full + j % R1));
                }
                issued1 = j + 1;
            }
            if (issued1 < n_tiles || *abort_flag) {
                // Winding down: wait (bounded) until every copy issued has landed.
                for (int j = (issued0 > R0 ? issued0 - R0 : 0); j < issued0; ++j)
                    wait_bounded(bar(C::kX0Full + j % R0), static_cast<uint32_t>(j / R0) & 1u, wd_drain, ROLE_LOAD, SITE_LOAD_DRAIN);
                for (int j = (issued1 > R1 ? issued1 - R1 : 0); j < issued1; ++j)
                    wait_bounded(bar(C::kX1Full + j % R1), static_cast<uint32_t>(j / R1) & 1u, wd_drain, ROLE_LOAD, SITE_LOAD_DRAIN);
                wait_bounded(bar(C::kFixFull), 0, wd_drain, ROLE_LOAD, SITE_LOAD_DRAIN);
            }
        }
        __syncwarp();
    } else if (warp == 8) {
        regs_decrease<kOtherRegs>();
        // ------------------------------------------------------------- MMA issuer
        if (n_tiles > 0) {
            constexpr uint32_t kIdescT = idesc_bf16_f32(kT, kT, false);
            constexpr uint32_t kIdescAcc = idesc_bf16_f32(kT, D, true);
            const uint32_t tT0 = tmem + C::kColT0, tT1 = tmem + C::kColT1;
            const uint32_t tT0b = tmem + C::kColAcc1;      // query CTA: the second T0
            const uint32_t tA0 = tmem + C::kColAcc0, tA1 = tmem + C::kColAcc1;

            // T = F X^T, both K-major, K = D channels.
            auto issue_t = [&](uint32_t tT, uint32_t f_addr, uint32_t x_addr) {
                const uint64_t df = sdesc_sw128(f_addr, 16, 1024), dx = sdesc_sw128(x_addr, 16, 1024);
                static_for<D / 16>([&](auto kk) {
                    constexpr uint32_t off = (kk.value >> 2) * C::kBlock + (kk.value & 3) * 32;
                    umma_ss_warp<off>(tT, df, dx, kIdescT, kk.value > 0 ? 1u : 0u);
                });
            };
            // ACC (+)= A X, A = bf16 pairs in TMEM (K columns 0-63 in the first 32
            // columns of T's first half, 64-127 in those of its second), X MN-major.
            auto issue_acc = [&](uint32_t tA, uint32_t tOp, uint32_t x_addr, bool accumulate) {
                const uint64_t dx = sdesc_sw128(x_addr, C::kBlock, 1024);
                static_for<kT / 16>([&](auto kk) {
                    umma_ts_warp<kk.value * 16 * 128>(tA, tOp + (kk.value >> 2) * 64 + (kk.value & 3) * 8, dx, kIdescAcc,
                                                      (accumulate || kk.value > 0) ? 1u : 0u);
                });
            };
            auto x0_full = [&](int j) {
                return wait_bounded_warp(bar(C::kX0Full + j % R0), static_cast<uint32_t>(j / R0) & 1u, wd, ROLE_MMA, SITE_X_FULL);
            };
            auto x1_full = [&](int j) {
                return wait_bounded_warp(bar(C::kX1Full + j % R1), static_cast<uint32_t>(j / R1) & 1u, wd, ROLE_MMA, SITE_X_FULL);
            };
            auto x0 = [&](int j) { return sX0 + j % R0 * TILE; };
            auto x1 = [&](int j) { return sX1 + j % R1 * TILE; };

            bool ok = wait_bounded_warp(bar(C::kFixFull), 0, wd, ROLE_MMA, SITE_FIX_FULL) && x0_full(0);
            if (ok) {
                tc_fence_after();
                issue_t(tT0, sF0, x0(0));
                umma_commit_warp(bar(C::kT0Full));
                ok = x1_full(0);
            }
            if (ok) {
                tc_fence_after();
                issue_t(tT1, sF1, x1(0));
                umma_commit_warp(bar(C::kT1Full));
                if (!KEY) umma_commit_warp(bar(C::kX1Empty));
            }
            for (int j = 0; ok && j < n_tiles; ++j) {
                const bool more = j + 1 < n_tiles;
                const uint32_t ph = static_cast<uint32_t>(j) & 1u;
                if constexpr (KEY) {
                    ok = wait_bounded_warp(bar(C::kP), ph, wd, ROLE_MMA, SITE_P_READY);
                    if (!ok) break;
                    tc_fence_after();
                    issue_acc(tA1, tT0, x1(j), j > 0);
                    umma_commit_warp(bar(C::kX1Empty + j % R1));
                    if (more) {
                        ok = x0_full(j + 1);
                        if (!ok) break;
                        tc_fence_after();
                        issue_t(tT0, sF0, x0(j + 1));
                        umma_commit_warp(bar(C::kT0Full));
                    }
                    ok = wait_bounded_warp(bar(C::kDS + (j & 1)), static_cast<uint32_t>(j >> 1) & 1u, wd, ROLE_MMA, SITE_DS_READY);
                    if (!ok) break;
                    tc_fence_after();
                    issue_acc(tA0, tT1, x0(j), j > 0);
                    umma_commit_warp(bar(C::kX0Empty + j % R0));
                    if (more) {
                        ok = x1_full(j + 1);
                        if (!ok) break;
                        tc_fence_after();
                        issue_t(tT1, sF1, x1(j + 1));
                        umma_commit_warp(bar(C::kT1Full));
                    }
                } else {
                    if (more) {
                        ok = x0_full(j + 1);
                        if (!ok) break;
                        tc_fence_after();
                        issue_t((j & 1) ? tT0 : tT0b, sF0, x0(j + 1));
                        umma_commit_warp(bar(C::kT0Full + ((j + 1) & 1)));
                        ok = x1_full(j + 1) && wait_bounded_warp(bar(C::kT1Read), ph, wd, ROLE_MMA, SITE_T1_READ);
                        if (!ok) break;
                        tc_fence_after();
                        issue_t(tT1, sF1, x1(j + 1));
                        umma_commit_warp(bar(C::kT1Full));
                        umma_commit_warp(bar(C::kX1Empty + (j + 1) % R1));
                    }
                    ok = wait_bounded_warp(bar(C::kDS + (j & 1)), static_cast<uint32_t>(j >> 1) & 1u, wd, ROLE_MMA, SITE_DS_READY);
                    if (!ok) break;
                    tc_fence_after();
                    issue_acc(tA0, (j & 1) ? tT0b : tT0, x0(j), j > 0);
                    umma_commit_warp(bar(C::kX0Empty + j % R0));
                }
                if (!more) umma_commit_warp(bar(C::kAccFinal));
            }
            // Every product issued must finish before TMEM is released.
            umma_commit_warp(bar(C::kDrain));
            wait_bounded_warp(bar(C::kDrain), 0, wd_drain, ROLE_MMA, SITE_BWD_DRAIN);
        }
        __syncwarp();
    } else {
        // ------------------------------------------------------- softmax warps
        regs_increase<kSoftmaxRegs>();
        const int g = warp >> 2;    // column half
        const int wq = warp & 3;    // TMEM lane quadrant
        const uint32_t lane_off = static_cast<uint32_t>(wq * 32) << 16;
        const uint32_t tT0 = tmem + lane_off + C::kColT0 + 64 * g;
        const uint32_t tT0b = tmem + lane_off + C::kColAcc1 + 64 * g;
        const uint32_t tT1 = tmem + lane_off + C::kColT1 + 64 * g;
        const float sl2 = a.scale_log2;
        const int row = row0 + wq * 32 + lane;      // this thread's row of the fixed tile
        bool ok = true;
        Stream<KEY> cur = stream;
        // query CTA: this row's statistics and mask words
        float nlse = 0.f, ndelta = 0.f;
        bool row_masked = false;
        const uint32_t* mrow = nullptr;
        if constexpr (!KEY) {
            if (n_tiles > 0) {      // without keys there are no statistics
                nlse = __ldg(stat + row);
                ndelta = __ldg(stat + static_cast<int64_t>(a.q_tiles) * kT + row);
            }
            if (MASK) {
                row_masked = row < a.mask_rows;
                mrow = a.mask + b * a.mask_sb + (row_masked ? row : 0) * a.mask_si;
            }
        }
        // 64 values -> 32 columns of bf16 pairs at t, in the layout they were read
        // (key CTA: the second half of the values are lanes 16-31)
        auto store_bf16 = [&](const float* v, uint32_t t) {
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                uint32_t pk[16];
#pragma unroll
                for (int i = 0; i < 16; ++i) pk[i] = pack_bf16x2(v[32 * c + 2 * i], v[32 * c + 2 * i + 1]);
                if constexpr (KEY) tmem_st_16x128b_x8(t + (static_cast<uint32_t>(16 * c) << 16), pk);
                else tmem_st16(t + c * 16, pk);
            }
        };

        for (int j = 0; j < n_tiles; ++j) {
            const int tile = cur.next();
            const uint32_t ph = static_cast<uint32_t>(j) & 1u;
            const int st = j % C::kStats;
            const uint32_t st_ph = static_cast<uint32_t>(j / C::kStats) & 1u;
            uint2 mw = make_uint2(~0u, ~0u);
            if (!KEY && MASK && row_masked) mw = __ldg(reinterpret_cast<const uint2*>(mrow + 4 * tile) + g);
            ok = KEY ? wait_bounded(bar(C::kT0Full), ph, wd, ROLE_SOFTMAX, SITE_T0_FULL)
                     : wait_bounded(bar(C::kT0Full + (j & 1)), static_cast<uint32_t>(j >> 1) & 1u, wd, ROLE_SOFTMAX, SITE_T0_FULL);
            // the statistics (and mask words) of this stage have landed
            if (KEY) ok = ok && wait_bounded(bar(C::kX1Full + j % R1), static_cast<uint32_t>(j / R1) & 1u, wd, ROLE_SOFTMAX, SITE_X_FULL);
            if (KEY && MASK) ok = ok && wait_bounded(bar(C::kMaskFull + st), st_ph, wd, ROLE_SOFTMAX, SITE_MASK_FULL);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            tc_fence_after();
            const uint32_t tS = (KEY || !(j & 1)) ? tT0 : tT0b;
            // P, then dS: 64 values a thread.  A query CTA's thread holds one row (its
            // statistics in registers) and 64 columns.  A key CTA's statistics go by
            // column: its thread holds four rows, lane / 4 + 8 i, and of every 8
            // columns the pair 2 (lane mod 4), so that it reads a quarter of them --
            // with a row a thread, broadcasting them from shared memory took half
            // of its bandwidth from the products (1.50 ms of key CTAs against 1.20).
            float p[64];
            const float2* nl = reinterpret_cast<const float2*>(smem + C::kStatOffset + st * C::kStatBytes) + 32 * g + (lane & 3);
            {
                uint32_t s0[32], s1[32];
                if constexpr (KEY) {
                    tmem_ld_16x256b_x8(tS, s0);
                    tmem_ld_16x256b_x8(tS + (16u << 16), s1);
                } else {
                    tmem_ld32(tS, s0);
                    tmem_ld32(tS + 32, s1);
                }
                tmem_ld_wait_dep(s0);
                reg_dep(s1);
#pragma unroll
                for (int c = 0; c < 32; c += 4) {
                    const float2 n = KEY ? nl[c] : make_float2(nlse, nlse);    // columns 2c .. 2c + 7 of this half
#pragma unroll
                    for (int i = 0; i < 4; i += 2) {
                        ffma2(p[c + i], p[c + i + 1], __uint_as_float(s0[c + i]), __uint_as_float(s0[c + i + 1]), sl2, n.x, n.y);
                        ffma2(p[32 + c + i], p[32 + c + i + 1], __uint_as_float(s1[c + i]), __uint_as_float(s1[c + i + 1]), sl2, n.x, n.y);
                    }
                }
            }
#pragma unroll
            for (int c = 0; c < 64; ++c) p[c] = ex2_approx(p[c]);
            if constexpr (MASK) {
                if constexpr (KEY) {
                    const uint2* m = reinterpret_cast<const uint2*>(smem + C::kMaskOffset + st * C::kMaskBytes) + wq * (kT / 2) + 32 * g + (lane & 3);
                    const int r = lane >> 2;
#pragma unroll
                    for (int c = 0; c < 32; c += 4) {
                        const uint2 w = m[c];
                        if (!((w.x >> r) & 1u)) p[c] = 0.f;
                        if (!((w.y >> r) & 1u)) p[c + 1] = 0.f;
                        if (!((w.x >> (r + 8)) & 1u)) p[c + 2] = 0.f;
                        if (!((w.y >> (r + 8)) & 1u)) p[c + 3] = 0.f;
                        if (!((w.x >> (r + 16)) & 1u)) p[32 + c] = 0.f;
                        if (!((w.y >> (r + 16)) & 1u)) p[32 + c + 1] = 0.f;
                        if (!((w.x >> (r + 24)) & 1u)) p[32 + c + 2] = 0.f;
                        if (!((w.y >> (r + 24)) & 1u)) p[32 + c + 3] = 0.f;
                    }
                } else {
#pragma unroll
                    for (int c = 0; c < 64; ++c)
                        if (!(((c < 32 ? mw.x : mw.y) >> (c & 31)) & 1u)) p[c] = 0.f;
                }
            }
            if constexpr (!KEY) {
                const int valid = a.kv_len - tile * kT - 64 * g;   // keys left in this half
                if (valid < 64) {
#pragma unroll
                    for (int c = 0; c < 64; ++c)
                        if (c >= valid) p[c] = 0.f;
                }
            }
            if constexpr (KEY) {
                store_bf16(p, tT0);
                tmem_st_wait();
                tc_fence_before();
                mbar_arrive(bar(C::kP));
            }
            // dS = P o (dP - delta), from the fp32 P
            ok = wait_bounded(bar(C::kT1Full), ph, wd, ROLE_SOFTMAX, SITE_T1_FULL);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            tc_fence_after();
            {
                uint32_t s0[32], s1[32];
                if constexpr (KEY) {
                    tmem_ld_16x256b_x8(tT1, s0);
                    tmem_ld_16x256b_x8(tT1 + (16u << 16), s1);
                } else {
                    tmem_ld32(tT1, s0);
                    tmem_ld32(tT1 + 32, s1);
                }
                tmem_ld_wait_dep(s0);
                reg_dep(s1);
                if constexpr (!KEY) {
                    tc_fence_before();
                    mbar_arrive(bar(C::kT1Read));
                }
#pragma unroll
                for (int c = 0; c < 32; c += 4) {
                    const float2 n = KEY ? nl[kT / 2 + c] : make_float2(ndelta, ndelta);
#pragma unroll
                    for (int i = 0; i < 4; i += 2) {
                        fadd2_mul2(p[c + i], p[c + i + 1], __uint_as_float(s0[c + i]), __uint_as_float(s0[c + i + 1]), n.x, n.y, p[c + i], p[c + i + 1]);
                        fadd2_mul2(p[32 + c + i], p[32 + c + i + 1], __uint_as_float(s1[c + i]), __uint_as_float(s1[c + i + 1]), n.x, n.y, p[32 + c + i], p[32 + c + i + 1]);
                    }
                }
            }
            store_bf16(p, KEY ? tT1 : tS);
            tmem_st_wait();
            tc_fence_before();
            mbar_arrive(bar(C::kDS + (j & 1)));
        }

        // ---------------------------------------------------------------- epilogue
        if (ok && n_tiles > 0) {
            ok = wait_bounded(bar(C::kAccFinal), 0, wd, ROLE_SOFTMAX, SITE_ACC_FINAL);
            ok = __all_sync(0xffffffffu, ok);
            if (ok) tc_fence_after();
        }
        if (ok) {
            // Key CTA: warps 0-3 write dV, warps 4-7 dK, all D channels; query CTA:
            // each half of the warps writes half of dQ's channels.  32-channel
            // chunks go through this warp's 4 KB of the idle fixed tiles, so that
            // stores leave as whole 128-byte lines.
            constexpr int kChunks = KEY ? D / 32 : D / 64;
            const int c0 = KEY ? 0 : g * kChunks;
            const uint32_t tA = tmem + lane_off + (KEY && g == 0 ? C::kColAcc1 : C::kColAcc0);
            const bool split = f > 1;
            const float mult = split ? 1.f : (KEY && g == 0 ? 1.f : a.scale);
            const int rows_valid = KEY ? a.kv_len : a.Nq;     // rows past it are zeros (key CTA)
            const int rows_out = KEY ? a.Nkv : a.Nq;
            void* const out = KEY ? (g == 0 ? a.dv : a.dk) : a.dq;
            const dit_strides4_t so = KEY ? (g == 0 ? a.sdv : a.sdk) : a.sdq;
            float* const part = KEY ? a.part_kv + (static_cast<int64_t>(slot) * 2 + g) * kT * D
                                    : a.part_q + static_cast<int64_t>(slot) * kT * D;
            float4* stg = reinterpret_cast<float4*>(smem + warp * 4096);
            const int k4 = lane & 7, r_sub = lane >> 3;
#pragma unroll 1
            for (int cc = c0; cc < c0 + kChunks; ++cc) {
                uint32_t o[32];
                if (n_tiles > 0) {
                    tmem_ld32(tA + cc * 32, o);
                    tmem_ld_wait_dep(o);
                } else {
#pragma unroll
                    for (int i = 0; i < 32; ++i) o[i] = 0u;
                }
                const bool zero_row = row >= rows_valid;
#pragma unroll
                for (int v4 = 0; v4 < 8; ++v4) {
                    float4 v = make_float4(__uint_as_float(o[4 * v4 + 0]) * mult, __uint_as_float(o[4 * v4 + 1]) * mult,
                                           __uint_as_float(o[4 * v4 + 2]) * mult, __uint_as_float(o[4 * v4 + 3]) * mult);
                    if (zero_row) v = make_float4(0.f, 0.f, 0.f, 0.f);
                    stg[lane * 8 + (v4 ^ (lane & 7))] = v;
                }
                __syncwarp();
#pragma unroll
                for (int it = 0; it < 8; ++it) {
                    const int r = it * 4 + r_sub;
                    const float4 v = stg[r * 8 + (k4 ^ (r & 7))];
                    const int tr = wq * 32 + r;
                    if (split) {
                        *reinterpret_cast<float4*>(part + tr * D + cc * 32 + 4 * k4) = v;
                    } else if (row0 + tr < rows_out) {
                        const int64_t off = b * so.b + static_cast<int64_t>(row0 + tr) * so.n + h * so.h + cc * 32 + 4 * k4;
                        if constexpr (OUT_BF16)
                            *reinterpret_cast<uint2*>(static_cast<uint16_t*>(out) + off) =
                                make_uint2(pack_bf16x2(v.x, v.y), pack_bf16x2(v.z, v.w));
                        else
                            *reinterpret_cast<float4*>(static_cast<float*>(out) + off) = v;
                    }
                }
                __syncwarp();
            }
        }
    }

    tc_fence_before();
    __syncthreads();
    if (warp == 8) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

template <int D, bool OUT_BF16, bool MASK>
__global__ void __launch_bounds__(kThreads, 1)
    attn_bwd_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                    const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ CUtensorMap tm_do,
                    const __grid_constant__ AttnBwdArgs a) {
    const int slot = static_cast<int>(blockIdx.x);
    if (slot < a.n_kv_ctas) bwd_body<D, true, OUT_BF16, MASK>(tm_k, tm_v, tm_q, tm_do, a, slot);
    else bwd_body<D, false, OUT_BF16, MASK>(tm_q, tm_do, tm_k, tm_v, a, slot - a.n_kv_ctas);
}

// stat[b*H + h][0][i] = -lse * log2(e) (-inf for rows without a key and rows
// past Nq, so that their P is 0), [1][i] = dlse - sum_d dO O.  One row per
// D / 8 lanes, 16 bytes of dO each; HBM-bound (reads dO and O once).
template <int D, bool OUT_BF16>
__global__ void __launch_bounds__(256) attn_bwd_stat_kernel(const AttnBwdStatArgs a) {
    constexpr int LPR = D / 8;
    const int64_t g = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
    const int64_t unit = g / LPR;
    const int c = static_cast<int>(g % LPR);
    const int64_t bh = unit / a.rows_pad;
    const int i = static_cast<int>(unit % a.rows_pad);
    if (bh >= static_cast<int64_t>(a.B) * a.H) return;     // a whole row's lanes (256 is a multiple of LPR)
    const int b = static_cast<int>(bh / a.H), h = static_cast<int>(bh % a.H);
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
        dst[a.rows_pad] = -s;
    }
}

// Sums the pieces' partials of one item in slot order and writes the gradient.
// blockIdx.y: 0 dv, 1 dk, 2 dq (those that were split).
template <int D, bool OUT_BF16>
__global__ void __launch_bounds__(256) attn_bwd_sum_kernel(const AttnBwdArgs a, int first) {
    const int which = static_cast<int>(blockIdx.y) + first;
    const bool key = which < 2;
    const int f = key ? a.f_kv : a.f_q;
    const int tiles = key ? a.kv_out_tiles : a.q_tiles;
    const int64_t g = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
    const int64_t unit = g / (D / 4);
    const int c4 = static_cast<int>(g % (D / 4));
    const int item = static_cast<int>(unit / kT), r = static_cast<int>(unit % kT);
    if (unit >= static_cast<int64_t>(a.B) * a.H * tiles * kT) return;
    const int row = (item % tiles) * kT + r;
    const int h = (item / tiles) % a.H, b = item / tiles / a.H;
    if (row >= (key ? a.Nkv : a.Nq)) return;
    const int64_t stride = static_cast<int64_t>(key ? 2 : 1) * kT * D;
    const float* p = (key ? a.part_kv + (static_cast<int64_t>(item) * f * 2 + which) * kT * D
                          : a.part_q + static_cast<int64_t>(item) * f * kT * D) + r * D + 4 * c4;
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
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg<D, MASK>::kSmemBytes);
    if (e != cudaSuccess) return e;
    kern<<<a.n_kv_ctas + a.n_q_ctas, kThreads, Cfg<D, MASK>::kSmemBytes, s>>>(tq, tk, tv, tdo, a);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_attn_bwd_stat(const AttnBwdStatArgs& a, int D, bool out_bf16, cudaStream_t s) {
    const int64_t threads = static_cast<int64_t>(a.B) * a.H * a.rows_pad * (D / 8);
    const unsigned blocks = static_cast<unsigned>((threads + 255) / 256);
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
    const int tiles = kv && q ? (a.kv_out_tiles > a.q_tiles ? a.kv_out_tiles : a.q_tiles) : (kv ? a.kv_out_tiles : a.q_tiles);
    const int64_t threads = static_cast<int64_t>(a.B) * a.H * tiles * kT * (D / 4);
    const dim3 grid(static_cast<unsigned>((threads + 255) / 256), (kv ? 2 : 0) + (q ? 1 : 0));
    const int first = kv ? 0 : 2;
    if (D == 128) {
        if (grad_bf16) attn_bwd_sum_kernel<128, true><<<grid, 256, 0, s>>>(a, first);
        else attn_bwd_sum_kernel<128, false><<<grid, 256, 0, s>>>(a, first);
    } else {
        if (grad_bf16) attn_bwd_sum_kernel<64, true><<<grid, 256, 0, s>>>(a, first);
        else attn_bwd_sum_kernel<64, false><<<grid, 256, 0, s>>>(a, first);
    }
    return cudaGetLastError();
}

}  // namespace dit

// layer_norm.cu -- layer norm of rows of C channels, forward and backward.
//
//   forward   mean = sum_c x / C,  rstd = 1 / sqrt(sum_c (x - mean)^2 / C + eps),
//             xh = (x - mean) rstd,  y = xh * weight + bias
//   backward  g = dy * weight,
//             dx = rstd * (g - sum_c g / C - xh * sum_c (g xh) / C),
//             dweight = sum_rows dy * xh,  dbias = sum_rows dy
// Without `center` the mean is 0 and its term of dx is absent (RMS norm).
// weight and bias are one vector, or one per batch entry (the modulation of a
// diffusion transformer's block).  All arithmetic is fp32; y and dx are
// rounded to their type once.
//
// HBM-bound: the forward pass reads x and writes y, the backward pass reads x
// and dy and writes dx (24,576 x 4,096 bf16: 68 us forward, 5.9 TB/s or 87% of a
// plain copy; 111 us backward, 80%, the parameters' sums included).  A row is
// held in the registers of `tpr` threads, at most 32 channels each, so the
// variance takes a second pass over registers and not over memory.  A thread
// keeps its channels while it walks over rows: their weights stay in registers,
// and so do the backward pass' sums over rows, which leave the block once, as
// one partial per block, summed in a fixed order by a second kernel (no atomics:
// results repeat bit for bit).  The next rows are on their way to shared memory
// while the current row is reduced.
#include <cuda_runtime.h>

#include <cstdint>

#include "internal.h"
#include "train.h"

namespace dit {
namespace {

constexpr int kMaxThreads = 512;
constexpr int kTwoRowThreads = 384;     // 168 registers a thread: two rows' values beside the sums over rows
// Cross-warp sums of a block, in 8 bytes a warp; a row's warps are padded to an
// even number (5 rows of 3 warps take 20).
constexpr int kSums = 24;

// Two fp32 numbers in a register pair: the kernels are bound by instructions as
// much as by memory, and packed operations halve the arithmetic.  Pairs are kept
// as 64-bit values throughout, so that none is packed twice.
using f2 = unsigned long long;
__device__ __forceinline__ f2 pk(float lo, float hi) {
    f2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ void unpk(f2 p, float& lo, float& hi) { asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(p)); }
__device__ __forceinline__ f2 add2(f2 a, f2 b) {
    f2 r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ f2 mul2(f2 a, f2 b) {
    f2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ f2 fma2(f2 a, f2 b, f2 c) {
    f2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ float sum2(f2 p) {
    float lo, hi;
    unpk(p, lo, hi);
    return lo + hi;
}
// A thread's channels of a row, NV loads of VEC, are NV * VEC / 2 pairs: two
// neighbours of one load, or with VEC = 1 the channels of two loads.

template <typename T, int VEC>
struct Row {   // VEC elements as loaded
    static constexpr int kBytes = static_cast<int>(sizeof(T)) * VEC;
    static constexpr int kWords = kBytes >= 4 ? kBytes / 4 : 1;
    uint32_t w[kWords];
    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int i = 0; i < kWords; ++i) w[i] = 0u;
    }
    __device__ __forceinline__ void load(const T* p) {
        if constexpr (kBytes >= 16) {
#pragma unroll
            for (int i = 0; i < kWords / 4; ++i) {
                const uint4 v = __ldcs(reinterpret_cast<const uint4*>(p) + i);
                w[4 * i] = v.x; w[4 * i + 1] = v.y; w[4 * i + 2] = v.z; w[4 * i + 3] = v.w;
            }
        } else if constexpr (kBytes == 8) {
            const uint2 v = __ldcs(reinterpret_cast<const uint2*>(p));
            w[0] = v.x; w[1] = v.y;
        } else if constexpr (kBytes == 4) {
            w[0] = __ldcs(reinterpret_cast<const uint32_t*>(p));
        } else {
            w[0] = __ldcs(reinterpret_cast<const unsigned short*>(p));
        }
    }
    __device__ __forceinline__ float one() const { return __uint_as_float(sizeof(T) == 4 ? w[0] : w[0] << 16); }
    // channels 2i and 2i + 1
    __device__ __forceinline__ f2 pair(int i) const {
        if constexpr (sizeof(T) == 4) return pk(__uint_as_float(w[2 * i]), __uint_as_float(w[2 * i + 1]));
        else return pk(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xFFFF0000u));
    }
};
// Pair k of a thread's NV loads.
template <typename T, int VEC, int NV>
__device__ __forceinline__ f2 pair_of(const Row<T, VEC> (&r)[NV], int k) {
    if constexpr (VEC == 1) return pk(r[2 * k].one(), r[2 * k + 1].one());
    else return r[k / (VEC / 2)].pair(k % (VEC / 2));
}
// Load i's channels from its pairs, rounded to T once.
template <typename T, int VEC, int NV>
__device__ __forceinline__ void store_row(T* p, int i, const f2 (&v)[NV * VEC / 2]) {
    using R = Row<T, VEC>;
    uint32_t w[R::kWords];
    if constexpr (VEC == 1) {
        float lo, hi;
        unpk(v[i / 2], lo, hi);
        const float x = (i & 1) ? hi : lo;
        if constexpr (sizeof(T) == 4) w[0] = __float_as_uint(x);
        else asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w[0]) : "f"(0.f), "f"(x));
    } else {
#pragma unroll
        for (int e = 0; e < VEC / 2; ++e) {
            float lo, hi;
            unpk(v[i * (VEC / 2) + e], lo, hi);
            if constexpr (sizeof(T) == 4) {
                w[2 * e] = __float_as_uint(lo);
                w[2 * e + 1] = __float_as_uint(hi);
            } else {
                asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w[e]) : "f"(hi), "f"(lo));
            }
        }
    }
    if constexpr (R::kBytes >= 16) {
#pragma unroll
        for (int e = 0; e < R::kWords / 4; ++e)
            __stcs(reinterpret_cast<uint4*>(p) + e, make_uint4(w[4 * e], w[4 * e + 1], w[4 * e + 2], w[4 * e + 3]));
    } else if constexpr (R::kBytes == 8) {
        __stcs(reinterpret_cast<uint2*>(p), make_uint2(w[0], w[1]));
    } else if constexpr (R::kBytes == 4) {
        __stcs(reinterpret_cast<uint32_t*>(p), w[0]);
    } else {
        __stcs(reinterpret_cast<unsigned short*>(p), static_cast<unsigned short>(w[0]));
    }
}

// A thread's own ring of P staged rows in shared memory, filled by asynchronous
// copies of its channels (no other thread reads them, so waiting for its own
// copies is all the synchronisation there is).  Loads of single bf16 channels
// are below the smallest asynchronous copy: those wait in registers, a row ahead.
// What a thread does not have is zeros in the ring, written once or where a row is
// missing, so that nothing is tested where rows are taken.
template <typename T, int VEC, int NV>
struct Ring {
    using R = Row<T, VEC>;
    static constexpr bool kAsync = R::kBytes >= 4;
    static constexpr int kChunk = R::kBytes < 16 ? R::kBytes : 16;    // bytes of one copy
    static constexpr int kChunks = R::kBytes < 16 ? 1 : R::kBytes / 16;
    static constexpr int kStageBytes = kAsync ? NV * kChunk * kChunks : 0;    // per thread
    uint32_t base;              // this thread's first chunk; chunks lie blockDim.x apart
    R reg[kAsync ? 1 : NV];
    __device__ __forceinline__ uint32_t slot(int stage, int i, int c) const {
        return base + static_cast<uint32_t>(((stage * NV + i) * kChunks + c) * blockDim.x) * kChunk;
    }
    __device__ __forceinline__ void init(void* smem) {
        base = static_cast<uint32_t>(__cvta_generic_to_shared(smem)) + threadIdx.x * kChunk;
    }
    __device__ __forceinline__ void fetch(int stage, int i, const T* p) {
        if constexpr (kAsync) {
#pragma unroll
            for (int c = 0; c < kChunks; ++c) {
                const char* src = reinterpret_cast<const char*>(p) + c * kChunk;
                if constexpr (kChunk == 16)
                    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(slot(stage, i, c)), "l"(src) : "memory");
                else
                    asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(slot(stage, i, c)), "l"(src), "n"(kChunk) : "memory");
            }
        } else {
            reg[i].load(p);
        }
    }
    // Zeros in place of a load: channels past the row's end, rows past the last.
    __device__ __forceinline__ void clear(int stage, int i) {
        if constexpr (kAsync) {
#pragma unroll
            for (int c = 0; c < kChunks; ++c) {
                if constexpr (kChunk == 16)
                    asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"(slot(stage, i, c)), "r"(0u) : "memory");
                else if constexpr (kChunk == 8)
                    asm volatile("st.shared.v2.u32 [%0], {%1, %1};" ::"r"(slot(stage, i, c)), "r"(0u) : "memory");
                else
                    asm volatile("st.shared.u32 [%0], %1;" ::"r"(slot(stage, i, c)), "r"(0u) : "memory");
            }
        } else {
            reg[i].zero();
        }
    }
    __device__ __forceinline__ R take(int stage, int i) const {
        if constexpr (kAsync) {
            R r;
#pragma unroll
            for (int c = 0; c < kChunks; ++c) {
                if constexpr (kChunk == 16)
                    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                                 : "=r"(r.w[4 * c]), "=r"(r.w[4 * c + 1]), "=r"(r.w[4 * c + 2]), "=r"(r.w[4 * c + 3])
                                 : "r"(slot(stage, i, c)) : "memory");
                else if constexpr (kChunk == 8)
                    asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(r.w[0]), "=r"(r.w[1]) : "r"(slot(stage, i, c)) : "memory");
                else
                    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(r.w[0]) : "r"(slot(stage, i, c)) : "memory");
            }
            return r;
        } else {
            return reg[i];
        }
    }
};
__device__ __forceinline__ void ring_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void ring_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

// Rows staged ahead: as many as fill some 128 bytes of shared memory a thread
// (64 KB for an SM's 512 threads), between 2 and 6.
constexpr int kStagedBytes = 128;
__host__ __device__ constexpr int ring_depth(int stage_bytes, bool async) {
    if (!async) return 1;
    const int p = kStagedBytes / stage_bytes;
    return p < 2 ? 2 : (p > 6 ? 6 : p);
}

// The threads of one row: `tpr` of them, a power of two up to 32 or else whole
// warps.  Sums over the row reach every thread in the same order.
// A forward block holds two rows of more than a warp at most, and names its
// barriers: a barrier named at run time takes all 16 of a block, and an SM has
// room for four such blocks.
template <bool FWD>
struct RowGroup {
    int tpr, t, id;             // threads per row, index in the row, row slot of the block
    int warps;                  // warps of a row (1 when tpr <= 32), at most 16
    int span;                   // the next power of two: across() adds over that many lanes
    float2* buf;                // [2][kSums]; zeroed for across_two(), which adds a row's padding too
    int pitch;                  // a row's place in it: its warps, rounded up to even
    int flip;
    __device__ RowGroup(int tpr_, float2* b)
        : tpr(tpr_), t(threadIdx.x % tpr_), id(threadIdx.x / tpr_), warps(tpr_ > 32 ? tpr_ >> 5 : 1),
          span(1), buf(b), pitch((warps + 1) & ~1), flip(0) {
        while (span < warps) span *= 2;
    }
    __device__ __forceinline__ void sync() const {
        if constexpr (!FWD) asm volatile("bar.sync %0, %1;" ::"r"(1 + id), "r"(tpr) : "memory");
        else if (id == 0) asm volatile("bar.sync 1, %0;" ::"r"(tpr) : "memory");
        else asm volatile("bar.sync 2, %0;" ::"r"(tpr) : "memory");
    }
    // Sum over the row's lanes of this warp.  Lanes of one warp may belong to
    // row slots that have run out of rows: every lane takes part in every sum.
    __device__ __forceinline__ float lanes(float v) const {
        if (tpr >= 32) {
#pragma unroll
            for (int o = 16; o >= 1; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
        } else {
            for (int o = tpr >> 1; o >= 1; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
        }
        return v;
    }
    // Two sums at once: lanes of the lower half end with the first, of the upper
    // half with the second (5 shuffles for both; whole warps only).
    __device__ __forceinline__ float lanes_two(float a, float b) const {
        const bool upper = (threadIdx.x & 16) != 0;
        float v = (upper ? b : a) + __shfl_xor_sync(0xffffffffu, upper ? a : b, 16);
#pragma unroll
        for (int o = 8; o >= 1; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
        return v;
    }
    // The sums of lanes_two over the row's warps, to every thread; of ROWS rows at once.
    template <int ROWS>
    __device__ __forceinline__ void across_two(const float (&v)[ROWS], f2 (&sum)[ROWS]) {
        float2* const b = buf + flip * kSums + id * ROWS * pitch;
        flip ^= 1;
        if ((threadIdx.x & 15) == 0) {
#pragma unroll
            for (int j = 0; j < ROWS; ++j) reinterpret_cast<float*>(b + j * pitch)[t >> 4] = v[j];
        }
        sync();
#pragma unroll
        for (int j = 0; j < ROWS; ++j) {
            const ulonglong2* p = reinterpret_cast<const ulonglong2*>(b + j * pitch);
            ulonglong2 q = p[0];
            sum[j] = add2(q.x, q.y);
            for (int w = 1; w < (pitch >> 1); ++w) {
                q = p[w];
                sum[j] = add2(sum[j], add2(q.x, q.y));
            }
        }
    }
    // Each warp's pair to the row's other warps: lane l gets that of warp
    // l mod span (0 past the last).  One barrier among the row's threads; the other buffer is
    // written next, so a second is not needed.
    __device__ __forceinline__ float2 exchange(float2 v) {
        float2* const b = buf + flip * kSums + id * pitch;
        flip ^= 1;
        if ((threadIdx.x & 31) == 0) b[t >> 5] = v;
        sync();
        const int w = threadIdx.x & (span - 1);
        return w < warps ? b[w] : make_float2(0.f, 0.f);
    }
    // Sum of what exchange() handed out, over the row's warps.
    __device__ __forceinline__ float across(float v) const {
        for (int o = span >> 1; o >= 1; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
        return v;
    }
};

// Element offset of row (b, n, h); rows that follow one another at one distance
// (the common case) take a multiply.
struct RowAt {
    dit_strides4_t s;
    bool flat;
    __device__ __forceinline__ int64_t operator()(const NormArgs& a, uint32_t row) const {
        if (flat) return static_cast<int64_t>(row) * (a.H == 1 ? s.n : s.h);
        uint32_t nh, h;
        const uint32_t b = a.div_nh.divmod(row, nh);
        const uint32_t n = a.div_h.divmod(nh, h);
        return b * s.b + n * s.n + h * s.h;
    }
    __device__ RowAt(const NormArgs& a, const dit_strides4_t& st) : s(st) {
        flat = (a.H == 1 || st.n == a.H * st.h) && (a.B == 1 || st.b == a.N * st.n);
    }
};

// A thread's weights (or biases), `other` where it has no channel or there are none.
template <int VEC, int NV>
__device__ __forceinline__ void load_params(const float* p, const bool (&live)[NV], const int (&col)[NV], float other,
                                            f2 (&v)[NV * VEC / 2]) {
    float f[NV * VEC];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
#pragma unroll
        for (int e = 0; e < VEC; ++e) f[i * VEC + e] = other;
        if (p == nullptr || !live[i]) continue;
        if constexpr (VEC == 8) {
            const float4 lo = __ldg(reinterpret_cast<const float4*>(p + col[i])), hi = __ldg(reinterpret_cast<const float4*>(p + col[i]) + 1);
            f[8 * i] = lo.x; f[8 * i + 1] = lo.y; f[8 * i + 2] = lo.z; f[8 * i + 3] = lo.w;
            f[8 * i + 4] = hi.x; f[8 * i + 5] = hi.y; f[8 * i + 6] = hi.z; f[8 * i + 7] = hi.w;
        } else if constexpr (VEC == 2) {
            const float2 x = __ldg(reinterpret_cast<const float2*>(p + col[i]));
            f[2 * i] = x.x;
            f[2 * i + 1] = x.y;
        } else {
            f[i] = __ldg(p + col[i]);
        }
    }
#pragma unroll
    for (int k = 0; k < NV * VEC / 2; ++k) v[k] = pk(f[2 * k], f[2 * k + 1]);
}

// grid (blocks, groups).  Every thread of a block makes the same number of
// rounds; a row slot past its last row runs along on zeros.
template <typename TX, typename TY, int VEC, int NV>
__global__ void __launch_bounds__(kMaxThreads) layer_norm_fwd_kernel(const NormArgs a, int tpr) {
    using RX = Ring<TX, VEC, NV>;
    constexpr int P = ring_depth(RX::kStageBytes, RX::kAsync);
    __shared__ __align__(16) float2 buf[2 * kSums];
    extern __shared__ __align__(16) uint8_t ring_mem[];
    RowGroup<true> g(tpr, buf);
    RX ring;
    ring.init(ring_mem);
    const RowAt x_at(a, a.sx), y_at(a, a.sy);
    const uint32_t slots = blockDim.x / tpr;
    const uint32_t step = gridDim.x * slots;
    const uint32_t row0 = blockIdx.y * a.rows_per_group;
    const uint32_t rounds = (a.rows_per_group - blockIdx.x * slots + step - 1) / step;   // >= 1: (blocks - 1) * slots < rows
    const uint32_t first = blockIdx.x * slots + g.id;
    bool live[NV];
    int col[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        col[i] = (i * tpr + g.t) * VEC;
        live[i] = col[i] < a.C;
    }
    auto fetch = [&](uint32_t k) {
        const uint32_t r = first + k * step;
        if (k < rounds && r < a.rows_per_group) {
            const TX* p = static_cast<const TX*>(a.x) + x_at(a, row0 + r);
#pragma unroll
            for (int i = 0; i < NV; ++i)
                if (live[i]) ring.fetch(k % P, i, p + col[i]);
        } else if (k < rounds) {
#pragma unroll
            for (int i = 0; i < NV; ++i) ring.clear(k % P, i);
        }
        ring_commit();
    };
#pragma unroll
    for (int i = 0; i < NV; ++i)
        if (!live[i])
            for (int k = 0; k < P; ++k) ring.clear(k, i);
    for (int k = 0; k < (RX::kAsync ? P - 1 : 1); ++k) fetch(k);
    constexpr int NP = NV * VEC / 2;
    f2 w[NP], bi[NP];
    load_params<VEC, NV>(a.weight ? a.weight + static_cast<int64_t>(blockIdx.y) * a.C : nullptr, live, col, 1.f, w);
    load_params<VEC, NV>(a.bias ? a.bias + static_cast<int64_t>(blockIdx.y) * a.C : nullptr, live, col, 0.f, bi);
    // Channels held by warp v of a row, 1 / that (0 for none): by this thread's
    // own warp, and by the warp whose pair exchange() hands this lane.
    auto held = [&](int v) {
        int n = 0;
        if (v >= g.warps) return 0.f;
#pragma unroll
        for (int i = 0; i < NV; ++i) n += min(max(a.C - (i * tpr + 32 * v) * VEC, 0), 32 * VEC);
        return static_cast<float>(n);
    };
    const float own_n = tpr > 32 ? held(g.t >> 5) : static_cast<float>(a.C);
    const float own_inv = own_n > 0.f ? 1.f / own_n : 0.f;
    const float got_n = tpr > 32 ? held(threadIdx.x & (g.span - 1)) : 0.f;
    const float got_inv = got_n > 0.f ? 1.f / got_n : 0.f;

    uint32_t r = first;
    for (uint32_t k = 0; k < rounds; ++k, r += step) {
        if constexpr (RX::kAsync) {
            fetch(k + P - 1);
            ring_wait<P - 1>();
        }
        const bool ok = r < a.rows_per_group;
        Row<TX, VEC> raw[NV];
#pragma unroll
        for (int i = 0; i < NV; ++i) raw[i] = ring.take(k % P, i);
        if constexpr (!RX::kAsync) fetch(k + 1);
        f2 x[NP];
#pragma unroll
        for (int e = 0; e < NP; ++e) x[e] = pair_of(raw, e);
        // This warp's mean and sum of squared deviations from it, then the row's
        // from all its warps': sum of (their deviations + n (their mean - mean)^2).
        float mean = 0.f, s = 0.f;
        if (a.center) {
            f2 t = 0ull;
#pragma unroll
            for (int e = 0; e < NP; ++e) t = add2(t, x[e]);
            s = g.lanes(sum2(t));
            mean = s * own_inv;
        }
        f2 u = 0ull;
#pragma unroll
        for (int e = 0; e < NP; ++e) {       // (channels a thread does not have stay 0)
            constexpr int kPer = VEC == 1 ? 1 : VEC / 2;     // pairs of a load
            const bool l0 = live[VEC == 1 ? 2 * e : e / kPer], l1 = live[VEC == 1 ? 2 * e + 1 : e / kPer];
            x[e] = add2(x[e], pk(l0 ? -mean : 0.f, l1 ? -mean : 0.f));
            u = fma2(x[e], x[e], u);
        }
        float q = g.lanes(sum2(u));
        float shift = 0.f;          // this warp's mean - the row's, still in x
        if (tpr > 32) {
            const float2 p = g.exchange(make_float2(s, q));
            q = p.y;
            if (a.center) {
                const float row_mean = g.across(p.x) * a.inv_c;
                const float d = fmaf(p.x, got_inv, -row_mean);
                q = fmaf(got_n * d, d, q);
                shift = mean - row_mean;
                mean = row_mean;
            }
            q = g.across(q);
        }
        const float rstd = 1.f / sqrtf(q * a.inv_c + a.eps);
        if (ok) {
            TY* const p = static_cast<TY*>(a.y) + y_at(a, row0 + r);
            const f2 r2 = pk(rstd, rstd), sr = pk(shift * rstd, shift * rstd);
            f2 v[NP];
#pragma unroll
            for (int e = 0; e < NP; ++e) v[e] = fma2(fma2(x[e], r2, sr), w[e], bi[e]);
#pragma unroll
            for (int i = 0; i < NV; ++i)
                if (live[i]) store_row<TY, VEC, NV>(p + col[i], i, v);
            if (g.t == 0) {
                if (a.center) a.mean[row0 + r] = mean;
                a.rstd[row0 + r] = rstd;
            }
        }
    }
}

// ROWS rows of a group of threads at a time: two where a block holds one such group,
// whose chain of loads, sums and barrier is then as long for two rows as for one.
template <typename TX, typename TY, int VEC, int NV, int ROWS>
__global__ void __launch_bounds__(ROWS == 1 ? kMaxThreads : kTwoRowThreads) layer_norm_bwd_kernel(const NormArgs a, int tpr) {
    using RX = Ring<TX, VEC, NV * ROWS>;
    using RD = Ring<TY, VEC, NV * ROWS>;
    constexpr int P = ring_depth(RX::kStageBytes + RD::kStageBytes, RX::kAsync && RD::kAsync);
    __shared__ __align__(16) float2 buf[2 * kSums];
    for (int i = threadIdx.x; i < 2 * kSums; i += blockDim.x) buf[i] = make_float2(0.f, 0.f);
    __syncthreads();
    extern __shared__ __align__(16) uint8_t ring_mem[];   // the rings; after the rows, [slots][tpr * NV * VEC] sums
    float* const acc = reinterpret_cast<float*>(ring_mem);
    if (threadIdx.x == 0) let_next();
    RowGroup<false> g(tpr, buf);
    RX rx;
    RD rd;
    rx.init(ring_mem);
    rd.init(ring_mem + P * RX::kStageBytes * blockDim.x);
    const RowAt x_at(a, a.sx), d_at(a, a.sdy), y_at(a, a.sy);
    const uint32_t slots = blockDim.x / tpr;
    const uint32_t step = gridDim.x * slots * ROWS;
    const uint32_t row0 = blockIdx.y * a.rows_per_group;
    const uint32_t rounds = (a.rows_per_group - blockIdx.x * slots * ROWS + step - 1) / step;
    const uint32_t first = (blockIdx.x * slots + g.id) * ROWS;
    bool live[NV];
    int col[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        col[i] = (i * tpr + g.t) * VEC;
        live[i] = col[i] < a.C;
    }
    float nmean[ROWS], nrstd[ROWS];
    auto stats = [&](uint32_t k) {       // of round k, read one round ahead
#pragma unroll
        for (int j = 0; j < ROWS; ++j) {
            const uint32_t r = first + k * step + j;
            const bool ok = k < rounds && r < a.rows_per_group;
            nmean[j] = ok && a.center ? __ldg(a.mean + row0 + r) : 0.f;
            nrstd[j] = ok ? __ldg(a.rstd + row0 + r) : 0.f;
        }
    };
    auto fetch = [&](uint32_t k) {
#pragma unroll
        for (int j = 0; j < ROWS; ++j) {
            const uint32_t r = first + k * step + j;
            if (k < rounds && r < a.rows_per_group) {
                const TX* p = static_cast<const TX*>(a.x) + x_at(a, row0 + r);
                const TY* d = static_cast<const TY*>(a.dy) + d_at(a, row0 + r);
#pragma unroll
                for (int i = 0; i < NV; ++i)
                    if (live[i]) {
                        rx.fetch(k % P, j * NV + i, p + col[i]);
                        rd.fetch(k % P, j * NV + i, d + col[i]);
                    }
            } else if (k < rounds) {
#pragma unroll
                for (int i = 0; i < NV; ++i) {
                    rx.clear(k % P, j * NV + i);
                    rd.clear(k % P, j * NV + i);
                }
            }
        }
        ring_commit();
    };
#pragma unroll
    for (int i = 0; i < NV * ROWS; ++i)
        if (!live[i % NV])
            for (int k = 0; k < P; ++k) {
                rx.clear(k, i);
                rd.clear(k, i);
            }
    constexpr bool kAsync = RX::kAsync && RD::kAsync;
    for (int k = 0; k < (kAsync ? P - 1 : 1); ++k) fetch(k);
    stats(0);
    constexpr int NP = NV * VEC / 2;
    f2 w[NP], dw[NP], db[NP];
    load_params<VEC, NV>(a.weight ? a.weight + static_cast<int64_t>(blockIdx.y) * a.C : nullptr, live, col, 1.f, w);
#pragma unroll
    for (int e = 0; e < NP; ++e) dw[e] = db[e] = 0ull;
    uint32_t r = first;
    for (uint32_t k = 0; k < rounds; ++k, r += step) {
        if constexpr (kAsync) {
            fetch(k + P - 1);
            ring_wait<P - 1>();
        } else {
            ring_wait<0>();
        }
        bool ok[ROWS];
        float rstd[ROWS], nm[ROWS];
        Row<TX, VEC> x[ROWS][NV];
        Row<TY, VEC> d[ROWS][NV];
#pragma unroll
        for (int j = 0; j < ROWS; ++j) {
            ok[j] = r + j < a.rows_per_group;
            rstd[j] = nrstd[j];
            nm[j] = -nmean[j];
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                x[j][i] = rx.take(k % P, j * NV + i);
                d[j][i] = rd.take(k % P, j * NV + i);
            }
        }
        if constexpr (!kAsync) fetch(k + 1);
        stats(k + 1);
        f2 xh[ROWS][NP], gr[ROWS][NP];      // xh and g, kept for dx
        f2 sum[ROWS];                       // of g and of g xh
        float both[ROWS];
#pragma unroll
        for (int j = 0; j < ROWS; ++j) {
            f2 s2 = 0ull, t2 = 0ull;
            const f2 r2 = pk(rstd[j], rstd[j]), m2 = pk(nm[j], nm[j]);
#pragma unroll
            for (int e = 0; e < NP; ++e) {
                const f2 dy = pair_of(d[j], e);
                // (the mean first: x rstd - mean rstd is off by 2^-24 |mean| rstd)
                xh[j][e] = mul2(add2(pair_of(x[j], e), m2), r2);
                gr[j][e] = mul2(dy, w[e]);
                s2 = add2(s2, gr[j][e]);
                t2 = fma2(gr[j][e], xh[j][e], t2);
                dw[e] = fma2(dy, xh[j][e], dw[e]);
                db[e] = add2(db[e], dy);
            }
            if (tpr > 32) both[j] = g.lanes_two(sum2(s2), sum2(t2));
            else sum[j] = pk(g.lanes(sum2(s2)), g.lanes(sum2(t2)));
        }
        if (tpr > 32) g.across_two(both, sum);
#pragma unroll
        for (int j = 0; j < ROWS; ++j) {
            float sg, st;
            unpk(sum[j], sg, st);
            if (!a.center) sg = 0.f;
            // dx = rstd g - rstd c1 - xh (rstd c2)
            const float n1 = -sg * a.inv_c * rstd[j], n2 = -st * a.inv_c * rstd[j];
            if (ok[j]) {
                TX* const p = static_cast<TX*>(a.y) + y_at(a, row0 + r + j);
                const f2 r2 = pk(rstd[j], rstd[j]), c1 = pk(n1, n1), c2 = pk(n2, n2);
                f2 v[NP];
#pragma unroll
                for (int e = 0; e < NP; ++e) v[e] = fma2(gr[j][e], r2, fma2(xh[j][e], c2, c1));
#pragma unroll
                for (int i = 0; i < NV; ++i)
                    if (live[i]) store_row<TX, VEC, NV>(p + col[i], i, v);
            }
        }
    }
    ring_wait<0>();
    // The block's sums: row slots added in order, then one partial per block
    // (the gradient itself when the group has one block).
    const int width = tpr * NV * VEC;
    auto leave = [&](f2 (&v)[NP], float* part, float* grad) {
        float* const out = gridDim.x == 1 ? grad + static_cast<int64_t>(blockIdx.y) * a.C
                                          : part + (static_cast<int64_t>(blockIdx.y) * gridDim.x + blockIdx.x) * a.C;
        float f[2 * NP];
#pragma unroll
        for (int e = 0; e < NP; ++e) unpk(v[e], f[2 * e], f[2 * e + 1]);
        if (slots == 1) {
#pragma unroll
            for (int i = 0; i < NV; ++i)
                if (live[i])
#pragma unroll
                    for (int e = 0; e < VEC; ++e) out[col[i] + e] = f[i * VEC + e];
            return;
        }
        __syncthreads();     // the rings (or the last sums) have been read
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int e = 0; e < VEC; ++e) acc[g.id * width + col[i] + e] = f[i * VEC + e];
        __syncthreads();
        for (int c = threadIdx.x; c < a.C; c += blockDim.x) {
            float t = 0.f;
            for (uint32_t k = 0; k < slots; ++k) t += acc[k * width + c];
            out[c] = t;
        }
    };
    if (a.want_w) leave(dw, a.part, a.dweight);
    if (a.want_b) leave(db, a.part + static_cast<int64_t>(a.groups) * gridDim.x * a.C, a.dbias);
}

// dweight / dbias [groups][C] = the sum over a group's `parts` partials, each
// column's in a fixed order: 32 interleaved sums, then those in order.
__global__ void __launch_bounds__(1024) layer_norm_param_sum_kernel(const NormArgs a, int parts) {
    __shared__ float s[32][33];
    after_previous();
    const int cx = threadIdx.x & 31, py = threadIdx.x >> 5;
    const int c = blockIdx.x * 32 + cx;
    const bool second = blockIdx.z != 0 || !a.want_w;
    float* const out = second ? a.dbias : a.dweight;
    const float* const p = a.part + (static_cast<int64_t>(second ? a.groups : 0) + blockIdx.y) * parts * a.C;
    float t = 0.f;
    if (c < a.C) {
#pragma unroll 4
        for (int k = py; k < parts; k += 32) t += __ldcs(p + static_cast<int64_t>(k) * a.C + c);
    }
    s[py][cx] = t;
    __syncthreads();
    if (py == 0 && c < a.C) {
#pragma unroll
        for (int k = 1; k < 32; ++k) t += s[k][cx];
        out[static_cast<int64_t>(blockIdx.y) * a.C + c] = t;
    }
}

template <typename TX, typename TY, int VEC, int NV>
cudaError_t fwd(const NormArgs& a, const NormPlan& p, cudaStream_t s) {
    using RX = Ring<TX, VEC, NV>;
    const int smem = ring_depth(RX::kStageBytes, RX::kAsync) * RX::kStageBytes * p.threads;
    auto kern = layer_norm_fwd_kernel<TX, TY, VEC, NV>;
    if (smem > 47 * 1024) {
        const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (e != cudaSuccess) return e;
    }
    kern<<<dim3(p.blocks, a.groups), p.threads, smem, s>>>(a, p.tpr);
    return cudaGetLastError();
}

template <typename TX, typename TY, int VEC, int NV, int ROWS>
cudaError_t bwd(const NormArgs& a, const NormPlan& p, cudaStream_t s) {
    using RX = Ring<TX, VEC, NV * ROWS>;
    using RD = Ring<TY, VEC, NV * ROWS>;
    const int depth = ring_depth(RX::kStageBytes + RD::kStageBytes, RX::kAsync && RD::kAsync);
    const int rings = (RX::kStageBytes + RD::kStageBytes) * depth * p.threads;
    const int sums = p.threads > p.tpr ? p.threads * NV * VEC * static_cast<int>(sizeof(float)) : 0;
    const int smem = rings > sums ? rings : sums;
    auto kern = layer_norm_bwd_kernel<TX, TY, VEC, NV, ROWS>;
    if (smem > 47 * 1024) {
        const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (e != cudaSuccess) return e;
    }
    kern<<<dim3(p.blocks, a.groups), p.threads, smem, s>>>(a, p.tpr);
    cudaError_t e = cudaGetLastError();
    const int wants = (a.want_w ? 1 : 0) + (a.want_b ? 1 : 0);
    if (e != cudaSuccess || p.blocks == 1 || wants == 0) return e;
    return launch_behind(layer_norm_param_sum_kernel, dim3((a.C + 31) / 32, a.groups, wants), 1024, 0, s, a, p.blocks);
}

template <typename TX, typename TY, bool BWD>
cudaError_t pick(const NormArgs& a, const NormPlan& p, cudaStream_t s) {
    if constexpr (BWD)
        if (p.two_rows) return bwd<TX, TY, 8, 2, 2>(a, p, s);
#define DIT_NORM_CASE(V, N) \
    if (p.vec == V && p.nv == N) {                                                                 \
        if constexpr (BWD) return bwd<TX, TY, V, N, 1>(a, p, s);                                   \
        else return fwd<TX, TY, V, N>(a, p, s);                                                    \
    }
    DIT_NORM_CASE(8, 1)
    DIT_NORM_CASE(8, 2)
    if constexpr (!BWD) DIT_NORM_CASE(8, 4)
    DIT_NORM_CASE(2, 4)
    DIT_NORM_CASE(2, 8)
    DIT_NORM_CASE(1, 8)
    DIT_NORM_CASE(1, 16)
#undef DIT_NORM_CASE
    return cudaErrorInvalidValue;
}

template <bool BWD>
cudaError_t pick_types(const NormArgs& a, const NormPlan& p, bool x_f32, bool y_f32, cudaStream_t s) {
    if (x_f32) return y_f32 ? pick<float, float, BWD>(a, p, s) : pick<float, uint16_t, BWD>(a, p, s);
    return y_f32 ? cudaErrorInvalidValue : pick<uint16_t, uint16_t, BWD>(a, p, s);
}

}  // namespace

// Channels a thread: forward 32 (16 without 16-byte loads), so that a row of
// 4,096 is four warps' and one of 1,024 a single warp's, without a barrier:
// 68 us for 24,576 x 4,096 bf16 against 101 with 16 a thread and 167 with 8;
// halved while rows are so few that the SMs would not get 512 threads each.
// Backward 16: its sums over rows hold two registers a channel (111 us there; 32
// spill), and 8 where rows are read channel by channel (24,576 x 4,095: 240 us
// against 550, whose prefetched row spills).
// A row's threads are whole warps and not a power of two: 24,576 x 2,560 takes
// 54 and 75 us (floor 37 and 56) against 61 and 101 with 128 and 256 threads.
// 512 threads an SM either way: forward in blocks of up to 128 (a row's threads
// when those are more), backward in one block, which leaves one partial (1,024
// threads an SM measured 127 us, for its partials).  Above 4,096 channels the
// backward pass has one group of threads on an SM; up to 6,144 it takes two rows
// at a time: 24,576 x 5,120 159 us (floor 111) against 188 one by one, 205 with 640
// threads of 8 channels and 240 with two rows of those.
NormPlan norm_plan(int C, uint32_t groups, uint32_t rows_per_group, int vec_max, int sms, bool backward) {
    NormPlan p;
    p.vec = vec_max;
    int per = backward || vec_max < 8 ? 16 : 32;
    if (backward && vec_max == 1 && C <= 8 * kMaxThreads) per = 8;
    const uint64_t rows = static_cast<uint64_t>(groups) * rows_per_group;
    while (per > 8 && rows * ((C + per - 1) / per) < static_cast<uint64_t>(sms) * 512 && C <= per / 2 * kMaxThreads) per /= 2;
    p.nv = per / p.vec;
    const int need_threads = (C + per - 1) / per;
    p.tpr = (need_threads + 31) / 32 * 32;
    if (need_threads <= 32)
        for (p.tpr = 1; p.tpr < need_threads;) p.tpr *= 2;
    // never more row slots than rows, but whole warps
    uint32_t slots = static_cast<uint32_t>((backward ? kMaxThreads : 128) / p.tpr);
    if (slots > rows_per_group) slots = rows_per_group;
    if (slots < 1) slots = 1;
    p.threads = (static_cast<int>(slots) * p.tpr + 31) / 32 * 32;
    slots = static_cast<uint32_t>(p.threads / p.tpr);
    p.two_rows = backward && p.vec == 8 && p.nv == 2 && p.tpr > kMaxThreads / 2 && p.tpr <= kTwoRowThreads && rows_per_group > 1;
    if (p.two_rows) slots *= 2;
    const uint64_t need = (rows_per_group + slots - 1) / slots;
    uint64_t blocks = (static_cast<uint64_t>(sms) * (512 / p.threads) + groups - 1) / groups;
    if (blocks > need) blocks = need;
    p.blocks = static_cast<int>(blocks < 1 ? 1 : blocks);
    return p;
}

cudaError_t launch_layer_norm_fwd(const NormArgs& a, const NormPlan& p, bool in_f32, bool out_f32, cudaStream_t s) {
    return pick_types<false>(a, p, in_f32, out_f32, s);
}

cudaError_t launch_layer_norm_bwd(const NormArgs& a, const NormPlan& p, bool in_f32, bool out_f32, cudaStream_t s) {
    return pick_types<true>(a, p, in_f32, out_f32, s);
}

}  // namespace dit

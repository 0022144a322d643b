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
// and dy and writes dx.  A row is held in the registers of `tpr` threads, at
// most 16 channels each, so the variance takes a second pass over registers
// and not over memory.  A thread keeps its channels while it walks over rows:
// their weights stay in registers, and so do the backward pass' sums over
// rows, which leave the block once, as one partial per block, summed in a
// fixed order by a second kernel (no atomics: results repeat bit for bit).
// The next row's loads are issued before the current row is reduced.
#include <cuda_runtime.h>

#include <cstdint>

#include "internal.h"
#include "train.h"

namespace dit {
namespace {

constexpr int kMaxThreads = 512;

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
    __device__ __forceinline__ float get(int i) const {
        if constexpr (sizeof(T) == 4) return __uint_as_float(w[i]);
        else return __uint_as_float((i & 1) ? (w[i >> 1] & 0xFFFF0000u) : (w[i >> 1] << 16));
    }
    static __device__ __forceinline__ void store(T* p, const float (&v)[VEC]) {
        Row r;
        if constexpr (sizeof(T) == 4) {
#pragma unroll
            for (int i = 0; i < VEC; ++i) r.w[i] = __float_as_uint(v[i]);
        } else {
#pragma unroll
            for (int i = 0; i < kWords; ++i) {
                const float lo = v[VEC > 1 ? 2 * i : 0], hi = VEC > 1 ? v[VEC > 1 ? 2 * i + 1 : 0] : 0.f;
                asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r.w[i]) : "f"(hi), "f"(lo));
            }
        }
        if constexpr (kBytes >= 16) {
#pragma unroll
            for (int i = 0; i < kWords / 4; ++i)
                __stcs(reinterpret_cast<uint4*>(p) + i, make_uint4(r.w[4 * i], r.w[4 * i + 1], r.w[4 * i + 2], r.w[4 * i + 3]));
        } else if constexpr (kBytes == 8) {
            __stcs(reinterpret_cast<uint2*>(p), make_uint2(r.w[0], r.w[1]));
        } else if constexpr (kBytes == 4) {
            __stcs(reinterpret_cast<uint32_t*>(p), r.w[0]);
        } else {
            __stcs(reinterpret_cast<unsigned short*>(p), static_cast<unsigned short>(r.w[0]));
        }
    }
};

// A thread's own ring of P staged rows in shared memory, filled by asynchronous
// copies of its channels (no other thread reads them, so waiting for its own
// copies is all the synchronisation there is).  Loads of single bf16 channels
// are below the smallest asynchronous copy: those are loaded when their row is
// due (a depth of one).
template <typename T, int VEC, int NV>
struct Ring {
    using R = Row<T, VEC>;
    static constexpr bool kAsync = R::kBytes >= 4;
    static constexpr int kChunk = R::kBytes < 16 ? R::kBytes : 16;    // bytes of one copy
    static constexpr int kChunks = kAsync ? R::kBytes / kChunk : 1;
    static constexpr int kStageBytes = NV * R::kBytes;                // per thread
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

// Rows staged ahead: as many as keep some 64 bytes a thread and direction in
// flight without holding more than half an SM's shared memory per 512 threads.
#ifndef DIT_NORM_STAGE_BYTES
#define DIT_NORM_STAGE_BYTES 128
#endif
__host__ __device__ constexpr int ring_depth(int stage_bytes, bool async) {
    if (!async) return 1;
    const int p = DIT_NORM_STAGE_BYTES / stage_bytes;
    return p < 2 ? 2 : (p > 6 ? 6 : p);
}

// Packed pairs of fp32 operations: the kernels are bound by instructions as
// much as by memory, and these halve the arithmetic.
__device__ __forceinline__ void add2(float& d0, float& d1, float a0, float a1, float b0, float b1) {
    asm("{\n\t.reg .b64 a, b;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\tadd.rn.f32x2 a, a, b;\n\tmov.b64 {%0, %1}, a;\n\t}"
        : "=f"(d0), "=f"(d1) : "f"(a0), "f"(a1), "f"(b0), "f"(b1));
}
__device__ __forceinline__ void mul2(float& d0, float& d1, float a0, float a1, float b0, float b1) {
    asm("{\n\t.reg .b64 a, b;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\tmul.rn.f32x2 a, a, b;\n\tmov.b64 {%0, %1}, a;\n\t}"
        : "=f"(d0), "=f"(d1) : "f"(a0), "f"(a1), "f"(b0), "f"(b1));
}
__device__ __forceinline__ void fma2(float& d0, float& d1, float a0, float a1, float b0, float b1, float c0, float c1) {
    asm("{\n\t.reg .b64 a, b, c;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\tmov.b64 c, {%6, %7};\n\tfma.rn.f32x2 a, a, b, c;\n\tmov.b64 {%0, %1}, a;\n\t}"
        : "=f"(d0), "=f"(d1) : "f"(a0), "f"(a1), "f"(b0), "f"(b1), "f"(c0), "f"(c1));
}

// The threads of one row: `tpr` of them (a power of two), whole warps when
// tpr > 32.  Sums over the row reach every thread in the same order.
struct RowGroup {
    int tpr, t, id;             // threads per row, index in the row, row slot of the block
    int warps;                  // warps of a row (1 when tpr <= 32)
    float2* buf;                // [2][kMaxThreads / 32] cross-warp partials
    int flip;
    __device__ RowGroup(int tpr_, float2* b)
        : tpr(tpr_), t(threadIdx.x & (tpr_ - 1)), id(threadIdx.x / tpr_), warps(tpr_ > 32 ? tpr_ >> 5 : 1), buf(b), flip(0) {}
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
    // Each warp's pair to the row's other warps: lane l gets that of warp
    // l mod warps.  One barrier among the row's threads; the other buffer is
    // written next, so a second is not needed.
    __device__ __forceinline__ float2 exchange(float2 v) {
        float2* const b = buf + flip * (kMaxThreads / 32);
        flip ^= 1;
        if ((threadIdx.x & 31) == 0) b[threadIdx.x >> 5] = v;
        asm volatile("bar.sync %0, %1;" ::"r"(1 + id), "r"(tpr) : "memory");
        return b[id * warps + (threadIdx.x & (warps - 1))];
    }
    // Sum of what exchange() handed out, over the row's warps.
    __device__ __forceinline__ float across(float v) const {
        for (int o = warps >> 1; o >= 1; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
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

template <int VEC>
__device__ __forceinline__ void load_params(const float* p, float (&v)[VEC]) {
    if constexpr (VEC == 8) {
        const float4 lo = __ldg(reinterpret_cast<const float4*>(p)), hi = __ldg(reinterpret_cast<const float4*>(p) + 1);
        v[0] = lo.x; v[1] = lo.y; v[2] = lo.z; v[3] = lo.w; v[4] = hi.x; v[5] = hi.y; v[6] = hi.z; v[7] = hi.w;
    } else if constexpr (VEC == 2) {
        const float2 x = __ldg(reinterpret_cast<const float2*>(p));
        v[0] = x.x; v[1] = x.y;
    } else {
        v[0] = __ldg(p);
    }
}

// grid (blocks, groups).  Every thread of a block makes the same number of
// rounds; a row slot past its last row runs along on zeros.
template <typename TX, typename TY, int VEC, int NV>
__global__ void __launch_bounds__(kMaxThreads) layer_norm_fwd_kernel(const NormArgs a, int tpr) {
    using RX = Ring<TX, VEC, NV>;
    constexpr int P = ring_depth(RX::kStageBytes, RX::kAsync);
    __shared__ float2 buf[2 * kMaxThreads / 32];
    extern __shared__ __align__(16) uint8_t ring_mem[];
    RowGroup g(tpr, buf);
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
        }
        ring_commit();
    };
    for (int k = 0; k < P - 1; ++k) fetch(k);
    float w[NV][VEC], bi[NV][VEC];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
#pragma unroll
        for (int e = 0; e < VEC; ++e) { w[i][e] = 1.f; bi[i][e] = 0.f; }
        if (live[i] && a.weight) load_params<VEC>(a.weight + static_cast<int64_t>(blockIdx.y) * a.C + col[i], w[i]);
        if (live[i] && a.bias) load_params<VEC>(a.bias + static_cast<int64_t>(blockIdx.y) * a.C + col[i], bi[i]);
    }
    // Channels held by warp v of a row, 1 / that (0 for none): by this thread's
    // own warp, and by the warp whose pair exchange() hands this lane.
    auto held = [&](int v) {
        int n = 0;
#pragma unroll
        for (int i = 0; i < NV; ++i) n += min(max(a.C - (i * tpr + 32 * v) * VEC, 0), 32 * VEC);
        return static_cast<float>(n);
    };
    const float own_n = tpr > 32 ? held(g.t >> 5) : static_cast<float>(a.C);
    const float own_inv = own_n > 0.f ? 1.f / own_n : 0.f;
    const float got_n = tpr > 32 ? held(threadIdx.x & (g.warps - 1)) : 0.f;
    const float got_inv = got_n > 0.f ? 1.f / got_n : 0.f;

    uint32_t r = first;
    for (uint32_t k = 0; k < rounds; ++k, r += step) {
        fetch(k + P - 1);
        ring_wait<P - 1>();
        const bool ok = r < a.rows_per_group;
        float x[NV][VEC];
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            if (ok && live[i]) {
                const Row<TX, VEC> v = ring.take(k % P, i);
#pragma unroll
                for (int e = 0; e < VEC; ++e) x[i][e] = v.get(e);
            } else {
#pragma unroll
                for (int e = 0; e < VEC; ++e) x[i][e] = 0.f;
            }
        }
        // This warp's mean and sum of squared deviations from it, then the row's
        // from all its warps': sum of (their deviations + n (their mean - mean)^2).
        float mean = 0.f, s = 0.f;
        if (a.center) {
            float s0 = 0.f, s1 = 0.f;
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                if constexpr (VEC == 1) s0 += x[i][0];
                else
#pragma unroll
                    for (int e = 0; e < VEC; e += 2) add2(s0, s1, s0, s1, x[i][e], x[i][e + 1]);
            }
            s = g.lanes(s0 + s1);
            mean = s * own_inv;
        }
        float q0 = 0.f, q1 = 0.f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            if constexpr (VEC == 1) {
                x[i][0] = live[i] ? x[i][0] - mean : 0.f;
                q0 = fmaf(x[i][0], x[i][0], q0);
            } else if (live[i]) {
#pragma unroll
                for (int e = 0; e < VEC; e += 2) {
                    add2(x[i][e], x[i][e + 1], x[i][e], x[i][e + 1], -mean, -mean);
                    fma2(q0, q1, x[i][e], x[i][e + 1], x[i][e], x[i][e + 1], q0, q1);
                }
            }
        }
        float q = g.lanes(q0 + q1);
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
            const float sr = shift * rstd;
#pragma unroll
            for (int i = 0; i < NV; ++i)
                if (live[i]) {
                    float v[VEC];
                    if constexpr (VEC == 1) {
                        v[0] = fmaf(fmaf(x[i][0], rstd, sr), w[i][0], bi[i][0]);
                    } else {
#pragma unroll
                        for (int e = 0; e < VEC; e += 2) {
                            fma2(v[e], v[e + 1], x[i][e], x[i][e + 1], rstd, rstd, sr, sr);
                            fma2(v[e], v[e + 1], v[e], v[e + 1], w[i][e], w[i][e + 1], bi[i][e], bi[i][e + 1]);
                        }
                    }
                    Row<TY, VEC>::store(p + col[i], v);
                }
            if (g.t == 0) {
                if (a.center) a.mean[row0 + r] = mean;
                a.rstd[row0 + r] = rstd;
            }
        }
    }
}

template <typename TX, typename TY, int VEC, int NV>
__global__ void __launch_bounds__(kMaxThreads) layer_norm_bwd_kernel(const NormArgs a, int tpr) {
    using RX = Ring<TX, VEC, NV>;
    using RD = Ring<TY, VEC, NV>;
    constexpr int P = ring_depth(RX::kStageBytes + RD::kStageBytes, RX::kAsync && RD::kAsync);
    __shared__ float2 buf[2 * kMaxThreads / 32];
    extern __shared__ __align__(16) uint8_t ring_mem[];   // the rings; after the rows, [slots][tpr * NV * VEC] sums
    float* const acc = reinterpret_cast<float*>(ring_mem);
    RowGroup g(tpr, buf);
    RX rx;
    RD rd;
    rx.init(ring_mem);
    rd.init(ring_mem + (RX::kAsync ? P * RX::kStageBytes * blockDim.x : 0));
    const RowAt x_at(a, a.sx), d_at(a, a.sdy), y_at(a, a.sy);
    const uint32_t slots = blockDim.x / tpr;
    const uint32_t step = gridDim.x * slots;
    const uint32_t row0 = blockIdx.y * a.rows_per_group;
    const uint32_t rounds = (a.rows_per_group - blockIdx.x * slots + step - 1) / step;
    const uint32_t first = blockIdx.x * slots + g.id;
    bool live[NV];
    int col[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        col[i] = (i * tpr + g.t) * VEC;
        live[i] = col[i] < a.C;
    }
    float nmean = 0.f, nrstd = 0.f;
    auto stats = [&](uint32_t k) {       // of round k, read one round ahead
        const uint32_t r = first + k * step;
        const bool ok = k < rounds && r < a.rows_per_group;
        nmean = ok && a.center ? __ldg(a.mean + row0 + r) : 0.f;
        nrstd = ok ? __ldg(a.rstd + row0 + r) : 0.f;
    };
    auto fetch = [&](uint32_t k) {
        const uint32_t r = first + k * step;
        if (k < rounds && r < a.rows_per_group) {
            const TX* p = static_cast<const TX*>(a.x) + x_at(a, row0 + r);
            const TY* d = static_cast<const TY*>(a.dy) + d_at(a, row0 + r);
#pragma unroll
            for (int i = 0; i < NV; ++i)
                if (live[i]) {
                    rx.fetch(k % P, i, p + col[i]);
                    rd.fetch(k % P, i, d + col[i]);
                }
        }
        ring_commit();
    };
    for (int k = 0; k < P - 1; ++k) fetch(k);
    stats(0);
    float w[NV][VEC], dw[NV][VEC], db[NV][VEC];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
#pragma unroll
        for (int e = 0; e < VEC; ++e) { w[i][e] = 1.f; dw[i][e] = 0.f; db[i][e] = 0.f; }
        if (live[i] && a.weight) load_params<VEC>(a.weight + static_cast<int64_t>(blockIdx.y) * a.C + col[i], w[i]);
    }
    uint32_t r = first;
    for (uint32_t k = 0; k < rounds; ++k, r += step) {
        fetch(k + P - 1);
        ring_wait<P - 1>();
        const bool ok = r < a.rows_per_group;
        const float rstd = nrstd, mr = -nmean * nrstd;
        stats(k + 1);
        float xh[NV][VEC], gr[NV][VEC];      // xh and g, kept for dx
        float s0 = 0.f, s1 = 0.f, t0 = 0.f, t1 = 0.f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            Row<TX, VEC> x;
            Row<TY, VEC> d;
            x.zero();
            d.zero();
            if (ok && live[i]) { x = rx.take(k % P, i); d = rd.take(k % P, i); }
            if constexpr (VEC == 1) {
                const float dy = d.get(0);
                xh[i][0] = fmaf(x.get(0), rstd, mr);
                gr[i][0] = dy * w[i][0];
                s0 += gr[i][0];
                t0 = fmaf(gr[i][0], xh[i][0], t0);
                dw[i][0] = fmaf(dy, xh[i][0], dw[i][0]);
                db[i][0] += dy;
            } else {
#pragma unroll
                for (int e = 0; e < VEC; e += 2) {
                    const float d0 = d.get(e), d1 = d.get(e + 1);
                    fma2(xh[i][e], xh[i][e + 1], x.get(e), x.get(e + 1), rstd, rstd, mr, mr);
                    mul2(gr[i][e], gr[i][e + 1], d0, d1, w[i][e], w[i][e + 1]);
                    add2(s0, s1, s0, s1, gr[i][e], gr[i][e + 1]);
                    fma2(t0, t1, gr[i][e], gr[i][e + 1], xh[i][e], xh[i][e + 1], t0, t1);
                    fma2(dw[i][e], dw[i][e + 1], d0, d1, xh[i][e], xh[i][e + 1], dw[i][e], dw[i][e + 1]);
                    add2(db[i][e], db[i][e + 1], db[i][e], db[i][e + 1], d0, d1);
                }
            }
        }
        float sg = a.center ? g.lanes(s0 + s1) : 0.f;
        float st = g.lanes(t0 + t1);
        if (tpr > 32) {
            const float2 p = g.exchange(make_float2(sg, st));
            if (a.center) sg = g.across(p.x);
            st = g.across(p.y);
        }
        // dx = rstd g - rstd c1 - xh (rstd c2)
        const float n1 = -sg * a.inv_c * rstd, n2 = -st * a.inv_c * rstd;
        if (ok) {
            TX* const p = static_cast<TX*>(a.y) + y_at(a, row0 + r);
#pragma unroll
            for (int i = 0; i < NV; ++i)
                if (live[i]) {
                    float v[VEC];
                    if constexpr (VEC == 1) {
                        v[0] = fmaf(gr[i][0], rstd, fmaf(xh[i][0], n2, n1));
                    } else {
#pragma unroll
                        for (int e = 0; e < VEC; e += 2) {
                            fma2(v[e], v[e + 1], xh[i][e], xh[i][e + 1], n2, n2, n1, n1);
                            fma2(v[e], v[e + 1], gr[i][e], gr[i][e + 1], rstd, rstd, v[e], v[e + 1]);
                        }
                    }
                    Row<TX, VEC>::store(p + col[i], v);
                }
        }
    }
    ring_wait<0>();
    // The block's sums: row slots added in order, then one partial per block
    // (the gradient itself when the group has one block).
    const int width = tpr * NV * VEC;
    auto leave = [&](float (&v)[NV][VEC], float* part, float* grad) {
        float* const out = gridDim.x == 1 ? grad + static_cast<int64_t>(blockIdx.y) * a.C
                                          : part + (static_cast<int64_t>(blockIdx.y) * gridDim.x + blockIdx.x) * a.C;
        if (slots == 1) {
#pragma unroll
            for (int i = 0; i < NV; ++i)
                if (live[i])
#pragma unroll
                    for (int e = 0; e < VEC; ++e) out[col[i] + e] = v[i][e];
            return;
        }
        __syncthreads();     // the rings (or the last sums) have been read
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int e = 0; e < VEC; ++e) acc[g.id * width + col[i] + e] = v[i][e];
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
// column's in a fixed order: 8 interleaved sums, then those in order.
__global__ void __launch_bounds__(256) layer_norm_param_sum_kernel(const NormArgs a, int parts) {
    __shared__ float s[8][33];
    const int cx = threadIdx.x & 31, py = threadIdx.x >> 5;
    const int c = blockIdx.x * 32 + cx;
    const bool second = blockIdx.z != 0 || !a.want_w;
    float* const out = second ? a.dbias : a.dweight;
    const float* const p = a.part + (static_cast<int64_t>(second ? a.groups : 0) + blockIdx.y) * parts * a.C;
    float t = 0.f;
    if (c < a.C)
        for (int k = py; k < parts; k += 8) t += __ldcs(p + static_cast<int64_t>(k) * a.C + c);
    s[py][cx] = t;
    __syncthreads();
    if (py == 0 && c < a.C) {
#pragma unroll
        for (int k = 1; k < 8; ++k) t += s[k][cx];
        out[static_cast<int64_t>(blockIdx.y) * a.C + c] = t;
    }
}

template <typename TX, typename TY, int VEC, int NV>
cudaError_t fwd(const NormArgs& a, const NormPlan& p, cudaStream_t s) {
    using RX = Ring<TX, VEC, NV>;
    const int smem = RX::kAsync ? ring_depth(RX::kStageBytes, true) * RX::kStageBytes * p.threads : 0;
    auto kern = layer_norm_fwd_kernel<TX, TY, VEC, NV>;
    if (smem > 47 * 1024) {
        const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (e != cudaSuccess) return e;
    }
    kern<<<dim3(p.blocks, a.groups), p.threads, smem, s>>>(a, p.tpr);
    return cudaGetLastError();
}

template <typename TX, typename TY, int VEC, int NV>
cudaError_t bwd(const NormArgs& a, const NormPlan& p, cudaStream_t s) {
    using RX = Ring<TX, VEC, NV>;
    using RD = Ring<TY, VEC, NV>;
    const int depth = ring_depth(RX::kStageBytes + RD::kStageBytes, RX::kAsync && RD::kAsync);
    const int rings = ((RX::kAsync ? RX::kStageBytes : 0) + (RD::kAsync ? RD::kStageBytes : 0)) * depth * p.threads;
    const int sums = p.threads > p.tpr ? p.threads * NV * VEC * static_cast<int>(sizeof(float)) : 0;
    const int smem = rings > sums ? rings : sums;
    auto kern = layer_norm_bwd_kernel<TX, TY, VEC, NV>;
    if (smem > 47 * 1024) {
        const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (e != cudaSuccess) return e;
    }
    kern<<<dim3(p.blocks, a.groups), p.threads, smem, s>>>(a, p.tpr);
    cudaError_t e = cudaGetLastError();
    const int wants = (a.want_w ? 1 : 0) + (a.want_b ? 1 : 0);
    if (e != cudaSuccess || p.blocks == 1 || wants == 0) return e;
    layer_norm_param_sum_kernel<<<dim3((a.C + 31) / 32, a.groups, wants), 256, 0, s>>>(a, p.blocks);
    return cudaGetLastError();
}

template <typename TX, typename TY, bool BWD>
cudaError_t pick(const NormArgs& a, const NormPlan& p, cudaStream_t s) {
#define DIT_NORM_CASE(V, N) \
    if (p.vec == V && p.nv == N) return BWD ? bwd<TX, TY, V, N>(a, p, s) : fwd<TX, TY, V, N>(a, p, s);
    DIT_NORM_CASE(8, 1)
    DIT_NORM_CASE(8, 2)
    DIT_NORM_CASE(8, 4)
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
// 70 us for 24,576 x 4,096 bf16 against 101 with 16 a thread and 167 with 8; halved
// while rows are so few that the SMs would not get 512 threads each.  Backward
// 16: its sums over rows hold two registers a channel (120 us there; 32 spill).
// 512 threads an SM either way: forward in blocks of 128 (a row's threads when
// those are more), backward in one block, which leaves one partial (1,024 threads
// an SM measured 127 us, for its partials).
NormPlan norm_plan(int C, uint32_t groups, uint32_t rows_per_group, int vec_max, int sms, bool backward) {
    NormPlan p;
    p.vec = vec_max;
    int per = backward || vec_max < 8 ? 16 : 32;
    const uint64_t rows = static_cast<uint64_t>(groups) * rows_per_group;
    while (per > 8 && rows * ((C + per - 1) / per) < static_cast<uint64_t>(sms) * 512 && C <= per / 2 * kMaxThreads) per /= 2;
    p.nv = per / p.vec;
    p.tpr = 1;
    while (p.tpr * per < C) p.tpr *= 2;
    p.threads = backward ? kMaxThreads : 128;
    if (p.threads < p.tpr) p.threads = p.tpr;
    // never more row slots than rows
    while (p.threads > 32 && p.threads > p.tpr && static_cast<uint32_t>(p.threads / p.tpr) > rows_per_group) p.threads /= 2;
    const uint32_t slots = static_cast<uint32_t>(p.threads / p.tpr);
    const uint64_t need = (rows_per_group + slots - 1) / slots;
    uint64_t blocks = (static_cast<uint64_t>(sms) * 512 / p.threads + groups - 1) / groups;
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

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

// The threads of one row: `tpr` of them (a power of two), warp-aligned when
// tpr > 32.  Sums over the row reach every thread in the same order.
struct RowGroup {
    int tpr, t, id;             // threads per row, index in the row, row slot of the block
    float2* buf;                // [2][kMaxThreads / 32] cross-warp partials
    int flip;
    __device__ RowGroup(int tpr_, float2* b) : tpr(tpr_), t(threadIdx.x & (tpr_ - 1)), id(threadIdx.x / tpr_), buf(b), flip(0) {}
    __device__ __forceinline__ float2 sum(float2 v) {
        const int lim = tpr < 32 ? tpr : 32;
        // lanes of one warp may belong to row slots that have run out of rows:
        // every lane of a block takes part in every sum
        for (int o = lim >> 1; o >= 1; o >>= 1) {
            v.x += __shfl_xor_sync(0xffffffffu, v.x, o);
            v.y += __shfl_xor_sync(0xffffffffu, v.y, o);
        }
        if (tpr > 32) {
            float2* const b = buf + flip * (kMaxThreads / 32);
            flip ^= 1;
            if ((threadIdx.x & 31) == 0) b[threadIdx.x >> 5] = v;
            __syncthreads();
            const int w0 = id * (tpr >> 5);
            v = b[w0];
            for (int w = 1; w < (tpr >> 5); ++w) {
                const float2 o = b[w0 + w];
                v.x += o.x;
                v.y += o.y;
            }
        }
        return v;
    }
};

__device__ __forceinline__ int64_t row_offset(const NormArgs& a, const dit_strides4_t& s, uint32_t row) {
    uint32_t nh, h;
    const uint32_t b = a.div_nh.divmod(row, nh);
    const uint32_t n = a.div_h.divmod(nh, h);
    return b * s.b + n * s.n + h * s.h;
}

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
    __shared__ float2 buf[2 * kMaxThreads / 32];
    RowGroup g(tpr, buf);
    const uint32_t slots = blockDim.x / tpr;
    const uint32_t step = gridDim.x * slots;
    const uint32_t row0 = blockIdx.y * a.rows_per_group;
    const uint32_t rounds = (a.rows_per_group - blockIdx.x * slots + step - 1) / step;   // >= 1: blocks * slots <= rows
    float w[NV][VEC], bi[NV][VEC];
    bool live[NV];
    int col[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        col[i] = (i * tpr + g.t) * VEC;
        live[i] = col[i] < a.C;
#pragma unroll
        for (int e = 0; e < VEC; ++e) { w[i][e] = 1.f; bi[i][e] = 0.f; }
        if (live[i] && a.weight) load_params<VEC>(a.weight + static_cast<int64_t>(blockIdx.y) * a.C + col[i], w[i]);
        if (live[i] && a.bias) load_params<VEC>(a.bias + static_cast<int64_t>(blockIdx.y) * a.C + col[i], bi[i]);
    }
    Row<TX, VEC> nx[NV];
    auto load = [&](uint32_t r) {
        const bool ok = r < a.rows_per_group;
        const TX* p = static_cast<const TX*>(a.x) + (ok ? row_offset(a, a.sx, row0 + r) : 0);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            if (ok && live[i]) nx[i].load(p + col[i]);
            else nx[i].zero();
        }
    };
    uint32_t r = blockIdx.x * slots + g.id;
    load(r);
    for (uint32_t k = 0; k < rounds; ++k, r += step) {
        Row<TX, VEC> x[NV];
#pragma unroll
        for (int i = 0; i < NV; ++i) x[i] = nx[i];
        if (k + 1 < rounds) load(r + step);
        float mean = 0.f;
        if (a.center) {
            float s = 0.f;
#pragma unroll
            for (int i = 0; i < NV; ++i)
#pragma unroll
                for (int e = 0; e < VEC; ++e) s += x[i].get(e);
            mean = g.sum(make_float2(s, 0.f)).x * a.inv_c;
        }
        float q = 0.f;
#pragma unroll
        for (int i = 0; i < NV; ++i)
            if (live[i])
#pragma unroll
                for (int e = 0; e < VEC; ++e) {
                    const float d = x[i].get(e) - mean;
                    q = fmaf(d, d, q);
                }
        const float var = g.sum(make_float2(q, 0.f)).x * a.inv_c;
        const float rstd = 1.f / sqrtf(var + a.eps);
        if (r < a.rows_per_group) {
            TY* const p = static_cast<TY*>(a.y) + row_offset(a, a.sy, row0 + r);
#pragma unroll
            for (int i = 0; i < NV; ++i)
                if (live[i]) {
                    float v[VEC];
#pragma unroll
                    for (int e = 0; e < VEC; ++e) v[e] = fmaf((x[i].get(e) - mean) * rstd, w[i][e], bi[i][e]);
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
    __shared__ float2 buf[2 * kMaxThreads / 32];
    extern __shared__ float acc[];      // [slots][tpr * NV * VEC], several row slots only
    RowGroup g(tpr, buf);
    const uint32_t slots = blockDim.x / tpr;
    const uint32_t step = gridDim.x * slots;
    const uint32_t row0 = blockIdx.y * a.rows_per_group;
    const uint32_t rounds = (a.rows_per_group - blockIdx.x * slots + step - 1) / step;
    float w[NV][VEC], dw[NV][VEC], db[NV][VEC];
    bool live[NV];
    int col[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        col[i] = (i * tpr + g.t) * VEC;
        live[i] = col[i] < a.C;
#pragma unroll
        for (int e = 0; e < VEC; ++e) { w[i][e] = 1.f; dw[i][e] = 0.f; db[i][e] = 0.f; }
        if (live[i] && a.weight) load_params<VEC>(a.weight + static_cast<int64_t>(blockIdx.y) * a.C + col[i], w[i]);
    }
    Row<TX, VEC> nx[NV];
    Row<TY, VEC> nd[NV];
    float nmean = 0.f, nrstd = 0.f;
    auto load = [&](uint32_t r) {
        const bool ok = r < a.rows_per_group;
        const TX* p = static_cast<const TX*>(a.x) + (ok ? row_offset(a, a.sx, row0 + r) : 0);
        const TY* d = static_cast<const TY*>(a.dy) + (ok ? row_offset(a, a.sdy, row0 + r) : 0);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            if (ok && live[i]) { nx[i].load(p + col[i]); nd[i].load(d + col[i]); }
            else { nx[i].zero(); nd[i].zero(); }
        }
        nmean = ok && a.center ? __ldg(a.mean + row0 + r) : 0.f;
        nrstd = ok ? __ldg(a.rstd + row0 + r) : 0.f;
    };
    uint32_t r = blockIdx.x * slots + g.id;
    load(r);
    for (uint32_t k = 0; k < rounds; ++k, r += step) {
        Row<TX, VEC> x[NV];
        Row<TY, VEC> d[NV];
#pragma unroll
        for (int i = 0; i < NV; ++i) { x[i] = nx[i]; d[i] = nd[i]; }
        const float mean = nmean, rstd = nrstd;
        if (k + 1 < rounds) load(r + step);
        float2 s = make_float2(0.f, 0.f);
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                const float xh = (x[i].get(e) - mean) * rstd, dy = d[i].get(e);
                const float gg = dy * w[i][e];
                s.x += gg;
                s.y = fmaf(gg, xh, s.y);
                dw[i][e] = fmaf(dy, xh, dw[i][e]);
                db[i][e] += dy;
            }
        s = g.sum(s);
        const float c1 = a.center ? s.x * a.inv_c : 0.f, c2 = s.y * a.inv_c;
        if (r < a.rows_per_group) {
            TX* const p = static_cast<TX*>(a.y) + row_offset(a, a.sy, row0 + r);
#pragma unroll
            for (int i = 0; i < NV; ++i)
                if (live[i]) {
                    float v[VEC];
#pragma unroll
                    for (int e = 0; e < VEC; ++e) {
                        const float xh = (x[i].get(e) - mean) * rstd;
                        v[e] = rstd * (fmaf(-xh, c2, d[i].get(e) * w[i][e]) - c1);
                    }
                    Row<TX, VEC>::store(p + col[i], v);
                }
        }
    }
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
        __syncthreads();
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
    layer_norm_fwd_kernel<TX, TY, VEC, NV><<<dim3(p.blocks, a.groups), p.threads, 0, s>>>(a, p.tpr);
    return cudaGetLastError();
}

template <typename TX, typename TY, int VEC, int NV>
cudaError_t bwd(const NormArgs& a, const NormPlan& p, cudaStream_t s) {
    const size_t smem = p.threads > p.tpr ? static_cast<size_t>(p.threads) * NV * VEC * sizeof(float) : 0;
    layer_norm_bwd_kernel<TX, TY, VEC, NV><<<dim3(p.blocks, a.groups), p.threads, smem, s>>>(a, p.tpr);
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

NormPlan norm_plan(int C, uint32_t groups, uint32_t rows_per_group, int vec_max, int sms, bool backward) {
    NormPlan p;
    p.vec = vec_max;
    // 8 channels a thread while a row then fits one block's 512 threads, else 16
    int per = C <= 8 * kMaxThreads ? 8 : 16;
    p.nv = per / p.vec;
    p.tpr = 1;
    while (p.tpr * per < C) p.tpr *= 2;
    // Blocks of several rows (256 threads; 512 when one row needs them), never
    // more row slots than rows.
    p.threads = p.tpr > 256 ? p.tpr : 256;
    while (p.threads > 32 && p.threads > p.tpr && static_cast<uint32_t>(p.threads / p.tpr) > rows_per_group) p.threads /= 2;
    if (p.threads < 32) p.threads = 32;
    const uint32_t slots = static_cast<uint32_t>(p.threads / p.tpr);
    const uint64_t need = (rows_per_group + slots - 1) / slots;
    // Backward: a block leaves a partial of C sums, so few, long-lived blocks;
    // forward: as many as are resident.
    const uint64_t resident = static_cast<uint64_t>(sms) * (backward ? 1024 : 2048) / p.threads;
    uint64_t blocks = (resident + groups - 1) / groups;
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

// rope.cu -- rotary positions of a strided [B, N, H, D] view.
//
// Pair i of the first 2 * pairs channels of every head turns by the angle
// theta = position * inv_freq_i:
//   (a, b) -> mscale * (a cos theta - b sin theta, a sin theta + b cos theta),
// with (a, b) = channels (2i, 2i+1) in the interleaved layout and
// (i, i + pairs) in the half layout; the other channels are copied.  The
// inverse turns by -theta, which is the gradient (the transpose).
//
// Angles: only theta / 2 pi modulo 1 matters, so inv_freq_i / 2 pi modulo 1 is
// held as a 64-bit fraction and multiplied by the integer position modulo
// 2^64 -- the wrap-around is the range reduction, exact at any 32-bit
// position (the fraction's rounding moves an angle by at most 2 pi * 2^-65
// per step, and the caller's fp64 frequency by 2^-53 of itself).  The upper
// 32 bits, rounded, go to sincospif as half turns in [-1, 1).
//
// HBM-bound: every element is read once and written once; positions are 4
// bytes a token.  A block takes `tokens` tokens: the cos/sin of their pairs
// are computed once into shared memory and used by all heads, while the first
// loads of x are already in flight.
#include <cuda_runtime.h>

#include <cstdint>

#include "internal.h"
#include "train.h"

namespace dit {
namespace {

constexpr int kThreads = 256;
constexpr int kUnroll = 4;              // units in flight per thread
constexpr int kMaxAngles = 2048;        // cos/sin pairs a block holds (16 KB)

template <typename T> struct IsF32 { static constexpr bool value = false; };
template <> struct IsF32<float> { static constexpr bool value = true; };

// `VEC` elements as raw 32-bit words (or one 16-bit element).
template <typename T, int VEC>
struct Pack {
    static constexpr int kBytes = static_cast<int>(sizeof(T)) * VEC;
    static constexpr int kWords = kBytes >= 4 ? kBytes / 4 : 1;
    uint32_t w[kWords];
    __device__ __forceinline__ void load(const T* p) {
        if constexpr (kBytes == 16) {
            const uint4 v = __ldcs(reinterpret_cast<const uint4*>(p));
            w[0] = v.x; w[1] = v.y; w[2] = v.z; w[3] = v.w;
        } else if constexpr (kBytes == 8) {
            const uint2 v = __ldcs(reinterpret_cast<const uint2*>(p));
            w[0] = v.x; w[1] = v.y;
        } else if constexpr (kBytes == 4) {
            w[0] = __ldcs(reinterpret_cast<const uint32_t*>(p));
        } else {
            w[0] = __ldcs(reinterpret_cast<const unsigned short*>(p));
        }
    }
    __device__ __forceinline__ void store(T* p) const {
        if constexpr (kBytes == 16) __stcs(reinterpret_cast<uint4*>(p), make_uint4(w[0], w[1], w[2], w[3]));
        else if constexpr (kBytes == 8) __stcs(reinterpret_cast<uint2*>(p), make_uint2(w[0], w[1]));
        else if constexpr (kBytes == 4) __stcs(reinterpret_cast<uint32_t*>(p), w[0]);
        else __stcs(reinterpret_cast<unsigned short*>(p), static_cast<unsigned short>(w[0]));
    }
    __device__ __forceinline__ float get(int i) const {
        if constexpr (IsF32<T>::value) return __uint_as_float(w[i]);
        else return __uint_as_float((i & 1) ? (w[i >> 1] & 0xFFFF0000u) : (w[i >> 1] << 16));
    }
    // elements 2i and 2i+1 (or the single one), rounded once to T
    __device__ __forceinline__ void put_all(const float (&v)[VEC]) {
        if constexpr (IsF32<T>::value) {
#pragma unroll
            for (int i = 0; i < VEC; ++i) w[i] = __float_as_uint(v[i]);
        } else {
#pragma unroll
            for (int i = 0; i < kWords; ++i) {
                const float lo = v[2 * i < VEC ? 2 * i : 0], hi = 2 * i + 1 < VEC ? v[2 * i + 1 < VEC ? 2 * i + 1 : 0] : 0.f;
                asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w[i]) : "f"(hi), "f"(lo));
            }
        }
    }
};

// One unit of work is VEC channels (interleaved: whole pairs, VEC >= 2, the
// pairs past the rotated ones passing through) or VEC pairs of the half layout
// (VEC channels of the first half and their partners), or VEC channels to copy.
// With VEC = 1 the HALF form takes single pairs of either layout.
template <typename T, bool HALF, int VEC>
__global__ void __launch_bounds__(kThreads) rope_kernel(const RopeArgs a, FastDiv div_units, FastDiv div_h,
                                                        FastDiv div_pairs, int rot_units, int tokens, int blocks_per_b) {
    __shared__ float2 cs[kMaxAngles];
    const int b = static_cast<int>(blockIdx.x) / blocks_per_b;
    const int n0 = (static_cast<int>(blockIdx.x) - b * blocks_per_b) * tokens;
    const int nt = min(tokens, a.N - n0);
    const T* const x = static_cast<const T*>(a.x) + b * a.sx.b + n0 * a.sx.n;
    T* const y = static_cast<T*>(a.y) + b * a.sy.b + n0 * a.sy.n;
    const uint32_t units = div_units.d;
    const uint32_t total = static_cast<uint32_t>(nt) * static_cast<uint32_t>(a.H) * units;

    struct Where { int n, u; int64_t ox, oy; };
    auto where = [&](uint32_t i) {
        uint32_t u, h;
        const uint32_t nh = div_units.divmod(i, u);
        const uint32_t n = div_h.divmod(nh, h);
        Where w;
        w.n = static_cast<int>(n);
        w.u = static_cast<int>(u);
        // channel of the unit: a half-layout copy unit starts behind both halves
        const int c = (!HALF || w.u < rot_units) ? w.u * (VEC == 1 ? a.lone_step : VEC)
                                                 : 2 * a.pairs + (w.u - rot_units) * VEC;
        w.ox = n * a.sx.n + h * a.sx.h + c;
        w.oy = n * a.sy.n + h * a.sy.h + c;
        return w;
    };
    const int partner = VEC == 1 ? a.lone_partner : a.pairs;
    Pack<T, VEC> p[kUnroll], q[kUnroll];
    auto load = [&](uint32_t i0) {
#pragma unroll
        for (int k = 0; k < kUnroll; ++k) {
            const uint32_t i = i0 + k * kThreads;
            if (i < total) {
                const Where w = where(i);
                p[k].load(x + w.ox);
                if (HALF && w.u < rot_units) q[k].load(x + w.ox + partner);
            }
        }
    };
    load(threadIdx.x);

    // cos/sin of every (token, pair) of this block
    for (uint32_t i = threadIdx.x; i < static_cast<uint32_t>(nt) * a.pairs; i += kThreads) {
        uint32_t pr;
        const uint32_t n = div_pairs.divmod(i, pr);
        int axis = 0;
#pragma unroll
        for (int k = 0; k + 1 < kRopeMaxAxes; ++k) axis += (k + 1 < a.axes && pr >= a.axis_end[k]) ? 1 : 0;
        const int64_t pos = a.offset + (a.pos != nullptr ? static_cast<int64_t>(__ldg(a.pos + b * a.pos_sb + static_cast<int64_t>(n0 + n) * a.axes + axis))
                                                        : static_cast<int64_t>(n0 + n));
        const uint64_t t = static_cast<uint64_t>(pos) * a.turns[pr] + 0x80000000ull;
        float s, c;
        sincospif(static_cast<float>(static_cast<int32_t>(t >> 32)) * 0x1p-31f, &s, &c);
        cs[i] = make_float2(c * a.mscale, (a.inverse ? -s : s) * a.mscale);
    }
    __syncthreads();

    for (uint32_t i0 = threadIdx.x; i0 < total; i0 += kUnroll * kThreads) {
        if (i0 != threadIdx.x) load(i0);
#pragma unroll
        for (int k = 0; k < kUnroll; ++k) {
            const uint32_t i = i0 + k * kThreads;
            if (i >= total) break;
            const Where w = where(i);
            const float2* row = cs + w.n * a.pairs;
            if constexpr (HALF) {
                if (w.u < rot_units) {
                    float lo[VEC], hi[VEC];
#pragma unroll
                    for (int e = 0; e < VEC; ++e) {
                        const float2 t = row[w.u * VEC + e];
                        const float f = p[k].get(e), g = q[k].get(e);
                        lo[e] = f * t.x - g * t.y;
                        hi[e] = f * t.y + g * t.x;
                    }
                    q[k].put_all(hi);
                    q[k].store(y + w.oy + partner);
                    p[k].put_all(lo);
                }
            } else {
                if (w.u < rot_units) {
                    float v[VEC];
#pragma unroll
                    for (int e = 0; e + 1 < VEC; e += 2) {
                        const int pr = (w.u * VEC + e) >> 1;
                        const float f = p[k].get(e), g = p[k].get(e + 1);
                        v[e] = f;
                        v[e + 1] = g;
                        if (pr < a.pairs) {
                            const float2 t = row[pr];
                            v[e] = f * t.x - g * t.y;
                            v[e + 1] = f * t.y + g * t.x;
                        }
                    }
                    p[k].put_all(v);
                }
            }
            p[k].store(y + w.oy);
        }
    }
}

template <typename T, bool HALF, int VEC>
cudaError_t launch_vec(const RopeArgs& a, cudaStream_t s) {
    // Units of one head: interleaved ceil(2 pairs / VEC) that rotate (the last may
    // hold pass-through pairs) then copies; half layout pairs / VEC and copies.
    const int rot = HALF ? a.pairs / VEC : (2 * a.pairs + VEC - 1) / VEC;
    const int units = HALF ? rot + (a.D - 2 * a.pairs) / VEC : a.D / VEC;
    // Tokens per block: enough units for several rounds of loads, angles within shared memory.
    const int64_t per_token = static_cast<int64_t>(units) * a.H;
    int64_t tokens = (2 * kUnroll * kThreads + per_token - 1) / per_token;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    // few tokens: one block each rather than fewer, fuller blocks
    const int64_t want = static_cast<int64_t>(a.B) * a.N / (2 * device_sm_count(dev));
    if (tokens > want) tokens = want;
    if (tokens > kMaxAngles / a.pairs) tokens = kMaxAngles / a.pairs;
    if (tokens > a.N) tokens = a.N;
    if (tokens < 1) tokens = 1;
    const int64_t blocks_per_b = (a.N + tokens - 1) / tokens;
    if (blocks_per_b * a.B > 0x7fffffffLL || tokens * per_token > 0x40000000LL) return cudaErrorInvalidValue;
    rope_kernel<T, HALF, VEC><<<static_cast<unsigned>(blocks_per_b * a.B), kThreads, 0, s>>>(
        a, FastDiv(units), FastDiv(a.H), FastDiv(a.pairs), rot, static_cast<int>(tokens), static_cast<int>(blocks_per_b));
    return cudaGetLastError();
}

template <typename T>
cudaError_t launch_t(const RopeArgs& a, bool half, int vec, cudaStream_t s) {
    constexpr int kMax = 16 / static_cast<int>(sizeof(T));
    if (half) {
        if constexpr (kMax == 8)
            if (vec == 8) return launch_vec<T, true, 8>(a, s);
        if (vec == 4) return launch_vec<T, true, 4>(a, s);
        if (vec == 2) return launch_vec<T, true, 2>(a, s);
        return launch_vec<T, true, 1>(a, s);
    }
    if constexpr (kMax == 8)
        if (vec == 8) return launch_vec<T, false, 8>(a, s);
    if (vec == 4) return launch_vec<T, false, 4>(a, s);
    return launch_vec<T, false, 2>(a, s);
}

}  // namespace

cudaError_t launch_rope(const RopeArgs& a, bool f32, bool half, int vec, cudaStream_t s) {
    return f32 ? launch_t<float>(a, half, vec, s) : launch_t<uint16_t>(a, half, vec, s);
}

}  // namespace dit

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
// 2^64 -- the wrap-around is the range reduction, exact at any position.  The
// fraction's own rounding (2^-65 of a turn) moves an angle by at most
// 2 pi 2^-65 a step: 2^-31 rad at 2^31, 2^-22 at 2^40.  The upper
// 32 bits, rounded, split into a quarter turn and a signed rest of at most an
// eighth, whose sine and cosine are their Taylor polynomials of degree 9 and 10
// (the first terms left out are below 2^-28 of an eighth turn's values).
//
// HBM-bound: every element is read once and written once; positions are 4
// bytes a token.  A block takes `tokens` tokens: the cos/sin of their pairs
// are computed once into shared memory and used by all heads, while the first
// loads of x are already in flight.  Measured, bf16, interleaved, 24,576 tokens
// x 64 heads x 128: 125 us, 6.4 TB/s (95% of a plain copy); the half layout 123
// us.  Two loads of a thread in flight were 134 us interleaved, eight 122; half
// layout units of two loads each: two in flight 121 us, four 139, eight 159.
// Blocks of 4 or 8 rounds were no faster, and slower in the half layout.
#include <cuda_runtime.h>

#include <cstdint>

#include "internal.h"
#include "train.h"

namespace dit {
namespace {

constexpr int kThreads = 256;
constexpr int kRounds = 2;              // rounds of units a block takes, where there is enough to do
constexpr int kMaxAngles = 2048;        // angles a block holds, cos and sin in fp32 (16 KB)

// The launch's index arithmetic.
struct RopeGrid {
    int units, rot_units;           // units of a head, those that rotate
    int wide_from, wide_at;         // copy units from this one on take 16 bytes, the first at this channel
    int step_u, step_h, step_n;     // kThreads units further
    int tokens, blocks_per_b, stride;
    FastDiv div_units, div_h, div_pairs;
};

__host__ __device__ constexpr int unroll(bool half) { return half ? 2 : 4; }

template <typename T> struct IsF32 { static constexpr bool value = false; };
template <> struct IsF32<float> { static constexpr bool value = true; };

// sin and cos of t / 2^32 turns.
__device__ __forceinline__ void sincos_turns(uint32_t t, float& sn, float& cs) {
    const uint32_t q = (t + 0x20000000u) >> 30;                        // nearest quarter turn
    const float x = static_cast<float>(static_cast<int32_t>(t - (q << 30))) * 1.4629180792671596e-9f;   // 2 pi / 2^32
    const float z = x * x;
    float s = fmaf(z, 1.f / 362880.f, -1.f / 5040.f);
    s = fmaf(z, s, 1.f / 120.f);
    s = fmaf(z, s, -1.f / 6.f);
    s = fmaf(z * x, s, x);
    float c = fmaf(z, -1.f / 3628800.f, 1.f / 40320.f);
    c = fmaf(z, c, -1.f / 720.f);
    c = fmaf(z, c, 1.f / 24.f);
    c = fmaf(z, c, -0.5f);
    c = fmaf(z, c, 1.f);
    const float a = (q & 1u) ? c : s, b = (q & 1u) ? s : c;
    sn = __uint_as_float(__float_as_uint(a) ^ ((q & 2u) << 30));
    cs = __uint_as_float(__float_as_uint(b) ^ (((q + 1u) & 2u) << 30));
}

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
// With VEC = 1 the HALF form takes single pairs of either layout.  Where the
// half layout's pairs are no multiple of 16 bytes but the heads are, its copy
// units are (13 pairs of 128 channels, 9,000 tokens x 32 heads: 47 us, with
// single-channel copies 109).  A thread's
// units are kThreads apart in (token, head, unit) order, so it steps from one to
// the next with additions (`step`) instead of dividing.
template <typename T, bool HALF, int VEC>
__global__ void __launch_bounds__(kThreads) rope_kernel(const __grid_constant__ RopeArgs a, const RopeGrid gr) {
    // units in flight per thread: a half-layout unit is two loads
    constexpr int kUnroll = unroll(HALF);
    constexpr int kFull = 16 / static_cast<int>(sizeof(T));
    constexpr bool kWide = HALF && VEC < kFull;
    extern __shared__ __align__(16) float angles[];     // cos [tokens][stride], then sin
    float* const cosv = angles;
    float* const sinv = angles + gr.tokens * gr.stride;
    const int b = static_cast<int>(blockIdx.x) / gr.blocks_per_b;
    const int n0 = (static_cast<int>(blockIdx.x) - b * gr.blocks_per_b) * gr.tokens;
    const int nt = min(gr.tokens, a.N - n0);
    const T* const x = static_cast<const T*>(a.x) + b * a.sx.b + n0 * a.sx.n;
    T* const y = static_cast<T*>(a.y) + b * a.sy.b + n0 * a.sy.n;
    const int partner = VEC == 1 ? a.lone_partner : a.pairs;

    struct At { int n, h, u; };
    auto channel = [&](int u) {     // a half-layout copy unit starts behind both halves
        if (kWide && u >= gr.wide_from) return gr.wide_at + (u - gr.wide_from) * kFull;
        return (!HALF || u < gr.rot_units) ? u * (VEC == 1 ? a.lone_step : VEC) : 2 * a.pairs + (u - gr.rot_units) * VEC;
    };
    auto advance = [&](At& t) {
        t.u += gr.step_u;
        t.h += gr.step_h;
        t.n += gr.step_n;
        if (t.u >= gr.units) { t.u -= gr.units; ++t.h; }
        if (t.h >= a.H) { t.h -= a.H; ++t.n; }
    };
    Pack<T, VEC> p[kUnroll], q[kUnroll];
    Pack<T, kFull> full[kUnroll];   // (kWide)
    At next;                        // the unit to load
    {
        const uint32_t nh = gr.div_units.div(threadIdx.x);
        next.u = static_cast<int>(threadIdx.x - nh * gr.div_units.d);
        next.n = static_cast<int>(gr.div_h.div(nh));
        next.h = static_cast<int>(nh - next.n * gr.div_h.d);
    }
    At cur = next;                  // the unit to rotate and store
    auto load = [&]() {
#pragma unroll
        for (int k = 0; k < kUnroll; ++k) {
            if (next.n < nt) {
                const T* s = x + (next.n * a.sx.n + next.h * a.sx.h + channel(next.u));
                if (kWide && next.u >= gr.wide_from) {
                    full[k].load(s);
                } else {
                    p[k].load(s);
                    if (HALF && next.u < gr.rot_units) q[k].load(s + partner);
                }
            }
            advance(next);
        }
    };
    load();

    // cos/sin of every (token, pair) of this block.  The table of turns is read
    // through a plain address: indexed as a parameter its 32 lanes' different
    // elements would be fetched one after another.
    const uint64_t* turns = a.turns;
    asm volatile("" : "+l"(turns));
    for (uint32_t i = threadIdx.x; i < static_cast<uint32_t>(nt * a.pairs); i += kThreads) {
        uint32_t pr;
        const uint32_t n = gr.div_pairs.divmod(i, pr);
        int axis = 0;
#pragma unroll
        for (int k = 0; k + 1 < kRopeMaxAxes; ++k) axis += (k + 1 < a.axes && pr >= a.axis_end[k]) ? 1 : 0;
        const uint64_t offset = static_cast<uint64_t>(a.offset);      // (the sum modulo 2^64, as the product)
        const uint64_t pos = a.pos != nullptr ? offset + static_cast<int64_t>(__ldg(a.pos + b * a.pos_sb + static_cast<int64_t>(n0 + n) * a.axes + axis))
                                              : offset + static_cast<uint32_t>(n0 + n);
        const uint64_t t = pos * turns[pr] + 0x80000000ull;
        float s, c;
        sincos_turns(static_cast<uint32_t>(t >> 32), s, c);
        cosv[n * gr.stride + pr] = c * a.mscale;
        sinv[n * gr.stride + pr] = (a.inverse ? -s : s) * a.mscale;
    }
    __syncthreads();

    while (cur.n < nt) {
#pragma unroll
        for (int k = 0; k < kUnroll; ++k) {
            if (cur.n < nt) {
                T* const d = y + (cur.n * a.sy.n + cur.h * a.sy.h + channel(cur.u));
                if (cur.u < gr.rot_units) {
                    constexpr int kPairs = HALF ? VEC : VEC / 2;
                    const int p0 = cur.n * gr.stride + cur.u * kPairs;
                    float c[kPairs], s[kPairs];
                    if constexpr (kPairs % 4 == 0) {      // stride is a multiple of 4
#pragma unroll
                        for (int e = 0; e < kPairs; e += 4) {
                            const float4 cv = *reinterpret_cast<const float4*>(cosv + p0 + e);
                            const float4 sv = *reinterpret_cast<const float4*>(sinv + p0 + e);
                            c[e] = cv.x; c[e + 1] = cv.y; c[e + 2] = cv.z; c[e + 3] = cv.w;
                            s[e] = sv.x; s[e + 1] = sv.y; s[e + 2] = sv.z; s[e + 3] = sv.w;
                        }
                    } else {
#pragma unroll
                        for (int e = 0; e < kPairs; ++e) { c[e] = cosv[p0 + e]; s[e] = sinv[p0 + e]; }
                    }
                    float lo[VEC], hi[VEC];
                    if constexpr (HALF) {
#pragma unroll
                        for (int e = 0; e < VEC; ++e) {
                            const float f = p[k].get(e), g = q[k].get(e);
                            lo[e] = f * c[e] - g * s[e];
                            hi[e] = f * s[e] + g * c[e];
                        }
                        q[k].put_all(hi);
                        q[k].store(d + partner);
                    } else {
#pragma unroll
                        for (int e = 0; e + 1 < VEC; e += 2) {
                            const float f = p[k].get(e), g = p[k].get(e + 1);
                            const bool turn = cur.u * kPairs + e / 2 < a.pairs;
                            lo[e] = turn ? f * c[e / 2] - g * s[e / 2] : f;
                            lo[e + 1] = turn ? f * s[e / 2] + g * c[e / 2] : g;
                        }
                    }
                    p[k].put_all(lo);
                }
                if (kWide && cur.u >= gr.wide_from) full[k].store(d);
                else p[k].store(d);
            }
            advance(cur);
        }
        load();
    }
}

template <typename T, bool HALF, int VEC>
cudaError_t launch_vec(const RopeArgs& a, cudaStream_t s) {
    // Units of one head: interleaved ceil(2 pairs / VEC) that rotate (the last may
    // hold pass-through pairs) then copies; half layout pairs / VEC and copies.
    const int rot = HALF ? a.pairs / VEC : (2 * a.pairs + VEC - 1) / VEC;
    constexpr int kFull = 16 / static_cast<int>(sizeof(T));
    int units = HALF ? rot + (a.D - 2 * a.pairs) / VEC : a.D / VEC;
    RopeGrid g;
    g.wide_from = units;
    g.wide_at = 0;
    if (HALF && VEC < kFull && a.wide) {
        g.wide_at = (2 * a.pairs + kFull - 1) / kFull * kFull;
        g.wide_from = rot + (g.wide_at - 2 * a.pairs) / VEC;
        units = g.wide_from + (a.D - g.wide_at) / kFull;
    }
    g.units = units;
    g.rot_units = rot;
    g.div_units = FastDiv(units);
    g.div_h = FastDiv(a.H);
    g.div_pairs = FastDiv(a.pairs);
    g.step_u = kThreads % units;
    g.step_h = kThreads / units % a.H;
    g.step_n = kThreads / units / a.H;
    g.stride = (a.pairs + 3) / 4 * 4;
    // Tokens per block: kRounds rounds of loads, angles within shared memory;
    // fewer while there are not two blocks an SM.
    const int64_t per_token = static_cast<int64_t>(units) * a.H;
    int64_t tokens = (kRounds * unroll(HALF) * kThreads + per_token - 1) / per_token;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const int64_t want = static_cast<int64_t>(a.B) * a.N / (2 * device_sm_count(dev));
    if (tokens > want) tokens = want;
    if (tokens > kMaxAngles / g.stride) tokens = kMaxAngles / g.stride;
    if (tokens > a.N) tokens = a.N;
    if (tokens < 1) tokens = 1;
    g.tokens = static_cast<int>(tokens);
    const int64_t blocks_per_b = (a.N + tokens - 1) / tokens;
    if (blocks_per_b * a.B > 0x7fffffffLL) return cudaErrorInvalidValue;
    g.blocks_per_b = static_cast<int>(blocks_per_b);
    rope_kernel<T, HALF, VEC><<<static_cast<unsigned>(blocks_per_b * a.B), kThreads, 2 * g.tokens * g.stride * sizeof(float), s>>>(a, g);
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

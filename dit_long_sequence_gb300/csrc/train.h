// train.h -- launch-side declarations of the training operators (attention
// backward, layer norm, rotary positions), shared by their kernels and the
// C-ABI layer (api_train.cu).  Not part of the public interface.
#pragma once

#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>

#include "dit_attn.h"
#include "fast_div.h"
#include "window_span.h"

namespace dit {

// ------------------------------------------------------------ launches

#ifdef __CUDACC__
// Launches a kernel that may be set up while the one before it on the stream
// ends (a programmatic dependent launch); it calls after_previous() before it
// touches anything the other wrote.  The other calls let_next() at its start:
// the next kernel's blocks then take what room is left, and the rest later.
template <typename... P, typename... A>
cudaError_t launch_behind(void (*kernel)(P...), dim3 grid, dim3 block, size_t smem, cudaStream_t s, const A&... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}
__device__ __forceinline__ void let_next() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void after_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
#endif

// ------------------------------------------------------------ layer norm

struct NormArgs {
    const void* x;
    const void* dy;             // backward only
    void* y;                    // forward: y, backward: dx
    dit_strides4_t sx, sdy, sy; // element strides (b, n, h), d contiguous
    uint32_t rows;              // B * N * H (< 2^31)
    uint32_t groups;            // parameter sets: B with per-batch parameters, else 1
    uint32_t rows_per_group;    // rows / groups
    FastDiv div_nh, div_h;      // row -> b, (n, h)
    int64_t B, N, H;
    int C;
    bool center;
    float eps, inv_c;
    const float* weight;        // [groups][C] or nullptr
    const float* bias;          // forward only
    float* mean;                // [rows] (written forward, read backward); unused without center
    float* rstd;                // [rows]
    float* part;                // backward: [2][groups][parts][C] partial dweight, dbias
    int want_w, want_b;         // backward: which parameter gradients are formed
    float *dweight, *dbias;     // backward: [groups][C]
};

// The launch shape both directions share: `vec` elements per load, `nv` loads
// per thread and row, `tpr` threads per row, `blocks` blocks per group.
struct NormPlan {
    int vec, nv, tpr, threads, blocks;
    bool two_rows;              // backward: a row group takes two rows at a time
};
NormPlan norm_plan(int C, uint32_t groups, uint32_t rows_per_group, int vec_max, int sms, bool backward);

cudaError_t launch_layer_norm_fwd(const NormArgs& a, const NormPlan& p, bool in_f32, bool out_f32, cudaStream_t s);
cudaError_t launch_layer_norm_bwd(const NormArgs& a, const NormPlan& p, bool in_f32, bool out_f32, cudaStream_t s);

// ------------------------------------------------------------ rotary positions

constexpr int kRopeMaxPairs = 128;
constexpr int kRopeMaxAxes = 4;

struct RopeArgs {
    const void* x;
    void* y;
    dit_strides4_t sx, sy;
    int B, N, H, D, pairs;      // pairs = rotary_dim / 2
    const int32_t* pos;         // [B or 1][N][axes], nullptr: the row index
    int64_t pos_sb;             // 0 shares the positions across the batch
    int axes;
    int64_t offset;
    float mscale;
    bool inverse;
    bool wide;                         // 16-byte copies are aligned wherever a head's channel is a multiple of them
    int lone_step, lone_partner;       // one-channel units: channel of pair i = i * step, its partner's distance
    uint8_t axis_end[kRopeMaxAxes];    // first pair past axis a
    uint64_t turns[kRopeMaxPairs];     // 2^64 * (inv_freq / 2 pi mod 1)
};

cudaError_t launch_rope(const RopeArgs& a, bool f32, bool half, int vec, cudaStream_t s);

// ------------------------------------------------------------ attention backward

struct OccArgs;      // of the mask's occupancy pre-pass
// launch_mask_occupancy beside the kernel before it on the stream: neither needs
// the other, and whoever waits for this one waits for both.
cudaError_t launch_mask_occupancy_behind(const OccArgs& a, cudaStream_t stream);

struct AttnBwdArgs {
    int B, Nq, Nkv, H, kv_len;
    int q_tiles, kv_tiles;      // ceil(Nq / 128), ceil(kv_len / 128)
    int kv_out_tiles;           // ceil(Nkv / 128): key tiles with rows to write (zeros past kv_len)
    float scale, scale_log2;
    const float* stat;          // [B*H][2][q_tiles * 128]: -lse * log2(e), -delta
    const uint32_t* mask;       // as AttnArgs
    int64_t mask_sb, mask_si;
    int mask_rows;
    const uint32_t* occ;
    int occ_words, occ_blocks;  // words per 256-row block, blocks per batch entry
    void *dq, *dk, *dv;
    dit_strides4_t sdq, sdk, sdv;
    // Key items (b, h, 128-key tile), each cut into f_kv ranges of query tiles,
    // and query items (b, h, 128-row tile), those from q_whole on cut into f_q
    // ranges of key tiles, over `grid` CTAs.  Pieces write fp32 partials
    // ([tile][piece][2][128][D] for dv, dk; [cut item][piece][128][D] for dq) that
    // a second kernel sums in piece order.
    int f_kv, f_q, q_whole;
    int n_kv_items, n_q_items;  // pieces counted
    // With a window (windowed) key items are (b, K/V head, tile), of which the leading
    // kv_cut tiles of every head come first, in f_kv pieces each (n_kv_cut in all).
    // Otherwise Hkv = H, and all key items are cut or none.
    bool windowed;
    Window window;
    int offset, Hkv, group;     // position of query 0, K/V heads, query heads of one
    int kv_cut, n_kv_cut;
    FastDiv div_hkv, div_group, div_kv_cut;
    FastDiv div_f_kv, div_f_q, div_kv_tiles, div_q_tiles, div_bh, div_h;   // item -> piece, tile, head (window: div_kv_tiles of the uncut tiles)
    int grid;
    unsigned int* counter;      // items handed out beyond the first `grid` (nullptr: every grid-th)
    bool wide;                  // gradients may be stored 32 bytes at a time
    float *part_kv, *part_q;
    unsigned int* status;
    unsigned long long timeout_ns;
    int dbg_rows_short;         // debug library: rows the bounds check takes off the streamed tensors
};

struct AttnBwdStatArgs {
    const void* out;
    const uint16_t* dout;
    dit_strides4_t so, sdo;
    const float *lse, *dlse;
    int B, Nq, H, rows_pad;     // rows_pad = q_tiles * 128
    float* stat;
    unsigned int* counter;      // set to zero for the main kernel
};

cudaError_t launch_attn_bwd_stat(const AttnBwdStatArgs& a, int D, bool out_bf16, cudaStream_t s);
cudaError_t launch_attn_bwd(const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv, const CUtensorMap& tdo,
                            const AttnBwdArgs& a, int D, bool grad_bf16, cudaStream_t s);
cudaError_t launch_attn_bwd_sum(const AttnBwdArgs& a, int D, bool grad_bf16, cudaStream_t s);

}  // namespace dit

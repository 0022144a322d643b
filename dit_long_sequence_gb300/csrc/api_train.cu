// api_train.cu -- the extern "C" entry points of the training operators
// (include/dit_attn.h): attention backward, layer norm, rotary positions.
//
// Host side only: argument / stride / alignment / placement checks before
// anything is enqueued, workspace layout, the kernel launches.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <cstring>
#include <initializer_list>
#include <utility>

#include "api_common.h"
#include "bwd_plan.h"
#include "dit_attn.h"
#include "internal.h"
#include "rope_turns.h"
#include "train.h"

using namespace dit;

namespace {

// Strides of an output: d contiguous, no two rows of a dimension at one place.
dit_status_t check_out_strides(const dit_strides4_t& s, int64_t B, int64_t N, int64_t H) {
    if (s.d != 1) return DIT_ERR_UNSUPPORTED;
    const int64_t st[3] = {s.b, s.n, s.h}, ext[3] = {B, N, H};
    for (int i = 0; i < 3; ++i)
        if (st[i] < 0 || st[i] >= (int64_t(1) << 39) || (ext[i] > 1 && st[i] == 0)) return DIT_ERR_INVALID_ARG;
    return DIT_OK;
}
// Strides of an input read with plain loads (0 broadcasts).
dit_status_t check_in_strides(const dit_strides4_t& s) {
    if (s.d != 1) return DIT_ERR_UNSUPPORTED;
    for (int64_t x : {s.b, s.n, s.h})
        if (x < 0 || x >= (int64_t(1) << 39)) return DIT_ERR_INVALID_ARG;
    return DIT_OK;
}
bool multiple(const dit_strides4_t& s, int64_t k) { return s.b % k == 0 && s.n % k == 0 && s.h % k == 0; }
bool on(const void* p, uintptr_t bytes) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0; }
bool known(dit_dtype_t t) { return t == DIT_BF16 || t == DIT_F32; }
uintptr_t size_of(dit_dtype_t t) { return t == DIT_F32 ? 4 : 2; }
// Two views that begin at one address place every row alike.
bool same_rows(const dit_strides4_t& s, const dit_strides4_t& t, int B, int N, int H) {
    return (B == 1 || s.b == t.b) && (N == 1 || s.n == t.n) && (H == 1 || s.h == t.h);
}

struct BwdMask {
    const uint32_t* bits;
    int64_t batch_stride, row_stride;
    int rows;
};

int64_t occ_bytes(int B, const BwdPlan& p) {
    return (static_cast<int64_t>(B) * ((p.q_tiles + 1) / 2) * ((p.kv_tiles + 31) / 32) * 4 + 255) / 256 * 256;
}

dit_status_t attn_bwd_common(const void* q, const void* k, const void* v, const void* out, dit_dtype_t out_dtype,
                             const float* lse, const void* dout, const float* dlse, const dit_attn_bwd_strides_t* st,
                             int B, int Nq, int Nkv, int H, int D, int key_valid_len, const BwdMask* mask, float scale,
                             void* dq, void* dk, void* dv, dit_dtype_t grad_dtype, void* workspace,
                             size_t workspace_bytes, dit_stream_t stream) {
    if (st == nullptr) return DIT_ERR_INVALID_ARG;
    if (B < 0 || Nq < 0 || Nkv < 0 || H < 0) return DIT_ERR_INVALID_ARG;
    if (key_valid_len < 0 || key_valid_len > Nkv) return DIT_ERR_INVALID_ARG;
    if (!(scale > 0.f) || !std::isfinite(scale)) return DIT_ERR_INVALID_ARG;
    if (!known(out_dtype) || !known(grad_dtype)) return DIT_ERR_INVALID_ARG;
    if (D != 64 && D != 128) return DIT_ERR_UNSUPPORTED;
    if (B > 65535 || H > 65535) return DIT_ERR_UNSUPPORTED;
    if (B == 0 || H == 0 || (Nq == 0 && Nkv == 0)) return DIT_OK;
    const bool any_keys = key_valid_len > 0 && Nq > 0;   // otherwise every gradient is zero
    if (Nq > 0 && dq == nullptr) return DIT_ERR_INVALID_ARG;
    if (Nkv > 0 && (dk == nullptr || dv == nullptr)) return DIT_ERR_INVALID_ARG;
    if (any_keys && (!q || !k || !v || !out || !lse || !dout)) return DIT_ERR_INVALID_ARG;

    dit_status_t e;
    const int64_t g_align = grad_dtype == DIT_F32 ? 4 : 8;
    if (Nq > 0) {
        if ((e = check_out_strides(st->dq, B, Nq, H)) != DIT_OK) return e;
        if (!multiple(st->dq, g_align) || !aligned16(dq)) return DIT_ERR_ALIGNMENT;
    }
    if (Nkv > 0) {
        if ((e = check_out_strides(st->dk, B, Nkv, H)) != DIT_OK) return e;
        if ((e = check_out_strides(st->dv, B, Nkv, H)) != DIT_OK) return e;
        if (!multiple(st->dk, g_align) || !multiple(st->dv, g_align) || !aligned16(dk) || !aligned16(dv))
            return DIT_ERR_ALIGNMENT;
    }
    CUtensorMap tq, tk, tv, tdo;
    for (CUtensorMap* m : {&tq, &tk, &tv, &tdo}) std::memset(m, 0, sizeof *m);
    if (any_keys) {
        for (const dit_strides4_t* s : {&st->q, &st->k, &st->v, &st->dout})
            if ((e = check_tma_strides(*s)) != DIT_OK) return e;
        if ((e = check_in_strides(st->o)) != DIT_OK) return e;
        if (!multiple(st->o, out_dtype == DIT_F32 ? 4 : 8)) return DIT_ERR_ALIGNMENT;
        if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(dout) || !aligned16(out)) return DIT_ERR_ALIGNMENT;
        if (!on(lse, 4) || !on(dlse, 4)) return DIT_ERR_ALIGNMENT;
    }
    // (views may interleave, so of the forbidden overlaps only a shared base is refused)
    const void* const grads[3] = {Nq > 0 ? dq : nullptr, Nkv > 0 ? dk : nullptr, Nkv > 0 ? dv : nullptr};
    for (int i = 0; i < 3; ++i) {
        if (grads[i] == nullptr) continue;
        for (int j = 0; j < i; ++j)
            if (grads[i] == grads[j]) return DIT_ERR_INVALID_ARG;
        for (const void* in : {q, k, v, out, dout, static_cast<const void*>(lse), static_cast<const void*>(dlse), static_cast<const void*>(workspace)})
            if (any_keys && grads[i] == in) return DIT_ERR_INVALID_ARG;
    }
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return DIT_ERR_CUDA;
    BwdPlan p = plan_attn_bwd(B, Nq, Nkv, H, D, any_keys ? key_valid_len : 0, device_sm_count(dev));
    const bool with_mask = mask != nullptr && mask->rows > 0 && any_keys;
    if (with_mask && p.q_whole > 0) {      // items of unknown lengths: none of the last ones is cut
        p.q_whole = p.query_items;
        p.f_q = 1;
    }
    // Items and partial tiles are counted in 32-bit ints on the device.
    if (p.key_items * p.f_kv + p.query_items * p.f_q > 0x7ffffff0LL - device_sm_count(dev) ||
        static_cast<int64_t>(B) * H * 128 * (p.q_tiles > p.kv_out_tiles ? p.q_tiles : p.kv_out_tiles) > (int64_t(1) << 37))
        return DIT_ERR_UNSUPPORTED;
    const int64_t need = p.stat_bytes + p.part_kv_bytes + p.part_q_bytes + (with_mask ? occ_bytes(B, p) : 0);
    if (any_keys) {
        if (workspace == nullptr || workspace_bytes < static_cast<size_t>(need)) return DIT_ERR_INVALID_ARG;
        if (!aligned16(workspace)) return DIT_ERR_ALIGNMENT;
    }
    if ((e = check_placement({any_keys ? q : nullptr, any_keys ? k : nullptr, any_keys ? v : nullptr,
                              any_keys ? out : nullptr, any_keys ? lse : nullptr, any_keys ? dout : nullptr,
                              any_keys ? dlse : nullptr, any_keys ? workspace : nullptr, Nq > 0 ? dq : nullptr,
                              Nkv > 0 ? dk : nullptr, Nkv > 0 ? dv : nullptr, with_mask ? mask->bits : nullptr},
                             stream)) != DIT_OK)
        return e;
    if (any_keys) {
        if ((e = encode_view(&tq, q, st->q, B, Nq, H, D)) != DIT_OK) return e;
        if ((e = encode_view(&tk, k, st->k, B, key_valid_len, H, D)) != DIT_OK) return e;
        if ((e = encode_view(&tv, v, st->v, B, key_valid_len, H, D)) != DIT_OK) return e;
        if ((e = encode_view(&tdo, dout, st->dout, B, Nq, H, D)) != DIT_OK) return e;
    }
    AttnBwdArgs a{};
    a.status = status_word(dev);
    if (a.status == nullptr) return DIT_ERR_CUDA;
    a.timeout_ns = kWatchdogNs;
#ifdef DIT_DEBUG
    if (debug_wait_limit_ns() != 0) a.timeout_ns = debug_wait_limit_ns();
    a.dbg_rows_short = static_cast<int>(std::min<int64_t>(debug_extent_shrink(), std::max(Nq, Nkv)));
#endif
    a.B = B;
    a.Nq = Nq;
    a.Nkv = Nkv;
    a.H = H;
    a.kv_len = any_keys ? key_valid_len : 0;
    a.q_tiles = p.q_tiles;
    a.kv_tiles = p.kv_tiles;
    a.kv_out_tiles = p.kv_out_tiles;
    a.scale = scale;
    a.scale_log2 = static_cast<float>(static_cast<double>(scale) * 1.4426950408889634);
    a.dq = dq;
    a.dk = dk;
    a.dv = dv;
    a.sdq = st->dq;
    a.sdk = st->dk;
    a.sdv = st->dv;
    a.f_kv = p.f_kv;
    a.f_q = p.f_q;
    a.q_whole = static_cast<int>(p.q_whole);
    a.n_kv_items = static_cast<int>(p.key_items * p.f_kv);
    a.n_q_items = static_cast<int>(p.q_whole + (p.query_items - p.q_whole) * p.f_q);
    auto div = [](int64_t d) { return FastDiv(static_cast<uint32_t>(d > 0 ? d : 1)); };
    a.div_f_kv = div(p.f_kv);
    a.div_f_q = div(p.f_q);
    a.div_kv_tiles = div(p.kv_out_tiles);
    a.div_q_tiles = div(p.q_tiles);
    a.div_bh = div(static_cast<int64_t>(B) * H);
    a.div_h = div(H);
    a.grid = std::min(device_sm_count(dev), a.n_kv_items + a.n_q_items);
    const int64_t wide = grad_dtype == DIT_F32 ? 8 : 16;
    a.wide = (Nq == 0 || (multiple(st->dq, wide) && on(dq, 32))) &&
             (Nkv == 0 || (multiple(st->dk, wide) && multiple(st->dv, wide) && on(dk, 32) && on(dv, 32)));
    const cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
    const bool grad_bf16 = grad_dtype == DIT_BF16;
    if (any_keys) {
        uint8_t* ws = static_cast<uint8_t*>(workspace);
        AttnBwdStatArgs s{};
        s.out = out;
        s.dout = static_cast<const uint16_t*>(dout);
        s.so = st->o;
        s.sdo = st->dout;
        s.lse = lse;
        s.dlse = dlse;
        s.B = B;
        s.Nq = Nq;
        s.H = H;
        s.rows_pad = p.q_tiles * 128;
        s.stat = reinterpret_cast<float*>(ws);
        a.stat = s.stat;
        s.counter = a.counter = reinterpret_cast<unsigned int*>(ws + p.stat_bytes - 256);    // behind the statistics
        a.part_kv = reinterpret_cast<float*>(ws + p.stat_bytes);
        a.part_q = reinterpret_cast<float*>(ws + p.stat_bytes + p.part_kv_bytes);
        OccArgs o{};
        if (with_mask) {
            a.mask = mask->bits;
            a.mask_sb = mask->batch_stride;
            a.mask_si = mask->row_stride;
            a.mask_rows = mask->rows;
            o.mask = mask->bits;
            o.mask_sb = mask->batch_stride;
            o.mask_si = mask->row_stride;
            o.mask_rows = mask->rows;
            o.B = B;
            o.Nq = Nq;
            o.kv_len = key_valid_len;
            o.n_kv_tiles = p.kv_tiles;
            o.row_blocks = (p.q_tiles + 1) / 2;
            o.occ_words = (p.kv_tiles + 31) / 32;
            o.occ = reinterpret_cast<uint32_t*>(ws + p.stat_bytes + p.part_kv_bytes + p.part_q_bytes);
            a.occ = o.occ;
            a.occ_words = o.occ_words;
            a.occ_blocks = o.row_blocks;
        }
        if (launch_attn_bwd_stat(s, D, out_dtype == DIT_BF16, cs) != cudaSuccess) return DIT_ERR_CUDA;
        if (with_mask && launch_mask_occupancy_behind(o, cs) != cudaSuccess) return DIT_ERR_CUDA;
    }
    if (launch_attn_bwd(tq, tk, tv, tdo, a, D, grad_bf16, cs) != cudaSuccess) return DIT_ERR_CUDA;
    return launch_attn_bwd_sum(a, D, grad_bf16, cs) == cudaSuccess ? DIT_OK : DIT_ERR_CUDA;
}

// ------------------------------------------------------------ layer norm

// Checks shared by both directions; `vec` receives the widest load every
// pointer, stride and C allow (8, 2 or 1 channels).
dit_status_t norm_common(int B, int N, int H, int C, int param_batches, dit_dtype_t x_dtype, dit_dtype_t y_dtype) {
    if (B < 0 || N < 0 || H < 0 || C < 0) return DIT_ERR_INVALID_ARG;
    if (!known(x_dtype) || !known(y_dtype)) return DIT_ERR_INVALID_ARG;
    if (x_dtype == DIT_BF16 && y_dtype == DIT_F32) return DIT_ERR_UNSUPPORTED;
    if (param_batches != 1 && param_batches != B) return DIT_ERR_INVALID_ARG;
    if (C > 8192 || B > 65535) return DIT_ERR_UNSUPPORTED;
    if (static_cast<double>(B) * N * H >= 2147483648.0) return DIT_ERR_UNSUPPORTED;
    return DIT_OK;
}

int norm_vec(int C, std::initializer_list<std::pair<const void*, dit_dtype_t>> ptrs,
             std::initializer_list<const dit_strides4_t*> strides) {
    for (int v : {8, 2}) {
        bool ok = C % v == 0;
        for (const auto& p : ptrs) ok = ok && on(p.first, std::min<uintptr_t>(16, v * size_of(p.second)));
        for (const dit_strides4_t* s : strides) ok = ok && multiple(*s, v);
        if (ok) return v;
    }
    return 1;
}

void norm_fill(NormArgs& a, int B, int N, int H, int C, int param_batches, bool center) {
    a.rows = static_cast<uint32_t>(B) * static_cast<uint32_t>(N) * static_cast<uint32_t>(H);
    a.groups = static_cast<uint32_t>(param_batches);
    a.rows_per_group = a.rows / a.groups;
    a.div_nh = FastDiv(static_cast<uint32_t>(N) * static_cast<uint32_t>(H));
    a.div_h = FastDiv(static_cast<uint32_t>(H));
    a.B = B;
    a.N = N;
    a.H = H;
    a.C = C;
    a.center = center;
    a.inv_c = 1.f / static_cast<float>(C);
}

}  // namespace

extern "C" {

size_t dit_attn_bwd_workspace_bytes(int B, int Nq, int Nkv, int H, int D, int key_valid_len, int masked) {
    if (B <= 0 || Nq <= 0 || H <= 0 || key_valid_len <= 0 || key_valid_len > Nkv || (D != 64 && D != 128)) return 0;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return 0;
    const BwdPlan p = plan_attn_bwd(B, Nq, Nkv, H, D, key_valid_len, device_sm_count(dev));
    return static_cast<size_t>(p.stat_bytes + p.part_kv_bytes + p.part_q_bytes + (masked ? occ_bytes(B, p) : 0));
}

dit_status_t dit_attn_bwd(const void* q, const void* k, const void* v, const void* out, dit_dtype_t out_dtype,
                          const float* lse, const void* dout, const float* dlse, const dit_attn_bwd_strides_t* strides,
                          int B, int Nq, int Nkv, int H, int D, int key_valid_len, float scale, void* dq, void* dk,
                          void* dv, dit_dtype_t grad_dtype, void* workspace, size_t workspace_bytes,
                          dit_stream_t stream) {
    return attn_bwd_common(q, k, v, out, out_dtype, lse, dout, dlse, strides, B, Nq, Nkv, H, D, key_valid_len, nullptr,
                           scale, dq, dk, dv, grad_dtype, workspace, workspace_bytes, stream);
}

dit_status_t dit_attn_bwd_masked(const void* q, const void* k, const void* v, const void* out, dit_dtype_t out_dtype,
                                 const float* lse, const void* dout, const float* dlse,
                                 const dit_attn_bwd_strides_t* strides, int B, int Nq, int Nkv, int H, int D,
                                 int key_valid_len, const uint32_t* mask, int64_t mask_batch_stride,
                                 int64_t mask_row_stride, int mask_rows, float scale, void* dq, void* dk, void* dv,
                                 dit_dtype_t grad_dtype, void* workspace, size_t workspace_bytes, dit_stream_t stream) {
    if (mask_rows < 0 || mask_rows > Nq) return DIT_ERR_INVALID_ARG;
    if (mask_rows > 0) {
        if (mask == nullptr) return DIT_ERR_INVALID_ARG;
        const int64_t words_read = 4 * ((static_cast<int64_t>(key_valid_len) + 127) / 128);
        if (mask_row_stride < words_read || mask_batch_stride < 0) return DIT_ERR_INVALID_ARG;
        if (mask_row_stride % 4 || mask_batch_stride % 4 || !aligned16(mask)) return DIT_ERR_ALIGNMENT;
    }
    const BwdMask m{mask, mask_batch_stride, mask_row_stride, mask_rows};
    return attn_bwd_common(q, k, v, out, out_dtype, lse, dout, dlse, strides, B, Nq, Nkv, H, D, key_valid_len, &m, scale,
                           dq, dk, dv, grad_dtype, workspace, workspace_bytes, stream);
}

dit_status_t dit_layer_norm_fwd(const void* x, dit_dtype_t x_dtype, const dit_strides4_t* x_strides, int B, int N, int H,
                                int C, const float* weight, const float* bias, int param_batches, float eps, int center,
                                void* y, dit_dtype_t y_dtype, const dit_strides4_t* y_strides, float* mean, float* rstd,
                                dit_stream_t stream) {
    dit_status_t e = norm_common(B, N, H, C, param_batches, x_dtype, y_dtype);
    if (e != DIT_OK) return e;
    if (!(eps >= 0.f) || !std::isfinite(eps)) return DIT_ERR_INVALID_ARG;
    if (B == 0 || N == 0 || H == 0 || C == 0) return DIT_OK;
    if (!x || !y || !rstd || !x_strides || !y_strides || (center && !mean)) return DIT_ERR_INVALID_ARG;
    if ((e = check_in_strides(*x_strides)) != DIT_OK) return e;
    if ((e = check_out_strides(*y_strides, B, N, H)) != DIT_OK) return e;
    if (!on(x, size_of(x_dtype)) || !on(y, size_of(y_dtype)) || !on(weight, 4) || !on(bias, 4) || !on(mean, 4) || !on(rstd, 4))
        return DIT_ERR_ALIGNMENT;
    if (x == y && (x_dtype != y_dtype || !same_rows(*x_strides, *y_strides, B, N, H))) return DIT_ERR_INVALID_ARG;
    if ((e = check_placement({x, y, weight, bias, center ? mean : nullptr, rstd}, stream)) != DIT_OK) return e;
    NormArgs a{};
    norm_fill(a, B, N, H, C, param_batches, center != 0);
    a.x = x;
    a.y = y;
    a.sx = *x_strides;
    a.sy = *y_strides;
    a.eps = eps;
    a.weight = weight;
    a.bias = bias;
    a.mean = mean;
    a.rstd = rstd;
    const int vec = norm_vec(C, {{x, x_dtype}, {y, y_dtype}, {weight, DIT_F32}, {bias, DIT_F32}}, {x_strides, y_strides});
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return DIT_ERR_CUDA;
    const NormPlan p = norm_plan(C, a.groups, a.rows_per_group, vec, device_sm_count(dev), false);
    return launch_layer_norm_fwd(a, p, x_dtype == DIT_F32, y_dtype == DIT_F32, reinterpret_cast<cudaStream_t>(stream)) ==
                   cudaSuccess
               ? DIT_OK
               : DIT_ERR_CUDA;
}

size_t dit_layer_norm_bwd_workspace_bytes(int B, int N, int H, int C, int param_batches) {
    if (norm_common(B, N, H, C, param_batches, DIT_F32, DIT_F32) != DIT_OK) return 0;
    if (B == 0 || N == 0 || H == 0 || C == 0) return 0;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return 0;
    const uint32_t rows = static_cast<uint32_t>(B) * static_cast<uint32_t>(N) * static_cast<uint32_t>(H);
    const uint32_t groups = static_cast<uint32_t>(param_batches);
    int blocks = 1;      // of whichever plan the pointers' alignment will allow
    for (int vec : {8, 2, 1}) blocks = std::max(blocks, norm_plan(C, groups, rows / groups, vec, device_sm_count(dev), true).blocks);
    return blocks > 1 ? static_cast<size_t>(2) * groups * blocks * C * sizeof(float) : 0;
}

dit_status_t dit_layer_norm_bwd(const void* dy, dit_dtype_t dy_dtype, const dit_strides4_t* dy_strides, const void* x,
                                dit_dtype_t x_dtype, const dit_strides4_t* x_strides, const float* mean,
                                const float* rstd, const float* weight, int B, int N, int H, int C, int param_batches,
                                int center, void* dx, const dit_strides4_t* dx_strides, float* dweight, float* dbias,
                                void* workspace, size_t workspace_bytes, dit_stream_t stream) {
    dit_status_t e = norm_common(B, N, H, C, param_batches, x_dtype, dy_dtype);
    if (e != DIT_OK) return e;
    if (C == 0) return DIT_OK;
    if (B == 0 || N == 0 || H == 0) {      // no rows: the sums over rows are zero
        int dev = 0;
        const cudaError_t found = cudaGetDevice(&dev);
        if (found == cudaErrorNoDevice || found == cudaErrorInsufficientDriver) {    // no memory that could hold them
            (void)cudaGetLastError();
            return DIT_OK;
        }
        if ((e = check_placement({dweight, dbias}, stream)) != DIT_OK) return e;
        const size_t bytes = static_cast<size_t>(param_batches) * C * sizeof(float);
        for (float* g : {dweight, dbias})
            if (g != nullptr && cudaMemsetAsync(g, 0, bytes, reinterpret_cast<cudaStream_t>(stream)) != cudaSuccess)
                return DIT_ERR_CUDA;
        return DIT_OK;
    }
    if (!x || !dy || !dx || !rstd || !x_strides || !dy_strides || !dx_strides || (center && !mean))
        return DIT_ERR_INVALID_ARG;
    if ((e = check_in_strides(*x_strides)) != DIT_OK) return e;
    if ((e = check_in_strides(*dy_strides)) != DIT_OK) return e;
    if ((e = check_out_strides(*dx_strides, B, N, H)) != DIT_OK) return e;
    if (!on(x, size_of(x_dtype)) || !on(dx, size_of(x_dtype)) || !on(dy, size_of(dy_dtype)) || !on(weight, 4) ||
        !on(mean, 4) || !on(rstd, 4) || !on(dweight, 4) || !on(dbias, 4))
        return DIT_ERR_ALIGNMENT;
    if ((dx == x && !same_rows(*dx_strides, *x_strides, B, N, H)) ||
        (dx == dy && (x_dtype != dy_dtype || !same_rows(*dx_strides, *dy_strides, B, N, H))) ||
        (dweight != nullptr && dweight == dbias))
        return DIT_ERR_INVALID_ARG;
    const bool wants = dweight != nullptr || dbias != nullptr;
    const size_t need = wants ? dit_layer_norm_bwd_workspace_bytes(B, N, H, C, param_batches) : 0;
    if (need > 0) {
        if (workspace == nullptr || workspace_bytes < need) return DIT_ERR_INVALID_ARG;
        if (!aligned16(workspace)) return DIT_ERR_ALIGNMENT;
    }
    if ((e = check_placement({x, dy, dx, weight, center ? mean : nullptr, rstd, dweight, dbias, need ? workspace : nullptr},
                             stream)) != DIT_OK)
        return e;
    NormArgs a{};
    norm_fill(a, B, N, H, C, param_batches, center != 0);
    a.x = x;
    a.dy = dy;
    a.y = dx;
    a.sx = *x_strides;
    a.sdy = *dy_strides;
    a.sy = *dx_strides;
    a.weight = weight;
    a.mean = const_cast<float*>(mean);
    a.rstd = const_cast<float*>(rstd);
    a.part = static_cast<float*>(workspace);
    a.want_w = dweight != nullptr;
    a.want_b = dbias != nullptr;
    a.dweight = dweight;
    a.dbias = dbias;
    const int vec = norm_vec(C, {{x, x_dtype}, {dx, x_dtype}, {dy, dy_dtype}, {weight, DIT_F32}},
                             {x_strides, dy_strides, dx_strides});
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return DIT_ERR_CUDA;
    const NormPlan p = norm_plan(C, a.groups, a.rows_per_group, vec, device_sm_count(dev), true);
    return launch_layer_norm_bwd(a, p, x_dtype == DIT_F32, dy_dtype == DIT_F32, reinterpret_cast<cudaStream_t>(stream)) ==
                   cudaSuccess
               ? DIT_OK
               : DIT_ERR_CUDA;
}

dit_status_t dit_rope_inv_freq(int pairs, double base, dit_rope_scaling_t scaling, double factor, double original_len,
                               double beta_fast, double beta_slow, double* inv_freq, float* mscale) {
    if (pairs < 1 || pairs > kRopeMaxPairs || inv_freq == nullptr || mscale == nullptr) return DIT_ERR_INVALID_ARG;
    if (!(base > 0.0) || !std::isfinite(base)) return DIT_ERR_INVALID_ARG;
    if (scaling < DIT_ROPE_PLAIN || scaling > DIT_ROPE_BY_PARTS) return DIT_ERR_INVALID_ARG;
    if (scaling != DIT_ROPE_PLAIN && (!(factor >= 1.0) || !std::isfinite(factor))) return DIT_ERR_INVALID_ARG;
    if (scaling == DIT_ROPE_BY_PARTS && (!(original_len > 0.0) || !std::isfinite(original_len) || !(beta_fast > beta_slow) ||
                                         !std::isfinite(beta_fast) || !std::isfinite(beta_slow)))
        return DIT_ERR_INVALID_ARG;
    double bb = base;
    if (scaling == DIT_ROPE_BASE && pairs > 1)
        bb = base * std::pow(factor, static_cast<double>(pairs) / (pairs - 1));
    for (int i = 0; i < pairs; ++i) {
        double w = std::pow(bb, -static_cast<double>(i) / pairs);
        if (scaling == DIT_ROPE_LINEAR) w /= factor;
        if (scaling == DIT_ROPE_BY_PARTS) {
            const double turns = original_len * w / 6.283185307179586476925;
            double keep = (turns - beta_slow) / (beta_fast - beta_slow);
            keep = keep < 0.0 ? 0.0 : (keep > 1.0 ? 1.0 : keep);
            w = keep * w + (1.0 - keep) * w / factor;
        }
        inv_freq[i] = w;
    }
    *mscale = scaling == DIT_ROPE_BY_PARTS ? static_cast<float>(0.1 * std::log(factor) + 1.0) : 1.f;
    return DIT_OK;
}

dit_status_t dit_rope(const void* x, dit_dtype_t dtype, const dit_strides4_t* x_strides, int B, int N, int H, int D,
                      int rotary_dim, dit_rope_layout_t layout, const double* inv_freq, const int* axis_pairs, int n_axes,
                      const int32_t* positions, int64_t positions_batch_stride, int64_t offset, float mscale, int inverse,
                      void* y, const dit_strides4_t* y_strides, dit_stream_t stream) {
    if (B < 0 || N < 0 || H < 0 || D < 0) return DIT_ERR_INVALID_ARG;
    if (!known(dtype) || (layout != DIT_ROPE_INTERLEAVED && layout != DIT_ROPE_HALF)) return DIT_ERR_INVALID_ARG;
    if (!std::isfinite(mscale)) return DIT_ERR_INVALID_ARG;
    if (rotary_dim < 2 || rotary_dim % 2 != 0 || rotary_dim > D) return DIT_ERR_INVALID_ARG;
    if (n_axes < 1 || inv_freq == nullptr || axis_pairs == nullptr) return DIT_ERR_INVALID_ARG;
    if (n_axes > kRopeMaxAxes || rotary_dim / 2 > kRopeMaxPairs || D > 1024) return DIT_ERR_UNSUPPORTED;
    const int pairs = rotary_dim / 2;
    RopeArgs a{};
    int at = 0;
    for (int i = 0; i < n_axes; ++i) {
        if (axis_pairs[i] < 0 || axis_pairs[i] > pairs - at) return DIT_ERR_INVALID_ARG;
        at += axis_pairs[i];
        a.axis_end[i] = static_cast<uint8_t>(at);
    }
    if (at != pairs) return DIT_ERR_INVALID_ARG;
    if (n_axes > 1 && positions == nullptr) return DIT_ERR_INVALID_ARG;
    if (positions_batch_stride < 0 || (positions != nullptr && positions_batch_stride != 0 &&
                                       positions_batch_stride < static_cast<int64_t>(N) * n_axes))
        return DIT_ERR_INVALID_ARG;
    for (int i = 0; i < pairs; ++i) {
        if (!std::isfinite(inv_freq[i])) return DIT_ERR_INVALID_ARG;
        a.turns[i] = turns_per_step(inv_freq[i]);
    }
    if (B == 0 || N == 0 || H == 0) return DIT_OK;
    if (!x || !y || !x_strides || !y_strides) return DIT_ERR_INVALID_ARG;
    if (H > 65535 || static_cast<int64_t>(B) * N > 0x7fffffffLL) return DIT_ERR_UNSUPPORTED;
    dit_status_t e;
    if ((e = check_in_strides(*x_strides)) != DIT_OK) return e;
    if ((e = check_out_strides(*y_strides, B, N, H)) != DIT_OK) return e;
    if (!on(x, size_of(dtype)) || !on(y, size_of(dtype)) || !on(positions, 4)) return DIT_ERR_ALIGNMENT;
    if (x == y && !same_rows(*x_strides, *y_strides, B, N, H)) return DIT_ERR_INVALID_ARG;
    if ((e = check_placement({x, y, positions}, stream)) != DIT_OK) return e;
    a.x = x;
    a.y = y;
    a.sx = *x_strides;
    a.sy = *y_strides;
    a.B = B;
    a.N = N;
    a.H = H;
    a.D = D;
    a.pairs = pairs;
    a.pos = positions;
    a.pos_sb = positions_batch_stride;
    a.axes = n_axes;
    a.offset = offset;
    a.mscale = mscale;
    a.inverse = inverse != 0;
    // The widest unit every pointer, stride and part of the head allows.
    const bool half = layout == DIT_ROPE_HALF;
    const int full = 16 / static_cast<int>(size_of(dtype));
    auto fits = [&](int v) {
        return on(x, v * size_of(dtype)) && on(y, v * size_of(dtype)) && multiple(*x_strides, v) && multiple(*y_strides, v) && D % v == 0;
    };
    a.wide = fits(full);
    int vec = full;
    while (vec > 1 && !(fits(vec) && (!half || pairs % vec == 0))) vec /= 2;
    // one channel at a time: the half layout's kernel serves both, by where a pair's two channels lie
    a.lone_step = half ? 1 : 2;
    a.lone_partner = half ? pairs : 1;
    return launch_rope(a, dtype == DIT_F32, half || vec == 1, vec, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess ? DIT_OK
                                                                                                             : DIT_ERR_CUDA;
}

}  // extern "C"

// api_window.cu -- the extern "C" entry points of windowed attention and the paged
// cache (include/dit_attn.h; the backward call is api_train.cu's).
//
// Host side only: argument / stride / alignment / placement checks before anything
// is enqueued, tensor maps, workspace layout, the kernel launches.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <cstring>
#include <initializer_list>

#include "api_common.h"
#include "dit_attn.h"
#include "internal.h"
#include "window.h"
#include "window_plan.h"

using namespace dit;

namespace {

constexpr int64_t kMaxTokens = int64_t(1) << 29;
constexpr int64_t kMaxItems = 0x7ffffff0;      // counted in 32-bit ints on the device

int64_t items_of(int B, int T, int H, int Hkv) {
    const int64_t rows = 2 * (128 / (H / Hkv));
    return static_cast<int64_t>(B) * Hkv * ((static_cast<int64_t>(T) + rows - 1) / rows);
}

// Sizes, window and scale that every form checks alike; `done`: nothing to compute.
dit_status_t check_common(int B, int T, int H, int Hkv, int D, const dit_window_t* window, float scale, bool& done) {
    done = false;
    if (B < 0 || T < 0 || H < 0 || Hkv < 0) return DIT_ERR_INVALID_ARG;
    if (!sound_window(window)) return DIT_ERR_INVALID_ARG;
    if (!(scale > 0.f) || !std::isfinite(scale)) return DIT_ERR_INVALID_ARG;
    if (D != 64 && D != 128) return DIT_ERR_UNSUPPORTED;
    if (B > 65535 || H > 65535 || T > kMaxTokens) return DIT_ERR_UNSUPPORTED;
    done = B == 0 || T == 0 || H == 0;
    if (done) return DIT_OK;
    if (Hkv == 0 || H % Hkv != 0) return DIT_ERR_INVALID_ARG;
    if (H / Hkv > 128 || items_of(B, T, H, Hkv) > kMaxItems) return DIT_ERR_UNSUPPORTED;
    return DIT_OK;
}

dit_status_t check_out(const void* out, dit_dtype_t type, const dit_strides4_t& so, const float* lse, int B, int T, int H) {
    if (out == nullptr || lse == nullptr) return DIT_ERR_INVALID_ARG;
    const dit_status_t e = check_out_strides(so, B, T, H);
    if (e != DIT_OK) return e;
    if (!multiple(so, type == DIT_F32 ? 4 : 8) || !aligned16(out) || !on(lse, 4)) return DIT_ERR_ALIGNMENT;
    return DIT_OK;
}

// Q as a map of five dimensions: channel, head of the group, token, K/V head, batch
// entry; a box is the whole tokens of a 128-row tile.
dit_status_t encode_q(CUtensorMap* map, const void* q, const dit_strides4_t& s, int B, int T, int H, int Hkv, int D, int tokens) {
    const uint64_t group = static_cast<uint64_t>(H / Hkv);
    const uint64_t dims[5] = {static_cast<uint64_t>(D), group, static_cast<uint64_t>(T), static_cast<uint64_t>(Hkv),
                              static_cast<uint64_t>(B)};
    const uint64_t st[4] = {static_cast<uint64_t>(s.h) * 2, static_cast<uint64_t>(s.n) * 2, static_cast<uint64_t>(s.h) * group * 2,
                            static_cast<uint64_t>(s.b) * 2};
    if (st[2] >= (uint64_t(1) << 40)) return DIT_ERR_INVALID_ARG;
    const uint32_t box[5] = {64, static_cast<uint32_t>(group), static_cast<uint32_t>(tokens), 1, 1};
    return encode_tiles(map, q, 5, dims, st, box);
}

void fill_common(WindowArgs& a, int B, int T, int H, int Hkv, const dit_window_t& window, float scale, void* out, dit_dtype_t type,
                 const dit_strides4_t& so, float* lse, int D) {
    a.B = B;
    a.T = T;
    a.H = H;
    a.Hkv = Hkv;
    a.group = H / Hkv;
    a.tokens = 128 / a.group;
    a.win = make_window(window);
    a.scale_log2 = static_cast<float>(static_cast<double>(scale) * 1.4426950408889634);
    a.out = out;
    a.out_bf16 = type == DIT_BF16;
    a.wide = multiple(so, a.out_bf16 ? 16 : 8) && on(out, 32);
    a.o_sb = so.b;
    a.o_sn = so.n;
    a.o_sh = so.h;
    a.lse = lse;
    a.n_blk = static_cast<int>((static_cast<int64_t>(T) + 2 * a.tokens - 1) / (2 * a.tokens));
    a.div_group = FastDiv(static_cast<uint32_t>(a.group));
    a.timeout_ns = kWatchdogNs;
    a.dbg_o_elems = static_cast<int64_t>(B - 1) * so.b + static_cast<int64_t>(T - 1) * so.n + static_cast<int64_t>(H - 1) * so.h + D;
#ifdef DIT_DEBUG
    if (debug_wait_limit_ns() != 0) a.timeout_ns = debug_wait_limit_ns();
    a.dbg_o_elems -= debug_extent_shrink();
    a.dbg_keys_short = static_cast<int>(std::min<int64_t>(debug_extent_shrink(), kMaxTokens));
#endif
}

struct GridPlan {
    int f = 1, late = 0;        // pieces of an item, blocks of a head that come last
};
// Attention over `kv_len` keys, queries from position `offset`.
GridPlan plan_of(int B, int T, int H, int Hkv, const dit_window_t& window, int offset, int kv_len, int sms) {
    const int rows = 2 * (128 / (H / Hkv));
    const Window w = make_window(window);
    const double mean = mean_key_tiles(w, T, rows, offset, kv_len);
    const double first = key_tiles(w, offset, offset + std::min(rows, T) - 1, kv_len).n;
    GridPlan p;
    p.f = plan_pieces(items_of(B, T, H, Hkv), mean, sms);
    p.late = late_blocks(first, mean, static_cast<int64_t>(B) * Hkv, (static_cast<int64_t>(T) + rows - 1) / rows, sms);
    return p;
}
// Settles the grid and the partials' place in the workspace.
dit_status_t set_grid(WindowArgs& a, const GridPlan& plan, int D, void* workspace, size_t workspace_bytes) {
    const int f = plan.f;
    const int64_t items = items_of(a.B, a.T, a.H, a.Hkv);
    a.part_rows = part_rows_of(a.T, a.group);
    order_items(a, plan.late);
    if (items * f > kMaxItems) return DIT_ERR_UNSUPPORTED;
    a.f = f;
    a.div_f = FastDiv(static_cast<uint32_t>(f));
    a.n_items = static_cast<int>(items * f);
    if (f > 1) {
        if (workspace == nullptr || workspace_bytes < static_cast<size_t>(pieces_bytes(items, f, a.part_rows, D))) return DIT_ERR_INVALID_ARG;
        if (!aligned16(workspace)) return DIT_ERR_ALIGNMENT;
        a.ws_o = static_cast<float*>(workspace);
        a.ws_lse = a.ws_o + items * f * a.part_rows * D;
    }
    return DIT_OK;
}

// A cache whose fields are in order; its capacity in tokens.
dit_status_t check_cache(const dit_paged_cache_t* c, int64_t& capacity) {
    if (c == nullptr || c->pages < 0 || c->page_size < 1 || c->table_width < 0 || c->table_stride < 0) return DIT_ERR_INVALID_ARG;
    if (c->page_size % 8 != 0) return DIT_ERR_UNSUPPORTED;
    capacity = static_cast<int64_t>(c->page_size) * c->table_width;
    if (capacity > 0x7fffff00LL || c->pages == 0x7fffffff) return DIT_ERR_UNSUPPORTED;
    if (c->kv_lens == nullptr) return DIT_ERR_INVALID_ARG;
    if (!on(c->kv_lens, 4)) return DIT_ERR_ALIGNMENT;
    if (capacity > 0 && c->pages > 0) {
        if (c->k == nullptr || c->v == nullptr || c->table == nullptr) return DIT_ERR_INVALID_ARG;
        dit_status_t e;
        if ((e = check_tma_strides(c->k_strides)) != DIT_OK || (e = check_tma_strides(c->v_strides)) != DIT_OK) return e;
        if (!aligned16(c->k) || !aligned16(c->v) || !on(c->table, 4)) return DIT_ERR_ALIGNMENT;
    }
    return DIT_OK;
}
int chunk_of(int page_size) {        // the largest power of two that divides the page, at most a key tile
    int c = 8;
    while (c < 128 && page_size % (2 * c) == 0) c *= 2;
    return c;
}
// One of the cache's tensors as a map (channel, row of a page, head, page); a box is
// `chunk` rows.
dit_status_t encode_pages(CUtensorMap* map, const void* base, const dit_strides4_t& s, const dit_paged_cache_t& c, int Hkv, int D, int chunk) {
    const uint64_t dims[4] = {static_cast<uint64_t>(D), static_cast<uint64_t>(c.page_size), static_cast<uint64_t>(Hkv),
                              static_cast<uint64_t>(c.pages)};
    const uint64_t st[3] = {static_cast<uint64_t>(s.n) * 2, static_cast<uint64_t>(s.h) * 2, static_cast<uint64_t>(s.b) * 2};
    const uint32_t box[4] = {64, static_cast<uint32_t>(chunk), 1, 1};
    return encode_tiles(map, base, 4, dims, st, box);
}
// The same over a cache, whose lengths the host does not know: as if every sequence
// filled its table row.
GridPlan paged_plan_of(int B, int T, int H, int Hkv, const dit_window_t& window, int64_t capacity, int sms) {
    const int len = static_cast<int>(capacity), tokens = 128 / (H / Hkv);
    if (T > tokens) return plan_of(B, T, H, Hkv, window, len - T, len, sms);
    GridPlan p;
    p.f = plan_pieces_few(items_of(B, T, H, Hkv), key_tiles(make_window(window), len - T, len - 1, len).n, sms);
    return p;
}

}  // namespace

extern "C" {

size_t dit_attn_fwd_window_workspace_bytes(int B, int Nq, int H, int Hkv, int D, int key_valid_len, const dit_window_t* window,
                                           int q_offset) {
    bool done;
    if (check_common(B, Nq, H, Hkv, D, window, 1.f, done) != DIT_OK || done || key_valid_len <= 0) return 0;
    if (key_valid_len > kMaxTokens || std::abs(static_cast<int64_t>(q_offset)) + Nq > kMaxTokens) return 0;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return 0;
    const int f = plan_of(B, Nq, H, Hkv, *window, q_offset, key_valid_len, device_sm_count(dev)).f;
    return static_cast<size_t>(pieces_bytes(items_of(B, Nq, H, Hkv), f, part_rows_of(Nq, H / Hkv), D));
}

dit_status_t dit_attn_fwd_window(const void* q, const void* k, const void* v, const dit_attn_strides_t* strides, int B, int Nq, int Nkv,
                                 int H, int Hkv, int D, int key_valid_len, const dit_window_t* window, int q_offset, float scale,
                                 void* out, dit_dtype_t out_dtype, float* lse, void* workspace, size_t workspace_bytes,
                                 dit_stream_t stream) {
    if (strides == nullptr || Nkv < 0 || key_valid_len < 0 || key_valid_len > Nkv) return DIT_ERR_INVALID_ARG;
    bool done;
    dit_status_t e = check_common(B, Nq, H, Hkv, D, window, scale, done);
    if (e != DIT_OK) return e;
    if (Nkv > kMaxTokens || std::abs(static_cast<int64_t>(q_offset)) + Nq > kMaxTokens) return DIT_ERR_UNSUPPORTED;
    if (!known(out_dtype)) return DIT_ERR_INVALID_ARG;
    if (done) return DIT_OK;
    if ((e = check_out(out, out_dtype, strides->o, lse, B, Nq, H)) != DIT_OK) return e;
    const bool any_keys = key_valid_len > 0;
    CUtensorMap tq, tk, tv;
    for (CUtensorMap* m : {&tq, &tk, &tv}) std::memset(m, 0, sizeof *m);
    if (any_keys) {
        if (!q || !k || !v) return DIT_ERR_INVALID_ARG;
        for (const dit_strides4_t* s : {&strides->q, &strides->k, &strides->v})
            if ((e = check_tma_strides(*s)) != DIT_OK) return e;
        if (!aligned16(q) || !aligned16(k) || !aligned16(v)) return DIT_ERR_ALIGNMENT;
        for (const void* in : {q, k, v, static_cast<const void*>(lse), static_cast<const void*>(workspace)})
            if (out == in) return DIT_ERR_INVALID_ARG;
    }
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return DIT_ERR_CUDA;
    WindowArgs a{};
    fill_common(a, B, Nq, H, Hkv, *window, scale, out, out_dtype, strides->o, lse, D);
    a.kv_len = key_valid_len;
    a.offset = q_offset;
    const GridPlan plan = any_keys ? plan_of(B, Nq, H, Hkv, *window, q_offset, key_valid_len, device_sm_count(dev)) : GridPlan{};
    if ((e = set_grid(a, plan, D, workspace, workspace_bytes)) != DIT_OK) return e;
    if ((e = check_placement({any_keys ? q : nullptr, any_keys ? k : nullptr, any_keys ? v : nullptr, out, lse, plan.f > 1 ? workspace : nullptr},
                             stream)) != DIT_OK)
        return e;
    if (any_keys) {
        if ((e = encode_q(&tq, q, strides->q, B, Nq, H, Hkv, D, a.tokens)) != DIT_OK) return e;
        if ((e = encode_view(&tk, k, strides->k, B, key_valid_len, Hkv, D)) != DIT_OK) return e;
        if ((e = encode_view(&tv, v, strides->v, B, key_valid_len, Hkv, D)) != DIT_OK) return e;
    }
    a.status = status_word(dev);
    if (a.status == nullptr) return DIT_ERR_CUDA;
    return launch_attn_window(tq, tk, tv, a, D, false, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess ? DIT_OK : DIT_ERR_CUDA;
}

dit_status_t dit_paged_append(const void* k, const dit_strides4_t* k_strides, const void* v, const dit_strides4_t* v_strides,
                              const dit_paged_cache_t* cache, const int32_t* new_lens, int B, int T, int Hkv, int D,
                              dit_stream_t stream) {
    if (B < 0 || T < 0 || Hkv < 0 || D < 0 || k_strides == nullptr || v_strides == nullptr) return DIT_ERR_INVALID_ARG;
    int64_t capacity;
    dit_status_t e = check_cache(cache, capacity);
    if (e != DIT_OK) return e;
    if (D % 8 != 0 || D > 1024 || B > 65535 || T > kMaxTokens) return DIT_ERR_UNSUPPORTED;
    if (B == 0 || T == 0 || Hkv == 0 || D == 0 || capacity == 0 || cache->pages == 0) return DIT_OK;
    const double units = static_cast<double>(B) * T * Hkv * (D / 8) * 2;
    if (units >= 2147483648.0) return DIT_ERR_UNSUPPORTED;
    if (k == nullptr || v == nullptr) return DIT_ERR_INVALID_ARG;
    if ((e = check_in_strides(*k_strides)) != DIT_OK || (e = check_in_strides(*v_strides)) != DIT_OK) return e;
    if (!on(k, 2) || !on(v, 2) || !on(new_lens, 4)) return DIT_ERR_ALIGNMENT;
    if (k == cache->k || k == cache->v || v == cache->k || v == cache->v || cache->k == cache->v) return DIT_ERR_INVALID_ARG;
    if ((e = check_placement({k, v, cache->k, cache->v, cache->table, cache->kv_lens, new_lens}, stream)) != DIT_OK) return e;
    AppendArgs a{};
    a.k = static_cast<const uint16_t*>(k);
    a.v = static_cast<const uint16_t*>(v);
    a.k_cache = static_cast<uint16_t*>(cache->k);
    a.v_cache = static_cast<uint16_t*>(cache->v);
    a.sk = *k_strides;
    a.sv = *v_strides;
    a.dk = cache->k_strides;
    a.dv = cache->v_strides;
    a.table = cache->table;
    a.kv_lens = cache->kv_lens;
    a.new_lens = new_lens;
    a.table_sb = cache->table_stride;
    a.capacity = capacity;
    a.T = T;
    a.pages = cache->pages;
    a.n = static_cast<uint32_t>(units);
    a.half = static_cast<uint32_t>(Hkv) * static_cast<uint32_t>(D / 8);
    a.div_parts = FastDiv(2 * a.half);
    a.div_t = FastDiv(static_cast<uint32_t>(T));
    a.div_d8 = FastDiv(static_cast<uint32_t>(D / 8));
    a.div_page = FastDiv(static_cast<uint32_t>(cache->page_size));
    const bool vec = aligned16(k) && aligned16(v) && multiple(a.sk, 8) && multiple(a.sv, 8);
    return launch_paged_append(a, vec, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess ? DIT_OK : DIT_ERR_CUDA;
}

size_t dit_attn_fwd_paged_workspace_bytes(int B, int T, int H, int Hkv, int D, int page_size, int table_width,
                                          const dit_window_t* window) {
    bool done;
    if (check_common(B, T, H, Hkv, D, window, 1.f, done) != DIT_OK || done || page_size <= 0 || table_width <= 0) return 0;
    const int64_t capacity = static_cast<int64_t>(page_size) * table_width;
    int dev = 0;
    if (capacity > 0x7fffff00LL || cudaGetDevice(&dev) != cudaSuccess) return 0;
    const int f = paged_plan_of(B, T, H, Hkv, *window, capacity, device_sm_count(dev)).f;
    return static_cast<size_t>(pieces_bytes(items_of(B, T, H, Hkv), f, part_rows_of(T, H / Hkv), D));
}

dit_status_t dit_attn_fwd_paged(const void* q, const dit_strides4_t* q_strides, const dit_paged_cache_t* cache, const int32_t* q_lens,
                                int B, int T, int H, int Hkv, int D, const dit_window_t* window, float scale, void* out,
                                dit_dtype_t out_dtype, const dit_strides4_t* out_strides, float* lse, void* workspace,
                                size_t workspace_bytes, dit_stream_t stream) {
    if (q_strides == nullptr || out_strides == nullptr) return DIT_ERR_INVALID_ARG;
    bool done;
    dit_status_t e = check_common(B, T, H, Hkv, D, window, scale, done);
    if (e != DIT_OK) return e;
    int64_t capacity;
    if ((e = check_cache(cache, capacity)) != DIT_OK) return e;
    if (!known(out_dtype)) return DIT_ERR_INVALID_ARG;
    if (done) return DIT_OK;
    if ((e = check_out(out, out_dtype, *out_strides, lse, B, T, H)) != DIT_OK) return e;
    if (!on(q_lens, 4)) return DIT_ERR_ALIGNMENT;
    const bool any_keys = capacity > 0 && cache->pages > 0;
    CUtensorMap tq, tk, tv;
    for (CUtensorMap* m : {&tq, &tk, &tv}) std::memset(m, 0, sizeof *m);
    if (any_keys) {
        if (q == nullptr) return DIT_ERR_INVALID_ARG;
        if ((e = check_tma_strides(*q_strides)) != DIT_OK) return e;
        if (!aligned16(q)) return DIT_ERR_ALIGNMENT;
        for (const void* in : {q, static_cast<const void*>(cache->k), static_cast<const void*>(cache->v), static_cast<const void*>(lse),
                               static_cast<const void*>(workspace)})
            if (out == in) return DIT_ERR_INVALID_ARG;
    }
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return DIT_ERR_CUDA;
    WindowArgs a{};
    fill_common(a, B, T, H, Hkv, *window, scale, out, out_dtype, *out_strides, lse, D);
    a.table = cache->table;
    a.table_sb = cache->table_stride;
    a.kv_lens = cache->kv_lens;
    a.q_lens = q_lens;
    a.n_pages = cache->pages;
    a.page = cache->page_size;
    a.chunk = chunk_of(cache->page_size);
    a.capacity = any_keys ? static_cast<int>(capacity) : 0;
    a.div_page = FastDiv(static_cast<uint32_t>(cache->page_size));
    const GridPlan plan = any_keys ? paged_plan_of(B, T, H, Hkv, *window, capacity, device_sm_count(dev)) : GridPlan{};
    if ((e = set_grid(a, plan, D, workspace, workspace_bytes)) != DIT_OK) return e;
    if ((e = check_placement({any_keys ? q : nullptr, any_keys ? cache->k : nullptr, any_keys ? cache->v : nullptr,
                              any_keys ? cache->table : nullptr, cache->kv_lens, q_lens, out, lse, plan.f > 1 ? workspace : nullptr},
                             stream)) != DIT_OK)
        return e;
    if (any_keys) {
        if ((e = encode_q(&tq, q, *q_strides, B, T, H, Hkv, D, a.tokens)) != DIT_OK) return e;
        if ((e = encode_pages(&tk, cache->k, cache->k_strides, *cache, Hkv, D, a.chunk)) != DIT_OK) return e;
        if ((e = encode_pages(&tv, cache->v, cache->v_strides, *cache, Hkv, D, a.chunk)) != DIT_OK) return e;
    }
    a.status = status_word(dev);
    if (a.status == nullptr) return DIT_ERR_CUDA;
    return launch_attn_window(tq, tk, tv, a, D, true, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess ? DIT_OK : DIT_ERR_CUDA;
}

}  // extern "C"

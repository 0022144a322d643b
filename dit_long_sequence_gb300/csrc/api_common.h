// api_common.h -- host-side pieces shared by the C-ABI files (api.cu,
// api_train.cu): placement and alignment checks, tensor maps, the device
// status word.  Defined in api.cu.
#pragma once

#include <cstdint>
#include <cuda.h>
#include <initializer_list>

#include "dit_attn.h"

namespace dit {

constexpr unsigned long long kWatchdogNs = 2000000000ull;  // 2 s per bounded wait

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// Device address of the status word in the current context, nullptr on failure.
unsigned int* status_word(int dev);

// Every buffer a kernel will touch must be memory of the current device (or
// managed memory), and the stream one of the current device's: a host address
// or another device's memory handed to a TMA copy or a store is refused here,
// before anything is enqueued, instead of faulting the GPU.  Null entries are
// skipped (the caller has already decided which buffers are required).
dit_status_t check_placement(std::initializer_list<const void*> ptrs, dit_stream_t stream);

// A [B, N, H, D] view as a 4-D TMA map (D, N, H, B) with 128-byte swizzle and
// a box of one swizzle column (64 bf16 or 128 E4M3 channels) by 128 rows.
// Rows n >= n_rows are outside the map and read as zeros.
dit_status_t encode_view(CUtensorMap* map, const void* base, const dit_strides4_t& s, int B, int n_rows, int H, int D,
                         bool fp8 = false);

// b, n, h strides of a TMA operand: positive, 16-byte multiples, < 2^39 elements.
dit_status_t check_tma_strides(const dit_strides4_t& s, bool fp8 = false);

// Strides of an output: d contiguous, no two rows of a dimension at one place.
inline dit_status_t check_out_strides(const dit_strides4_t& s, int64_t B, int64_t N, int64_t H) {
    if (s.d != 1) return DIT_ERR_UNSUPPORTED;
    const int64_t st[3] = {s.b, s.n, s.h}, ext[3] = {B, N, H};
    for (int i = 0; i < 3; ++i)
        if (st[i] < 0 || st[i] >= (int64_t(1) << 39) || (ext[i] > 1 && st[i] == 0)) return DIT_ERR_INVALID_ARG;
    return DIT_OK;
}
// Strides of an input read with plain loads (0 broadcasts).
inline dit_status_t check_in_strides(const dit_strides4_t& s) {
    if (s.d != 1) return DIT_ERR_UNSUPPORTED;
    for (int64_t x : {s.b, s.n, s.h})
        if (x < 0 || x >= (int64_t(1) << 39)) return DIT_ERR_INVALID_ARG;
    return DIT_OK;
}
inline bool multiple(const dit_strides4_t& s, int64_t k) { return s.b % k == 0 && s.n % k == 0 && s.h % k == 0; }
inline bool on(const void* p, uintptr_t bytes) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0; }
inline bool known(dit_dtype_t t) { return t == DIT_BF16 || t == DIT_F32; }
inline uintptr_t size_of(dit_dtype_t t) { return t == DIT_F32 ? 4 : 2; }
// Two views that begin at one address place every row alike.
inline bool same_rows(const dit_strides4_t& s, const dit_strides4_t& t, int B, int N, int H) {
    return (B == 1 || s.b == t.b) && (N == 1 || s.n == t.n) && (H == 1 || s.h == t.h);
}

// A tiled map of bf16 elements: `rank` dimensions innermost first, strides in bytes
// of all but the first, 128-byte swizzle, a box of 64 channels.  Elements outside
// are read as zeros.
dit_status_t encode_tiles(CUtensorMap* map, const void* base, int rank, const uint64_t* dims, const uint64_t* strides,
                          const uint32_t* box);

#ifdef DIT_DEBUG
// The wait limit (0: the default) and the extent shrink dit_debug_configure set.
unsigned long long debug_wait_limit_ns();
int64_t debug_extent_shrink();
#endif

}  // namespace dit

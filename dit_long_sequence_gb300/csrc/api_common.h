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

#ifdef DIT_DEBUG
// The wait limit (0: the default) and the extent shrink dit_debug_configure set.
unsigned long long debug_wait_limit_ns();
int64_t debug_extent_shrink();
#endif

}  // namespace dit

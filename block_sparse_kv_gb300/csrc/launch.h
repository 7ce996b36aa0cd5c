// Host-side helpers shared by the kernel launchers of libbskv.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <atomic>

#include "common.cuh"
#include "internal.h"

namespace bskv {

bskv_status cuda_check(cudaError_t e, const char* what);
bskv_status status_args(dev::StatusArgs* out);

// cuTensorMapEncodeTiled through the runtime's driver entry point (no -lcuda link).
// dims/strides are innermost first; strides_bytes has rank-1 entries (dim 1 upward).
bskv_status encode_tiled(CUtensorMap* map, CUtensorMapDataType dt, int rank, const void* base,
                         const uint64_t* dims, const uint64_t* strides_bytes,
                         const uint32_t* box, CUtensorMapSwizzle swizzle);

// Pointers and strides (bytes) of a 4-bit paged cache: codes {page, K/V, head, slot}, scales
// {page, K/V, head} (a slot's scales contiguous, slots contiguous).
bskv_status check_fp4_cache(const char* who, const void* kv_codes, const int64_t* codes_strides,
                            const void* kv_scales, const int64_t* scales_strides);

// Merge the split-KV partial states of a decode plan into out / lse (zero-filling units without
// tokens): slot_rows query heads per unit, units_per_request units per request.
bskv_status launch_state_merge(const bskv_plan* plan, const int32_t* meta, float* ws_o,
                               float* ws_lse, void* out, const int64_t* out_strides, float* lse,
                               int units_per_request, int slot_rows, cudaStream_t stream);

// Allow a kernel `bytes` of dynamic shared memory on the current device, asking the runtime only
// when it has not been allowed as much there before.
bskv_status allow_smem(const void* kernel, size_t bytes, std::atomic<int> (&allowed)[64], const char* what);

// Checks that the two runs of a block-sparse plan share.
bskv_status check_blocks_run(const char* who, const bskv_plan* plan, const int32_t* batch_indices,
                             const int32_t* positions, const int32_t* kv_indptr, const int32_t* kv_indices,
                             int32_t batch, const int32_t* blocks, const void* float_ws, size_t float_ws_bytes);

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

inline int32_t meta_word(const bskv_plan* p, int h) { return p->meta[size_t(h)]; }

}  // namespace bskv

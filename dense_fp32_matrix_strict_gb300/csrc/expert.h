// expert.h — what the expert-layer entry points share (router, grouped
// products, 4-bit matrix-vector products): element types, the status bit of
// a bad offset or expert index, argument helpers.
#pragma once

#include <cstdint>

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "sgemm.h"
#include "sgemm_internal.h"

namespace sg {

// Status bit (beside those of sgemm_kernel.cuh): an offset or an expert
// index read on the device was out of range; the kernel skipped it.
constexpr int STATUS_BAD_INDEX = 32;

constexpr int64_t kMaxDim = 0x7fffffff;              // of what only int64 arithmetic touches
// Of sizes that the product kernels count in 32 bits. They step past a size by
// a tile, or in the streaming kernel by a slab of at most 8192 k.
constexpr int64_t kMaxGroupedDim = SGEMM_GROUPED_MAX_DIM;
constexpr int64_t kMaxOffset = int64_t{1} << 59;     // elements; fits in int64 bytes
constexpr int kMaxGroups = 1024;                     // experts of one call

inline bool ptr_aligned(const void* p, uintptr_t a) {
    return (reinterpret_cast<uintptr_t>(p) % a) == 0;
}

inline size_t type_bytes(int type) { return type == SGEMM_TYPE_BF16 ? 2 : 4; }

// [lo, hi) byte ranges overlap.
inline bool ranges_overlap(const void* a, int64_t a_bytes, const void* b, int64_t b_bytes) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return a_bytes > 0 && b_bytes > 0 && x < y + static_cast<uintptr_t>(b_bytes) &&
           y < x + static_cast<uintptr_t>(a_bytes);
}

// Bytes spanned by rows x cols elements with row stride ld.
inline int64_t span_bytes(int64_t rows, int64_t cols, int64_t ld, size_t elem) {
    return rows > 0 && cols > 0 ? ((rows - 1) * ld + cols) * static_cast<int64_t>(elem) : 0;
}

__device__ __forceinline__ float load_f32(const float* p) { return *p; }
__device__ __forceinline__ float load_f32(const __nv_bfloat16* p) { return __bfloat162float(*p); }
__device__ __forceinline__ void store_f32(float* p, float v) { *p = v; }
// One rounding (to nearest even) of the 32-bit result to the output's type.
__device__ __forceinline__ void store_f32(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }

}  // namespace sg

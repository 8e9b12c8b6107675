// grouped_internal.h — the kernels behind the grouped entry points.
#pragma once

#include "grouped.cuh"

namespace sg {
namespace grouped {

// All take something to sum (K and rows above zero). The first two load by
// TMA: x and w with bases, row and matrix strides on 16 bytes (launch_f32's
// forward w only if w_tma says so).
// bfloat16 on the tensor cores; forward and weight gradient.
cudaError_t launch_bf16(const Params& p, bool wgrad, const DeviceInfo* dev, cudaStream_t stream);
// float in FP32 FMAs; forward and weight gradient.
cudaError_t launch_f32(const Params& p, bool wgrad, const DeviceInfo* dev, cudaStream_t stream);
// Forward of float groups of a few rows, any alignment.
cudaError_t launch_skinny(const Params& p, const DeviceInfo* dev, cudaStream_t stream);

// Parts it splits sums into.
int skinny_parts(const Params& p, const DeviceInfo* dev);

// What a tile kernel's last round is about: workers, tiles (an upper bound:
// the groups' sizes are not known), blocks of k of a sum (the mean), fewest to
// a piece, fewest worth a second kernel; when a round is then cut (see
// TailRule); bytes of a slot.
struct Tail {
    int64_t workers = 0, items = 0, blocks = 0, min_blocks = 0, worth = 0;
    TailRule rule;
    size_t slot_bytes = 0;
};
Tail bf16_tail(const Params& p, bool wgrad, const DeviceInfo* dev);
Tail f32_tail(const Params& p, bool wgrad, const DeviceInfo* dev);

}  // namespace grouped
}  // namespace sg

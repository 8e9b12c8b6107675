// The kernels of w4_matvec.cuh for bfloat16 tokens, rows of weights on any byte.
#include "w4_matvec.cuh"

namespace sg {
namespace w4 {

int run_bf16_bytes(const __nv_bfloat16* x, const __nv_bfloat16* scales, __nv_bfloat16* y, Params p, int group,
                  const DeviceInfo* dev, cudaMemPool_t pool, cudaStream_t stream) {
    return run<__nv_bfloat16, 1>(x, scales, y, p, group, dev, pool, stream);
}

}  // namespace w4
}  // namespace sg

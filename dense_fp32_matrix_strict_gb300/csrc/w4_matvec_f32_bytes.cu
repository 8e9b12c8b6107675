// The kernels of w4_matvec.cuh for float tokens, rows of weights on any byte.
#include "w4_matvec.cuh"

namespace sg {
namespace w4 {

int run_f32_bytes(const float* x, const float* scales, float* y, Params p, int group,
                  const DeviceInfo* dev, cudaMemPool_t pool, cudaStream_t stream) {
    return run<float, 1>(x, scales, y, p, group, dev, pool, stream);
}

}  // namespace w4
}  // namespace sg

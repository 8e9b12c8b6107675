// w4_matvec.cu — the entry point of the products with 4-bit weights (the kernel
// and its launch: w4_matvec.cuh, compiled for each type and alignment in a file
// of its own).
#include "w4_matvec.cuh"

namespace sg {
namespace w4 {
// Rows of weights that start on 16 bytes, on 4, anywhere.
template <typename X>
using Run = int(const X* x, const X* scales, X* y, Params p, int group, const DeviceInfo* dev,
                cudaMemPool_t pool, cudaStream_t stream);
Run<float> run_f32, run_f32_words, run_f32_bytes;
Run<__nv_bfloat16> run_bf16, run_bf16_words, run_bf16_bytes;

}  // namespace w4
}  // namespace sg

using namespace sg;

extern "C" int sgemv_w4(int type, int64_t pairs, int64_t repeat, int64_t N, int64_t K,
                        int64_t group, const void* X, int64_t ldx, const uint8_t* Q, int64_t ldq,
                        int64_t stride_q, const void* scales, const uint8_t* zeros,
                        int64_t num_experts, const int32_t* experts, void* Y, int64_t ldy,
                        cudaStream_t stream) {
    using namespace sg::w4;
    if (type != SGEMM_TYPE_F32 && type != SGEMM_TYPE_BF16) return SGEMM_ERR_INVALID_VALUE;
    if (group != 32 && group != 64 && group != 128) return SGEMM_ERR_INVALID_VALUE;
    if (pairs < 0 || N < 0 || K < 0 || pairs > 65535 || N > kMaxGroupedDim || K > SGEMV_W4_MAX_K ||
        repeat < 1 || pairs % repeat != 0)
        return SGEMM_ERR_INVALID_VALUE;
    const int64_t bytes = (K + 1) / 2, groups = (K + group - 1) / group;
    const int64_t xrows = pairs / repeat;
    if (ldx < (K > 1 ? K : 1) || ldq < (bytes > 1 ? bytes : 1) || ldy < (N > 1 ? N : 1))
        return SGEMM_ERR_INVALID_VALUE;
    if ((xrows > 0 && ldx > kMaxOffset / xrows) || (N > 0 && ldq > kMaxOffset / N) ||
        (pairs > 0 && ldy > kMaxOffset / pairs))
        return SGEMM_ERR_INVALID_VALUE;
    int64_t copies = 1;
    if (experts != nullptr) {
        if (num_experts < 1 || num_experts > kMaxDim || !ptr_aligned(experts, 4) || stride_q < 0 ||
            stride_q > kMaxOffset / num_experts)
            return SGEMM_ERR_INVALID_VALUE;
        copies = num_experts;
    }
    if (pairs == 0 || N == 0) return SGEMM_OK;
    const size_t es = type_bytes(type);
    if (Y == nullptr || !ptr_aligned(Y, es)) return SGEMM_ERR_INVALID_VALUE;
    const int64_t y_span = span_bytes(pairs, N, ldy, es);
    if (K > 0) {
        if (X == nullptr || Q == nullptr || scales == nullptr || !ptr_aligned(X, es) ||
            !ptr_aligned(scales, es))
            return SGEMM_ERR_INVALID_VALUE;
        if (ranges_overlap(Y, y_span, X, span_bytes(xrows, K, ldx, es)) ||
            ranges_overlap(Y, y_span, Q, (copies - 1) * stride_q + span_bytes(N, bytes, ldq, 1)) ||
            ranges_overlap(Y, y_span, scales, copies * N * groups * static_cast<int64_t>(es)) ||
            (zeros != nullptr && ranges_overlap(Y, y_span, zeros, copies * N * groups)))
            return SGEMM_ERR_INVALID_VALUE;
    }
    if (experts != nullptr && ranges_overlap(Y, y_span, experts, pairs * 4))
        return SGEMM_ERR_INVALID_VALUE;
    const DeviceInfo* dev = nullptr;
    int rc = device_info(&dev);
    if (rc != SGEMM_OK) return rc;
    int* status = nullptr;
    cudaMemPool_t pool = nullptr;
    if ((rc = device_memory_handles(dev, &status, &pool)) != SGEMM_OK) return rc;
    if (K == 0) {
        const cudaError_t e = cudaMemset2DAsync(Y, static_cast<size_t>(ldy) * es, 0,
                                                static_cast<size_t>(N) * es,
                                                static_cast<size_t>(pairs), stream);
        return e == cudaSuccess ? SGEMM_OK : cuda_fail(e, SGEMM_ERR_CUDA);
    }
    Params p;
    std::memset(&p, 0, sizeof(p));
    p.N = static_cast<int>(N);
    p.K = static_cast<int>(K);
    p.groups = static_cast<int>(groups);
    p.units = static_cast<int>((K + UNIT_K - 1) / UNIT_K);
    p.tiles = static_cast<int>((N + 15) / 16);
    p.pairs = pairs;
    p.repeat = repeat;
    p.ldx = ldx;
    p.ldq = ldq;
    p.stride_q = experts != nullptr ? stride_q : 0;
    p.ldy = ldy;
    p.q = Q;
    p.zeros = zeros;
    p.experts = experts;
    p.num_experts = static_cast<int>(copies);
    auto rows_on = [&](int bytes) {
        return ptr_aligned(Q, bytes) && ldq % bytes == 0 && (experts == nullptr || stride_q % bytes == 0);
    };
    p.q_end = Q + (copies - 1) * p.stride_q + span_bytes(N, bytes, ldq, 1);
    // A unit starts UNIT_K / group elements after the last: rows of scales
    // (and zeros) have to start on 4 bytes, too.
    p.meta4 = ptr_aligned(scales, 4) && groups * static_cast<int64_t>(es) % 4 == 0 &&
              (zeros == nullptr || (ptr_aligned(zeros, 4) && groups % 4 == 0));
    p.status = status;
    const int place = rows_on(16) ? 0 : rows_on(4) ? 1 : 2;
    if (type == SGEMM_TYPE_BF16) {
        constexpr Run<__nv_bfloat16>* RUNS[3] = {run_bf16, run_bf16_words, run_bf16_bytes};
        return RUNS[place](static_cast<const __nv_bfloat16*>(X), static_cast<const __nv_bfloat16*>(scales),
                           static_cast<__nv_bfloat16*>(Y), p, static_cast<int>(group), dev, pool,
                           stream);
    }
    constexpr Run<float>* RUNS[3] = {run_f32, run_f32_words, run_f32_bytes};
    return RUNS[place](static_cast<const float*>(X), static_cast<const float*>(scales),
                       static_cast<float*>(Y), p, static_cast<int>(group), dev, pool, stream);
}

// grouped.cu — matrix products grouped by expert with ragged sizes: the entry
// points, the choice of a kernel, and the small kernels beside the products.
//
//   forward / input gradient:  Y[r] = alpha * X[r] op(W_g) + beta * Y[r]
//   weight gradient:           D_g = alpha * P_g^T Q_g + beta * D_g
// where group g holds the rows offsets[g] .. offsets[g + 1], known on the
// device only: one launch covers all groups, its blocks walk the tiles that
// the offsets give.
#include <cstring>

#include "grouped.cuh"
#include "grouped_internal.h"

namespace sg {
namespace grouped {

// Calls without a sum (alpha == 0, K == 0, no rows at all): beta times the rows
// of Y that belong to a group, or times every D_g. 32 rows x 256 columns per
// item, neighbouring threads on neighbouring columns; bound by its bytes.
constexpr int SCALE_ROWS = 32, SCALE_COLS = 256;

template <typename O, bool WGRAD>
__global__ void __launch_bounds__(SCALE_COLS) scale_kernel(const Params p) {
    extern __shared__ int sched_sm[];
    const Schedule sch = build_schedule(p, SCALE_ROWS, sched_sm);
    const int strips = (p.N + SCALE_COLS - 1) / SCALE_COLS;
    const int tiles_m = (p.K + SCALE_ROWS - 1) / SCALE_ROWS;      // weight gradient: K is M
    const int64_t items =
        strips * (WGRAD ? static_cast<int64_t>(p.groups) * tiles_m : static_cast<int64_t>(sch.start[p.groups]));
    for (int64_t item = blockIdx.x; item < items; item += gridDim.x) {
        const int64_t t = item / strips;
        const int n = static_cast<int>(item - t * strips) * SCALE_COLS + threadIdx.x;
        if (n >= p.N) continue;
        int64_t row, end;
        O* y = static_cast<O*>(p.y) + n;
        if (WGRAD) {
            const int64_t g = t / tiles_m;
            y += g * p.stride_y;
            row = (t - g * tiles_m) * SCALE_ROWS;
            end = p.K;
        } else {
            const int place = place_of(sch, p.groups, static_cast<int>(t));
            const int g = sch.perm[place];
            row = sch.off[g] + (t - sch.start[place]) * SCALE_ROWS;
            end = sch.off[g + 1];
        }
        end = min(end, row + SCALE_ROWS);
#pragma unroll 4
        for (; row < end; ++row) {
            O* o = y + row * p.ldy;
            store_f32(o, p.beta != 0.0f ? fmaf(p.beta, load_f32(o), 0.0f) : 0.0f);
        }
    }
}

// dst (rows x ldd, a multiple of 16 bytes) <- src (rows x cols, row stride lds,
// any alignment), for `mats` matrices; padding columns get zeros. With offsets,
// the matrices of groups without rows are left out. A thread writes 16 bytes.
// Two such kernels run side by side and the product's prologue beside them:
// the second ends only when the first has, so waiting for it is enough.
template <typename T>
__global__ void __launch_bounds__(256) pack_kernel(const T* __restrict__ src, int64_t lds,
                                                   int64_t stride, T* __restrict__ dst, int64_t ldd,
                                                   int64_t rows, int64_t cols, int mats,
                                                   const int* offsets) {
    constexpr int V = 16 / sizeof(T);
    griddep_launch_dependents();
    const int64_t pieces = ldd / V;
    const int64_t per = rows * pieces;
    for (int m = blockIdx.y; m < mats; m += gridDim.y) {
        if (offsets != nullptr && offsets[m + 1] <= offsets[m]) continue;
        const T* s0 = src + m * stride;
        T* d0 = dst + m * rows * ldd;
        for (int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; i < per;
             i += static_cast<int64_t>(gridDim.x) * 256) {
            const int64_t r = i / pieces, c = (i - r * pieces) * V;
            const T* s = s0 + r * lds + c;
            __align__(16) T v[V];
#pragma unroll
            for (int j = 0; j < V; ++j) v[j] = c + j < cols ? s[j] : T(0.0f);
            *reinterpret_cast<uint4*>(d0 + r * ldd + c) = *reinterpret_cast<const uint4*>(v);
        }
    }
    griddep_wait();
}

// One operand that TMA cannot read in place: rows x cols, mats of them.
struct Packed {
    bool on = false;
    int64_t rows = 0, cols = 0, mats = 1, ld = 0;
    size_t bytes = 0;
};

Packed plan_pack(const void* ptr, int64_t rows, int64_t cols, int64_t mats, int64_t ld,
                 int64_t stride, int64_t vec) {
    Packed k;
    const int64_t far = int64_t{1} << 37;             // TMA's limit on strides
    k.on = !ptr_aligned(ptr, 16) || ld % vec != 0 || ld >= far ||
           (mats > 1 && (stride % vec != 0 || stride >= far));
    k.rows = rows;
    k.cols = cols;
    k.mats = mats;
    k.ld = (cols + vec - 1) / vec * vec;
    k.bytes = k.on ? (static_cast<size_t>(mats) * rows * k.ld * (16 / vec) + 255) & ~size_t{255} : 0;
    return k;
}

cudaError_t pack(int type, const Packed& k, const void* src, int64_t ld, int64_t stride, void* dst,
                 const int* offsets, const DeviceInfo* dev, cudaStream_t stream, bool pdl) {
    const int64_t vec = type == SGEMM_TYPE_BF16 ? 8 : 4;
    const int64_t blocks = (k.rows * (k.ld / vec) + 255) / 256;
    const int64_t most = 16 * static_cast<int64_t>(dev->sm_count);
    const dim3 grid(static_cast<unsigned>(blocks < most ? blocks : most),
                    static_cast<unsigned>(k.mats < 1024 ? k.mats : 1024));
    if (type == SGEMM_TYPE_BF16)
        return launch_kernel(pack_kernel<__nv_bfloat16>, grid, dim3(256), 0, stream, pdl, 1,
                             static_cast<const __nv_bfloat16*>(src), ld, stride,
                             static_cast<__nv_bfloat16*>(dst), k.ld, k.rows, k.cols,
                             static_cast<int>(k.mats), offsets);
    return launch_kernel(pack_kernel<float>, grid, dim3(256), 0, stream, pdl, 1,
                         static_cast<const float*>(src), ld, stride, static_cast<float*>(dst), k.ld,
                         k.rows, k.cols, static_cast<int>(k.mats), offsets);
}

// Joins the parts of the streaming kernel's split sums, in order: y = alpha *
// sum + beta * y. ws holds [part][row][N]; only rows of valid groups are read
// and written.
constexpr int JOIN_ROWS = 4;

__global__ void __launch_bounds__(256) join_kernel(const float* __restrict__ ws, const Params p) {
    extern __shared__ int sched_sm[];
    const Schedule sch = build_schedule(p, JOIN_ROWS, sched_sm);
    const int strips = (p.N + 255) / 256;
    griddep_wait();                                    // (the offsets are older than the kernel before)
    const int64_t tiles = sch.start[p.groups];
    for (int64_t i = blockIdx.x; i < tiles * strips; i += gridDim.x) {
        const int64_t t = i / strips;
        const int n = static_cast<int>(i - t * strips) * 256 + threadIdx.x;
        const int place = place_of(sch, p.groups, static_cast<int>(t));
        const int g = sch.perm[place];
        const int64_t row = sch.off[g] + (t - sch.start[place]) * JOIN_ROWS;
        const int64_t end = sch.off[g + 1];
        if (n >= p.N) continue;
#pragma unroll
        for (int j = 0; j < JOIN_ROWS; ++j) {
            if (row + j >= end) break;
            const float* at = ws + (row + j) * p.N + n;
            float v = 0.0f;
#pragma unroll 4
            for (int q = 0; q < p.parts; ++q) v += at[q * p.part_stride];
            float* o = static_cast<float*>(p.y) + (row + j) * p.ldy + n;
            v *= p.alpha;
            *o = p.beta != 0.0f ? fmaf(p.beta, *o, v) : v;
        }
    }
}

// Mean rows per group up to which float takes the streaming kernel (against
// 32-row tiles; 32 groups of 10, 2048 x 2048, W stored N x K: 199 and 212 us,
// of 12: 209 and 211, uneven groups and unaligned W sooner; W stored K x N, of
// 9: 184 and 171). The mean is all that the host knows: where one group holds
// most rows, W is read once for every 8 of them (1024 rows, 2048 x 2048, all in
// one of 128 groups: 414 us stored N x K, 380 K x N, from L2; a call with that
// group alone takes tiles, 178 and 155).
constexpr int64_t skinny_rows(int opw) { return opw ? 10 : 8; }
// Rounds of tiles from which on the last one is left as it is: cutting it
// gains half a round in the mean and costs a second kernel.
constexpr int64_t kCutRounds = 5;

cudaError_t run_skinny(Params p, const DeviceInfo* dev, cudaMemPool_t pool, cudaStream_t stream) {
    p.parts = skinny_parts(p, dev);
    p.part_stride = 0;
    void* ws = nullptr;
    if (p.parts > 1) {
        const int64_t part = p.rows * static_cast<int64_t>(p.N);
        if (cudaMallocFromPoolAsync(&ws, static_cast<size_t>(p.parts * part) * 4, pool, stream) !=
            cudaSuccess) {
            (void)cudaGetLastError();
            p.parts = 1;
        } else {
            p.part_stride = part;
        }
    }
    if (p.parts == 1) return launch_skinny(p, dev, stream);
    Params q = p;
    q.y = ws;
    q.ldy = p.N;
    q.alpha = 1.0f;
    q.beta = 0.0f;
    cudaError_t e = launch_skinny(q, dev, stream);
    if (e == cudaSuccess) {
        const int64_t used = p.rows < p.groups ? p.rows : p.groups;
        const int64_t work = (p.rows / JOIN_ROWS + used) * ((p.N + 255) / 256);
        const int64_t most = 8 * static_cast<int64_t>(dev->sm_count);
        e = launch_kernel(join_kernel, dim3(static_cast<unsigned>(work < most ? work : most)), dim3(256),
                          schedule_ints(p.groups) * sizeof(int), stream, pdl_enabled(), 1,
                          static_cast<const float*>(ws), p);
    }
    cudaFreeAsync(ws, stream);
    return e;
}

// Copies that the product cannot do without and slots that it can: without
// memory for the copies the call fails, without slots the last round stays
// uncut.
cudaError_t run(int type, int out, bool wgrad, Params p, const DeviceInfo* dev, cudaMemPool_t pool,
                cudaStream_t stream) {
    const bool half = type == SGEMM_TYPE_BF16;
    const int64_t vec = half ? 8 : 4;
    p.y_vec = ptr_aligned(p.y, 16) && p.ldy % 4 == 0 && p.stride_y % 4 == 0;
    p.parts = 1;
    p.part_stride = 0;
    p.tail_ws = nullptr;
    p.pdl = 0;
    if (p.K == 0 || p.rows == 0 || p.x == nullptr) {
        void (*const scale)(Params) =
            wgrad ? (out == SGEMM_TYPE_BF16 ? &scale_kernel<__nv_bfloat16, true> : &scale_kernel<float, true>)
                  : (half ? &scale_kernel<__nv_bfloat16, false> : &scale_kernel<float, false>);
        return launch_kernel(scale, dim3(4 * dev->sm_count), dim3(SCALE_COLS),
                             schedule_ints(p.groups) * sizeof(int), stream, false, 1, p);
    }
    if (!wgrad && !half && p.rows <= p.groups * skinny_rows(p.opw)) return run_skinny(p, dev, pool, stream);
    const Packed kx = plan_pack(p.x, p.rows, p.K, 1, p.ldx, 0, vec);
    Packed kw = wgrad ? plan_pack(p.w, p.rows, p.N, 1, p.ldw, 0, vec)
                      : plan_pack(p.w, p.opw ? p.N : p.K, p.opw ? p.K : p.N, p.groups, p.ldw,
                                  p.stride_w, vec);
    p.w_tma = !kw.on;
    if (!wgrad && !half) {
        kw.on = false;                                 // read in place
        kw.bytes = 0;
    }
    const Tail t = half ? bf16_tail(p, wgrad, dev) : f32_tail(p, wgrad, dev);
    bool cut = t.items < kCutRounds * t.workers && t.blocks >= t.worth;
    const size_t copies = kx.bytes + kw.bytes, slots = 2 * static_cast<size_t>(t.workers) * t.slot_bytes;
    void* ws = nullptr;
    cudaError_t e = cudaSuccess;
    if (cut && cudaMallocFromPoolAsync(&ws, copies + slots, pool, stream) != cudaSuccess) {
        (void)cudaGetLastError();
        cut = false;
    }
    if (!cut && copies > 0) e = cudaMallocFromPoolAsync(&ws, copies, pool, stream);
    if (e != cudaSuccess) return e;
    unsigned char* at = static_cast<unsigned char*>(ws);
    if (kx.on) {
        e = pack(type, kx, p.x, p.ldx, 0, at, nullptr, dev, stream, false);
        p.x = at;
        p.ldx = kx.ld;
    }
    if (kw.on && e == cudaSuccess) {
        void* w2 = at + kx.bytes;
        e = pack(type, kw, p.w, p.ldw, p.stride_w, w2, wgrad ? nullptr : p.offsets, dev, stream,
                 kx.on && pdl_enabled());
        p.w = w2;
        p.ldw = kw.ld;
        p.stride_w = kw.rows * kw.ld;
    }
    p.pdl = (kx.on || kw.on) && pdl_enabled();
    if (cut) p.tail_ws = reinterpret_cast<float*>(at + copies);
    if (e == cudaSuccess)
        e = half ? launch_bf16(p, wgrad, dev, stream) : launch_f32(p, wgrad, dev, stream);
    if (ws != nullptr) cudaFreeAsync(ws, stream);
    return e;
}

int launch(int type, int out, bool wgrad, const Params& p, const DeviceInfo* dev, cudaMemPool_t pool,
           cudaStream_t stream) {
    const cudaError_t e = run(type, out, wgrad, p, dev, pool, stream);
    if (e == cudaSuccess) return SGEMM_OK;
    (void)cudaGetLastError();
    return cuda_fail(e, e == cudaErrorMemoryAllocation ? SGEMM_ERR_CUDA : SGEMM_ERR_LAUNCH);
}

bool dims_ok(int64_t groups, int64_t rows, int64_t a, int64_t b) {
    return groups >= 0 && groups <= kMaxGroups && rows >= 0 && rows <= kMaxGroupedDim && a >= 0 &&
           a <= kMaxGroupedDim && b >= 0 && b <= kMaxGroupedDim;
}

bool ld_ok(int64_t rows, int64_t cols, int64_t ld) {
    return ld >= (cols > 1 ? cols : 1) && (rows == 0 || ld <= kMaxOffset / rows);
}

// The copies of a matrix for every group do not overlap one another and
// their offsets fit.
bool stride_ok(int64_t groups, int64_t rows, int64_t cols, int64_t ld, int64_t stride) {
    if (stride < 0 || (groups > 0 && stride > kMaxOffset / groups)) return false;
    return groups < 2 || rows == 0 || cols == 0 || stride >= (rows - 1) * ld + cols;
}

}  // namespace grouped
}  // namespace sg

using namespace sg;

extern "C" int sgemm_grouped(int opw, int type, int64_t groups, int64_t rows, int64_t N, int64_t K,
                             float alpha, const void* X, int64_t ldx, const void* W, int64_t ldw,
                             int64_t stride_w, const int32_t* offsets, float beta, void* Y,
                             int64_t ldy, cudaStream_t stream) {
    using namespace sg::grouped;
    if ((opw != SGEMM_OP_N && opw != SGEMM_OP_T) ||
        (type != SGEMM_TYPE_F32 && type != SGEMM_TYPE_BF16) || !dims_ok(groups, rows, N, K))
        return SGEMM_ERR_INVALID_VALUE;
    const int64_t wr = opw ? N : K, wc = opw ? K : N;
    if (!ld_ok(rows, K, ldx) || !ld_ok(wr, wc, ldw) || !ld_ok(rows, N, ldy) ||
        !stride_ok(groups, wr, wc, ldw, stride_w))
        return SGEMM_ERR_INVALID_VALUE;
    if (groups == 0 || rows == 0 || N == 0) return SGEMM_OK;
    const size_t es = type_bytes(type);
    const bool reads = alpha != 0.0f && K > 0;
    if (Y == nullptr || !ptr_aligned(Y, es) || offsets == nullptr || !ptr_aligned(offsets, 4))
        return SGEMM_ERR_INVALID_VALUE;
    const int64_t y_span = span_bytes(rows, N, ldy, es);
    if (ranges_overlap(Y, y_span, offsets, (groups + 1) * 4)) return SGEMM_ERR_INVALID_VALUE;
    if (reads) {
        if (X == nullptr || W == nullptr || !ptr_aligned(X, es) || !ptr_aligned(W, es))
            return SGEMM_ERR_INVALID_VALUE;
        const int64_t w_span = (groups - 1) * stride_w * static_cast<int64_t>(es) +
                               span_bytes(wr, wc, ldw, es);
        if (ranges_overlap(Y, y_span, X, span_bytes(rows, K, ldx, es)) ||
            ranges_overlap(Y, y_span, W, w_span))
            return SGEMM_ERR_INVALID_VALUE;
    }
    const DeviceInfo* dev = nullptr;
    int rc = device_info(&dev);
    if (rc != SGEMM_OK) return rc;
    int* status = nullptr;
    cudaMemPool_t pool = nullptr;
    if ((rc = device_memory_handles(dev, &status, &pool)) != SGEMM_OK) return rc;
    Params p;
    std::memset(&p, 0, sizeof(p));
    p.groups = static_cast<int>(groups);
    p.rows = rows;
    p.N = static_cast<int>(N);
    p.K = reads ? static_cast<int>(K) : 0;
    p.offsets = offsets;
    p.x = X;
    p.w = W;
    p.y = Y;
    p.ldx = ldx;
    p.ldw = ldw;
    p.stride_w = stride_w;
    p.ldy = ldy;
    p.alpha = alpha;
    p.beta = beta;
    p.opw = opw;
    p.out_bf16 = type == SGEMM_TYPE_BF16;
    p.timeout_ns = wait_timeout_ns();
    p.status = status;
    return launch(type, type, false, p, dev, pool, stream);
}

extern "C" int sgemm_grouped_wgrad(int type, int64_t groups, int64_t rows, int64_t M, int64_t N,
                                   float alpha, const void* P, int64_t ldp, const void* Q,
                                   int64_t ldq, const int32_t* offsets, float beta, int out_type,
                                   void* D, int64_t ldd, int64_t stride_d, cudaStream_t stream) {
    using namespace sg::grouped;
    if ((type != SGEMM_TYPE_F32 && type != SGEMM_TYPE_BF16) ||
        (out_type != SGEMM_TYPE_F32 && out_type != type) || !dims_ok(groups, rows, M, N))
        return SGEMM_ERR_INVALID_VALUE;
    if (!ld_ok(rows, M, ldp) || !ld_ok(rows, N, ldq) || !ld_ok(M, N, ldd) ||
        !stride_ok(groups, M, N, ldd, stride_d))
        return SGEMM_ERR_INVALID_VALUE;
    if (groups == 0 || M == 0 || N == 0) return SGEMM_OK;
    const size_t es = type_bytes(type), os = type_bytes(out_type);
    const bool reads = alpha != 0.0f && rows > 0;
    if (D == nullptr || !ptr_aligned(D, os) || offsets == nullptr || !ptr_aligned(offsets, 4))
        return SGEMM_ERR_INVALID_VALUE;
    const int64_t d_span = (groups - 1) * stride_d * static_cast<int64_t>(os) +
                           span_bytes(M, N, ldd, os);
    if (ranges_overlap(D, d_span, offsets, (groups + 1) * 4)) return SGEMM_ERR_INVALID_VALUE;
    if (reads) {
        if (P == nullptr || Q == nullptr || !ptr_aligned(P, es) || !ptr_aligned(Q, es) ||
            ranges_overlap(D, d_span, P, span_bytes(rows, M, ldp, es)) ||
            ranges_overlap(D, d_span, Q, span_bytes(rows, N, ldq, es)))
            return SGEMM_ERR_INVALID_VALUE;
    }
    const DeviceInfo* dev = nullptr;
    int rc = device_info(&dev);
    if (rc != SGEMM_OK) return rc;
    int* status = nullptr;
    cudaMemPool_t pool = nullptr;
    if ((rc = device_memory_handles(dev, &status, &pool)) != SGEMM_OK) return rc;
    Params p;
    std::memset(&p, 0, sizeof(p));
    p.groups = static_cast<int>(groups);
    p.rows = rows;
    p.N = static_cast<int>(N);
    p.K = static_cast<int>(M);
    p.offsets = offsets;
    p.x = reads ? P : nullptr;
    p.w = Q;
    p.y = D;
    p.ldx = ldp;
    p.ldw = ldq;
    p.ldy = ldd;
    p.stride_y = stride_d;
    p.alpha = alpha;
    p.beta = beta;
    p.out_bf16 = out_type == SGEMM_TYPE_BF16;
    p.timeout_ns = wait_timeout_ns();
    p.status = status;
    return launch(type, out_type, true, p, dev, pool, stream);
}

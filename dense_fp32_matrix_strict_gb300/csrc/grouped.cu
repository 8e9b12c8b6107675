// grouped.cu — matrix products grouped by expert with ragged sizes: the entry
// points, and a kernel that takes every layout.
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

// 64 x 64 tiles, 16 k at a time through shared memory, 4 x 4 outputs per
// thread in FP32 FMAs. Element strides describe the operands, so any base,
// leading dimension and orientation is taken.
constexpr int ST = 64, SK = 16;

template <typename T, typename O, bool WGRAD>
__global__ void __launch_bounds__(256) simple_kernel(const Params p) {
    extern __shared__ int sched_sm[];
    __shared__ float as[SK][ST + 4], bs[SK][ST + 4];
    const Schedule sch = build_schedule(p, ST, sched_sm);
    const T* x = static_cast<const T*>(p.x);
    const T* w = static_cast<const T*>(p.w);
    O* y = static_cast<O*>(p.y);
    const int tiles_n = (p.N + ST - 1) / ST;
    const int tiles_m = (p.K + ST - 1) / ST;            // weight gradient: K is M
    const int64_t items = WGRAD ? static_cast<int64_t>(p.groups) * tiles_m * tiles_n
                                : static_cast<int64_t>(sch.start[p.groups]) * tiles_n;
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    for (int64_t item = blockIdx.x; item < items; item += gridDim.x) {
        int g, i0, depth;
        int64_t row0, row_end;
        const int j0 = static_cast<int>(item % tiles_n) * ST;
        if (WGRAD) {
            const int64_t m = item / tiles_n;
            g = static_cast<int>(m / tiles_m);
            i0 = static_cast<int>(m % tiles_m) * ST;
            row0 = sch.off[g];
            // Empty, refused, or alpha == 0.
            row_end = p.x == nullptr ? row0 : row0 + max(0, group_rows(sch, p.rows, g));
            depth = static_cast<int>(row_end - row0);
        } else {
            const int t = static_cast<int>(item / tiles_n);
            const int place = place_of(sch, p.groups, t);
            g = sch.perm[place];
            i0 = 0;
            row0 = sch.off[g] + static_cast<int64_t>(t - sch.start[place]) * ST;
            row_end = sch.off[g + 1];
            depth = p.K;
        }
        const T* wg = WGRAD ? w : w + g * p.stride_w;
        float acc[4][4] = {};
        for (int k0 = 0; k0 < depth; k0 += SK) {
            for (int e = threadIdx.x; e < ST * SK; e += 256) {
                float a = 0.0f, b = 0.0f;
                if (WGRAD) {
                    const int i = e % ST, k = e / ST;
                    if (k0 + k < depth) {
                        if (i0 + i < p.K) a = load_f32(x + (row0 + k0 + k) * p.ldx + i0 + i);
                        if (j0 + i < p.N) b = load_f32(w + (row0 + k0 + k) * p.ldw + j0 + i);
                    }
                    as[k][i] = a;
                    bs[k][i] = b;
                } else {
                    const int k = e % SK, i = e / SK;
                    if (k0 + k < depth && row0 + i < row_end)
                        a = load_f32(x + (row0 + i) * p.ldx + k0 + k);
                    as[k][i] = a;
                    const int kb = p.opw ? k : e / ST, jb = p.opw ? i : e % ST;
                    if (k0 + kb < depth && j0 + jb < p.N)
                        b = load_f32(p.opw ? wg + (j0 + jb) * p.ldw + k0 + kb
                                           : wg + (k0 + kb) * p.ldw + j0 + jb);
                    bs[kb][jb] = b;
                }
            }
            __syncthreads();
#pragma unroll
            for (int k = 0; k < SK; ++k) {
                const float4 a = *reinterpret_cast<const float4*>(&as[k][4 * ty]);
                const float4 b = *reinterpret_cast<const float4*>(&bs[k][4 * tx]);
                const float av[4] = {a.x, a.y, a.z, a.w}, bv[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(av[i], bv[j], acc[i][j]);
            }
            __syncthreads();
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int64_t r = WGRAD ? i0 + 4 * ty + i : row0 + 4 * ty + i;
            if (r >= (WGRAD ? static_cast<int64_t>(p.K) : row_end)) continue;
            O* out = y + (WGRAD ? g * p.stride_y : 0) + r * p.ldy;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int n = j0 + 4 * tx + j;
                if (n >= p.N) continue;
                float v = depth > 0 ? p.alpha * acc[i][j] : 0.0f;   // (empty: whatever alpha is)
                if (p.beta != 0.0f) v = fmaf(p.beta, load_f32(out + n), v);
                store_f32(out + n, v);
            }
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

using SimpleKernel = void (*)(Params);

SimpleKernel simple_for(int type, int out, bool wgrad) {
    if (type == SGEMM_TYPE_F32)
        return wgrad ? &simple_kernel<float, float, true> : &simple_kernel<float, float, false>;
    if (!wgrad) return &simple_kernel<__nv_bfloat16, __nv_bfloat16, false>;
    return out == SGEMM_TYPE_BF16 ? &simple_kernel<__nv_bfloat16, __nv_bfloat16, true>
                                  : &simple_kernel<__nv_bfloat16, float, true>;
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
// 9: 184 and 171).
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

cudaError_t run(int type, int out, bool wgrad, Params p, const DeviceInfo* dev, cudaMemPool_t pool,
                cudaStream_t stream) {
    const bool half = type == SGEMM_TYPE_BF16;
    const bool reads = p.K > 0 && p.rows > 0 && p.x != nullptr;
    const int64_t vec = half ? 8 : 4;
    p.y_vec = ptr_aligned(p.y, 16) && p.ldy % 4 == 0 && p.stride_y % 4 == 0;
    p.parts = 1;
    p.part_stride = 0;
    p.tail_ws = nullptr;
    p.pdl = 0;
    if (reads) {
        if (!wgrad && !half && p.rows <= p.groups * skinny_rows(p.opw)) return run_skinny(p, dev, pool, stream);
        const Packed kx = plan_pack(p.x, p.rows, p.K, 1, p.ldx, 0, vec);
        Packed kw = wgrad ? plan_pack(p.w, p.rows, p.N, 1, p.ldw, 0, vec)
                          : plan_pack(p.w, p.opw ? p.N : p.K, p.opw ? p.K : p.N, p.groups, p.ldw,
                                      p.stride_w, vec);
        p.w_tma = !kw.on;
        if (!wgrad && !half) {
            kw.on = false;                             // read in place
            kw.bytes = 0;
        }
        const Tail t = half ? bf16_tail(p, wgrad, dev) : f32_tail(p, wgrad, dev);
        const bool cut = t.items < kCutRounds * t.workers && t.blocks >= t.worth;
        const size_t slots = cut ? 2 * static_cast<size_t>(t.workers) * t.slot_bytes : 0;
        void* ws = nullptr;
        const size_t bytes = kx.bytes + kw.bytes + slots;
        if (bytes == 0 || cudaMallocFromPoolAsync(&ws, bytes, pool, stream) == cudaSuccess) {
            unsigned char* at = static_cast<unsigned char*>(ws);
            cudaError_t e = cudaSuccess;
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
            if (cut) p.tail_ws = reinterpret_cast<float*>(at + kx.bytes + kw.bytes);
            if (e == cudaSuccess)
                e = half ? launch_bf16(p, wgrad, dev, stream) : launch_f32(p, wgrad, dev, stream);
            if (ws != nullptr) cudaFreeAsync(ws, stream);
            return e;
        }
        // No workspace: the kernel that takes any layout.
        (void)cudaGetLastError();
    }
    const size_t smem = schedule_ints(p.groups) * sizeof(int);
    return launch_kernel(simple_for(type, out, wgrad), dim3(4 * dev->sm_count), dim3(256), smem, stream,
                         false, 1, p);
}

int launch(int type, int out, bool wgrad, const Params& p, const DeviceInfo* dev, cudaMemPool_t pool,
           cudaStream_t stream) {
    const cudaError_t e = run(type, out, wgrad, p, dev, pool, stream);
    if (e == cudaSuccess) return SGEMM_OK;
    (void)cudaGetLastError();
    return cuda_fail(e, SGEMM_ERR_LAUNCH);
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

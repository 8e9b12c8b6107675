// route.cu — the router of an expert layer: top-k of each token's logits,
// softmax weights, and the stable grouping of the (token, choice) pairs by
// expert that the grouped products take; and the gradient of the logits.
//
// Forward, for token t with logits l[t][0..E):
//   the `top` experts of the largest logits, ties to the lowest index, a
//   logit of -inf or NaN never chosen (expert -1, weight 0 in its place);
//   weight = exp(l - m) / S with m = max l and S the sum of exp(l - m) over
//   all experts, or (renorm) over the chosen ones.
// Pairs p = t * top + j are numbered by expert, then by p: place[p] is the
// row of pair p, order[row] its inverse, offsets[e] the first row of expert e.
//
// route_topk_kernel: one warp per token, a lane holds E / 32 logits as
// order-preserving 32-bit keys, and the choices come one by one from warp
// maxima, and warp minima of the index among equal keys (redux). Every choice
// sets one bit per token in a shared mask per expert, so the rank of a pair
// among its block's tokens is a population count: no order of atomics shows
// in the result.
//   Up to 256 tokens: one cluster of up to 8 blocks does it all; the blocks
// read one another's counts through distributed shared memory.
//   More: a block walks a contiguous chunk of tokens, 128 at a time, and
// leaves its counts; route_place_kernel sums the chunks' counts before its own
// (at most 152 rows of E, from L2), scans the experts' totals, and turns ranks
// into rows.
#include <climits>
#include <cstring>

#include "expert.h"
#include "kernels.h"

namespace sg {
namespace route {

constexpr int WARPS = 32;                 // tokens of one step of a block
constexpr int THREADS = 32 * WARPS;
constexpr int MAX_TOP = 32;

constexpr int STEP = 128;                 // tokens between two barriers: 4 per warp
constexpr int WORDS = STEP / 32;
constexpr int CLUSTER = 8;
constexpr int64_t CLUSTER_TOKENS = 32 * CLUSTER;

// Counts per chunk, padded to rows of 16 bytes.
__host__ __device__ constexpr int padded_experts(int E) { return (E + 3) & ~3; }

struct Params {
    int64_t T;
    int E, top, renorm;
    int64_t ldl;
    int vec;                 // rows of logits allow loads of four
    float* weights;          // T x top
    int* experts;            // T x top
    int* offsets;            // E + 1
    int* order;              // T * top
    int* place;              // T x top
    int* counts;             // chunks x padded_experts(E) (null when one cluster does the call)
    int chunk, chunks;       // tokens per block, blocks
};

// Four neighbouring logits; -inf past E.
__device__ __forceinline__ void load4(const float* p, int n, bool vec, float (&v)[4]) {
    if (vec && n >= 4) {
        const float4 x = *reinterpret_cast<const float4*>(p);
        v[0] = x.x;
        v[1] = x.y;
        v[2] = x.z;
        v[3] = x.w;
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = i < n ? p[i] : -INFINITY;
    }
}
__device__ __forceinline__ void load4(const __nv_bfloat16* p, int n, bool vec, float (&v)[4]) {
    if (vec && n >= 4) {
        const uint2 x = *reinterpret_cast<const uint2*>(p);
        v[0] = __uint_as_float(x.x << 16);
        v[1] = __uint_as_float(x.x & 0xffff0000u);
        v[2] = __uint_as_float(x.y << 16);
        v[3] = __uint_as_float(x.y & 0xffff0000u);
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = i < n ? __bfloat162float(p[i]) : -INFINITY;
    }
}
__device__ __forceinline__ void store4(float* p, int n, bool vec, const float (&v)[4]) {
    if (vec && n >= 4) {
        *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (i < n) p[i] = v[i];
    }
}
__device__ __forceinline__ void store4(__nv_bfloat16* p, int n, bool vec, const float (&v)[4]) {
    if (vec && n >= 4) {
        __nv_bfloat162 h[2] = {__floats2bfloat162_rn(v[0], v[1]), __floats2bfloat162_rn(v[2], v[3])};
        *reinterpret_cast<uint2*>(p) = *reinterpret_cast<const uint2*>(h);
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (i < n) store_f32(p + i, v[i]);
    }
}

// Monotonic key of a logit: larger float, larger key. -inf, and NaN with it,
// gets KEY_NONE, and no key from KEY_NONE down is ever chosen. `x` comes from
// plain_logit, which makes NaN -inf and -0 the same as +0.
constexpr uint32_t KEY_NONE = 0x007fffffu;
__device__ __forceinline__ float plain_logit(float x) { return fmaxf(x, -INFINITY) + 0.0f; }
__device__ __forceinline__ uint32_t key_of(float x) {
    const uint32_t b = __float_as_uint(x);
    return b ^ (static_cast<uint32_t>(static_cast<int32_t>(b) >> 31) | 0x80000000u);
}
__device__ __forceinline__ float logit_of(uint32_t key) {
    return __uint_as_float(key ^ ((key >> 31) ? 0x80000000u : 0xffffffffu));
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// Exclusive scan over threads of one int each; returns the exclusive prefix
// and leaves the total in *total. `tmp` holds THREADS / 32 + 1 ints.
__device__ int block_scan(int v, int* tmp, int* total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    if (lane == 31) tmp[warp] = x;
    __syncthreads();
    if (warp == 0) {
        int s = tmp[lane];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, s, o);
            if (lane >= o) s += y;
        }
        tmp[lane] = s;
    }
    __syncthreads();
    const int base = warp > 0 ? tmp[warp - 1] : 0;
    *total = tmp[WARPS - 1];
    return base + x - v;
}

// Turns the ranks left in place[] into rows for pairs [lo, hi) and fills
// order[]; base[e] is the first row of the chunk's pairs of expert e.
__device__ void place_pairs(const Params& p, int64_t lo, int64_t hi, const int* base) {
    for (int64_t i = lo + threadIdx.x; i < hi; i += THREADS) {
        const int e = p.experts[i];
        int row = -1;
        if (e >= 0) {
            row = base[e] + p.place[i];
            p.order[row] = static_cast<int>(i);
        }
        p.place[i] = row;
    }
}

// The choices of one token: lane j gets the expert of choice j (-1: none) and
// its key; returns the largest key. Every lane keeps its two best keys at
// hand: a choice is a warp maximum of the best ones and a warp minimum of the
// index among equal ones, and the lane that loses its best brings up the next.
// Only a lane that loses a third looks through its keys again.
template <int VPL>
__device__ __forceinline__ uint32_t choose(const uint32_t (&key)[VPL], int top, int lane,
                                           int& my_expert, uint32_t& my_key) {
    my_expert = -1;
    my_key = KEY_NONE;
    // Best and next of this lane; of equal keys the lower slot first.
    uint32_t best = 0u, next = 0u;
    int at = 0, then = 0;
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
        const bool first = key[i] > best, second = key[i] > next;
        then = first ? at : second ? i : then;
        next = first ? best : second ? key[i] : next;
        at = first ? i : at;
        best = first ? key[i] : best;
    }
    auto expert_of = [&](int slot) { return (slot >> 2) * 128 + lane * 4 + (slot & 3); };
    uint32_t top_key = KEY_NONE;
    int left = 2;                                         // choices until this lane looks again
    for (int j = 0; j < top; ++j) {
        const uint32_t k = __reduce_max_sync(0xffffffffu, best);
        if (j == 0) top_key = k;
        if (k <= KEY_NONE) break;
        const uint32_t e = best == k ? static_cast<uint32_t>(expert_of(at)) : UINT_MAX;
        const uint32_t low = __reduce_min_sync(0xffffffffu, e);
        if (lane == j) {
            my_key = k;
            my_expert = static_cast<int>(low);
        }
        if (e == low) {
            const uint32_t last = best;
            const int last_at = at;
            best = next;
            at = then;
            if (--left == 0 || (left < 0)) {
                // The two kept are gone: the largest key after (last, last_at).
                best = 0u;
#pragma unroll
                for (int i = 0; i < VPL; ++i) {
                    const bool after = key[i] < last || (key[i] == last && i > last_at);
                    if (after && key[i] > best) {
                        best = key[i];
                        at = i;
                    }
                }
            }
        }
    }
    return top_key;
}

template <typename L, int VPL>
__global__ void __launch_bounds__(THREADS) route_topk_kernel(const L* __restrict__ logits,
                                                             const Params p) {
    extern __shared__ uint32_t sm[];
    uint32_t* mask = sm;                                  // WORDS x E: tokens of the step, by expert
    int* run = reinterpret_cast<int*>(sm + WORDS * p.E);  // E: pairs of the chunk so far
    __shared__ int tmp[WARPS + 1];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    for (int i = threadIdx.x; i < (WORDS + 1) * p.E; i += THREADS) sm[i] = 0u;
    __syncthreads();
    if (p.counts != nullptr) griddep_launch_dependents();
    const int64_t t_lo = static_cast<int64_t>(blockIdx.x) * p.chunk;
    const int64_t t_hi = min(p.T, t_lo + p.chunk);
    for (int64_t t0 = t_lo; t0 < t_hi; t0 += STEP) {
        int expert[WORDS];                                // lane j: choice j of the warp's tokens
#pragma unroll
        for (int w = 0; w < WORDS; ++w) {
            const int64_t t = t0 + w * 32 + warp;         // bit `warp` of word w
            expert[w] = -1;
            if (t >= t_hi) continue;
            const L* row = logits + t * p.ldl + lane * 4;
            float x[VPL];
            uint32_t key[VPL];
#pragma unroll
            for (int h = 0; h < VPL / 4; ++h) {
                float v[4];
                load4(row + h * 128, p.E - h * 128 - lane * 4, p.vec != 0, v);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    x[4 * h + i] = plain_logit(v[i]);
                    key[4 * h + i] = key_of(x[4 * h + i]);
                }
            }
            uint32_t my_key;
            const uint32_t first = choose<VPL>(key, p.top, lane, expert[w], my_key);
            const float m = logit_of(first);
            const float raised = expert[w] >= 0 ? expf(logit_of(my_key) - m) : 0.0f;
            float sum = raised;
            if (!p.renorm && first > KEY_NONE) {
                sum = 0.0f;
#pragma unroll
                for (int i = 0; i < VPL; ++i) sum += expf(x[i] - m);
            }
            sum = warp_sum(sum);
            if (lane < p.top) {
                p.weights[t * p.top + lane] = expert[w] >= 0 ? raised / sum : 0.0f;
                p.experts[t * p.top + lane] = expert[w];
                if (expert[w] >= 0) atomicOr(&mask[w * p.E + expert[w]], 1u << warp);
            }
        }
        __syncthreads();
#pragma unroll
        for (int w = 0; w < WORDS; ++w) {
            const int64_t t = t0 + w * 32 + warp;
            if (t >= t_hi || lane >= p.top) continue;
            int rank = -1;
            const int e = expert[w];
            if (e >= 0) {
                rank = run[e] + __popc(mask[w * p.E + e] & ((1u << warp) - 1u));
#pragma unroll
                for (int v = 0; v < w; ++v) rank += __popc(mask[v * p.E + e]);
            }
            p.place[t * p.top + lane] = rank;
        }
        __syncthreads();
        for (int e = threadIdx.x; e < p.E; e += THREADS) {
            int c = 0;
#pragma unroll
            for (int w = 0; w < WORDS; ++w) {
                c += __popc(mask[w * p.E + e]);
                mask[w * p.E + e] = 0u;
            }
            run[e] += c;
        }
        __syncthreads();
    }
    if (p.counts != nullptr) {
        const int padded = padded_experts(p.E);
        for (int e = threadIdx.x; e < padded; e += THREADS)
            p.counts[static_cast<int64_t>(blockIdx.x) * padded + e] = e < p.E ? run[e] : 0;
        return;
    }
    // One cluster: the blocks' counts, then the experts' first rows, then the
    // pairs of this block's tokens.
    cluster_sync();
    int all = 0, before = 0;
    if (threadIdx.x < p.E) {
        const uint32_t at = smem_u32(run + threadIdx.x);
        for (int c = 0; c < p.chunks; ++c) {
            int v;
            asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(mapa_shared(at, c)) : "memory");
            all += v;
            if (c < static_cast<int>(blockIdx.x)) before += v;
        }
    }
    cluster_sync();                                       // every block has read `run`
    int total = 0;
    const int first = block_scan(all, tmp, &total);
    if (threadIdx.x < p.E) {
        run[threadIdx.x] = first + before;
        if (blockIdx.x == 0) p.offsets[threadIdx.x] = first;
    }
    if (blockIdx.x == 0 && threadIdx.x == 0) p.offsets[p.E] = total;
    __syncthreads();
    const int64_t pairs = p.T * p.top;
    place_pairs(p, t_lo * p.top, max(t_lo, t_hi) * p.top, run);
    if (blockIdx.x == 0)
        for (int64_t i = total + threadIdx.x; i < pairs; i += THREADS) p.order[i] = -1;
}

__global__ void __launch_bounds__(THREADS) route_place_kernel(const Params p) {
    extern __shared__ __align__(16) uint32_t sm[];
    const int padded = padded_experts(p.E);
    int4* part = reinterpret_cast<int4*>(sm);             // 2 x slices x padded / 4: totals, before
    int* base = reinterpret_cast<int*>(part + 2 * THREADS);
    __shared__ int tmp[WARPS + 1];
    griddep_wait();
    // Slices of padded / 4 threads share the chunks' rows of counts, 16 bytes
    // a load, most of them in flight at once: the kernel is a chain of a few
    // L2 latencies.
    const int width = padded / 4, slices = THREADS / width;
    const int slice = threadIdx.x / width, col = threadIdx.x - slice * width;
    if (slice < slices) {
        int4 all = make_int4(0, 0, 0, 0), before = all;
        const int4* rows = reinterpret_cast<const int4*>(p.counts) + col;
#pragma unroll 10
        for (int c = slice; c < p.chunks; c += slices) {
            const int4 v = rows[static_cast<int64_t>(c) * width];
            all = make_int4(all.x + v.x, all.y + v.y, all.z + v.z, all.w + v.w);
            if (c < static_cast<int>(blockIdx.x))
                before = make_int4(before.x + v.x, before.y + v.y, before.z + v.z, before.w + v.w);
        }
        part[slice * width + col] = all;
        part[THREADS + slice * width + col] = before;
    }
    __syncthreads();
    int all = 0, before = 0;
    if (threadIdx.x < p.E) {
        const int* totals = reinterpret_cast<const int*>(part);
        for (int s = 0; s < slices; ++s) {
            all += totals[s * padded + threadIdx.x];
            before += totals[4 * THREADS + s * padded + threadIdx.x];
        }
    }
    int total = 0;
    const int first = block_scan(all, tmp, &total);
    if (threadIdx.x < p.E) {
        base[threadIdx.x] = first + before;
        if (blockIdx.x == 0) p.offsets[threadIdx.x] = first;
    }
    if (blockIdx.x == 0 && threadIdx.x == 0) p.offsets[p.E] = total;
    __syncthreads();
    const int64_t pairs = p.T * p.top;
    const int64_t lo = static_cast<int64_t>(blockIdx.x) * p.chunk * p.top;
    place_pairs(p, lo, min(pairs, lo + static_cast<int64_t>(p.chunk) * p.top), base);
    for (int64_t i = total + static_cast<int64_t>(blockIdx.x) * THREADS + threadIdx.x; i < pairs;
         i += static_cast<int64_t>(gridDim.x) * THREADS)
        p.order[i] = -1;
}

// Gradient of the logits from the gradient of the weights: with p the softmax
// over all experts, or (renorm) over the chosen ones and 0 elsewhere, and
// s = sum_j dw_j p[e_j],
//     dl[e] = p[e] * ((dw_j if e = e_j else 0) - s).
// A choice without an expert, or whose logit is -inf or NaN, takes no part: its
// dw_j may be NaN.
// One warp per token, the probabilities recomputed from the logits; reads the
// logits once and writes the gradient once: bandwidth bound.
constexpr int BWD_WARPS = 8;

template <typename L, int VPL>
__global__ void __launch_bounds__(32 * BWD_WARPS)
route_backward_kernel(const L* __restrict__ logits, const int64_t T, const int E, const int top,
                      const int renorm, const int64_t ldl, const int vec,
                      const int* __restrict__ experts, const float* __restrict__ dweights,
                      L* __restrict__ dlogits, const int64_t ldd, const int out_vec, int* status) {
    const int lane = threadIdx.x & 31;
    const int64_t step = static_cast<int64_t>(gridDim.x) * BWD_WARPS;
    for (int64_t t = static_cast<int64_t>(blockIdx.x) * BWD_WARPS + (threadIdx.x >> 5); t < T;
         t += step) {
        const L* row = logits + t * ldl;
        L* out = dlogits + t * ldd;
        int my_expert = -1;
        float dw = 0.0f;
        if (lane < top) {
            my_expert = experts[t * top + lane];
            dw = dweights[t * top + lane];
            if (my_expert >= E) {
                atomicOr(status, STATUS_BAD_INDEX);
                my_expert = -1;
            }
        }
        float x[VPL], m = -INFINITY;
        // The chosen logits, and for the softmax over all the others too.
        const float own = my_expert >= 0 ? load_f32(row + my_expert) : -INFINITY;
        const bool able = own > -INFINITY;                // not -inf, not NaN
        if (!renorm) {
#pragma unroll
            for (int h = 0; h < VPL / 4; ++h) {
                float v[4];
                const int e = h * 128 + lane * 4;
                load4(row + e, E - e, vec != 0, v);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    x[4 * h + i] = plain_logit(v[i]);
                    m = fmaxf(m, x[4 * h + i]);
                }
            }
        } else {
            m = able ? own : -INFINITY;
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
        const bool some = m > -INFINITY;
        float mine = able && some ? expf(own - m) : 0.0f;
        float sum = mine;
        if (!renorm) {
            sum = 0.0f;
#pragma unroll
            for (int i = 0; i < VPL; ++i) {
                x[i] = some ? expf(x[i] - m) : 0.0f;
                sum += x[i];
            }
        }
        sum = warp_sum(sum);
        // (An infinite logit makes the sum NaN, which is kept as in the weights.)
        const float scale = sum == 0.0f ? 0.0f : 1.0f / sum;
        mine *= scale;
        // Without an expert anything may stand in dw. (Asked here: before the
        // row's loads it costs 1.2 us of 10.)
        const float s = warp_sum(able ? dw * mine : 0.0f);
#pragma unroll
        for (int h = 0; h < VPL / 4; ++h) {
            float v[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) v[i] = renorm ? 0.0f : -x[4 * h + i] * scale * s;
            const int e = h * 128 + lane * 4;
            store4(out + e, E - e, out_vec != 0, v);
        }
        // The same warp's later stores to the same addresses win.
        __syncwarp();
        if (able) store_f32(out + my_expert, mine * (dw - s));
    }
}

template <typename L>
using TopkKernel = void (*)(const L*, Params);

template <typename L>
TopkKernel<L> topk_kernel(int E) {
    if (E <= 128) return &route_topk_kernel<L, 4>;
    if (E <= 256) return &route_topk_kernel<L, 8>;
    if (E <= 512) return &route_topk_kernel<L, 16>;
    return &route_topk_kernel<L, 32>;
}

template <typename L>
auto backward_kernel(int E) {
    if (E <= 128) return &route_backward_kernel<L, 4>;
    if (E <= 256) return &route_backward_kernel<L, 8>;
    if (E <= 512) return &route_backward_kernel<L, 16>;
    return &route_backward_kernel<L, 32>;
}

template <typename L>
bool rows_of_four(const void* p, int64_t ld) {
    return ptr_aligned(p, 4 * sizeof(L)) && ld % 4 == 0;
}

template <typename L>
int run_forward(const L* logits, Params p, int sms, cudaMemPool_t pool, cudaStream_t stream) {
    p.vec = rows_of_four<L>(logits, p.ldl);
    const size_t smem = (WORDS + 1) * static_cast<size_t>(p.E) * sizeof(int);
    if (p.T <= CLUSTER_TOKENS) {
        p.chunks = static_cast<int>(p.T < CLUSTER ? p.T : CLUSTER);
        p.chunk = static_cast<int>((p.T + p.chunks - 1) / p.chunks);
        p.counts = nullptr;
        const cudaError_t e = launch_kernel(topk_kernel<L>(p.E), dim3(p.chunks), dim3(THREADS), smem,
                                            stream, false, p.chunks, logits, p);
        if (e == cudaSuccess) return SGEMM_OK;
        (void)cudaGetLastError();
        return cuda_fail(e, SGEMM_ERR_LAUNCH);
    }
    const int64_t per = (p.T + sms - 1) / sms;
    p.chunk = static_cast<int>(per);
    p.chunks = static_cast<int>((p.T + p.chunk - 1) / p.chunk);
    void* ws = nullptr;
    cudaError_t e = cudaMallocFromPoolAsync(&ws, static_cast<size_t>(p.chunks) * padded_experts(p.E) * sizeof(int), pool,
                                            stream);
    if (e != cudaSuccess) {
        (void)cudaGetLastError();
        return cuda_fail(e, SGEMM_ERR_CUDA);
    }
    p.counts = static_cast<int*>(ws);
    e = launch_kernel(topk_kernel<L>(p.E), dim3(p.chunks), dim3(THREADS), smem, stream, false, 1, logits,
                      p);
    if (e == cudaSuccess) {
        const size_t sm2 = 2 * THREADS * sizeof(int4) + static_cast<size_t>(p.E) * sizeof(int);
        e = launch_kernel(route_place_kernel, dim3(p.chunks), dim3(THREADS), sm2, stream,
                          pdl_enabled(), 1, p);
    }
    cudaFreeAsync(ws, stream);
    if (e != cudaSuccess) {
        (void)cudaGetLastError();
        return cuda_fail(e, SGEMM_ERR_LAUNCH);
    }
    return SGEMM_OK;
}

int check(int type, int64_t T, int64_t E, int64_t top, int renorm, const void* logits, int64_t ldl) {
    if (type != SGEMM_TYPE_F32 && type != SGEMM_TYPE_BF16) return SGEMM_ERR_INVALID_VALUE;
    if (renorm != 0 && renorm != 1) return SGEMM_ERR_INVALID_VALUE;
    if (T < 0 || E < 1 || E > kMaxGroups || top < 1 || top > MAX_TOP || top > E)
        return SGEMM_ERR_INVALID_VALUE;
    if (T > kMaxDim / top || ldl < E || (T > 0 && ldl > kMaxOffset / T)) return SGEMM_ERR_INVALID_VALUE;
    if (T > 0 && (logits == nullptr || !ptr_aligned(logits, type_bytes(type))))
        return SGEMM_ERR_INVALID_VALUE;
    return SGEMM_OK;
}

bool int_ptr_ok(const void* p) { return p != nullptr && ptr_aligned(p, 4); }

}  // namespace route
}  // namespace sg

using namespace sg;

extern "C" int sgemm_route(int type, int64_t T, int64_t E, int64_t top, int renorm,
                           const void* logits, int64_t ldl, float* weights, int32_t* experts,
                           int32_t* offsets, int32_t* order, int32_t* place, cudaStream_t stream) {
    using namespace sg::route;
    int rc = check(type, T, E, top, renorm, logits, ldl);
    if (rc != SGEMM_OK) return rc;
    if (!int_ptr_ok(offsets)) return SGEMM_ERR_INVALID_VALUE;
    if (T > 0) {
        const void* outs[5] = {weights, experts, order, place, offsets};
        const int64_t n = T * top * 4;
        const int64_t bytes[5] = {n, n, n, n, (E + 1) * 4};
        const int64_t in = span_bytes(T, E, ldl, type_bytes(type));
        for (int i = 0; i < 5; ++i) {
            if (!int_ptr_ok(outs[i]) || ranges_overlap(outs[i], bytes[i], logits, in))
                return SGEMM_ERR_INVALID_VALUE;
            for (int j = 0; j < i; ++j)
                if (ranges_overlap(outs[i], bytes[i], outs[j], bytes[j]))
                    return SGEMM_ERR_INVALID_VALUE;
        }
    }
    const DeviceInfo* dev = nullptr;
    if ((rc = device_info(&dev)) != SGEMM_OK) return rc;
    int* status = nullptr;
    cudaMemPool_t pool = nullptr;
    if ((rc = device_memory_handles(dev, &status, &pool)) != SGEMM_OK) return rc;
    if (T == 0) {
        const cudaError_t e = cudaMemsetAsync(offsets, 0, static_cast<size_t>(E + 1) * 4, stream);
        return e == cudaSuccess ? SGEMM_OK : cuda_fail(e, SGEMM_ERR_CUDA);
    }
    Params p;
    std::memset(&p, 0, sizeof(p));
    p.T = T;
    p.E = static_cast<int>(E);
    p.top = static_cast<int>(top);
    p.renorm = renorm;
    p.ldl = ldl;
    p.weights = weights;
    p.experts = experts;
    p.offsets = offsets;
    p.order = order;
    p.place = place;
    if (type == SGEMM_TYPE_BF16)
        return run_forward(static_cast<const __nv_bfloat16*>(logits), p, dev->sm_count, pool, stream);
    return run_forward(static_cast<const float*>(logits), p, dev->sm_count, pool, stream);
}

extern "C" int sgemm_route_backward(int type, int64_t T, int64_t E, int64_t top, int renorm,
                                    const void* logits, int64_t ldl, const int32_t* experts,
                                    const float* dweights, void* dlogits, int64_t ldd,
                                    cudaStream_t stream) {
    using namespace sg::route;
    int rc = check(type, T, E, top, renorm, logits, ldl);
    if (rc != SGEMM_OK) return rc;
    if (ldd < E || (T > 0 && ldd > kMaxOffset / T)) return SGEMM_ERR_INVALID_VALUE;
    if (T == 0) return SGEMM_OK;
    const size_t es = type_bytes(type);
    if (!int_ptr_ok(experts) || !int_ptr_ok(dweights) || dlogits == nullptr ||
        !ptr_aligned(dlogits, es))
        return SGEMM_ERR_INVALID_VALUE;
    const int64_t out = span_bytes(T, E, ldd, es);
    if (ranges_overlap(dlogits, out, logits, span_bytes(T, E, ldl, es)) ||
        ranges_overlap(dlogits, out, experts, T * top * 4) ||
        ranges_overlap(dlogits, out, dweights, T * top * 4))
        return SGEMM_ERR_INVALID_VALUE;
    const DeviceInfo* dev = nullptr;
    if ((rc = device_info(&dev)) != SGEMM_OK) return rc;
    int* status = nullptr;
    cudaMemPool_t pool = nullptr;
    if ((rc = device_memory_handles(dev, &status, &pool)) != SGEMM_OK) return rc;
    const int64_t want = (T + BWD_WARPS - 1) / BWD_WARPS;
    const int64_t most = static_cast<int64_t>(dev->sm_count) * 8;
    const dim3 grid(static_cast<unsigned>(want < most ? want : most));
    const int e32 = static_cast<int>(E), k32 = static_cast<int>(top);
    cudaError_t e;
    if (type == SGEMM_TYPE_BF16)
        e = launch_kernel(backward_kernel<__nv_bfloat16>(e32), grid, dim3(32 * BWD_WARPS), 0, stream,
                          false, 1, static_cast<const __nv_bfloat16*>(logits), T, e32, k32, renorm,
                          ldl, static_cast<int>(rows_of_four<__nv_bfloat16>(logits, ldl)), experts,
                          dweights, static_cast<__nv_bfloat16*>(dlogits), ldd,
                          static_cast<int>(rows_of_four<__nv_bfloat16>(dlogits, ldd)), status);
    else
        e = launch_kernel(backward_kernel<float>(e32), grid, dim3(32 * BWD_WARPS), 0, stream, false, 1,
                          static_cast<const float*>(logits), T, e32, k32, renorm, ldl,
                          static_cast<int>(rows_of_four<float>(logits, ldl)), experts, dweights,
                          static_cast<float*>(dlogits), ldd,
                          static_cast<int>(rows_of_four<float>(dlogits, ldd)), status);
    if (e != cudaSuccess) {
        (void)cudaGetLastError();
        return cuda_fail(e, SGEMM_ERR_LAUNCH);
    }
    return SGEMM_OK;
}

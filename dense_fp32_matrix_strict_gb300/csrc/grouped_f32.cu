// grouped_f32.cu — the grouped products of float operands: strict FP32, every
// product accumulated by single-rounding FMAs on the CUDA cores (packed, two
// per instruction).
//
// A CTA computes BM x 128 tiles of a group. One producer thread brings 32 k of
// both operands by TMA through a ring of stages; a W whose base or strides are
// not multiples of 16 bytes comes by plain loads of all four producer warps
// instead, 32 per thread and stage in flight at once (an aligned copy of all
// experts' W first costs more: 12 experts of 1531 x 5120, 4093 rows, 1302
// against 1219 us). Eight consumer warps hold 8 x 8 outputs per thread (four
// warps 8 x 4 in the 32-row tiles) as pairs of neighbouring columns, X's (P's)
// value in both halves of the FMA's other operand. Operands lie in shared
// memory as they lie in HBM: K-major (32 k of a row in 128 bytes, 128-byte
// swizzle: a 16-byte read brings 4 k of one row), or MN-major (a k's 128
// columns: a 16-byte read brings two pairs), both read without bank conflicts.
// Where W is stored N x K both operands are K-major and the pair is (even k,
// odd k) of one output instead: two partial sums, added at the end, and no
// register is moved (58 TFLOP/s; zipping columns to pairs first 37).
// What bounds the tiles is shared memory beside the FMAs: 16 values read per
// lane and k for 64 FMAs keep both nearly full (65 to 68 of 80 TFLOP/s); the
// 32-row tiles read 12 for 32.
// The weight gradient's sum runs over a group's rows: the consumers stop at
// the last of them, so the next group's rows in the same block are never
// touched. Rows of X past the group's end are other groups' rows: they reach
// only outputs that are not written.
#include <atomic>
#include <cstring>

#include "grouped_internal.h"

namespace sg {
namespace grouped {
namespace f32 {

constexpr int BN = 128, BK = 32;
constexpr int PRODUCERS = 4;                          // warps
// Consumer warps: 4 x 2 of 8 x 8 outputs per thread, or for 32-row tiles
// 1 x 4 of 8 x 4.
__host__ __device__ constexpr int consumers(int bm) { return bm == 128 ? 8 : 4; }
__host__ __device__ constexpr int threads_of(int bm) { return 32 * (consumers(bm) + PRODUCERS); }
constexpr int B_BYTES = BN * BK * 4;                  // 16 KB
// Row tiles that share a pass over the columns. (Bound by FMAs: bands of 1 to 64
// take the same time within 1 %.)
constexpr int BAND = 16;

__host__ __device__ constexpr int a_bytes(int bm) { return bm * BK * 4; }
__host__ __device__ constexpr int stages_of(int bm) { return bm == 128 ? 6 : 5; }
__host__ __device__ constexpr int ctas_of(int bm) { return bm == 128 ? 1 : 2; }
// Registers per thread of the 128-row tiles: a block is launched with 168 for
// each of its 384 threads; the producers hand theirs to the consumers, within
// that total. (Plain loads need more of them.)
__host__ __device__ constexpr int regs_producer(bool tma) { return tma ? 40 : 56; }
__host__ __device__ constexpr int regs_consumer(bool tma) { return tma ? 232 : 224; }
static_assert(256 * regs_consumer(true) + 128 * regs_producer(true) <= 384 * 168, "registers");
static_assert(256 * regs_consumer(false) + 128 * regs_producer(false) <= 384 * 168, "registers");
__host__ __device__ constexpr int smem_fixed(int bm) { return 1024 + stages_of(bm) * (a_bytes(bm) + B_BYTES) + 256; }
static_assert(smem_fixed(128) + (schedule_ints(kMaxGroups) + WALK_INTS) * 4 <= 227 * 1024, "shared memory");
static_assert(2 * (smem_fixed(32) + 1024) <= 227 * 1024, "two CTAs per SM");

enum { W_NK = 0, W_KN = 1, WGRAD = 2 };               // the layouts

__device__ __forceinline__ float2 as_float2(unsigned long long v) {
    return make_float2(__uint_as_float(static_cast<uint32_t>(v)),
                       __uint_as_float(static_cast<uint32_t>(v >> 32)));
}
__device__ __forceinline__ void fma2(unsigned long long& c, unsigned long long a,
                                     unsigned long long b) {
    const float2 r = __ffma2_rn(as_float2(a), as_float2(b), as_float2(c));
    c = (static_cast<unsigned long long>(__float_as_uint(r.y)) << 32) | __float_as_uint(r.x);
}
__device__ __forceinline__ unsigned long long pack2(float lo, float hi) {
    return (static_cast<unsigned long long>(__float_as_uint(hi)) << 32) | __float_as_uint(lo);
}
__device__ __forceinline__ void unpack2(unsigned long long v, float& lo, float& hi) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
// 16 bytes of shared memory as two packed pairs, or four floats.
__device__ __forceinline__ void lds_pairs(const uint8_t* at, unsigned long long& x,
                                          unsigned long long& y) {
    const ulonglong2 v = *reinterpret_cast<const ulonglong2*>(at);
    x = v.x;
    y = v.y;
}
__device__ __forceinline__ float4 lds4(const uint8_t* at) {
    return *reinterpret_cast<const float4*>(at);
}
__device__ __forceinline__ void tma_load_3d(uint32_t dst, const void* desc, uint32_t bar, int32_t x,
                                            int32_t y, int32_t z) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4, %5}], [%2];"
        :: "r"(dst), "l"(reinterpret_cast<uint64_t>(desc)), "r"(bar), "r"(x), "r"(y), "r"(z)
        : "memory");
}

__device__ __forceinline__ bool wait_for(uint32_t bar, uint32_t parity, unsigned long long limit,
                                         const Params& p, int code) {
    if (mbar_try_wait(bar, parity)) return true;
    const uint64_t t0 = globaltimer_ns();
    for (;;) {
#pragma unroll 1
        for (int i = 0; i < 16; ++i)
            if (mbar_try_wait(bar, parity)) return true;
        if (globaltimer_ns() - t0 > limit) {
            atomicOr(p.status, code);
            return false;
        }
    }
}
__device__ __forceinline__ bool wait_bar(uint32_t bar, uint32_t parity, const Params& p, int code) {
    return wait_for(bar, parity, p.timeout_ns, p, code);
}

// An output tile: rows row0 .. row0 + valid of Y (forward) or mrow .. of D
// (weight gradient), columns col .. col + 128; the sum's length is depth.
struct Item {
    int g, col, mrow, row0, valid, depth;
    int k0, k1;                      // this piece's k
};

// Items that share a row tile (forward), or a group (weight gradient).
template <int MODE, int BM>
__device__ __forceinline__ int items_per(const Params& p) {
    const int tiles_c = (p.N + BN - 1) / BN;
    return MODE == WGRAD ? tiles_c * ((p.K + BM - 1) / BM) : tiles_c;
}

template <int MODE, int BM>
__device__ __forceinline__ Item item_at(const Params& p, const Schedule& s, const Piece& piece) {
    Item it;
    const int i = piece.item;
    const int tiles_c = (p.N + BN - 1) / BN;
    int place, first, tiles;
    if (MODE == WGRAD) {
        tiles = (p.K + BM - 1) / BM;
        place = i / (tiles * tiles_c);
        first = place * tiles * tiles_c;
    } else {
        place = place_of(s, p.groups, i / tiles_c);
        first = s.start[place] * tiles_c;
        tiles = s.start[place + 1] - s.start[place];
    }
    const TileAt at = tile_at(i, first, tiles, tiles_c, BAND, place);
    it.g = s.perm[place];
    it.col = at.c * BN;
    const int rows = max(0, group_rows(s, p.rows, it.g));
    it.row0 = s.off[it.g];
    if (MODE == WGRAD) {
        it.mrow = at.t * BM;
        it.depth = rows;
        it.valid = min(BM, p.K - it.mrow);
    } else {
        it.mrow = 0;
        it.row0 += at.t * BM;
        it.valid = min(BM, rows - at.t * BM);
        it.depth = p.K;
    }
    it.k0 = piece.kb * BK;
    it.k1 = piece.ke < 0 ? it.depth : min(it.depth, piece.ke * BK);
    return it;
}

// W's tile by plain loads, 128 threads, 32 loads of each in flight; rows and
// columns past the ends become zeros. K-major (128 rows x 32 k, 128-byte
// swizzle; src: row 0, k 0), a warp reads 128 bytes of a row at a time:
__device__ __forceinline__ void copy_k_major(uint8_t* dst, const float* src, int64_t ld, int rows,
                                             int ks, int t) {
    const int k = t & 31, r0 = t >> 5;
    const float* at = src + r0 * ld + k;
    if (k >= ks) rows = 0;
    float v[32];
#pragma unroll
    for (int j = 0; j < 32; ++j) {
        v[j] = r0 + 4 * j < rows ? *at : 0.0f;
        at += 4 * ld;
    }
#pragma unroll
    for (int j = 0; j < 32; ++j) {
        const int r = r0 + 4 * j;
        *reinterpret_cast<float*>(dst + r * 128 + ((((k >> 2) ^ (r & 7)) << 4) | ((k & 3) << 2))) = v[j];
    }
}
// MN-major (32 k x 128 columns; src: k 0, column 0), a thread takes a column:
__device__ __forceinline__ void copy_mn_major(uint8_t* dst, const float* src, int64_t ld, int ks,
                                              int cols, int t) {
    const float* at = src + t;
    if (t >= cols) ks = 0;
    float v[32];
#pragma unroll
    for (int k = 0; k < 32; ++k) {
        v[k] = k < ks ? *at : 0.0f;
        at += ld;
    }
#pragma unroll
    for (int k = 0; k < 32; ++k) *reinterpret_cast<float*>(dst + (k * 128 + t) * 4) = v[k];
}

template <int MODE, int BM, bool B_TMA>
__global__ void __launch_bounds__(threads_of(BM), ctas_of(BM))
tile_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
            const Params p) {
    constexpr int STAGES = stages_of(BM), CONSUMERS = consumers(BM);
    constexpr int TM = 8, WN = BM == 128 ? 2 : 4, TN = 16 / WN;    // per thread; warps along the columns
    constexpr int A_BYTES = a_bytes(BM), STAGE_BYTES = A_BYTES + B_BYTES;
    extern __shared__ __align__(16) uint8_t smem_raw[];
    uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    const uint32_t s0 = smem_u32(smem);
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + STAGES * STAGE_BYTES);
    const uint32_t full0 = smem_u32(bars), empty0 = full0 + 8 * STAGES;
    int* sched_sm = reinterpret_cast<int*>(smem + STAGES * STAGE_BYTES + 256);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int s = 0; s < STAGES; ++s) {
            mbar_init(full0 + 8 * s, B_TMA ? 1 : 1 + 32 * PRODUCERS);
            mbar_init(empty0 + 8 * s, CONSUMERS);
        }
        fence_barrier_init();
    }
    const Schedule sch = build_schedule(p, BM, sched_sm);
    Walk<MODE != WGRAD> walk(p, sch, reinterpret_cast<WalkPlan*>(sched_sm + schedule_ints(p.groups)),
                             items_per<MODE, BM>(p), BK, blockIdx.x);
    Piece piece;
    if (p.tail_ws != nullptr) griddep_launch_dependents();
    griddep_wait();                                    // for packed operands

    if (warp >= CONSUMERS) {
        if (BM == 128)
            asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" :: "n"(regs_producer(B_TMA)));
        const int t = threadIdx.x - 32 * CONSUMERS;
        if (B_TMA && t != 0) return;
        if (t == 0) {
            tma_prefetch_desc(&tmA);
            if (B_TMA) tma_prefetch_desc(&tmB);
        }
        int s = 0, issued = 0;
        uint32_t ph = 0;
        bool ok = true;
        while (ok && walk.next(piece)) {
            const Item it = item_at<MODE, BM>(p, sch, piece);
            for (int k = it.k0; k < it.k1; k += BK) {
                if (!wait_bar(empty0 + 8 * s, ph ^ 1u, p, STATUS_PRODUCER_TIMEOUT)) {
                    ok = false;
                    break;
                }
                const uint32_t bar = full0 + 8 * s, a = s0 + s * STAGE_BYTES, b = a + A_BYTES;
                if (t == 0) {
                    mbar_arrive_expect_tx(bar, B_TMA ? STAGE_BYTES : A_BYTES);
                    if (MODE == WGRAD) tma_load_3d(a, &tmA, bar, it.mrow, it.row0 + k, 0);
                    else tma_load_3d(a, &tmA, bar, k, it.row0, 0);
                    if (B_TMA) {
                        if (MODE == WGRAD) tma_load_3d(b, &tmB, bar, it.col, it.row0 + k, 0);
                        else if (MODE == W_NK) tma_load_3d(b, &tmB, bar, k, it.col, it.g);
                        else tma_load_3d(b, &tmB, bar, it.col, k, it.g);
                    }
                }
                if (!B_TMA) {
                    uint8_t* dst = smem + s * STAGE_BYTES + A_BYTES;
                    const float* w = static_cast<const float*>(p.w) + it.g * p.stride_w;
                    if (MODE == W_NK)
                        copy_k_major(dst, w + it.col * p.ldw + k, p.ldw, p.N - it.col, it.depth - k, t);
                    else
                        copy_mn_major(dst, w + k * p.ldw + it.col, p.ldw, it.depth - k, p.N - it.col, t);
                    mbar_arrive(bar);
                }
                ++issued;
                if (++s == STAGES) { s = 0; ph ^= 1u; }
            }
        }
        // The copies land before the block can end, whoever gave up waiting
        // (the consumers may have gone) and however short the limit is.
        if (t == 0) {
            const int n = issued < STAGES ? issued : STAGES;
            for (int j = 0; j < n; ++j) {
                if (--s < 0) { s = STAGES - 1; ph ^= 1u; }
                wait_for(full0 + 8 * s, ph, max(p.timeout_ns, LAND_NS), p, STATUS_DRAIN_TIMEOUT);
            }
        }
        return;
    }

    if (BM == 128)
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" :: "n"(regs_consumer(B_TMA)));
    const int wr = warp / WN, wc = warp % WN, lr = lane >> 3, lc = lane & 7;
    int s = 0;
    uint32_t ph = 0;
    bool ok = true;
    while (ok && walk.next(piece)) {
        const Item it = item_at<MODE, BM>(p, sch, piece);
        // Pairs of columns, or (W stored N x K) of partial sums per column.
        constexpr int ACC = MODE == W_NK ? TN : TN / 2;
        // Warps whose rows all lie past the tile's last one have nothing to do
        // but to pass the stages on: a tile of up to 64 rows takes half the time.
        const bool busy = wr * 32 < it.valid;
        unsigned long long acc[TM][ACC];
#pragma unroll
        for (int r = 0; r < TM; ++r)
#pragma unroll
            for (int c = 0; c < ACC; ++c) acc[r][c] = 0ull;
        for (int k = it.k0; k < it.k1; k += BK) {
            if (!wait_bar(full0 + 8 * s, ph, p, STATUS_CONSUMER_TIMEOUT)) {
                ok = false;
                break;
            }
            const uint8_t* a0 = smem + s * STAGE_BYTES;
            const uint8_t* b0 = a0 + A_BYTES;
            if (busy) {
            if constexpr (MODE == WGRAD) {
                // a: [k][BM], b: [k][128]; rows 4 lr + {0..3} and + 16 of the
                // warp's 32, columns 4 lc + {0..3} and + 32 of its 64.
                const uint8_t* pa = a0 + (wr * 32 + 4 * lr) * 4;
                const uint8_t* pb = b0 + (wc * 8 * TN + 4 * lc) * 4;
                const int n = min(BK, it.depth - k);
                auto step = [&](int kk) {
                    unsigned long long b[ACC];
#pragma unroll
                    for (int h = 0; h < ACC / 2; ++h)
                        lds_pairs(pb + kk * BN * 4 + 128 * h, b[2 * h], b[2 * h + 1]);
#pragma unroll
                    for (int h = 0; h < TM / 4; ++h) {
                        const float4 a = lds4(pa + kk * BM * 4 + h * 64);
                        const float av[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
                        for (int q = 0; q < 4; ++q) {
                            const unsigned long long aa = pack2(av[q], av[q]);
#pragma unroll
                            for (int c = 0; c < ACC; ++c) fma2(acc[4 * h + q][c], aa, b[c]);
                        }
                    }
                };
                if (n == BK) {
#pragma unroll
                    for (int kk = 0; kk < BK; ++kk) step(kk);
                } else {
#pragma unroll 1
                    for (int kk = 0; kk < n; ++kk) step(kk);
                }
            } else if constexpr (MODE == W_KN) {
                // a: rows lr + 4 q of 32 k, swizzled (row % 8 = lr + 4 (q % 2));
                // b: [k][128], columns 4 lc + {0..3} (and + 32) of the warp's 8 TN.
                const uint8_t* pa = a0 + (wr * 32 + lr) * 128;
                const uint8_t* pb = b0 + (wc * 8 * TN + 4 * lc) * 4;
#pragma unroll
                for (int c4 = 0; c4 < BK / 4; ++c4) {
                    const int sw = (c4 ^ lr) << 4;
                    float a[TM][4];
#pragma unroll
                    for (int q = 0; q < TM; ++q) {
                        const float4 v = lds4(pa + q * 512 + (sw ^ ((q & 1) << 6)));
                        a[q][0] = v.x;
                        a[q][1] = v.y;
                        a[q][2] = v.z;
                        a[q][3] = v.w;
                    }
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk) {
                        unsigned long long b[ACC];
#pragma unroll
                        for (int h = 0; h < ACC / 2; ++h)
                            lds_pairs(pb + (4 * c4 + kk) * BN * 4 + 128 * h, b[2 * h], b[2 * h + 1]);
#pragma unroll
                        for (int q = 0; q < TM; ++q) {
                            const unsigned long long aa = pack2(a[q][kk], a[q][kk]);
#pragma unroll
                            for (int c = 0; c < ACC; ++c) fma2(acc[q][c], aa, b[c]);
                        }
                    }
                }
            } else {
                // a as above; b: columns lc + 8 c of 32 k (row % 8 = lc). Pairs
                // are (even k, odd k); four columns at a time.
                const uint8_t* pa = a0 + (wr * 32 + lr) * 128;
                const uint8_t* pb = b0 + (wc * 8 * TN + lc) * 128;
#pragma unroll
                for (int c4 = 0; c4 < BK / 4; ++c4) {
                    const int sa = (c4 ^ lr) << 4, sb = (c4 ^ lc) << 4;
#pragma unroll
                    for (int h = 0; h < TN / 4; ++h) {
                        unsigned long long b[4][2];
#pragma unroll
                        for (int c = 0; c < 4; ++c)
                            lds_pairs(pb + (4 * h + c) * 1024 + sb, b[c][0], b[c][1]);
#pragma unroll
                        for (int q = 0; q < TM; ++q) {
                            unsigned long long x, y;
                            lds_pairs(pa + q * 512 + (sa ^ ((q & 1) << 6)), x, y);
#pragma unroll
                            for (int c = 0; c < 4; ++c) fma2(acc[q][4 * h + c], x, b[c][0]);
#pragma unroll
                            for (int c = 0; c < 4; ++c) fma2(acc[q][4 * h + c], y, b[c][1]);
                        }
                    }
                }
            }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(empty0 + 8 * s);
            if (++s == STAGES) { s = 0; ph ^= 1u; }
        }
        if (!ok) break;
        // Outputs: alpha * sum + beta * y, or a piece's sums to a slot of BM x BN.
        const bool cut = piece.slot >= 0;
        const int64_t ld = cut ? BN : p.ldy;
        // (An empty sum is zero whatever alpha is.)
        const float alpha = cut ? 1.0f : MODE == WGRAD && it.depth == 0 ? 0.0f : p.alpha;
        const float beta = cut ? 0.0f : p.beta;
        const int cols = cut ? BN : p.N - it.col;
        const bool vec = (cut || p.y_vec) && beta == 0.0f && cols >= BN;
        float* base = cut ? p.tail_ws + static_cast<int64_t>(piece.slot) * BM * BN
                          : static_cast<float*>(p.y) + it.col +
                                (MODE == WGRAD ? it.g * p.stride_y + it.mrow * p.ldy : it.row0 * p.ldy);
#pragma unroll
        for (int r = 0; r < TM; ++r) {
            const int row = wr * 32 +
                            (MODE == WGRAD ? (r / 4) * 16 + 4 * lr + r % 4 : lr + 4 * r);
            if (row >= it.valid) continue;
            float* out = base + row * ld;
            float v[TN];
            int at[TN];
#pragma unroll
            for (int c = 0; c < TN; ++c) {
                float lo, hi;
                unpack2(acc[r][MODE == W_NK ? c : c / 2], lo, hi);
                v[c] = MODE == W_NK ? lo + hi : (c & 1) ? hi : lo;
                at[c] = wc * 8 * TN + (MODE == W_NK ? lc + 8 * c : (c / 4) * 32 + 4 * lc + c % 4);
                v[c] *= alpha;
            }
            if (MODE != W_NK && vec) {
#pragma unroll
                for (int h = 0; h < TN; h += 4)
                    *reinterpret_cast<float4*>(out + at[h]) = make_float4(v[h], v[h + 1], v[h + 2], v[h + 3]);
            } else {
#pragma unroll
                for (int c = 0; c < TN; ++c) {
                    if (at[c] < cols) {
                        float* o = out + at[c];
                        *o = beta != 0.0f ? fmaf(beta, *o, v[c]) : v[c];
                    }
                }
            }
        }
    }
}

// Adds the pieces of the cut tiles, a strip of 4 rows of one tile at a time.
constexpr int JOIN_ROWS = 4;

template <int MODE, int BM>
__global__ void __launch_bounds__(BN) tail_kernel(const Params p) {
    extern __shared__ int sched_sm[];
    const Schedule sch = build_schedule(p, BM, sched_sm);
    const Walk<MODE != WGRAD> walk(p, sch, reinterpret_cast<WalkPlan*>(sched_sm + schedule_ints(p.groups)),
                                   items_per<MODE, BM>(p), BK, 0);
    const int tiles = (MODE == WGRAD ? p.groups : sch.start[p.groups]) * walk.w.per - walk.w.full;
    griddep_wait();                                    // (the offsets are older than the kernel before)
    constexpr int STRIPS = BM / JOIN_ROWS;
    Piece piece;
    piece.kb = 0;
    piece.ke = -1;
    for (int i = blockIdx.x; i < tiles * STRIPS; i += gridDim.x) {
        const int strip = i % STRIPS;
        int first, n, lo, hi;
        piece.item = walk.tile_number(i / STRIPS, first, n);
        if (!tile_pieces(walk, first, n, lo, hi)) continue;
        const Item it = item_at<MODE, BM>(p, sch, piece);
        const int col = it.col + threadIdx.x;
        if (col >= p.N) continue;
        float* out = static_cast<float*>(p.y) + col +
                     (MODE == WGRAD ? it.g * p.stride_y + it.mrow * p.ldy : it.row0 * p.ldy);
        const int r0 = strip * JOIN_ROWS, rows = it.valid - r0;
        if (rows <= 0) continue;
        const float* at = p.tail_ws + r0 * BN + threadIdx.x;
        float v[JOIN_ROWS] = {};
#pragma unroll 4
        for (int c = lo; c <= hi; ++c) {
            const float* piece_at = at + static_cast<int64_t>(slot_of(c, lo)) * BM * BN;
#pragma unroll
            for (int r = 0; r < JOIN_ROWS; ++r)
                if (r < rows) v[r] += piece_at[r * BN];
        }
#pragma unroll
        for (int r = 0; r < JOIN_ROWS; ++r) {
            if (r >= rows) continue;
            float* o = out + (r0 + r) * p.ldy;
            const float x = p.alpha * v[r];
            *o = p.beta != 0.0f ? fmaf(p.beta, *o, x) : x;
        }
    }
}

bool encode_3d(CUtensorMap* map, const void* base, int64_t x, int64_t y, int64_t z, int64_t ld,
               int64_t stride, int box_x, int box_y, bool swizzle) {
    cuuint64_t dims[3] = {static_cast<cuuint64_t>(x), static_cast<cuuint64_t>(y),
                          static_cast<cuuint64_t>(z)};
    cuuint64_t strides[2] = {static_cast<cuuint64_t>(ld) * 4, static_cast<cuuint64_t>(stride) * 4};
    cuuint32_t box[3] = {static_cast<cuuint32_t>(box_x), static_cast<cuuint32_t>(box_y), 1};
    cuuint32_t step[3] = {1, 1, 1};
    return tensor_map_encoder()(map, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 3, const_cast<void*>(base),
                                dims, strides, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE,
                                swizzle ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_NONE,
                                CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int MODE, int BM, bool B_TMA = true>
cudaError_t launch_tile(const Params& p0, const Tail& t, const DeviceInfo* dev, cudaStream_t stream) {
    Params p = p0;
    CUtensorMap a, b;
    std::memset(&b, 0, sizeof(b));
    bool ok;
    if (MODE == WGRAD) {
        ok = encode_3d(&a, p.x, p.K, p.rows, 1, p.ldx, p.ldx, BM, BK, false) &&
             encode_3d(&b, p.w, p.N, p.rows, 1, p.ldw, p.ldw, BN, BK, false);
    } else {
        // One matrix has no stride to speak of; the map wants one.
        const int64_t stride = p.groups > 1 ? p.stride_w : p.ldw;
        ok = encode_3d(&a, p.x, p.K, p.rows, 1, p.ldx, p.ldx, BK, BM, true) &&
             (!B_TMA ? true
              : MODE == W_NK ? encode_3d(&b, p.w, p.K, p.N, p.groups, p.ldw, stride, BK, BN, true)
                             : encode_3d(&b, p.w, p.N, p.K, p.groups, p.ldw, stride, BN, BK, false));
    }
    if (!ok || t.items > 0x3fffffff) return cudaErrorInvalidValue;
    const size_t sched = (schedule_ints(p.groups) + WALK_INTS) * sizeof(int);
    static std::atomic<int> ready[64];
    if (!ready[dev->device].load(std::memory_order_acquire)) {
        const cudaError_t e = cudaFuncSetAttribute(tile_kernel<MODE, BM, B_TMA>,
                                                   cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                   smem_fixed(BM) + (schedule_ints(kMaxGroups) + WALK_INTS) * 4);
        if (e != cudaSuccess) return e;
        ready[dev->device].store(1, std::memory_order_release);
    }
    const int64_t workers = p.tail_ws == nullptr && t.items < t.workers ? t.items : t.workers;
    p.workers = static_cast<int>(workers);
    p.tail_min = static_cast<int>(t.min_blocks);
    p.tail_rule = t.rule;
    cudaError_t e = launch_kernel(tile_kernel<MODE, BM, B_TMA>, dim3(static_cast<unsigned>(workers)),
                                  dim3(threads_of(BM)), smem_fixed(BM) + sched, stream, p.pdl != 0, 1, a, b, p);
    if (e == cudaSuccess && p.tail_ws != nullptr)
        e = launch_kernel(tail_kernel<MODE, BM>, dim3(static_cast<unsigned>(8 * dev->sm_count)), dim3(BN),
                          sched, stream, pdl_enabled(), 1, p);
    return e;
}

}  // namespace f32

bool f32_short(const Params& p) { return p.rows <= static_cast<int64_t>(p.groups) * 48; }

Tail f32_tail(const Params& p, bool wgrad, const DeviceInfo* dev) {
    using namespace f32;
    Tail t;
    const int bm = !wgrad && f32_short(p) ? 32 : 128;
    t.workers = static_cast<int64_t>(dev->sm_count) * ctas_of(bm);
    t.slot_bytes = bm * BN * 4;
    const int64_t tiles_c = (p.N + BN - 1) / BN;
    const int64_t used = p.rows < p.groups ? p.rows : p.groups;
    t.items = wgrad ? p.groups * tiles_c * ((p.K + bm - 1) / bm) : (p.rows / bm + used) * tiles_c;
    t.blocks = ((wgrad ? p.rows / used : p.K) + BK - 1) / BK;
    t.min_blocks = bm == 32 ? 8 : 3;
    t.worth = bm == 32 ? 16 : 6;                      // about 10 us
    // Whole and cut, us: 8 tiles of 128 rows, K = 256, 33 and 27, K = 4096, 361
    // and 45; 136 of 152 tiles, K = 2048, 191 and 194, K = 4096, 365 and 350;
    // weight gradients over 256 rows, 8 tiles 27 and 24, 64 tiles 28 and 32;
    // 64 of 304 tiles of 32 rows, K = 1024, 33 and 26, 272 tiles 56 and 62.
    t.rule = bm == 32 ? TailRule{7, 3, 8} : wgrad ? TailRule{4, 4, 12} : TailRule{3, 2, 8};
    return t;
}

template <int MODE>
cudaError_t launch_forward(const Params& p, const DeviceInfo* dev, cudaStream_t stream) {
    using namespace f32;
    const Tail t = f32_tail(p, false, dev);
    if (p.w_tma)
        return f32_short(p) ? launch_tile<MODE, 32, true>(p, t, dev, stream)
                            : launch_tile<MODE, 128, true>(p, t, dev, stream);
    return f32_short(p) ? launch_tile<MODE, 32, false>(p, t, dev, stream)
                        : launch_tile<MODE, 128, false>(p, t, dev, stream);
}

cudaError_t launch_f32(const Params& p, bool wgrad, const DeviceInfo* dev, cudaStream_t stream) {
    using namespace f32;
    if (wgrad) return launch_tile<WGRAD, 128>(p, f32_tail(p, true, dev), dev, stream);
    return p.opw ? launch_forward<W_NK>(p, dev, stream) : launch_forward<W_KN>(p, dev, stream);
}

}  // namespace grouped
}  // namespace sg

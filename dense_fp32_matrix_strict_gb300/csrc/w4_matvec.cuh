// w4_matvec.cuh — products of a few tokens with weights held in 4 bits and a
// scale (and zero point) per group of inputs, optionally one expert's weights
// per token: the single-token form of an expert layer.
//
//   y[p][n] = sum_k x[p / repeat][k] * s[n][k / G] * (q[n][k] - z[n][k / G])
//
// with the weights of expert experts[p]. Bandwidth bound: every byte of q is
// read once per token chunk; all else is small beside it.
//
// Mathematics. Per group the kernel forms sum_k x (q - z) and scales that
// sum once, in FP32. q - z is a small integer, exact in BF16; a BF16 x is
// itself, and an FP32 x is the exact sum of three BF16 pieces (8 + 8 + 8
// significand bits, split by truncation). So the tensor cores' BF16 x BF16
// products are exact and only the FP32 sums round: an FP32 token keeps FP32
// accuracy at the price of three columns of the MMA instead of one.
//
// Layout. mma.sync m16n8k16: 16 weight rows, 8 columns (tokens, or pieces of
// tokens), 16 inputs. mma.sync and not tcgen05: the weights pass through
// registers to be unpacked and the A operand can stay there, while tcgen05
// would send the unpacked weights (4x the bytes) back through shared memory
// or TMEM; the tensor pipe is far from the bound either way. A warp owns 16
// rows and a strided set of units of 512 inputs (16 x 256 bytes), copied by
// cp.async, with its scales and zero points, into its own ring in
// shared memory, so that no barrier and no load's latency stands in the stream. A lane reads 32-bit words of 8 weights;
// four masks (two of them of the word shifted by 8) pick the pairs of nibbles
// (i, i + 4) and one packed BF16 FMA turns each into a pair of q - z, see
// unpack_pair. x is stored in the same order (0, 4, 1, 5, 2, 6, 3, 7 in each
// 8), so one 16-byte read feeds two MMAs. The order of k inside a group does
// not matter to the sum.
#pragma once

#include <atomic>
#include <cstring>

#include "expert.h"
#include "kernels.h"

namespace sg {
namespace w4 {

constexpr int UNIT_K = 512;                        // inputs of one unit
constexpr int ROW_BYTES = UNIT_K / 2;              // 256
constexpr int MAX_SMEM = 227 * 1024;
constexpr int MAX_STAGES = 4;

// A ring slot: 16 rows of weights, then their scales and zero points
// (UNIT_K / group of each per row), then, where rows start off 16 bytes, the
// rows' last pieces (see load_unit).
__host__ __device__ constexpr int edge_at(int elem, int group) {
    return 16 * ROW_BYTES + 16 * (UNIT_K / group) * (elem + 1);
}
__host__ __device__ constexpr int slot_bytes(int elem, int group, int align) {
    return edge_at(elem, group) + (align == 1 ? 16 * 16 : 0);
}

// Where 16-byte piece c of row r lies in the row: xored so that what a warp
// reads at once, GROUP / 32 words of each of 4 lanes and 8 rows, falls into
// 32 different banks.
template <int GROUP>
__device__ __forceinline__ int piece_at(int r, int c) {
    return GROUP == 128 ? c ^ ((r & 1) << 2) : GROUP == 64 ? c ^ ((r & 3) << 1) : c ^ (r & 7);
}

struct Params {
    int N, K, groups;                   // groups of inputs per row
    int units;                          // ceil(K / UNIT_K)
    int slab;                           // units of one slab (blockIdx.z)
    float* ws;                          // slab x pair x N: sums of slabs (null: one slab)
    int kw;                             // warps that share a row tile's units
    int tiles;                          // ceil(N / 16)
    int stages;                         // ring slots per warp, 2 .. MAX_STAGES
    int tokens_per;                     // tokens of one chunk (blockIdx.y)
    int64_t pairs, repeat;
    int64_t ldx, ldq, stride_q, ldy;
    const uint8_t* q;
    const uint8_t* q_end;               // one past the last byte of all weights
    const uint8_t* zeros;               // null: 8 everywhere
    const int* experts;                 // null: one set of weights
    int num_experts;
    int x_vec;                          // x's rows start on 16 bytes
    int meta4;                          // a unit's scales (and zeros) start on 4 bytes in every row
    int* status;
};

__device__ __forceinline__ void cp_async_16(uint32_t dst, const void* src, uint32_t bytes) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" :: "r"(dst), "l"(src), "r"(bytes)
                 : "memory");
}
__device__ __forceinline__ void cp_async_word(uint32_t dst, const void* src, uint32_t bytes) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" :: "r"(dst), "l"(src), "r"(bytes)
                 : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// All but the newest n groups of this thread have landed.
__device__ __forceinline__ void cp_async_wait(int n) {
    if (n >= 3) asm volatile("cp.async.wait_group 3;" ::: "memory");
    else if (n == 2) asm volatile("cp.async.wait_group 2;" ::: "memory");
    else asm volatile("cp.async.wait_group 1;" ::: "memory");
}

// d = a * b, and c += a * b.
__device__ __forceinline__ void mma_first(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                          uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 "
                 "{%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
                 : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.0f));
}
__device__ __forceinline__ void mma_next(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 "
                 "{%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Unpacking by BF16 arithmetic. The bits of a nibble read as a BF16 number are
// a multiple of the nibble: in bits 0-3 of the half word q * 2^-133, in bits
// 4-7 q * 2^-129 (BF16's subnormals and its first binade are equally spaced,
// so the nibble's top bit, which falls into the exponent, counts right). One
// packed FMA then makes (q - z) * 2^-6, exactly, from a masked word: `mul` is
// 2^127 or 2^123 and `off` is -z * 2^-6, twice each.
constexpr uint32_t MASK_LO = 0x000f000fu, MASK_HI = 0x00f000f0u;
constexpr uint32_t MUL_LO = 0x7f007f00u, MUL_HI = 0x7d007d00u;
constexpr float UNPACK_SCALE = 64.0f;

__device__ __forceinline__ uint32_t unpack_pair(uint32_t bits, uint32_t mul, uint32_t off) {
    uint32_t v;
    asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(v) : "r"(bits), "r"(mul), "r"(off));
    return v;
}
// -z * 2^-6 as two BF16 numbers, for any byte: its bits are z * 2^-133, from
// z = 128 on in the first binade, and q - z stays within 8 bits.
__device__ __forceinline__ uint32_t zero_pair(uint32_t z) {
    return unpack_pair(z * 0x00010001u, 0xff00ff00u, 0x80008000u);
}

// Copies unit u of row tile `row0` into a ring slot: 16 rows x 16 pieces of
// 16 bytes, 8 per lane, and the rows' scales and zero points. Bytes past a
// row's end and rows past N become zeros. Rows that start on 4 bytes come in
// words (10 float tokens, 6720 x 6184: 35.6 against 41 us by loads through
// registers); others as the 17 aligned pieces that hold them, in plain order,
// the last at `edge`, and align_unit puts the bytes in their places when they
// have landed (3 float tokens, 4093 x 1531, cold: 15.0 against 17.1 us). A
// kernel for each: chosen at run time they cost the first 0.6 us of 9.4.
template <typename X, int GROUP, bool ZEROS, int ALIGN>
__device__ __forceinline__ void load_unit(const Params& p, const uint8_t* q, const X* sc,
                                          const uint8_t* zr, int row0, int u, uint8_t* slot,
                                          int lane) {
    constexpr int GU = UNIT_K / GROUP;                 // groups of a unit
    const int row_bytes = (p.K + 1) >> 1;
    const int byte0 = u * ROW_BYTES;
    const int g0 = u * GU, gs = min(GU, p.groups - g0);
    uint8_t* s_sc = slot + 16 * ROW_BYTES;
    uint8_t* s_zr = s_sc + 16 * GU * sizeof(X);
    const int half = lane >> 4, c = lane & 15;         // rows half, half + 2, ...; piece c
    const int have = max(0, min(16, row_bytes - byte0 - 16 * c));
    const int rows = p.N - row0;
    const uint8_t* src = q + static_cast<int64_t>(row0 + half) * p.ldq + byte0 + 16 * c;
    if constexpr (ALIGN == 16) {
        const uint32_t dst = smem_u32(slot) + half * ROW_BYTES;
        const int64_t step = 2 * p.ldq;
        if (rows >= 16 && (u + 1) * ROW_BYTES <= row_bytes) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                cp_async_16(dst + 2 * i * ROW_BYTES + 16 * piece_at<GROUP>(2 * i + half, c), src, 16u);
                src += step;
            }
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int r = 2 * i + half;
                const bool in = r < rows && have > 0;
                cp_async_16(dst + 2 * i * ROW_BYTES + 16 * piece_at<GROUP>(r, c), in ? src : q,
                            in ? static_cast<uint32_t>(have) : 0u);
                src += step;
            }
        }
    } else if constexpr (ALIGN == 4) {
        // Two words of 4 bytes per lane and row.
        const uint32_t dst = smem_u32(slot) + 4 * (lane & 3);
        const uint8_t* at = q + static_cast<int64_t>(row0) * p.ldq + byte0 + 4 * lane;
        const int have0 = max(0, min(4, row_bytes - byte0 - 4 * lane));
        const int have1 = max(0, min(4, row_bytes - byte0 - 128 - 4 * lane));
#pragma unroll
        for (int r = 0; r < 16; ++r) {
            const uint32_t n0 = r < rows ? have0 : 0, n1 = r < rows ? have1 : 0;
            cp_async_word(dst + r * ROW_BYTES + 16 * piece_at<GROUP>(r, lane >> 2), n0 > 0 ? at : q, n0);
            cp_async_word(dst + r * ROW_BYTES + 16 * piece_at<GROUP>(r, 8 + (lane >> 2)),
                          n1 > 0 ? at + 128 : q, n1);
            at += p.ldq;
        }
    } else {
        uint8_t* edge = s_zr + 16 * GU;
        const int need = max(0, min(ROW_BYTES, row_bytes - byte0));
        auto piece = [&](int r, int c) {
            const uint8_t* first = q + static_cast<int64_t>(row0 + r) * p.ldq + byte0;
            const uint8_t* at = first - (reinterpret_cast<uintptr_t>(first) & 15) + 16 * c;
            uint8_t* to = c < 16 ? slot + r * ROW_BYTES + 16 * c : edge + 16 * r;
            if (r >= rows || at >= first + need) return;
            if (at >= p.q) {
                const int64_t left = p.q_end - at;
                cp_async_16(smem_u32(to), at, left < 16 ? static_cast<uint32_t>(left) : 16u);
            } else {                                   // the first bytes of all
                for (int i = static_cast<int>(p.q - at); i < 16; ++i)
                    if (at + i < p.q_end) to[i] = at[i];
            }
        };
#pragma unroll
        for (int i = 0; i < 8; ++i) piece(2 * i + half, c);
        if (lane < 16) piece(lane, 16);
    }
    if (p.meta4) {
        constexpr int WORDS = GU * static_cast<int>(sizeof(X)) / 4;        // per row
#pragma unroll
        for (int i = 0; i < (16 * WORDS + 31) / 32; ++i) {
            const int e = i * 32 + lane, r = e / WORDS, c = e % WORDS * 4;
            if (16 * WORDS < 32 && r >= 16) continue;
            const int have = row0 + r < p.N ? max(0, min(4, gs * static_cast<int>(sizeof(X)) - c)) : 0;
            const uint8_t* src = reinterpret_cast<const uint8_t*>(
                                     sc + (have > 0 ? static_cast<int64_t>(row0 + r) * p.groups + g0 : 0)) +
                                 (have > 0 ? c : 0);
            cp_async_word(smem_u32(s_sc + r * GU * sizeof(X) + c), src, static_cast<uint32_t>(have));
        }
        if (ZEROS) {
            constexpr int ZW = GU / 4;
#pragma unroll
            for (int i = 0; i < (16 * ZW + 31) / 32; ++i) {
                const int e = i * 32 + lane, r = e / ZW, c = e % ZW * 4;
                if (16 * ZW < 32 && r >= 16) continue;
                const int have = row0 + r < p.N ? max(0, min(4, gs - c)) : 0;
                cp_async_word(smem_u32(s_zr + r * GU + c),
                              zr + (have > 0 ? static_cast<int64_t>(row0 + r) * p.groups + g0 + c : 0),
                              static_cast<uint32_t>(have));
            }
        }
    } else {
#pragma unroll
        for (int i = 0; i < 16 * GU / 32; ++i) {
            const int e = i * 32 + lane, r = e / GU, c = e % GU;
            const bool in = row0 + r < p.N && c < gs;
            const int64_t at = in ? static_cast<int64_t>(row0 + r) * p.groups + g0 + c : 0;
            reinterpret_cast<X*>(s_sc)[e] = sc[at];
            if (ZEROS) s_zr[e] = zr[at];
        }
    }
}

// The rows of a landed unit to their places: 16 bytes from two pieces that
// lie side by side, zeros past the row's end and N. Four row pairs at a time,
// each read before any of it is written.
template <int GROUP>
__device__ __forceinline__ void align_unit(const Params& p, const uint8_t* q, int row0, int u,
                                           uint8_t* slot, const uint8_t* edge, int lane) {
    const int half = lane >> 4, c = lane & 15;
    const int have = max(0, min(16, ((p.K + 1) >> 1) - u * ROW_BYTES - 16 * c));
    uint32_t keep[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const int left = have - 4 * j;
        keep[j] = left >= 4 ? 0xffffffffu : left <= 0 ? 0u : (1u << (8 * left)) - 1u;
    }
#pragma unroll
    for (int i0 = 0; i0 < 8; i0 += 4) {
        uint4 out[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int r = 2 * (i0 + i) + half;
            const uint32_t shift =
                static_cast<uint32_t>(reinterpret_cast<uintptr_t>(q) + static_cast<uintptr_t>(row0 + r) * p.ldq);
            const uint8_t* at = slot + r * ROW_BYTES + 16 * c;
            const uint4 lo = *reinterpret_cast<const uint4*>(at);
            const uint4 hi = *reinterpret_cast<const uint4*>(c < 15 ? at + 16 : edge + 16 * r);
            // Two words on, one word on, then bytes.
            const bool two = (shift & 8) != 0, one = (shift & 4) != 0;
            const uint32_t w0 = two ? lo.z : lo.x, w1 = two ? lo.w : lo.y, w2 = two ? hi.x : lo.z,
                           w3 = two ? hi.y : lo.w, w4 = two ? hi.z : hi.x, w5 = two ? hi.w : hi.y;
            const uint32_t v0 = one ? w1 : w0, v1 = one ? w2 : w1, v2 = one ? w3 : w2,
                           v3 = one ? w4 : w3, v4 = one ? w5 : w4;
            const uint32_t bits = 8 * (shift & 3);
            const bool in = row0 + r < p.N;
            out[i].x = in ? __funnelshift_r(v0, v1, bits) & keep[0] : 0u;
            out[i].y = in ? __funnelshift_r(v1, v2, bits) & keep[1] : 0u;
            out[i].z = in ? __funnelshift_r(v2, v3, bits) & keep[2] : 0u;
            out[i].w = in ? __funnelshift_r(v3, v4, bits) & keep[3] : 0u;
        }
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int r = 2 * (i0 + i) + half;
            *reinterpret_cast<uint4*>(slot + r * ROW_BYTES + 16 * piece_at<GROUP>(r, c)) = out[i];
        }
    }
    __syncwarp();
}

// 8 inputs from 16-byte loads (one by one each would touch all the lines that
// the 32 lanes' pieces lie in: 10 bfloat16 tokens, 14336 x 4096, 23.2 against
// 21.9 us).
__device__ __forceinline__ void load_8(const float* p, float (&v)[8]) {
    const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
}
__device__ __forceinline__ void load_8(const __nv_bfloat16* p, float (&v)[8]) {
    const uint4 a = *reinterpret_cast<const uint4*>(p);
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[2 * i] = __uint_as_float(w[i] << 16);
        v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
}

// The BF16 pieces of x[k] of `units` units from unit u0 on, k in the unpacking
// order, as columns: column c = token * PIECES + piece at x_sm + c * pitch.
template <typename X, int GROUP, int THREADS>
__device__ void stage_x(const Params& p, const X* x, int64_t pair0, int tokens, int u0, int units,
                        uint16_t* x_sm, int pitch) {
    constexpr int PIECES = sizeof(X) == 4 ? 3 : 1;
    const int eights = units * (UNIT_K / 8);
    for (int e = threadIdx.x; e < tokens * eights; e += THREADS) {
        const int t = e / eights, k = (e - t * eights) * 8;
        const X* row = x + (pair0 + t) / p.repeat * p.ldx + u0 * UNIT_K;
        const int left = p.K - u0 * UNIT_K;
        // The 8 inputs of word w of lane l (of 4) of a group: at w * 32 + l * 8.
        constexpr int WORDS = GROUP / 32;
        const int in = k & (GROUP - 1);
        const int at = (k - in) + (in / 8 % WORDS) * 32 + in / 8 / WORDS * 8;
        uint16_t* col = x_sm + static_cast<int64_t>(t) * PIECES * pitch + at;
        float v[8];
        if (p.x_vec && k + 8 <= left) {
            load_8(row + k, v);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = k + i < left ? load_f32(row + k + i) : 0.0f;
        }
        uint32_t piece[PIECES][8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const uint32_t hi = __float_as_uint(v[i]) & 0xffff0000u;
            if (PIECES == 1) {
                piece[0][i] = hi;
            } else {
                // An infinity or NaN is its own first piece.
                const bool fine = (hi & 0x7f800000u) != 0x7f800000u;
                const float r1 = fine ? v[i] - __uint_as_float(hi) : 0.0f;
                const uint32_t mid = __float_as_uint(r1) & 0xffff0000u;
                // (A NaN whose payload would be cut off keeps a quiet one.)
                piece[0][i] = !fine && v[i] != v[i] ? 0x7fc00000u : hi;
                piece[PIECES > 1 ? 1 : 0][i] = mid;
                piece[PIECES > 1 ? 2 : 0][i] = __float_as_uint(r1 - __uint_as_float(mid));
            }
        }
#pragma unroll
        for (int pc = 0; pc < PIECES; ++pc) {
            // Order 0, 4, 1, 5, 2, 6, 3, 7.
            uint32_t w[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) w[i] = (piece[pc][i] >> 16) | (piece[pc][i + 4] & 0xffff0000u);
            *reinterpret_cast<uint4*>(col + pc * pitch) = make_uint4(w[0], w[1], w[2], w[3]);
        }
    }
}

// NT: MMA column tiles of 8. GROUP: inputs per scale. ALIGN: bytes that rows of
// weights start on, 16, 4 or 1.
template <typename X, int NT, int GROUP, int WARPS, bool ZEROS, int ALIGN>
__global__ void __launch_bounds__(32 * WARPS, 1) w4_kernel(const X* __restrict__ x,
                                                           const X* __restrict__ scales,
                                                           X* __restrict__ y, const Params p) {
    constexpr int PIECES = sizeof(X) == 4 ? 3 : 1, THREADS = 32 * WARPS;
    constexpr int SLOT = slot_bytes(sizeof(X), GROUP, ALIGN), GU = UNIT_K / GROUP;
    extern __shared__ __align__(16) uint8_t smem[];
    if (p.ws != nullptr) griddep_launch_dependents();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    uint8_t* ring = smem + warp * p.stages * SLOT;
    const int pitch = p.slab * UNIT_K + 32;
    uint16_t* x_sm = reinterpret_cast<uint16_t*>(smem + WARPS * p.stages * SLOT);

    // This block's tokens and weights.
    const int64_t pair0 = static_cast<int64_t>(blockIdx.y) * p.tokens_per;
    const int tokens = static_cast<int>(min(static_cast<int64_t>(p.tokens_per), p.pairs - pair0));
    const int cols = tokens * PIECES;
    float* part = reinterpret_cast<float*>(x_sm + p.tokens_per * PIECES * pitch);   // 2 x warp x column x 16
    int expert = 0;
    if (p.experts != nullptr) {                       // tokens_per is 1
        expert = p.experts[pair0];
        if (expert < 0 || expert >= p.num_experts) {
            if (expert >= p.num_experts && threadIdx.x == 0) atomicOr(p.status, STATUS_BAD_INDEX);
            // No expert: a row of zeros.
            const int64_t step = static_cast<int64_t>(gridDim.x) * THREADS;
            for (int64_t n = static_cast<int64_t>(blockIdx.x) * THREADS + threadIdx.x; n < p.N; n += step) {
                if (p.ws != nullptr) p.ws[(blockIdx.z * p.pairs + pair0) * p.N + n] = 0.0f;
                else store_f32(y + pair0 * p.ldy + n, 0.0f);
            }
            return;
        }
    }
    const uint8_t* q = p.q + static_cast<int64_t>(expert) * p.stride_q;
    const int64_t meta0 = static_cast<int64_t>(expert) * p.N * p.groups;
    const X* sc = scales + meta0;
    const uint8_t* zr = ZEROS ? p.zeros + meta0 : nullptr;

    // Row tiles: the block takes `side` tiles at a time, kw warps on each.
    const int kw = p.kw, side = WARPS / kw;
    const int part_k = warp % kw, my_side = warp / kw;
    const int steps = (p.tiles + side - 1) / side;
    const int u0 = static_cast<int>(blockIdx.z) * p.slab, units = min(p.slab, p.units - u0);
    const int my_units = part_k < units ? (units - part_k + kw - 1) / kw : 0;
    const int my_steps = blockIdx.x < steps ? (steps - blockIdx.x + gridDim.x - 1) / gridDim.x : 0;
    const int total = my_units * my_steps;            // units this warp streams

    // The next unit to load: its step, its place in the step, its slot.
    int l_step = 0, l_unit = 0, l_slot = 0, l_count = 0;
    auto issue = [&]() {
        if (l_count < total) {
            const int tile = (blockIdx.x + l_step * gridDim.x) * side + my_side;
            load_unit<X, GROUP, ZEROS, ALIGN>(p, q, sc, zr, tile * 16, u0 + part_k + l_unit * kw,
                                              ring + l_slot * SLOT, lane);
            ++l_count;
            if (++l_unit == my_units) { l_unit = 0; ++l_step; }
            if (++l_slot == p.stages) l_slot = 0;
        }
        cp_async_commit();
    };
    for (int i = 0; i < p.stages - 1; ++i) issue();
    stage_x<X, GROUP, THREADS>(p, x, pair0, tokens, u0, units, x_sm, pitch);
    __syncthreads();

    const int g = lane >> 2, t4 = lane & 3;
    int slot_at = 0;
    for (int s = 0; s < my_steps; ++s) {
        float acc[NT][4];
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[j][i] = 0.0f;
        for (int u = 0; u < my_units; ++u) {
            issue();
            cp_async_wait(p.stages - 1);
            __syncwarp();
            uint8_t* slot = ring + slot_at * SLOT;
            const X* s_sc = reinterpret_cast<const X*>(slot + 16 * ROW_BYTES);
            const uint8_t* s_zr = slot + 16 * ROW_BYTES + 16 * GU * sizeof(X);
            if (ALIGN == 1)
                align_unit<GROUP>(p, q, ((blockIdx.x + s * gridDim.x) * side + my_side) * 16,
                                  u0 + part_k + u * kw, slot, slot + edge_at(sizeof(X), GROUP), lane);
            const int k0 = (part_k + u * kw) * UNIT_K;
            const int gs = min(GU, p.groups - (u0 + part_k + u * kw) * GU);
            const uint16_t* x_at[NT];
#pragma unroll
            for (int j = 0; j < NT; ++j)               // columns past the last: its values, dropped
                x_at[j] = x_sm + min(j * 8 + g, cols - 1) * pitch + k0 + t4 * 8;
            auto group = [&](int gr) {
                constexpr int WORDS = GROUP / 32;      // of 8 weights, per lane and row
                const float s0 = load_f32(s_sc + g * GU + gr);
                const float s1 = load_f32(s_sc + (g + 8) * GU + gr);
                uint32_t off0 = 0xbe00be00u, off1 = 0xbe00be00u;      // -8 * 2^-6
                if (ZEROS) {
                    off0 = zero_pair(s_zr[g * GU + gr]);
                    off1 = zero_pair(s_zr[(g + 8) * GU + gr]);
                }
                // Bytes GROUP / 2 * gr + 4 WORDS * t4 of rows g and g + 8.
                const int byte = GROUP / 2 * gr + 4 * WORDS * t4;
                const uint8_t* at = slot + g * ROW_BYTES + 16 * piece_at<GROUP>(g, byte >> 4) + (byte & 15);
                uint32_t w0[WORDS], w1[WORDS];
                if constexpr (WORDS == 4) {
                    const uint4 v0 = *reinterpret_cast<const uint4*>(at);
                    const uint4 v1 = *reinterpret_cast<const uint4*>(at + 8 * ROW_BYTES);
                    w0[0] = v0.x; w0[1] = v0.y; w0[2] = v0.z; w0[3] = v0.w;
                    w1[0] = v1.x; w1[1] = v1.y; w1[2] = v1.z; w1[3] = v1.w;
                } else if constexpr (WORDS == 2) {
                    const uint2 v0 = *reinterpret_cast<const uint2*>(at);
                    const uint2 v1 = *reinterpret_cast<const uint2*>(at + 8 * ROW_BYTES);
                    w0[0] = v0.x; w0[1] = v0.y;
                    w1[0] = v1.x; w1[1] = v1.y;
                } else {
                    w0[0] = *reinterpret_cast<const uint32_t*>(at);
                    w1[0] = *reinterpret_cast<const uint32_t*>(at + 8 * ROW_BYTES);
                }
                float c[NT][4];
#pragma unroll
                for (int st = 0; st < WORDS; ++st) {
                    const uint32_t h0 = w0[st] >> 8, h1 = w1[st] >> 8;
                    const uint32_t a[4] = {unpack_pair(w0[st] & MASK_LO, MUL_LO, off0),
                                           unpack_pair(w1[st] & MASK_LO, MUL_LO, off1),
                                           unpack_pair(w0[st] & MASK_HI, MUL_HI, off0),
                                           unpack_pair(w1[st] & MASK_HI, MUL_HI, off1)};
                    const uint32_t b[4] = {unpack_pair(h0 & MASK_LO, MUL_LO, off0),
                                           unpack_pair(h1 & MASK_LO, MUL_LO, off1),
                                           unpack_pair(h0 & MASK_HI, MUL_HI, off0),
                                           unpack_pair(h1 & MASK_HI, MUL_HI, off1)};
#pragma unroll
                    for (int j = 0; j < NT; ++j) {
                        const uint4 xv = *reinterpret_cast<const uint4*>(x_at[j] + gr * GROUP + st * 32);
                        if (st == 0) mma_first(c[j], a, xv.x, xv.y);
                        else mma_next(c[j], a, xv.x, xv.y);
                        mma_next(c[j], b, xv.z, xv.w);
                    }
                }
#pragma unroll
                for (int j = 0; j < NT; ++j) {
                    acc[j][0] = fmaf(s0, c[j][0], acc[j][0]);
                    acc[j][1] = fmaf(s0, c[j][1], acc[j][1]);
                    acc[j][2] = fmaf(s1, c[j][2], acc[j][2]);
                    acc[j][3] = fmaf(s1, c[j][3], acc[j][3]);
                }
            };
            if (gs == GU) {
#pragma unroll
                for (int gr = 0; gr < GU; ++gr) group(gr);
            } else {
#pragma unroll 1
                for (int gr = 0; gr < gs; ++gr) group(gr);
            }
            __syncwarp();                              // the slot may be refilled
            if (++slot_at == p.stages) slot_at = 0;
        }
        // Join the warps of a row tile, and the pieces of a token, in a fixed
        // order. Only a tile's kw warps wait for one another, and two buffers
        // taken in turn spare the second barrier.
        float* sums = part + (s & 1) * WARPS * cols * 16;
        float* mine = sums + warp * cols * 16;
#pragma unroll
        for (int j = 0; j < NT; ++j) {
            const int c0 = j * 8 + 2 * t4;
            if (c0 < cols) {
                mine[c0 * 16 + g] = acc[j][0];
                mine[c0 * 16 + g + 8] = acc[j][2];
            }
            if (c0 + 1 < cols) {
                mine[(c0 + 1) * 16 + g] = acc[j][1];
                mine[(c0 + 1) * 16 + g + 8] = acc[j][3];
            }
        }
        if (kw == 1) __syncwarp();
        else named_bar_sync(1 + my_side, 32 * kw);
        const float* tile = sums + my_side * kw * cols * 16;
        for (int i = part_k * 32 + lane; i < tokens * 16; i += 32 * kw) {
            const int r = i & 15, t = i >> 4;
            const int n = ((blockIdx.x + s * gridDim.x) * side + my_side) * 16 + r;
            float v = 0.0f;
            for (int pc = PIECES - 1; pc >= 0; --pc)
                for (int w = 0; w < kw; ++w) v += tile[(w * cols + t * PIECES + pc) * 16 + r];
            if (n >= p.N) continue;
            if (p.ws != nullptr) p.ws[(blockIdx.z * p.pairs + pair0 + t) * p.N + n] = v * UNPACK_SCALE;
            else store_f32(y + (pair0 + t) * p.ldy + n, v * UNPACK_SCALE);
        }
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
}

template <typename X>
using Kernel = void (*)(const X*, const X*, X*, Params);

// Sets *kernel, allowed all of an SM's shared memory. The limit belongs to the
// function, not to a launch: it is set once per device and to one size, so that
// host threads whose calls need different amounts cannot take it from one
// another.
template <typename X, int NT, int GROUP, int WARPS, bool ZEROS, int ALIGN>
cudaError_t prepare(int device, Kernel<X>* kernel) {
    static std::atomic<bool> ready[64] = {};           // (device_info admits indexes below 64)
    *kernel = &w4_kernel<X, NT, GROUP, WARPS, ZEROS, ALIGN>;
    if (ready[device].load(std::memory_order_acquire)) return cudaSuccess;
    const cudaError_t e =
        cudaFuncSetAttribute(*kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, MAX_SMEM);
    if (e == cudaSuccess) ready[device].store(true, std::memory_order_release);
    return e;
}

template <typename X, int NT, int WARPS, bool ZEROS, int ALIGN>
cudaError_t pick_group(int group, int device, Kernel<X>* kernel) {
    return group == 32   ? prepare<X, NT, 32, WARPS, ZEROS, ALIGN>(device, kernel)
           : group == 64 ? prepare<X, NT, 64, WARPS, ZEROS, ALIGN>(device, kernel)
                         : prepare<X, NT, 128, WARPS, ZEROS, ALIGN>(device, kernel);
}

template <typename X, bool ZEROS, int ALIGN>
cudaError_t pick(bool wide, int64_t cols, int group, int device, Kernel<X>* kernel) {
    if (wide)
        return cols <= 8 ? pick_group<X, 1, 16, ZEROS, ALIGN>(group, device, kernel)
                         : pick_group<X, 2, 16, ZEROS, ALIGN>(group, device, kernel);
    return cols <= 8    ? pick_group<X, 1, 8, ZEROS, ALIGN>(group, device, kernel)
           : cols <= 16 ? pick_group<X, 2, 8, ZEROS, ALIGN>(group, device, kernel)
                        : pick_group<X, 4, 8, ZEROS, ALIGN>(group, device, kernel);
}

// y = the slabs' sums, in order.
template <typename X>
__global__ void __launch_bounds__(256) join_kernel(const Params p, X* __restrict__ y, int slabs) {
    griddep_wait();
    const int64_t total = p.pairs * p.N;
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; i < total;
         i += static_cast<int64_t>(gridDim.x) * 256) {
        float v = 0.0f;
#pragma unroll 4
        for (int z = 0; z < slabs; ++z) v += p.ws[z * total + i];
        const int64_t pair = i / p.N;
        store_f32(y + pair * p.ldy + (i - pair * p.N), v);
    }
}

// Blocks of 16 warps with up to four slots each keep most of what an SM reads
// in flight from the start; many columns take eight warps. As many tokens go
// through a block as four column tiles hold, so that the weights are unpacked
// once for all of them; where their inputs exceed shared memory, k is taken in
// slabs by blocks of their own and the slabs' sums are joined by a second
// kernel (10 float tokens, 6720 x 6184: 40 us when this came; three tokens at a
// time with all of k took 82).
template <typename X, int ALIGN>
int run(const X* x, const X* scales, X* y, Params p, int group, const DeviceInfo* dev,
        cudaMemPool_t pool, cudaStream_t stream) {
    constexpr int PIECES = sizeof(X) == 4 ? 3 : 1;
    const int sms = dev->sm_count;
    const int slot = slot_bytes(sizeof(X), group, ALIGN);
    auto need = [&](int warps, int stages, int64_t cols, int64_t units) {
        return static_cast<int64_t>(warps) * stages * slot + cols * ((units * UNIT_K + 32) * 2 + warps * 128);
    };
    int64_t per = 32 / PIECES;                         // tokens per chunk: four column tiles
    if (p.experts != nullptr) per = 1;
    if (per > p.pairs) per = p.pairs;
    const int64_t chunks = (p.pairs + per - 1) / per;
    per = (p.pairs + chunks - 1) / chunks;             // equal chunks
    const int64_t cols = per * PIECES;
    p.tokens_per = static_cast<int>(per);
    // Slabs of equal length, and the warps that share a row tile's units: the
    // choice of the least cost, in quarters of the time that eight warps take
    // for a unit each. A block's time is its steps' (the units of the busiest
    // warp, which take half as long again among sixteen warps, and a quarter
    // for joining) and that to bring in x (a pass of all threads); a second
    // kernel costs as much as three units. (With the fewest slabs that fit and
    // as many warps to a tile as it has units 16 bfloat16 tokens, 6720 x 6184,
    // take 33.5 us, not 22.9, 16 float tokens 65.7, not 47.9, and 8 bfloat16
    // tokens, 1024 x 8192, 21.2, not 13.4.)
    constexpr int64_t JOIN_COST = 12;
    int64_t fewest = 1, slabs = 1, best = INT64_MAX, gx = 1;
    auto slab_of = [&](int64_t n) { return (p.units + n - 1) / n; };
    while (need(8, 2, cols, slab_of(fewest)) > MAX_SMEM) ++fewest;
    int warps = 8;
    for (int64_t n = fewest; n <= fewest + 3 && n <= p.units; ++n) {
        const int64_t slab = slab_of(n), parts = (p.units + slab - 1) / slab;
        const int w = cols <= 16 && need(16, 2, cols, slab) <= MAX_SMEM ? 16 : 8;
        int64_t most = sms / (chunks * parts);
        if (most < 1) most = 1;
        for (int kw = 1; kw <= w; kw *= 2) {
            const int64_t steps = (p.tiles + w / kw - 1) / (w / kw), x = most < steps ? most : steps;
            const int64_t waves = (chunks * parts * x + sms - 1) / sms;
            const int64_t step = (w == 16 ? 6 : 4) * ((slab + kw - 1) / kw) + 1;
            const int64_t fill = per * slab * (UNIT_K / 8) / (32 * w);
            const int64_t cost = waves * ((steps + x - 1) / x * step + fill) + (parts > 1 ? JOIN_COST : 0);
            // Of equals the one that keeps more SMs busy (3 tokens, 4093 x 1536:
            // 6.2 against 7.6 us).
            if (cost > best || (cost == best && x * parts <= gx * slabs)) continue;
            best = cost;
            warps = w;
            slabs = parts;
            gx = x;
            p.slab = static_cast<int>(slab);
            p.kw = kw;
        }
    }
    if (chunks > 65535 || slabs > 65535) return SGEMM_ERR_INVALID_VALUE;
    const bool wide = warps == 16;
    p.stages = 2;
    while (p.stages < MAX_STAGES && need(warps, p.stages + 1, cols, p.slab) <= MAX_SMEM) ++p.stages;
    p.x_vec = ptr_aligned(x, 16) && p.ldx * static_cast<int64_t>(sizeof(X)) % 16 == 0;
    void* ws = nullptr;
    cudaError_t e;
    if (slabs > 1) {
        e = cudaMallocFromPoolAsync(&ws, static_cast<size_t>(slabs * p.pairs * p.N) * 4, pool, stream);
        if (e != cudaSuccess) {
            (void)cudaGetLastError();
            return cuda_fail(e, SGEMM_ERR_CUDA);
        }
    }
    p.ws = static_cast<float*>(ws);
    Kernel<X> kernel = nullptr;
    e = p.zeros != nullptr ? pick<X, true, ALIGN>(wide, cols, group, dev->device, &kernel)
                           : pick<X, false, ALIGN>(wide, cols, group, dev->device, &kernel);
    const size_t smem = static_cast<size_t>(need(warps, p.stages, cols, p.slab));
    if (e == cudaSuccess)
        e = launch_kernel(kernel,
                          dim3(static_cast<unsigned>(gx), static_cast<unsigned>(chunks),
                               static_cast<unsigned>(slabs)),
                          dim3(32 * warps), smem, stream, false, 1, x, scales, y, p);
    if (e == cudaSuccess && slabs > 1) {
        const int64_t blocks = (p.pairs * p.N + 255) / 256, most = 8 * static_cast<int64_t>(sms);
        e = launch_kernel(join_kernel<X>, dim3(static_cast<unsigned>(blocks < most ? blocks : most)),
                          dim3(256), 0, stream, pdl_enabled(), 1, p, y, static_cast<int>(slabs));
    }
    if (ws != nullptr) cudaFreeAsync(ws, stream);
    if (e != cudaSuccess) {
        (void)cudaGetLastError();
        return cuda_fail(e, SGEMM_ERR_LAUNCH);
    }
    return SGEMM_OK;
}

}  // namespace w4
}  // namespace sg

// grouped_bf16.cu — the grouped products of bfloat16 operands on the
// 5th-generation tensor cores (tcgen05, FP32 accumulators in TMEM).
//
// Two CTAs of a cluster share one tile of 256 x 256 through
// tcgen05.mma.cta_group::2. The M side of the MMA is the dimension that is
// contiguous in the output (the weight's output features; Q's columns in the
// weight gradient), the N side its rows (a group's rows; P's columns):
//   * few rows per expert cost few MMA columns, not 256 padded rows: the N
//     extent of a tile is the group's rows left, rounded up to 32, so ragged
//     groups waste at most 31 rows and decode steps stream the weights with
//     almost no arithmetic;
//   * a lane of TMEM is an output column, so 32 lanes write consecutive
//     elements of an output row and nothing is transposed on the way out.
// Operands come in by TMA with the 128-byte swizzle in the layout they have:
// K-major (64 k of a row in 128 bytes) or MN-major (64 columns of a k), the
// descriptors tell the MMA which: nothing is transposed. (An operand whose base
// or strides TMA cannot take arrives as an aligned copy, made before.)
//
// Roles per CTA: warp 0 TMA producer, warp 1 (of rank 0) MMA issuer, the next
// eight or sixteen epilogue, and in the weight gradient one more: its sums run
// over a group's rows, whose last block of 64 also brings rows of the next
// group. That block lands on a barrier of its own, the last warp overwrites
// the foreign rows in both operands with zeros and only then releases it to
// the MMA (zeroing one operand would let 0 * NaN through). Whole blocks know
// nothing of this: an arrival of the peer's producer on every stage, for one
// barrier with one count, costs more than half of the rate (700 against 1570
// TFLOP/s).
//
// Per stage a CTA holds 128 x 64 of each side (32 KB); six stages; two
// accumulators of 256 columns, so the epilogue of one tile runs beside the
// MMAs of the next.
#include <atomic>
#include <climits>
#include <cstring>

#include "grouped.cuh"
#include "grouped_internal.h"

namespace sg {
namespace grouped {
namespace bf16 {

constexpr int TILE = 256, HALF = 128, BK = 64;
constexpr int STAGES = 6;
constexpr int OP_BYTES = HALF * BK * 2;               // 16 KB per operand and CTA
constexpr int STAGE_BYTES = 2 * OP_BYTES;
constexpr int BOX_BYTES = OP_BYTES / 2;               // 64 columns x 64 k, MN-major
constexpr int TMEM_COLS = 2 * TILE;
constexpr int ROW_STEP = 32;                          // N extent granule of a pair
// Row tiles that share a pass over the columns. More keep too many rows in L2
// (2 uneven groups of 4096 rows in all, 4096 x 14336: 315 us, bands of 16 352,
// of 32 362), fewer read W more often (8 x 2048 rows, 14336 x 4096: 1043, bands
// of 2 1100, of 1 1221).
constexpr int BAND = 8;
// Epilogue warps. The weight gradient's tiles are short (a group's rows over
// 64 blocks) and large (FP32 out), its epilogue is what they wait for, and that
// is a chain of latencies: twice the warps (202 against 224 us, 32 experts of
// 64 rows, 4096 x 2048).
__host__ __device__ constexpr int epi_warps(bool wgrad) { return wgrad ? 16 : 8; }
constexpr int PART_K = 512;                           // rows summed in one accumulator (weight gradient)
__host__ __device__ constexpr int threads_of(bool wgrad) { return 32 * (2 + epi_warps(wgrad) + (wgrad ? 1 : 0)); }
constexpr int SMEM_FIXED = 1024 + STAGES * STAGE_BYTES + 512;
static_assert(SMEM_FIXED + (schedule_ints(kMaxGroups) + WALK_INTS) * 4 <= 227 * 1024, "shared memory");

// Instruction descriptor of kind::f16 without N: D FP32 (bits 4-5), A and B
// BF16 (bits 7-9, 10-12), MN-major flags (bits 15, 16), M >> 4 = 16 (bits
// 24-28); N >> 3 goes to bits 17-22.
__host__ __device__ constexpr uint32_t idesc_base(bool a_mn, bool b_mn) {
    return (1u << 4) | (1u << 7) | (1u << 10) | (static_cast<uint32_t>(a_mn) << 15) |
           (static_cast<uint32_t>(b_mn) << 16) | (static_cast<uint32_t>(TILE >> 4) << 24);
}

// Shared-memory descriptors with the 128-byte swizzle (bits 61-63 = 2),
// version 1 (bit 46). K-major: rows of 128 bytes, 1024 bytes between 8-row
// groups (stride offset). MN-major: k rows of 128 bytes (64 columns), 1024
// bytes between groups of 8 k (stride offset), one box between columns 0..63
// and 64..127 (leading offset).
template <bool MN>
__device__ __forceinline__ uint64_t smem_desc(uint32_t addr) {
    uint64_t d = static_cast<uint64_t>((addr >> 4) & 0x3FFFu);
    d |= static_cast<uint64_t>(MN ? BOX_BYTES >> 4 : 1) << 16;
    d |= static_cast<uint64_t>(1024u >> 4) << 32;
    d |= static_cast<uint64_t>(1u) << 46;
    d |= static_cast<uint64_t>(2u) << 61;
    return d;
}
// Advance of a descriptor by 16 k, in 16-byte units.
template <bool MN>
__host__ __device__ constexpr uint64_t k16_step() { return MN ? (16 * 128) >> 4 : 32 >> 4; }

__device__ __forceinline__ void mma_pair(uint32_t d_tmem, uint64_t a, uint64_t b, uint32_t idesc,
                                         uint32_t acc) {
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
                 "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}"
                 :: "r"(d_tmem), "l"(a), "l"(b), "r"(idesc), "r"(acc) : "memory");
}
__device__ __forceinline__ void commit_pair_mc(uint32_t bar, uint16_t mask) {
    asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster"
                 ".multicast::cluster.b64 [%0], %1;" :: "r"(bar), "h"(mask) : "memory");
}
__device__ __forceinline__ void commit_pair(uint32_t bar) {
    asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 [%0];"
                 :: "r"(bar) : "memory");
}
// 3-D TMA load into this CTA; the bytes complete on the barrier at cluster
// address bar, which may be in either CTA of the pair. x is a multiple of 64
// elements (128 bytes).
__device__ __forceinline__ void tma_load_3d_pair(uint32_t dst, const void* desc, uint32_t bar,
                                                 int32_t x, int32_t y, int32_t z) {
    asm volatile(
        "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4, %5}], [%2];"
        :: "r"(dst), "l"(reinterpret_cast<uint64_t>(desc)), "r"(bar), "r"(x), "r"(y), "r"(z)
        : "memory");
}
__device__ __forceinline__ void fence_before() {
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void fence_after() {
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}
// Arrive on a barrier at a cluster address for a TMEM accumulator that has been
// read. No write of this thread is handed over: what orders the reads before
// the peer's next MMAs is the pair of tcgen05 fences around a relaxed arrival
// of cluster scope and its wait. (A release at cluster scope would wait for the
// stores of the tile before: 265 us instead of 216, 32 experts of 256 rows,
// 4096 x 2048.)
__device__ __forceinline__ void arrive_read(uint32_t cluster_addr) {
    asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" :: "r"(cluster_addr)
                 : "memory");
}
// 32 consecutive FP32 columns of this thread's TMEM lane.
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, float (&v)[32]) {
    uint32_t r[32];
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x32.b32 "
                 "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
                 "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]),
                   "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]),
                   "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]),
                   "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
                   "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]),
                   "=r"(r[30]), "=r"(r[31])
                 : "r"(taddr));
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
    for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
}

// 16 of them.
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, float (&v)[16]) {
    uint32_t r[16];
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x16.b32 "
                 "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]),
                   "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]),
                   "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
                 : "r"(taddr));
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(r[i]);
}

// A thread of the pair gave up a wait. (Static: its address costs the main
// loops no register.)
__device__ __forceinline__ uint32_t* gave_up() {
    __shared__ uint32_t word;
    return &word;
}

// Bounded wait; on giving up sets the status bit and gave_up in both CTAs, and
// returns false. Acquires at cluster scope (the peer's threads arrive on some
// of the barriers).
__device__ __forceinline__ void give_up(const Params& p, int code) {
    atomicOr(p.status, code);
#pragma unroll 1
    for (uint32_t r = 0; r < 2; ++r)
        asm volatile("st.relaxed.cluster.shared::cluster.u32 [%0], %1;"
                     :: "r"(mapa_shared(smem_u32(gave_up()), r)), "r"(1u) : "memory");
}
__device__ __forceinline__ bool wait_bar(uint32_t bar, uint32_t parity, const Params& p, int code) {
    if (mbar_try_wait_cluster(bar, parity)) return true;
    const uint64_t t0 = globaltimer_ns();
    for (;;) {
#pragma unroll 1
        for (int i = 0; i < 16; ++i)
            if (mbar_try_wait_cluster(bar, parity)) return true;
        if (globaltimer_ns() - t0 > p.timeout_ns) {
            give_up(p, code);
            return false;
        }
    }
}
// The same for all lanes of a warp, which decide together: what follows is
// warp-collective, and one lane's clock may pass the limit where another's
// does not.
__device__ __forceinline__ bool warp_wait_bar(uint32_t bar, uint32_t parity, const Params& p, int code) {
    bool done = mbar_try_wait_cluster(bar, parity);
    if (__all_sync(0xffffffffu, done)) return true;
    const uint64_t t0 = globaltimer_ns();
    do {
#pragma unroll 1
        for (int i = 0; i < 16; ++i) {
            done = done || mbar_try_wait_cluster(bar, parity);
            if (__all_sync(0xffffffffu, done)) return true;
        }
    } while (__all_sync(0xffffffffu, globaltimer_ns() - t0 <= p.timeout_ns));
    if ((threadIdx.x & 31) == 0) give_up(p, code);
    return false;
}

// One output tile. Forward: group g, rows row0 .. row0 + valid (at most 256),
// M side at column col. Weight gradient: group g, M side at column col of Q, N
// side at column ncol of P, `depth` rows from row0.
struct Item {
    int g, col, ncol;
    int row0, valid, width;          // width: N extent, a multiple of 32
    int depth;                       // k of the sum over all parts
    int kb, ke;                      // this piece's blocks of the sum
};

// Items that share a row tile (forward), or a group (weight gradient).
template <bool WGRAD>
__device__ __forceinline__ int items_per(const Params& p) {
    const int tiles_c = (p.N + TILE - 1) / TILE;
    return WGRAD ? tiles_c * ((p.K + TILE - 1) / TILE) : tiles_c;
}

template <bool WGRAD>
__device__ __forceinline__ Item item_at(const Params& p, const Schedule& s, const Piece& piece) {
    Item it;
    const int i = piece.item;
    const int tiles_c = (p.N + TILE - 1) / TILE;
    int place, first, tiles;         // the group's place, first item, tiles on the N side
    if (WGRAD) {
        tiles = (p.K + TILE - 1) / TILE;
        place = i / (tiles * tiles_c);
        first = place * tiles * tiles_c;
    } else {
        place = place_of(s, p.groups, i / tiles_c);
        first = s.start[place] * tiles_c;
        tiles = s.start[place + 1] - s.start[place];
    }
    const TileAt at = tile_at(i, first, tiles, tiles_c, BAND, place);
    it.g = s.perm[place];
    it.col = at.c * TILE;
    const int rows = max(0, group_rows(s, p.rows, it.g));
    it.row0 = s.off[it.g];
    if (WGRAD) {
        it.ncol = at.t * TILE;
        it.depth = rows;
        it.valid = min(TILE, p.K - it.ncol);
        it.width = TILE;
    } else {
        // The group's rows in equal tiles, rounded up to the granule.
        const int high = ((rows + tiles - 1) / tiles + ROW_STEP - 1) / ROW_STEP * ROW_STEP;
        it.ncol = 0;
        it.row0 += at.t * high;
        it.valid = max(0, min(high, rows - at.t * high));
        it.width = max(ROW_STEP, (it.valid + ROW_STEP - 1) / ROW_STEP * ROW_STEP);
        it.depth = p.K;
    }
    it.kb = piece.kb;
    it.ke = piece.ke < 0 ? (it.depth + BK - 1) / BK : min(piece.ke, (it.depth + BK - 1) / BK);
    return it;
}

// Accumulators a tile's sum is split into. The tensor cores' FP32 sums are
// truncated at every step, an error that grows with the number of steps; a
// weight gradient in FP32 sums over thousands of rows, so its sum is taken
// PART_K rows at a time and the parts are added by FP32 adds in registers.
// Forward results are rounded to bfloat16, far above that error.
template <bool WGRAD>
__device__ __forceinline__ int part_count(const Item& it) {
    if (it.ke == it.kb) return 0;
    return WGRAD ? ((it.ke - it.kb) * BK + PART_K - 1) / PART_K : 1;
}

// alpha * v + beta * y to up to 32 rows of one output column.
template <typename O>
__device__ __forceinline__ void write_rows(O* out, int64_t ld, float alpha, float beta, int rows,
                                           const float* v) {
    if (beta == 0.0f) {
        if (rows >= 32) {
#pragma unroll
            for (int j = 0; j < 32; ++j) {
                store_f32(out, alpha * v[j]);
                out += ld;
            }
        } else {
#pragma unroll
            for (int j = 0; j < 32; ++j) {
                if (j < rows) store_f32(out, alpha * v[j]);
                out += ld;
            }
        }
    } else {
#pragma unroll
        for (int j = 0; j < 32; ++j) {
            if (j < rows) store_f32(out, fmaf(beta, load_f32(out), alpha * v[j]));
            out += ld;
        }
    }
}

template <bool A_MN, bool WGRAD, typename O>
__global__ void __launch_bounds__(threads_of(WGRAD), 1)
pair_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
            const __grid_constant__ CUtensorMap tmB64, const __grid_constant__ CUtensorMap tmB32,
            const __grid_constant__ CUtensorMap tmB16, const Params p) {
    constexpr bool B_MN = WGRAD;
    constexpr int EPI_WARPS = epi_warps(WGRAD), SPAN = 4 * TILE / EPI_WARPS;   // columns per epilogue warp
    extern __shared__ __align__(16) uint8_t smem_raw[];
    uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    const uint32_t s0 = smem_u32(smem);
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + STAGES * STAGE_BYTES);
    const uint32_t full0 = smem_u32(bars), empty0 = full0 + 8 * STAGES;
    const uint32_t land0 = empty0 + 8 * STAGES, clean0 = land0 + 8 * STAGES;
    const uint32_t accf0 = clean0 + 8 * STAGES, acce0 = accf0 + 16, done_bar = acce0 + 16;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 4 * STAGES + 5);
    int* sched_sm = reinterpret_cast<int*>(smem + STAGES * STAGE_BYTES + 512);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = cluster_ctarank();
    const bool leader = rank == 0;
    if (threadIdx.x == 0) {
        for (int s = 0; s < STAGES; ++s) {
            // "full" (used in rank 0): armed by rank 0's producer for both
            // CTAs' bytes. "land", "clean" (rank 0's): a partial last block of
            // the weight gradient, its bytes in each CTA and both CTAs' last warps.
            mbar_init(full0 + 8 * s, 1);
            mbar_init(empty0 + 8 * s, 1);
            mbar_init(land0 + 8 * s, 1);
            mbar_init(clean0 + 8 * s, 2);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(accf0 + 8 * b, 1);
            mbar_init(acce0 + 8 * b, 2 * EPI_WARPS);      // both CTAs' epilogue warps (rank 0's)
        }
        mbar_init(done_bar, 1);
        *gave_up() = 0;
        fence_barrier_init();
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;"
                     :: "r"(smem_u32(tmem_slot)), "r"(TMEM_COLS) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    }
    const Schedule sch = build_schedule(p, TILE, sched_sm);
    fence_before();
    __syncthreads();
    fence_after();
    const uint32_t tmem = *tmem_slot;
    cluster_sync();

    Walk<!WGRAD> walk(p, sch, reinterpret_cast<WalkPlan*>(sched_sm + schedule_ints(p.groups)),
                      items_per<WGRAD>(p), BK, static_cast<int>(cluster_id_x()));
    Piece piece;
    if (p.tail_ws != nullptr) griddep_launch_dependents();
    griddep_wait();                                    // for packed operands
    const uint32_t full_r0 = mapa_shared(full0, 0);

    if (warp == 0) {
        if (lane == 0) {
            tma_prefetch_desc(&tmA);
            tma_prefetch_desc(&tmB);
            if (!WGRAD) {
                tma_prefetch_desc(&tmB64);
                tma_prefetch_desc(&tmB32);
                tma_prefetch_desc(&tmB16);
            }
            int s = 0;
            uint32_t ph = 0;
            bool ok = true;
            while (ok && walk.next(piece)) {
                const Item it = item_at<WGRAD>(p, sch, piece);
                const int a_col = it.col + static_cast<int>(rank) * HALF;
                const int b_half = it.width / 2;
                const int b_at = (WGRAD ? it.ncol : it.row0) + static_cast<int>(rank) * b_half;
                const uint32_t bytes = OP_BYTES + (WGRAD ? OP_BYTES : b_half * BK * 2);
                for (int kb = it.kb; kb < it.ke; ++kb) {
                    if (!wait_bar(empty0 + 8 * s, ph ^ 1u, p, STATUS_PRODUCER_TIMEOUT)) {
                        ok = false;
                        break;
                    }
                    uint32_t bar = full_r0 + 8 * s;
                    if (WGRAD && (kb + 1) * BK > it.depth) {
                        // The last, partial block: its bytes complete on
                        // "land", "full" only keeps its phase.
                        bar = mapa_shared(land0 + 8 * s, rank);
                        mbar_arrive_expect_tx(land0 + 8 * s, bytes);
                        if (leader) mbar_arrive(full0 + 8 * s);
                    } else if (leader) {
                        mbar_arrive_expect_tx(full0 + 8 * s, 2 * bytes);
                    }
                    const uint32_t a = s0 + s * STAGE_BYTES, b = a + OP_BYTES;
                    const int k = kb * BK;
                    if (A_MN) {
                        const int y = WGRAD ? it.row0 + k : k, z = WGRAD ? 0 : it.g;
                        tma_load_3d_pair(a, &tmA, bar, a_col, y, z);
                        tma_load_3d_pair(a + BOX_BYTES, &tmA, bar, a_col + 64, y, z);
                    } else {
                        tma_load_3d_pair(a, &tmA, bar, k, a_col, it.g);
                    }
                    if (WGRAD) {
                        tma_load_3d_pair(b, &tmB, bar, b_at, it.row0 + k, 0);
                        tma_load_3d_pair(b + BOX_BYTES, &tmB, bar, b_at + 64, it.row0 + k, 0);
                    } else if (it.width == TILE) {
                        tma_load_3d_pair(b, &tmB, bar, k, b_at, 0);
                    } else {
                        // Boxes of 64, 32 and 16 rows: the bits of the half's height.
                        int h = 0;
                        if (b_half & 64) {
                            tma_load_3d_pair(b, &tmB64, bar, k, b_at, 0);
                            h = 64;
                        }
                        if (b_half & 32) {
                            tma_load_3d_pair(b + h * BK * 2, &tmB32, bar, k, b_at + h, 0);
                            h += 32;
                        }
                        if (b_half & 16) tma_load_3d_pair(b + h * BK * 2, &tmB16, bar, k, b_at + h, 0);
                    }
                    if (++s == STAGES) { s = 0; ph ^= 1u; }
                }
            }
        }
    } else if (warp == 1) {
        if (leader && lane == 0) {
            int s = 0, n = 0;
            uint32_t ph = 0, cleaned = 0;               // cleaned: phases of "clean"
            bool ok = true;
            while (ok && walk.next(piece)) {
                const Item it = item_at<WGRAD>(p, sch, piece);
                const int parts = part_count<WGRAD>(it);
                const uint32_t idesc =
                    idesc_base(A_MN, B_MN) | (static_cast<uint32_t>(it.width >> 3) << 17);
                int kb = it.kb;
                for (int c = 0; c < parts && ok; ++c, ++n) {
                    const int b = n & 1;
                    const uint32_t acc_phase = static_cast<uint32_t>((n >> 1) & 1);
                    if (!wait_bar(acce0 + 8 * b, acc_phase ^ 1u, p, STATUS_CONSUMER_TIMEOUT)) {
                        ok = false;
                        break;
                    }
                    fence_after();
                    const uint32_t d = tmem + static_cast<uint32_t>(b * TILE);
                    const int end = WGRAD ? min(it.ke, kb + PART_K / BK) : it.ke;
                    uint32_t more = 0;
                    for (; kb < end; ++kb) {
                        if (!wait_bar(full0 + 8 * s, ph, p, STATUS_CONSUMER_TIMEOUT)) {
                            ok = false;
                            break;
                        }
                        if (WGRAD && (kb + 1) * BK > it.depth) {
                            if (!wait_bar(clean0 + 8 * s, (cleaned >> s) & 1u, p, STATUS_CONSUMER_TIMEOUT)) {
                                ok = false;
                                break;
                            }
                            cleaned ^= 1u << s;
                        }
                        fence_after();
                        const uint32_t st = s0 + s * STAGE_BYTES;
                        const uint64_t da = smem_desc<A_MN>(st), db = smem_desc<B_MN>(st + OP_BYTES);
#pragma unroll
                        for (int kk = 0; kk < BK / 16; ++kk) {
                            mma_pair(d, da + kk * k16_step<A_MN>(), db + kk * k16_step<B_MN>(), idesc,
                                     more);
                            more = 1u;
                        }
                        commit_pair_mc(empty0 + 8 * s, 0x3);
                        if (++s == STAGES) { s = 0; ph ^= 1u; }
                    }
                    if (ok) commit_pair_mc(accf0 + 8 * b, 0x3);
                }
            }
            // Every MMA issued has finished before the TMEM is freed.
            commit_pair(done_bar);
            wait_bar(done_bar, 0, p, STATUS_DRAIN_TIMEOUT);
        }
    } else if (warp < 2 + EPI_WARPS) {
        // Epilogue: warp w reads TMEM lanes 32 (w % 4) .. + 31, which are
        // output columns; every four warps take SPAN of the tile's output rows
        // (TMEM columns).
        const int wq = warp & 3;
        const int c0 = (warp - 2) / 4 * SPAN;
        const uint32_t acce_r0 = mapa_shared(acce0, 0);
        const uint32_t lanes = tmem + (static_cast<uint32_t>(32 * wq) << 16);
        int n = 0;
        bool ok = true;
        while (ok && walk.next(piece)) {
            const Item it = item_at<WGRAD>(p, sch, piece);
            // Columns ch .. ch + 31 of the accumulator to this thread's column
            // of the output, or of a slot of TILE x TILE for a piece of a tile.
            auto write = [&](int ch, const float* v) {
                const int in_tile = static_cast<int>(rank) * HALF + 32 * wq + lane;
                const int col = it.col + in_tile;
                const int rows = col < p.N ? it.valid - c0 - ch : 0;
                const bool cut = piece.slot >= 0;
                // (An empty sum is zero whatever alpha is.)
                const float alpha = WGRAD && it.depth == 0 ? 0.0f : p.alpha;
                float* slot = p.tail_ws + static_cast<int64_t>(piece.slot) * TILE * TILE +
                              (c0 + ch) * TILE + in_tile;
                O* out = static_cast<O*>(p.y) + (col < p.N ? col : 0) + (c0 + ch) * p.ldy +
                         (WGRAD ? it.g * p.stride_y + it.ncol * p.ldy : it.row0 * p.ldy);
                if constexpr (sizeof(O) == 4) {
                    write_rows(cut ? slot : reinterpret_cast<float*>(out), cut ? TILE : p.ldy,
                               cut ? 1.0f : alpha, cut ? 0.0f : p.beta, rows, v);
                } else if (cut) {
                    write_rows(slot, TILE, 1.0f, 0.0f, rows, v);
                } else {
                    write_rows(out, p.ldy, alpha, p.beta, rows, v);
                }
            };
            const int parts = part_count<WGRAD>(it);
            if constexpr (WGRAD) {
                // Join the parts of the sum in registers, then write.
                float acc[SPAN];
#pragma unroll
                for (int j = 0; j < SPAN; ++j) acc[j] = 0.0f;
                for (int c = 0; c < parts; ++c, ++n) {
                    const int b = n & 1;
                    if (!warp_wait_bar(accf0 + 8 * b, static_cast<uint32_t>((n >> 1) & 1), p,
                                       STATUS_CONSUMER_TIMEOUT)) {
                        ok = false;
                        break;
                    }
                    fence_after();
#pragma unroll
                    for (int ch = 0; ch < SPAN; ch += 16) {
                        float v[16];
                        tmem_ld16(lanes + static_cast<uint32_t>(b * TILE + c0 + ch), v);
#pragma unroll
                        for (int j = 0; j < 16; ++j) acc[ch + j] += v[j];
                    }
                    fence_before();
                    __syncwarp();
                    if (lane == 0) arrive_read(acce_r0 + 8 * b);
                }
                if (!ok) break;
#pragma unroll
                for (int ch = 0; ch < SPAN; ch += 32)
                    write(ch, &acc[ch]);
            } else {
                const int b = n & 1;
                if (parts > 0) {
                    if (!warp_wait_bar(accf0 + 8 * b, static_cast<uint32_t>((n >> 1) & 1), p,
                                       STATUS_CONSUMER_TIMEOUT))
                        break;
                    ++n;
                    fence_after();
                }
                for (int ch = 0; ch < SPAN && c0 + ch < it.width; ch += 32) {
                    float v[32];
                    __syncwarp();
                    tmem_ld32(lanes + static_cast<uint32_t>(b * TILE + c0 + ch), v);
                    write(ch, v);
                }
                if (parts > 0) {
                    fence_before();
                    __syncwarp();
                    if (lane == 0) arrive_read(acce_r0 + 8 * b);
                }
            }
        }
    } else if (WGRAD) {
        // The last warp: zeros over the rows of a last block that are not the group's.
        int s = 0;
        uint32_t phases = 0;
        while (walk.next(piece)) {
            const Item it = item_at<WGRAD>(p, sch, piece);
            if (it.ke == it.kb) continue;
            s = (s + it.ke - it.kb - 1) % STAGES;
            const int left = it.depth - (it.ke - 1) * BK;
            if (left < BK) {
                if (!warp_wait_bar(land0 + 8 * s, (phases >> s) & 1u, p, STATUS_CONSUMER_TIMEOUT)) break;
                phases ^= 1u << s;
                // Four boxes of 64 k rows of 128 bytes; a k row stays one
                // 128-byte line under the swizzle.
                uint8_t* st = smem + s * STAGE_BYTES;
                for (int c = left * 128 + lane * 16; c < BK * 128; c += 512)
#pragma unroll
                    for (int box = 0; box < 4; ++box)
                        *reinterpret_cast<uint4*>(st + box * BOX_BYTES + c) = make_uint4(0, 0, 0, 0);
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                __syncwarp();
                if (lane == 0) {
                    if (leader) mbar_arrive(clean0 + 8 * s);
                    else mbar_arrive_remote(mapa_shared(clean0 + 8 * s, 0));
                }
            }
            s = (s + 1) % STAGES;
        }
    }

    // Single exit: every role is done (or gave up after its bounded waits);
    // rank 0's MMA thread has seen its last MMA finish, and the cluster
    // barrier makes the peer wait for that before the TMEM of both is freed.
    // If a wait was given up, no barrier vouches for the copies and MMAs of
    // either CTA (rank 1's bytes complete on rank 0's barriers, and one
    // producer may be stages ahead of the other): both CTAs stay LAND_NS.
    fence_before();
    __syncthreads();
    cluster_sync();
    fence_after();
    if (*static_cast<volatile uint32_t*>(gave_up()) != 0) {
        const uint64_t t0 = globaltimer_ns();
        while (globaltimer_ns() - t0 < LAND_NS) __nanosleep(1000);
    }
    if (warp == 1) {
        __syncwarp();
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;"
                     :: "r"(tmem), "r"(TMEM_COLS) : "memory");
    }
    cluster_sync();
}

// Adds the pieces of the cut tiles, a strip of 4 rows of one tile at a time.
constexpr int JOIN_ROWS = 4;

template <bool WGRAD, typename O>
__global__ void __launch_bounds__(256) tail_kernel(const Params p) {
    extern __shared__ int sched_sm[];
    const Schedule sch = build_schedule(p, TILE, sched_sm);
    const Walk<!WGRAD> walk(p, sch, reinterpret_cast<WalkPlan*>(sched_sm + schedule_ints(p.groups)),
                            items_per<WGRAD>(p), BK, 0);
    const int tiles = (WGRAD ? p.groups : sch.start[p.groups]) * walk.w.per - walk.w.full;
    griddep_wait();                                    // (the offsets are older than the kernel before)
    constexpr int STRIPS = TILE / JOIN_ROWS;
    Piece piece;
    piece.kb = 0;
    piece.ke = -1;
    for (int i = blockIdx.x; i < tiles * STRIPS; i += gridDim.x) {
        const int strip = i % STRIPS;
        int first, n, lo, hi;
        piece.item = walk.tile_number(i / STRIPS, first, n);
        if (!tile_pieces(walk, first, n, lo, hi)) continue;
        const Item it = item_at<WGRAD>(p, sch, piece);
        const int col = it.col + threadIdx.x;
        if (col >= p.N) continue;
        O* out = static_cast<O*>(p.y) + col +
                 (WGRAD ? it.g * p.stride_y + it.ncol * p.ldy : it.row0 * p.ldy);
        const int r0 = strip * JOIN_ROWS, rows = it.valid - r0;
        if (rows <= 0) continue;
        const float* at = p.tail_ws + r0 * TILE + threadIdx.x;
        float v[JOIN_ROWS] = {};
#pragma unroll 4
        for (int c = lo; c <= hi; ++c) {
            const float* piece_at = at + static_cast<int64_t>(slot_of(c, lo)) * TILE * TILE;
#pragma unroll
            for (int r = 0; r < JOIN_ROWS; ++r)
                if (r < rows) v[r] += piece_at[r * TILE];
        }
#pragma unroll
        for (int r = 0; r < JOIN_ROWS; ++r) {
            if (r >= rows) continue;
            O* o = out + (r0 + r) * p.ldy;
            const float x = p.alpha * v[r];
            store_f32(o, p.beta != 0.0f ? fmaf(p.beta, load_f32(o), x) : x);
        }
    }
}

// dims x: inner (contiguous), y, z; strides of y and z in elements.
bool encode_3d(CUtensorMap* map, const void* base, int64_t x, int64_t y, int64_t z, int64_t ld,
               int64_t stride, int box_x, int box_y) {
    cuuint64_t dims[3] = {static_cast<cuuint64_t>(x), static_cast<cuuint64_t>(y),
                          static_cast<cuuint64_t>(z)};
    cuuint64_t strides[2] = {static_cast<cuuint64_t>(ld) * 2, static_cast<cuuint64_t>(stride) * 2};
    cuuint32_t box[3] = {static_cast<cuuint32_t>(box_x), static_cast<cuuint32_t>(box_y), 1};
    cuuint32_t step[3] = {1, 1, 1};
    return tensor_map_encoder()(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base),
                                dims, strides, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE,
                                CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

using PairKernel = void (*)(CUtensorMap, CUtensorMap, CUtensorMap, CUtensorMap, CUtensorMap, Params);

// Clusters of two that the GPU runs at once; 0 if it cannot. Set up once per
// device and kernel.
int clusters_of(PairKernel kernel, int which, const DeviceInfo* dev, size_t smem) {
    static std::atomic<int> known[4][64];
    int n = known[which][dev->device].load(std::memory_order_acquire);
    if (n != 0) return n < 0 ? 0 : n;
    n = -1;
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             SMEM_FIXED + (schedule_ints(kMaxGroups) + WALK_INTS) * 4) == cudaSuccess) {
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(2);
        cfg.blockDim = dim3(threads_of(which == 2 || which == 3));
        cfg.dynamicSmemBytes = smem;
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = 2;
        attr[0].val.clusterDim.y = 1;
        attr[0].val.clusterDim.z = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        int most = 0;
        if (cudaOccupancyMaxActiveClusters(&most, kernel, &cfg) == cudaSuccess && most > 0) n = most;
    }
    (void)cudaGetLastError();
    known[which][dev->device].store(n, std::memory_order_release);
    return n < 0 ? 0 : n;
}

}  // namespace bf16

Tail bf16_tail(const Params& p, bool wgrad, const DeviceInfo* dev) {
    using namespace bf16;
    Tail t;
    t.workers = dev->sm_count / 2;
    t.slot_bytes = TILE * TILE * 4;
    const int64_t tiles_c = (p.N + TILE - 1) / TILE;
    const int64_t used = p.rows < p.groups ? p.rows : p.groups;
    t.items = wgrad ? p.groups * tiles_c * ((p.K + TILE - 1) / TILE) : (p.rows / TILE + used) * tiles_c;
    t.blocks = ((wgrad ? p.rows / used : p.K) + BK - 1) / BK;
    t.min_blocks = 8;
    // Below this a tile takes no longer than the second kernel (4 x 64 rows,
    // 1024 x 1024: 15.1 us whole, 18.0 in halves; 1 x 64 rows, 4096 x 4096:
    // 32.2 whole, 21.1 in quarters).
    t.worth = 32;
    // A slot's bytes grow with a tile's rows, and W of many pairs comes at HBM's
    // rate whether they share tiles or not (K = 8192, us whole and cut: 4 tiles
    // of 32 rows 58 and 22, of 256 rows 46 and 27; 32 tiles of 32 rows 58 and
    // 49, of 256 rows 56 and 58; 60 tiles of 32 rows 66 and 77, of 256 rows 68
    // and 88). Tiles of more than 160 rows never gained above a half.
    const int64_t mean = wgrad ? p.K : p.rows / used;
    const int high = static_cast<int>(mean < TILE ? mean : TILE);
    t.rule = TailRule{10, 35 + high * high / 800, high <= 160 ? 55 + high / 8 : INT_MAX};
    return t;
}

cudaError_t launch_bf16(const Params& p0, bool wgrad, const DeviceInfo* dev, cudaStream_t stream) {
    using namespace bf16;
    Params p = p0;
    PairKernel kernel;
    int which;
    CUtensorMap a, b, b64, b32, b16;
    bool ok;
    if (wgrad) {
        which = p.out_bf16 ? 2 : 3;
        kernel = p.out_bf16 ? &pair_kernel<true, true, __nv_bfloat16> : &pair_kernel<true, true, float>;
        ok = encode_3d(&a, p.w, p.N, p.rows, 1, p.ldw, p.ldw, 64, BK) &&
             encode_3d(&b, p.x, p.K, p.rows, 1, p.ldx, p.ldx, 64, BK);
        b64 = b32 = b16 = b;
    } else {
        which = p.opw ? 0 : 1;
        kernel = p.opw ? &pair_kernel<false, false, __nv_bfloat16>
                       : &pair_kernel<true, false, __nv_bfloat16>;
        // One matrix has no stride to speak of; the map wants one.
        const int64_t stride = p.groups > 1 ? p.stride_w : p.ldw;
        ok = p.opw ? encode_3d(&a, p.w, p.K, p.N, p.groups, p.ldw, stride, BK, HALF)
                   : encode_3d(&a, p.w, p.N, p.K, p.groups, p.ldw, stride, 64, BK);
        ok = ok && encode_3d(&b, p.x, p.K, p.rows, 1, p.ldx, p.ldx, BK, HALF) &&
             encode_3d(&b64, p.x, p.K, p.rows, 1, p.ldx, p.ldx, BK, 64) &&
             encode_3d(&b32, p.x, p.K, p.rows, 1, p.ldx, p.ldx, BK, 32) &&
             encode_3d(&b16, p.x, p.K, p.rows, 1, p.ldx, p.ldx, BK, 16);
    }
    const Tail t = bf16_tail(p, wgrad, dev);
    if (!ok || t.items > 0x3fffffff) return cudaErrorInvalidValue;
    const size_t sched = (schedule_ints(p.groups) + WALK_INTS) * sizeof(int);
    const int clusters = clusters_of(kernel, which, dev, SMEM_FIXED + sched);
    if (clusters <= 0) return cudaErrorInvalidConfiguration;
    int64_t workers = clusters < t.workers ? clusters : t.workers;
    if (p.tail_ws == nullptr && t.items < workers) workers = t.items;
    p.workers = static_cast<int>(workers);
    p.tail_min = static_cast<int>(t.min_blocks);
    p.tail_rule = t.rule;
    cudaError_t e = launch_kernel(kernel, dim3(static_cast<unsigned>(2 * workers)), dim3(threads_of(wgrad)),
                                  SMEM_FIXED + sched, stream, p.pdl != 0, 2, a, b, b64, b32, b16, p);
    if (e == cudaSuccess && p.tail_ws != nullptr) {
        void (*join)(Params) = wgrad ? (p.out_bf16 ? &tail_kernel<true, __nv_bfloat16>
                                                   : &tail_kernel<true, float>)
                                     : &tail_kernel<false, __nv_bfloat16>;
        e = launch_kernel(join, dim3(static_cast<unsigned>(8 * dev->sm_count)), dim3(256), sched, stream,
                          pdl_enabled(), 1, p);
    }
    return e;
}

}  // namespace grouped
}  // namespace sg

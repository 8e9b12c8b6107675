// grouped.cuh — the schedule that the grouped kernels share: which rows each
// expert has, read and checked on the device, and which tile an item is.
#pragma once

#include "expert.h"
#include "kernels.h"

namespace sg {
namespace grouped {

// When the last round of tiles is cut: whole it lasts as long as its longest
// sum, cut it lasts a worker's share, and what that saves, in blocks of k, has
// to reach the price of slots and joining. The price grows with the part r of
// the workers that have a whole tile (the rest of the GPU's bandwidth is idle
// then, and a tile alone is faster): base + slope * r up to a half, above that
// `over`.
struct TailRule {
    int base, slope, over;
};

// What every grouped kernel takes. Forward (and input gradient): output rows
// off[g] .. off[g+1] are X's rows times W_g (opw: 0 stored K x N, 1 stored
// N x K). Weight gradient: D_g (M x N) = P^T Q over those rows; P is in x
// (M columns), Q in w (N columns), K is M.
struct Params {
    int groups;
    int64_t rows;
    int N, K;
    const int* offsets;
    const void* x;
    const void* w;
    void* y;
    int64_t ldx, ldw, stride_w, ldy, stride_y;
    float alpha, beta;
    int opw;
    int out_bf16;
    int y_vec;                      // y rows allow 16-byte stores
    int w_vec, x_vec;               // rows allow 16-byte loads
    int w_tma;                      // w can be read by TMA
    int pdl;                        // host: launch behind this call's packing kernels
    // streaming kernel: sums split over `parts` items each (few strips, long
    // sums); part q goes to y + q * part_stride, FP32, for join_kernel.
    int parts;
    int64_t part_stride;
    // tile kernels: blocks (pairs of blocks) at work; and where the last,
    // partial round of tiles is split evenly over all of them (see Walk), the
    // slots of the split tiles' sums, two per worker, and the fewest blocks of
    // k to take apart. tail_ws null: not split.
    int workers;
    float* tail_ws;
    int tail_min;
    TailRule tail_rule;
    unsigned long long timeout_ns;
    int* status;
};

// A block that gives up a bounded wait stays until what it has in flight has
// landed, however short the caller's limit is: this long without a barrier to
// tell, thousands of times what a copy or an MMA takes.
constexpr unsigned long long LAND_NS = 20000000ull;

// Shared-memory schedule: off[0..groups], the groups by falling number of
// rows (perm), and start[0..groups], the row tiles of at most `per` rows
// before the group at each place of that order. A group whose offsets do not
// satisfy 0 <= off[g] <= off[g+1] <= rows counts as empty and sets
// STATUS_BAD_INDEX, so no later address depends on it. All threads call it;
// ends synchronised.
//
// Blocks take items round robin, forth and back (item_of), large groups first:
// a work queue's balance, nearly, without its counter. Groups are sorted, not
// tiles: a group's tiles are of one height, or its last one is lower, and the
// heights of neighbouring groups differ (256 rows make one tile of 256, 259 two
// of 160), so a round's items are not all of one cost. By the tiles' heights
// the busiest of 76 pairs has 4.4 % more than the mean (16384 rows over 8 uneven
// groups, 14336 columns) or 8.3 % (8192 rows over 32, 4096 columns). Above
// kSortGroups groups there are many items per block and the order is left as it
// is (the ranking is quadratic).
constexpr int kSortGroups = 256;

struct Schedule {
    int* off;
    int* start;
    int* perm;
};
__host__ __device__ constexpr int schedule_ints(int groups) { return 3 * (groups + 1); }   // and WALK_INTS

__device__ __forceinline__ int group_rows(const Schedule& s, int64_t rows, int g) {
    const int lo = s.off[g], hi = s.off[g + 1];
    return lo < 0 || hi < lo || hi > rows ? -1 : hi - lo;
}

__device__ __forceinline__ Schedule build_schedule(const Params& p, int per, int* sm) {
    Schedule s{sm, sm + p.groups + 1, sm + 2 * (p.groups + 1)};
    for (int g = threadIdx.x; g <= p.groups; g += blockDim.x) s.off[g] = p.offsets[g];
    __syncthreads();
    for (int g = threadIdx.x; g < p.groups; g += blockDim.x) {
        const int mine = group_rows(s, p.rows, g);
        if (mine < 0 && blockIdx.x == 0) atomicOr(p.status, STATUS_BAD_INDEX);
        int rank = g;
        if (p.groups <= kSortGroups) {
            rank = 0;
            for (int h = 0; h < p.groups; ++h) {
                const int other = group_rows(s, p.rows, h);
                rank += other > mine || (other == mine && h < g);
            }
        }
        s.perm[rank] = g;
    }
    __syncthreads();
    if (threadIdx.x < 32) {
        const int lane = threadIdx.x;
        int base = 0;
        for (int i0 = 0; i0 < p.groups; i0 += 32) {
            const int i = i0 + lane;
            int tiles = 0;
            if (i < p.groups) {
                const int n = group_rows(s, p.rows, s.perm[i]);
                tiles = n > 0 ? (n - 1) / per + 1 : 0;
            }
            int x = tiles;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int v = __shfl_up_sync(0xffffffffu, x, o);
                if (lane >= o) x += v;
            }
            if (i < p.groups) s.start[i] = base + x - tiles;
            base += __shfl_sync(0xffffffffu, x, 31);
        }
        if (lane == 0) s.start[p.groups] = base;
    }
    __syncthreads();
    return s;
}

// The place in the order of row tile `t` (start[i] <= t < start[i+1]).
__device__ __forceinline__ int place_of(const Schedule& s, int groups, int t) {
    int lo = 0, hi = groups;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (s.start[mid] <= t) lo = mid;
        else hi = mid;
    }
    return lo;
}

// The blocks [lo, hi) of a sum of `blocks` that part q of `parts` takes.
__device__ __forceinline__ void part_range(int blocks, int parts, int q, int& lo, int& hi) {
    const int per = (blocks + parts - 1) / parts;
    lo = min(blocks, q * per);
    hi = min(blocks, lo + per);
}

// Worker w's item in round r, of `workers`.
__device__ __forceinline__ int item_of(int r, int w, int workers) {
    return r * workers + ((r & 1) ? workers - 1 - w : w);
}

// What a worker does, tile by tile: whole tiles in rounds, then its share of
// the last round. When the tiles do not fill the last round (or the only
// one) and TailRule finds it worth it, its blocks of k, all tiles' in a row,
// are cut into equal shares: a worker takes the end of one tile, perhaps whole
// ones, and the start of another. The sums of cut tiles go to slots (2 w: a piece that starts inside
// its tile, 2 w + 1: one that starts with it), and a second kernel adds a
// tile's pieces in the order of k. Every worker, and that kernel, computes the
// same cut from the offsets.
// UNIFORM: all sums are equally long (forward); else a group's tiles sum over
// its rows (weight gradient), in blocks of bk.
struct Piece {
    int item, kb, ke, slot;          // blocks [kb, ke) of the tile; slot -1: all of them
};

// What does not change, in shared memory: the main loops have no registers to
// spare for it.
struct WalkPlan {
    int per, blocks, bk;             // items of a row tile (of a group); blocks of a sum
    int full;                        // whole items [0, full)
    int share, u, end;               // a worker's blocks of the cut round; its first, its last
};
constexpr int WALK_INTS = sizeof(WalkPlan) / sizeof(int);

template <bool UNIFORM>
struct Walk {
    const Params& p;
    const Schedule& s;
    const WalkPlan& w;
    int round, u;

    // All threads call it; `plan` is WALK_INTS of shared memory.
    __device__ __forceinline__ Walk(const Params& p_, const Schedule& s_, WalkPlan* plan, int per,
                                    int bk, int me)
        : p(p_), s(s_), w(*plan), round(0), u(0) {
        if (threadIdx.x == 0) {
            const int items = (UNIFORM ? s.start[p.groups] : p.groups) * per;
            plan->per = per;
            plan->bk = bk;
            plan->blocks = UNIFORM ? (p.K + bk - 1) / bk : 0;
            plan->full = items;
            plan->u = plan->end = 0;
            plan->share = 1;
            const int rest = items % p.workers;
            if (p.tail_ws != nullptr && rest != 0) {
                int longest = plan->blocks;
                int64_t all = static_cast<int64_t>(rest) * plan->blocks;
                if (!UNIFORM) {
                    longest = 0;
                    for (int i = items - rest; i < items;) {
                        const int place = i / per, n = (place + 1) * per - i, b = blocks_at(place);
                        all += static_cast<int64_t>(n) * b;
                        longest = max(longest, b);
                        i += n;
                    }
                }
                const int64_t share = max(static_cast<int64_t>(p.tail_min), (all + p.workers - 1) / p.workers);
                const TailRule& r = p.tail_rule;
                const int price = 2 * rest <= p.workers ? r.base + r.slope * rest / p.workers : r.over;
                if (all <= (1 << 30) && longest - share >= max(1, price)) {
                    plan->share = static_cast<int>(share);
                    plan->full = items - rest;
                    plan->u = static_cast<int>(min(all, me * share));
                    plan->end = static_cast<int>(min(all, me * share + share));
                }
            }
        }
        __syncthreads();
        u = w.u;
    }
    __device__ __forceinline__ int me() const {
        return static_cast<int>(blockIdx.x) / (static_cast<int>(gridDim.x) / p.workers);
    }
    // Blocks of a sum at a place of the order; an empty sum counts as one.
    __device__ __forceinline__ int blocks_at(int place) const {
        return UNIFORM ? w.blocks : max(1, (group_rows(s, p.rows, s.perm[place]) + w.bk - 1) / w.bk);
    }
    // The cut tile that unit `at` lies in, the first unit and the number of its blocks.
    __device__ __forceinline__ int tile_of(int at, int& first, int& n) const {
        if (UNIFORM) {
            const int j = at / w.blocks;
            first = j * w.blocks;
            n = w.blocks;
            return w.full + j;
        }
        first = 0;
        for (int i = w.full;;) {
            const int place = i / w.per, count = (place + 1) * w.per - i;
            n = blocks_at(place);
            const int span = count * n;
            if (at < first + span || place + 1 >= p.groups) {
                const int j = (at - first) / n;
                first += j * n;
                return i + j;
            }
            first += span;
            i += count;
        }
    }
    // The same for the j-th cut tile.
    __device__ __forceinline__ int tile_number(int j, int& first, int& n) const {
        first = 0;
        if (UNIFORM) {
            first = j * w.blocks;
            n = w.blocks;
        } else {
            for (int i = w.full; i <= w.full + j;) {
                const int place = i / w.per, count = min((place + 1) * w.per, w.full + j) - i;
                n = blocks_at(place);
                first += count * n;
                i += count == 0 ? w.per : count;
            }
        }
        return w.full + j;
    }
    __device__ __forceinline__ bool next(Piece& q) {
        if (static_cast<int64_t>(round) * p.workers < w.full) {
            q.item = item_of(round, me(), p.workers);
            ++round;
            if (q.item < w.full) {
                q.kb = 0;
                q.ke = -1;
                q.slot = -1;
                return true;
            }
            return false;                              // (only without a cut round)
        }
        if (u >= w.end) return false;
        int first, n;
        q.item = tile_of(u, first, n);
        q.kb = u - first;
        q.ke = min(n, w.end - first);
        q.slot = q.kb > 0 ? 2 * me() : q.ke < n ? 2 * me() + 1 : -1;
        if (q.slot < 0) q.ke = -1;
        u = first + (q.ke < 0 ? n : q.ke);
        return true;
    }
};

// The workers [lo, hi] that hold pieces of the cut tile of units [first,
// first + n); false if it is whole.
template <bool UNIFORM>
__device__ __forceinline__ bool tile_pieces(const Walk<UNIFORM>& w, int first, int n, int& lo,
                                            int& hi) {
    lo = first / w.w.share;
    hi = (first + n - 1) / w.w.share;
    return lo != hi;
}
// Slot of worker c's piece of a tile whose first piece is worker lo's.
__device__ __forceinline__ int slot_of(int c, int lo) { return c == lo ? 2 * c + 1 : 2 * c; }

// An output tile in units of tiles: place i of the order, N-side tile t of the
// group's `rows` ones, column tile c. Bands of `band` row tiles share a pass
// over the columns, row tiles fastest: the columns' operand is then read once
// per band from HBM, and the band's rows stay in L2.
struct TileAt {
    int place, t, c;
};
__device__ __forceinline__ TileAt tile_at(int item, int first, int rows, int tiles_c, int band,
                                          int place) {
    const int r = item - first;
    const int b = r / (band * tiles_c);
    const int high = min(band, rows - b * band);
    const int q = r - b * band * tiles_c;
    return TileAt{place, b * band + q % high, q / high};
}

}  // namespace grouped
}  // namespace sg

// ep_tiles.h — device helpers of the expert products: tiles of rows that are
// grouped by expert, copies from memory to LDS and the wavefronts' meetings.
#pragma once

#include "ep_rows8.h"

namespace ep {

// Row tiles of bm rows that M rows in G groups can need at most.
__host__ __device__ inline int64_t max_tiles(int64_t M, int32_t G, int bm) {
    return M / bm + (G < M ? (int64_t)G : M);
}

// The rows of a tile of `bm` rows, tiles counted over the groups in order.
struct RowTile {
    int32_t g;        // group; -1: no such tile
    int64_t first;    // first row of the tile
    int32_t count;    // its rows, 1 .. bm
};

__device__ inline int64_t clamp_row(int64_t r, int64_t M) { return r < 0 ? 0 : r > M ? M : r; }

// A step of find_tile: lane l has the first row `lo` and the `n` rows of group g0 + l.
// Whether `tile` is one of theirs (or one that overlapping groups leave out: r->g is
// -1 then), *before* the tiles of the groups before g0, which gets theirs added.
__device__ inline bool find_in(int64_t lo, int64_t n, int g0, int64_t* before, int64_t tile, int bm,
                               RowTile* r) {
    const int lane = lane_id();
    const int t = (int)((n + bm - 1) / bm);
    int sum = t;   // inclusive scan: at most M < 2^31 tiles where the offsets are in order
#pragma unroll
    for (int o = 1; o < kWave; o *= 2) {
        const int up = __shfl_up(sum, o);
        sum += lane >= o ? up : 0;
    }
    const uint64_t here = __ballot(tile < *before + sum);
    if (here) {
        const int l = __builtin_ctzll(here);
        const int in = (int)(tile - *before) - (bcast(sum, l) - bcast(t, l));
        // overlapping groups can wrap the sum: such a tile is left out
        if (in < 0 || in >= bcast(t, l)) return true;
        r->g = g0 + l;
        r->first = (int64_t)bcast((int32_t)lo, l) + (int64_t)in * bm;
        const int64_t left = (int64_t)bcast((int32_t)n, l) - (int64_t)in * bm;
        r->count = (int)(left < bm ? left : bm);
        return true;
    }
    *before += bcast(sum, kWave - 1);
    return false;
}

// Called by whole wavefronts: lane l looks at group g0 + l, 64 groups a step.
// Offsets outside [0, M] or decreasing are clamped, so that a tile's rows are
// always rows of the buffers (check_groups reports them).
__device__ inline RowTile find_tile(const int32_t* off, int G, int64_t M, int64_t tile, int bm) {
    RowTile r{-1, 0, 0};
    int64_t before = 0;   // tiles of the groups before g0
    for (int g0 = 0; g0 < G; g0 += kWave) {
        const int g = g0 + lane_id();
        int64_t lo = 0, n = 0;
        if (g < G) {
            lo = clamp_row(off[g], M);
            n = clamp_row(off[g + 1], M) - lo;
            n = n < 0 ? 0 : n;
        }
        if (find_in(lo, n, g0, &before, tile, bm, &r)) return r;
    }
    return r;
}

// Tiles of all groups.
__device__ inline int64_t count_tiles(const int32_t* off, int G, int64_t M, int bm) {
    int64_t all = 0;
    for (int g0 = 0; g0 < G; g0 += kWave) {
        const int g = g0 + lane_id();
        int t = 0;
        if (g < G) {
            const int64_t n = clamp_row(off[g + 1], M) - clamp_row(off[g], M);
            t = n > 0 ? (int)((n + bm - 1) / bm) : 0;
        }
#pragma unroll
        for (int o = 1; o < kWave; o *= 2) t += __shfl_xor(t, o);
        all += bcast(t, 0);
    }
    return all;
}

// Decreasing or negative offsets, and rows beyond M, by the first workgroup.
__device__ inline void check_groups(const int32_t* off, int G, int64_t M, int32_t* st) {
    for (int g = (int)threadIdx.x; g <= G; g += (int)blockDim.x) {
        const int32_t o = off[g];
        if (o < 0 || (g > 0 && o < off[g - 1])) set_error(st, EP_ERR_INVALID_ARG);
        if (o > M) set_error(st, EP_ERR_CAPACITY);
    }
}

typedef __attribute__((address_space(3))) void* LdsPtr;

// Sixteen bytes a lane from offset `lane_at` + `at` of a buffer to LDS: 64 lanes
// to 1 KB from `lds` on; `at` and `lds` are the same for the wavefront.
__device__ inline void to_lds(__amdgpu_buffer_rsrc_t p, uint32_t lane_at, uint32_t at,
                              uint8_t* lds) {
    __builtin_amdgcn_raw_ptr_buffer_load_lds(p, (LdsPtr)lds, 16, (int)lane_at, (int)at, 0, 0);
}

// Waits until at most VM of the wavefront's memory operations and LDS of its
// LDS reads are under way (each kind ends in its order), then for the other
// wavefronts.  (__syncthreads would wait for all the copies.)
template <int VM, int LDS>
__device__ inline void meet() {
    asm volatile("" ::: "memory");
    // gfx9 encoding: vmcnt in bits 3:0 and 15:14, expcnt 6:4 at its maximum,
    // lgkmcnt 11:8
    __builtin_amdgcn_s_waitcnt((VM & 15) | (VM >> 4 << 14) | 0x70 | LDS << 8);
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
}

// A workgroup's share of the tiles.  Workgroups go to the eight XCDs in turn:
// each XCD gets one run of the tiles, ordered so that the 32 it has at a time
// are 5 row tiles x 6 or 7 column tiles, whose operands its L2 shares (8-bit, 8192 x
// 8192 x 7168: 480 us against 486, 496, 486, 500 for 3, 4, 6 and 8; bf16, the same forward
// 656 us against 659, 652, 655, 653, 4 experts of 8192 x 8192 with 960 rows each 411
// against 418, 386, 394, 392, their weights' gradient 430 against 436, 448, 437, 458).
constexpr int kBand = 5;
struct TileShare {
    int64_t row_tiles, first;   // first: this workgroup's; the next ones follow `step` apart
    int32_t count, step, n_tiles;

    __device__ TileShare(int64_t row_tiles_, int n_tiles_) {
        row_tiles = row_tiles_;
        n_tiles = n_tiles_;
        const int64_t all = row_tiles * n_tiles, per = all / 8, extra = all % 8;
        const int xcd = (int)(blockIdx.x % 8u), slot = (int)(blockIdx.x / 8u);
        step = (int)(gridDim.x / 8u);
        const int64_t run = per + (xcd < extra);
        first = xcd * per + (xcd < extra ? xcd : extra) + slot;
        count = slot < run ? (int)((run - slot + step - 1) / step) : 0;
    }

    // row tile and column tile of the workgroup's i-th tile
    __device__ void place(int i, int64_t* m, int* n) const {
        const int64_t at = first + (int64_t)i * step, wide = kBand * (int64_t)n_tiles;
        const int64_t band = at / wide;
        const int in = (int)(at - band * wide);
        const int64_t left = row_tiles - band * kBand;
        const int rows = (int)(left < kBand ? left : kBand);
        *m = band * kBand + in % rows;
        *n = in / rows;
    }
};

}  // namespace ep

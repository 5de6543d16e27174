// Rows in groups of any length (gfx950): sequences of a packed batch, rows of
// experts.
//
// Groups are offsets[q] <= r < offsets[q + 1] on the device (or equal
// lengths), within n rows; what lies before the first and past the last is in
// no group.  With those two as groups of their own, bounds b_0 = 0 <= b_1 =
// offsets[0] <= ... <= b_{count + 2} = n, tiles of T rows are numbered so that
// group j's first is b_j / T + j: that many tiles suffice, as
// ceil(l / T) <= (b + l) / T - b / T + 1, and a tile's group is found by a
// search in the bounds.  Each offset is cut to [0, n], so whatever the array
// holds, tiles stay within the rows.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

namespace lx {

struct RaggedTile {
    int64_t group;   // -1: rows of no group
    int64_t row;     // first row
    int64_t index;   // tile of its group
    int64_t first;   // the group's first row
    int64_t end;     // past its last
    int rows;        // of the tile; <= 0: no such tile
};

struct Ragged {
    const int32_t* offsets;  // [count + 1], or null: groups of `length` rows
    int64_t count, n, length;

    __host__ __device__ int64_t units(int tile) const { return n / tile + count + 2; }

    // b_j, 0 <= j <= count + 2
    __device__ __forceinline__ int64_t bound(int64_t j) const
    {
        if (j <= 0) return 0;
        if (j > count + 1) return n;
        const int64_t b = offsets ? (int64_t)offsets[j - 1] : (j - 1) * length;
        return b < 0 ? 0 : b > n ? n : b;
    }

    // Tile `unit` of T rows; the same answer in every lane of a wave (all lanes must call).
    __device__ __forceinline__ RaggedTile find(int64_t unit, int T) const
    {
        const int lane = threadIdx.x & 63;
        // the last j in [lo, lo + span) with b_j / T + j <= unit; j = lo always is one
        int64_t lo = 0, span = count + 2;
        while (span > 1) {
            const int64_t step = (span + 63) / 64;
            const int64_t j = lo + lane * step;
            const bool ok = lane * step < span && bound(j) / T + j <= unit;
            const uint64_t m = __ballot(ok);
            // ascending offsets give a run of ones; whatever they hold, take its end
            const int k = __builtin_ctzll(~m | (1ull << 63)) - 1;
            const int at = m == ~0ull ? 63 : (k < 0 ? 0 : k);
            lo += at * step;
            span = span - at * step < step ? span - at * step : step;
        }
        RaggedTile t;
        t.first = bound(lo);
        t.end = bound(lo + 1);
        t.index = unit - (t.first / T + lo);
        t.row = t.first + t.index * T;
        const int64_t left = t.end - t.row;
        t.rows = t.index < 0 || left <= 0 ? 0 : left < T ? (int)left : T;
        t.group = lo >= 1 && lo <= count ? lo - 1 : -1;
        return t;
    }
};

}  // namespace lx

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

// A value that is the same in all lanes, in scalar registers.
__device__ __forceinline__ int uniform(int x) { return __builtin_amdgcn_readfirstlane(x); }
__device__ __forceinline__ int64_t uniform(int64_t x)
{
    return (int64_t)(((uint64_t)(uint32_t)uniform((int)((uint64_t)x >> 32)) << 32) | (uint32_t)uniform((int)x));
}

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
        lo = uniform(lo);
        t.first = uniform(bound(lo));
        t.end = uniform(bound(lo + 1));
        t.index = unit - (t.first / T + lo);
        t.row = t.first + t.index * T;
        const int64_t left = t.end - t.row;
        t.rows = t.index < 0 || left <= 0 ? 0 : left < T ? (int)left : T;
        t.group = lo >= 1 && lo <= count ? lo - 1 : -1;
        return t;
    }

    // Tiles of T rows without gaps in their numbers: the groups', one after
    // the other, then those of rows of no group.  Their sums over the groups
    // are worked out by each wave (count at most 4096, all lanes must call).
    struct Dense {
        int up_to;           // tiles up to the end of this lane's run of groups
        int inside, outside; // tiles of groups, and of rows of no group
    };
    __device__ __forceinline__ int64_t length_of(int64_t g) const
    {
        const int64_t l = g < count ? bound(g + 2) - bound(g + 1) : 0;
        return l > 0 ? l : 0;
    }
    __device__ __forceinline__ static int scan(int x)
    {
        const int lane = threadIdx.x & 63;
#pragma unroll
        for (int d = 1; d < 64; d *= 2) {
            const int below = __shfl_up(x, d);
            if (lane >= d) x += below;
        }
        return x;
    }
    __device__ __forceinline__ Dense dense(int T) const
    {
        const int per = (int)((count + 63) / 64), lane = threadIdx.x & 63;
        int tiles = 0;
        for (int i = 0; i < per; ++i) tiles += (int)((length_of(lane * per + i) + T - 1) / T);
        Dense d;
        d.up_to = scan(tiles);
        d.inside = uniform(__shfl(d.up_to, 63));
        d.outside = uniform((int)((bound(1) + T - 1) / T + (n - bound(count + 1) + T - 1) / T));
        return d;
    }
    __device__ __forceinline__ RaggedTile dense_tile(const Dense& d, int k, int T) const
    {
        const int per = (int)((count + 63) / 64), lane = threadIdx.x & 63;
        const uint64_t past = __ballot(d.up_to > k);
        const int run = past ? __builtin_ctzll(past) : 63;
        const int below = __shfl(d.up_to, run > 0 ? run - 1 : 0);
        k -= run > 0 ? below : 0;
        const int in_run = scan(lane < per ? (int)((length_of(run * per + lane) + T - 1) / T) : 0);
        const uint64_t at = __ballot(in_run > k);
        const int i = at ? __builtin_ctzll(at) : 0;
        const int under = __shfl(in_run, i > 0 ? i - 1 : 0);
        k -= i > 0 ? under : 0;
        RaggedTile t;
        t.group = uniform(run * per + i);
        t.first = uniform(bound(t.group + 1));
        t.end = t.first + uniform(length_of(t.group));
        t.index = uniform(k);
        t.row = t.first + t.index * T;
        const int64_t left = t.end - t.row;
        t.rows = t.group >= count || left <= 0 ? 0 : left < T ? (int)left : T;
        return t;
    }
    // Tile k of the rows of no group.
    __device__ __forceinline__ RaggedTile outside_tile(int k, int T) const
    {
        const int64_t head = bound(1), heads = (head + T - 1) / T;
        RaggedTile t;
        t.group = -1;
        t.first = k < heads ? 0 : uniform(bound(count + 1));
        t.end = k < heads ? head : n;
        t.index = k < heads ? k : k - heads;
        t.row = t.first + t.index * T;
        const int64_t left = t.end - t.row;
        t.rows = left <= 0 ? 0 : left < T ? (int)left : T;
        return t;
    }
};

}  // namespace lx

// Device parts shared by the gated recurrence and its backward pass.
//
// Along the rows (tokens) of one sequence, for every channel,
//     h_t = a_t h_{t-1} + x_t,   a_t = exp(g_t),
// the causal half of the operator's scan with its decays given per token: an
// affine map per row, composed along rows.  Rows are cut into tiles of
// kRecurTile rows by kRecurCols channels, one workgroup each.  A thread has V
// neighbouring channels of L consecutive rows in registers; the LR threads
// of a row group cover the tile's channels, 4 V groups its rows:
//     V = 4: 16 lanes x 16 groups of 8 rows, loads of 8 bytes (half types)
//     V = 1: 64 lanes x  4 groups of 32 rows, for rows without alignment
// A decay of exactly zero forgets the state, whatever it held (inf and NaN
// too): 0 * h is never formed.  The first row of a sequence is such a row,
// with a h0 added to x, so one form serves packed and single sequences.
// States, decays and sums are float32.
#pragma once
#include "lx_device.h"
#include "lx_internal.h"
#include "lx_types.h"

namespace lx {

constexpr int kRecurThreads = 256;

template <int V>
struct RecurLayout {
    static constexpr int kLanes = kRecurCols / V;               // threads per row
    static constexpr int kGroups = kRecurThreads / kLanes;      // row groups
    static constexpr int kRows = kRecurTile / kGroups;          // rows per thread
};

// e^g by the hardware's base-2 exponential (1 ulp), which flushes results
// below 2^-126: those are made 2^64 larger and scaled back, so only an e^g
// below the smallest float32 is 0 and forgets the state.
__device__ __forceinline__ float decay_of(float g)
{
    const float p = g * 1.44269504088896341f;
    const bool low = p < -126.f;
    const float e = __builtin_amdgcn_exp2f(low ? p + 64.f : p);
    return low ? e * 0x1p-64f : e;
}

// a h + x, forgetting h where a is 0.
__device__ __forceinline__ float step_of(float a, float h, float x) { return a == 0.f ? x : fmaf(a, h, x); }

// What is special about a tile's rows.
struct RecurRows {
    int start[kRecurTile];  // sequence whose first row this is; -1: none; -2: a row of no sequence
    int last[kRecurTile];   // sequence whose last row this is; -1: none
    int any;                // whether any row is special
};

// Index of the first of n values that is not below `key` (values ascend),
// 64 probes at a time; the same in every lane.  For values in any order the
// result is still in [0, n].
__device__ __forceinline__ int64_t lower_bound64(const int32_t* v, int64_t n, int64_t key)
{
    int64_t lo = 0, hi = n;
    while (lo < hi) {
        const int64_t step = (hi - lo + kWave - 1) / kWave;
        const int64_t at = lo + (int64_t)lane_id() * step;
        const bool below = at < hi && (int64_t)v[at] < key;
        const int c = __popcll(__ballot(below));
        if (c == 0) break;
        const int64_t next = lo + (int64_t)c * step;
        lo += (int64_t)(c - 1) * step + 1;
        if (next < hi) hi = next;
        if (step == 1) break;
    }
    return lo;
}

// Fills R for the tile of rows [t0, t0 + kRecurTile).  All threads; ends
// with a barrier.
__device__ __forceinline__ void recur_rows(const RecurArgs& A, int64_t t0, RecurRows& R)
{
    const int tid = threadIdx.x;
    if (tid == 0) R.any = 0;
    if (tid < kRecurTile) {
        const int64_t t = t0 + tid;
        int start = -1, last = -1;
        if (t >= A.n) {
            start = -2;
        } else if (!A.offsets) {
            const int64_t q = A.seqs == 1 ? 0 : t / A.seq_len;
            const int64_t at = t - q * A.seq_len;
            if (at == 0) start = (int)q;
            if (at == A.seq_len - 1) last = (int)q;
        } else if (t < (int64_t)A.offsets[0] || t >= (int64_t)A.offsets[A.seqs]) {
            start = -2;
        }
        R.start[tid] = start;
        R.last[tid] = last;
    }
    __syncthreads();
    if (A.offsets && tid < kWave) {
        // one wave: the offsets in [t0, t0 + kRecurTile], 64 at a time
        const int64_t end = t0 + kRecurTile;
        for (int64_t q0 = lower_bound64(A.offsets, A.seqs + 1, t0); q0 <= A.seqs; q0 += kWave) {
            const int64_t q = q0 + tid;
            const int64_t o = q <= A.seqs ? (int64_t)A.offsets[q] : end + 1;
            if (o >= t0 && o <= end) {
                // the last of several equal offsets starts the one sequence that is not empty
                if (q < A.seqs && o < end && (int64_t)A.offsets[q + 1] > o) R.start[o - t0] = (int)q;
                if (q > 0 && o > t0 && (int64_t)A.offsets[q - 1] < o) R.last[o - 1 - t0] = (int)(q - 1);
            }
            if (__ballot(o > end)) break;
        }
    }
    __syncthreads();
    if (tid < kRecurTile && (R.start[tid] != -1 || R.last[tid] != -1)) R.any = 1;
    __syncthreads();
}

// Raw rows of one array: L rows of V channels, zero outside.
template <int V, int L, class T>
__device__ __forceinline__ void load_rows(const void* base, int64_t ld, int64_t row0, int64_t n, int64_t col, bool in,
                                          float (&out)[L][V])
{
    const T* p = (const T*)base + row0 * ld + col;
    if (in && row0 + L <= n) {
#pragma unroll
        for (int j = 0; j < L; ++j) load_vec<V>(p + j * ld, out[j]);
    } else {
#pragma unroll
        for (int j = 0; j < L; ++j) {
            if (in && row0 + j < n) {
                load_vec<V>(p + j * ld, out[j]);
            } else {
#pragma unroll
                for (int v = 0; v < V; ++v) out[j][v] = 0.f;
            }
        }
    }
}

template <int V, int L, class T>
__device__ __forceinline__ void store_rows(void* base, int64_t ld, int64_t row0, int64_t n, int64_t col, bool in,
                                           const float (&val)[L][V])
{
    T* p = (T*)base + row0 * ld + col;
    if (in && row0 + L <= n) {
#pragma unroll
        for (int j = 0; j < L; ++j) store_vec<V>(p + j * ld, val[j]);
    } else if (in) {
#pragma unroll
        for (int j = 0; j < L; ++j)
            if (row0 + j < n) store_vec<V>(p + j * ld, val[j]);
    }
}

// A thread's rows of x and decays.  SH: one decay serves the V channels.
template <class T, class TG, int V, bool SH>
struct RecurThread {
    static constexpr int L = RecurLayout<V>::kRows;
    static constexpr int D = SH ? 1 : V;
    float x[L][V], a[L][D];
    int64_t row0, col;
    int r0, lane, group;  // first row within the tile, thread of the row, row group
    bool in;              // channels inside the width

    __device__ __forceinline__ void load(const RecurArgs& A, int64_t tile, int ct)
    {
        lane = (int)threadIdx.x % RecurLayout<V>::kLanes;
        group = (int)threadIdx.x / RecurLayout<V>::kLanes;
        r0 = group * L;
        row0 = tile * kRecurTile + r0;
        col = (int64_t)ct * kRecurCols + lane * V;
        in = col < A.width;
        load_rows<V, L, T>(A.x, A.ldx, row0, A.n, col, in, x);
        load_rows<D, L, TG>(A.g, A.ldg, row0, A.n, SH ? col / A.per : col, in, a);
    }
    __device__ __forceinline__ void decays()
    {
#pragma unroll
        for (int j = 0; j < L; ++j)
#pragma unroll
            for (int d = 0; d < D; ++d) a[j][d] = decay_of(a[j][d]);
    }
    // first rows of sequences take h0 in and forget what came before; rows of
    // no sequence are 0
    __device__ __forceinline__ void special(const RecurArgs& A, const RecurRows& R)
    {
#pragma unroll
        for (int j = 0; j < L; ++j) {
            const int q = R.start[r0 + j];
            if (q == -1) continue;
            float h[V];
#pragma unroll
            for (int v = 0; v < V; ++v) h[v] = 0.f;
            if (q >= 0 && A.h0 && in) load_vec<V>(A.h0 + (int64_t)q * A.width + col, h);
#pragma unroll
            for (int v = 0; v < V; ++v) x[j][v] = q < 0 ? 0.f : step_of(a[j][SH ? 0 : v], h[v], x[j][v]);
#pragma unroll
            for (int d = 0; d < D; ++d) a[j][d] = 0.f;
        }
    }
};

}  // namespace lx

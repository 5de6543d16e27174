// Tokens sorted by expert and back (gfx950).
//
// Slot s = t K + k of token t asks for expert id[s].  A stable counting sort
// by id gives every kept slot its place among the rows ordered by expert:
//     place[s] = #{s' : id[s'] < id[s]} + #{s' < s : id[s'] = id[s]},
// order[place[s]] = s, offsets[e] = #{s' : id[s'] < e}.  It is the zero-
// temperature limit of the operator (equality of keys routes values) with
// whole numbers as keys.  Ids outside [0, E) are dropped slots: place -1, no
// row; order is -1 past the last row.  No atomics on global memory, so the
// result does not depend on the order in which workgroups run.
//
// Ranking: a workgroup takes a tile of consecutive slots, each wave a quarter
// of them in order, 64 at a time; lanes of one id find each other by ballots
// over the id's bits and count the lanes below, a counter per wave and id in
// LDS carries the rest.  Up to kRouteSingle slots one launch does everything
// (bound by its latency, 4 us, 11 with the host's part); above, tiles of
// kRouteTile slots are counted, their counts scanned along the tiles (E
// columns of `tiles` counts) and the slots placed, three launches.  A wave's
// rounds wait for each other's counters, so shorter tiles, more of them at a
// time, are faster: 2^20 slots, 256 experts, 28 us of kernels at 4096 slots a
// tile, 22 at 2048 (5 counting, 4 scanning, 12 placing), 26 at 1024 (the scan
// grows).  What is left is the placing's chain of counters and its scattered
// 4-byte writes.
//
// The data movement has one thread per token and 16 bytes of its row (at any
// address; the last thread of a row takes its last 16 bytes, some of them a
// second time), so a token's row is read (written) once and its K copies are
// in flight together:
//     dispatch      xs[place[t,k]] = x[t]
//     combine       y[t] = sum_k w[t,k] ys[place[t,k]]
//     combine_grad  dys[place[t,k]] = w[t,k] dy[t], dw[t,k] = <dy[t], ys[place[t,k]]>
// and is bound by memory.  Rows by expert are moved past the caches: an array
// of them is read or written once here, in scattered pieces, and filling the
// caches with it makes the next kernel wait for their write-back (dispatch
// and combine of 65536 rows of 4 KB: 61 + 92 us through the caches, 58 + 54
// past them; 8192 rows followed by a product that reads them all: 30.6 us,
// 23.2).  Sums are float32 in ascending k; a dropped slot's
// weight and row are never used, whatever they hold.
#include "lx_device.h"
#include "lx_internal.h"
#include "lx_types.h"

namespace lx {

namespace {

constexpr int kRouteThreads = 256;
constexpr int kRouteWaves = kRouteThreads / kWave;

__device__ __forceinline__ int route_id(const void* ids, int wide, int64_t s, int experts)
{
    const int64_t id = wide ? ((const int64_t*)ids)[s] : (int64_t)((const int32_t*)ids)[s];
    return id >= 0 && id < experts ? (int)id : -1;
}

// Counts of a tile: hist[tile][experts].
__global__ __launch_bounds__(kRouteThreads) void lx_route_count(RouteArgs A)
{
    extern __shared__ uint32_t s_cnt[];
    const int E = A.experts;
    for (int e = threadIdx.x; e < E; e += kRouteThreads) s_cnt[e] = 0;
    __syncthreads();
    const int64_t s0 = (int64_t)blockIdx.x * kRouteTile + threadIdx.x;
#pragma unroll
    for (int j = 0; j < kRouteTile / kRouteThreads; ++j) {
        const int64_t s = s0 + j * kRouteThreads;
        const int id = s < A.n ? route_id(A.ids, A.wide, s, E) : -1;
        if (id >= 0) atomicAdd(&s_cnt[id], 1u);
    }
    __syncthreads();
    uint32_t* h = A.hist + (int64_t)blockIdx.x * E;
    for (int e = threadIdx.x; e < E; e += kRouteThreads) h[e] = s_cnt[e];
}

// Exclusive scan of hist along the tiles, in place; total[e] the column sum.
// A workgroup has 16 columns by 64 runs of 8 tiles.
constexpr int kColThreads = 1024;
constexpr int kCols = 16;
constexpr int kRuns = kColThreads / kCols;
constexpr int kRunLen = 8;
__global__ __launch_bounds__(kColThreads) void lx_route_scan(RouteArgs A)
{
    __shared__ uint32_t s_run[kRuns][kCols];
    __shared__ uint32_t s_tot[kCols];
    const int E = A.experts;
    const int col = threadIdx.x % kCols, run = threadIdx.x / kCols;
    const int e = (int)blockIdx.x * kCols + col;
    uint32_t carry = 0;
    for (int64_t t0 = 0; t0 < A.tiles; t0 += kRuns * kRunLen) {
        uint32_t v[kRunLen], sum = 0;
#pragma unroll
        for (int i = 0; i < kRunLen; ++i) {
            const int64_t t = t0 + run * kRunLen + i;
            v[i] = t < A.tiles && e < E ? A.hist[t * E + e] : 0u;
            sum += v[i];
        }
        s_run[run][col] = sum;
        __syncthreads();
        if (threadIdx.x < kCols) {
            uint32_t acc = carry;
#pragma unroll 8
            for (int r = 0; r < kRuns; ++r) {
                const uint32_t c = s_run[r][threadIdx.x];
                s_run[r][threadIdx.x] = acc;
                acc += c;
            }
            s_tot[threadIdx.x] = acc;
        }
        __syncthreads();
        uint32_t acc = s_run[run][col];
        carry = s_tot[col];
#pragma unroll
        for (int i = 0; i < kRunLen; ++i) {
            const int64_t t = t0 + run * kRunLen + i;
            if (t < A.tiles && e < E) A.hist[t * E + e] = acc;
            acc += v[i];
        }
        __syncthreads();
    }
    if (run == 0 && e < E) A.total[e] = carry;
}

// Exclusive scan over the experts of s_base (counts in, first places out);
// thread i owns a run of `per` experts.  Returns the sum of all counts.
__device__ __forceinline__ uint32_t scan_experts(uint32_t* s_base, uint32_t* s_wave, int E)
{
    const int per = (E + kRouteThreads - 1) / kRouteThreads;
    const int e0 = (int)threadIdx.x * per;
    uint32_t sum = 0;
    for (int i = 0; i < per; ++i)
        if (e0 + i < E) sum += s_base[e0 + i];
    const int lane = lane_id(), w = (int)threadIdx.x / kWave;
    uint32_t inc = sum;
#pragma unroll
    for (int d = 1; d < kWave; d <<= 1) {
        const uint32_t o = (uint32_t)__shfl_up((int)inc, d);
        if (lane >= d) inc += o;
    }
    if (lane == kWave - 1) s_wave[w] = inc;
    __syncthreads();
    uint32_t before = inc - sum, all = 0;
#pragma unroll
    for (int i = 0; i < kRouteWaves; ++i) {
        if (i < w) before += s_wave[i];
        all += s_wave[i];
    }
    for (int i = 0; i < per; ++i) {
        if (e0 + i < E) {
            const uint32_t c = s_base[e0 + i];
            s_base[e0 + i] = before;
            before += c;
        }
    }
    __syncthreads();
    return all;
}

// Ranks a tile and writes place and order.  BITS: bits that tell the ids
// apart.  SINGLE: the only tile, whose counts are all there is.
// LDS: cnt[waves][E], base[E].
template <int BITS, bool SINGLE>
__global__ __launch_bounds__(kRouteThreads) void lx_route_place(RouteArgs A)
{
    constexpr int kTile = SINGLE ? kRouteSingle : kRouteTile;
    constexpr int kRounds = kTile / kRouteThreads;  // of 64 slots per wave
    extern __shared__ uint32_t s_dyn[];
    __shared__ uint32_t s_wave[kRouteWaves];
    const int E = A.experts;
    uint32_t* cnt = s_dyn;
    uint32_t* base = s_dyn + kRouteWaves * E;
    const int tid = threadIdx.x, lane = lane_id(), w = tid / kWave;
    const int64_t tile = blockIdx.x, tile0 = tile * kTile;
    const int64_t left = A.n - tile0;
    const int room = (int)(left < kTile ? left : kTile);  // slots of this tile
    const int w0 = w * (kTile / kRouteWaves);

    int id[kRounds];
#pragma unroll
    for (int j = 0; j < kRounds; ++j) {
        const int i = w0 + j * kWave + lane;
        id[j] = i < room ? route_id(A.ids, A.wide, tile0 + i, E) : -1;
    }
    for (int e = tid; e < kRouteWaves * E; e += kRouteThreads) cnt[e] = 0;
    if (!SINGLE)
        for (int e = tid; e < E; e += kRouteThreads) base[e] = A.total[e];
    __syncthreads();

    // rank within the wave's quarter, 64 slots at a time; one wave alone
    // touches its counters, in order
    uint32_t rank[kRounds];
    uint32_t* mine = cnt + w * E;
#pragma unroll
    for (int j = 0; j < kRounds; ++j) {
        rank[j] = 0;
        if (w0 + j * kWave < room) {
            const uint64_t kept = __ballot(id[j] >= 0);
            const uint64_t same = match_bits<BITS>((uint32_t)id[j]) & kept;
            if (id[j] >= 0) {
                const uint32_t below = count_below(same);
                const uint32_t old = mine[id[j]];
                rank[j] = old + below;
                if (below == 0) mine[id[j]] = old + (uint32_t)__popcll(same);
            }
            // the next round's lanes read what this round's first lanes wrote
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        }
    }
    __syncthreads();

    // counts per wave -> first rank of each wave within the tile
    for (int e = tid; e < E; e += kRouteThreads) {
        uint32_t acc = 0;
#pragma unroll
        for (int i = 0; i < kRouteWaves; ++i) {
            const uint32_t c = cnt[i * E + e];
            cnt[i * E + e] = acc;
            acc += c;
        }
        if (SINGLE) base[e] = acc;
    }
    __syncthreads();
    const uint32_t total = scan_experts(base, s_wave, E);
    if (tile == 0) {
        for (int e = tid; e < E; e += kRouteThreads) A.offsets[e] = (int32_t)base[e];
        if (tid == 0) A.offsets[E] = (int32_t)total;
    }
    if (!SINGLE) {
        __syncthreads();
        for (int e = tid; e < E; e += kRouteThreads) base[e] += A.hist[tile * E + e];
        __syncthreads();
    }
#pragma unroll
    for (int j = 0; j < kRounds; ++j) {
        const int i = w0 + j * kWave + lane;
        if (i < room) {
            int p = -1;
            if (id[j] >= 0) {
                p = (int)(base[id[j]] + cnt[w * E + id[j]] + rank[j]);
                A.order[p] = (int32_t)(tile0 + i);
            }
            A.place[tile0 + i] = p;
            if (tile0 + i >= (int64_t)total) A.order[tile0 + i] = -1;  // a row past the last kept slot
        }
    }
}

// Rows past the last kept slot, `kept` .. n - 1: at most K per token, row
// kept + t + i T for i = 0, 1, ... by token t's threads.
template <int V, class T>
__device__ __forceinline__ void zero_tail(const MoveArgs& A, T* rows, int64_t ld, int64_t kept, int64_t t)
{
    float z[V];
#pragma unroll
    for (int i = 0; i < V; ++i) z[i] = 0.f;
    for (int64_t r = (kept < 0 ? 0 : kept) + t; r < A.tokens * A.slots; r += A.tokens) store_vec<V>(rows + r * ld, z);
}

// First column of group i of V: the last one ends with the row.
template <int V>
__device__ __forceinline__ int64_t group_col(const MoveArgs& A, int i)
{
    const int64_t at = (int64_t)i * V;
    return at < A.width - V ? at : A.width - V;
}

// Token and first column of this thread: the flat index over
// [tokens][groups], divided in 64 bits once per workgroup and in 32 bits per
// thread.  False past the last token.
template <int V>
__device__ __forceinline__ bool token_group(const MoveArgs& A, int64_t* t, int64_t* at)
{
    const int64_t i0 = group_id<256>() * 256;
    const int64_t t0 = i0 / A.groups;
    const uint32_t rest = (uint32_t)(i0 - t0 * A.groups) + threadIdx.x;
    const uint32_t more = rest / (uint32_t)A.groups;
    *t = t0 + more;
    *at = group_col<V>(A, (int)(rest - more * (uint32_t)A.groups));
    return *t < A.tokens;
}

// Rows of KC slots of a token, from slot k0 on; -1 where there is none.
template <int KC>
__device__ __forceinline__ void slot_rows(const MoveArgs& A, int64_t t, int64_t k0, int (&row)[KC])
{
    const int64_t rows = A.tokens * A.slots;
    const int32_t* place = A.place + t * A.slots + k0;
#pragma unroll
    for (int k = 0; k < KC; ++k) {
        const int r = k0 + k < A.slots ? place[k] : -1;
        row[k] = r >= 0 && r < rows ? r : -1;
    }
}

// KC: slots whose rows are in flight together; more are done KC at a time.
template <int V, class T, int KC>
__global__ __launch_bounds__(256) void lx_dispatch(MoveArgs A)
{
    int64_t t, at;
    if (!token_group<V>(A, &t, &at)) return;
    const Pack<T, V> v = load_pack<V>((const T*)A.in + t * A.ld_in + at);
    const int64_t kept = A.offsets[A.experts];
    T* xs = (T*)A.out + at;
    for (int64_t k0 = 0; k0 < A.slots; k0 += KC) {
        int row[KC];
        slot_rows<KC>(A, t, k0, row);
#pragma unroll
        for (int k = 0; k < KC; ++k)
            if (row[k] >= 0) store_once<V>(xs + row[k] * A.ld_out, v);
    }
    zero_tail<V>(A, xs, A.ld_out, kept, t);
}

// 16384 tokens x 2 rows of 4096 bf16: 62 us, 6.5 TB/s.
template <int V, class T, int KC>
__global__ __launch_bounds__(256) void lx_combine(MoveArgs A)
{
    int64_t t, at;
    if (!token_group<V>(A, &t, &at)) return;
    const T* ys = (const T*)A.in + at;
    float acc[V];
#pragma unroll
    for (int q = 0; q < V; ++q) acc[q] = 0.f;
    for (int64_t k0 = 0; k0 < A.slots; k0 += KC) {
        int row[KC];
        float w[KC];
        Pack<T, V> v[KC];
        slot_rows<KC>(A, t, k0, row);
#pragma unroll
        for (int k = 0; k < KC; ++k) {
            const bool kept = row[k] >= 0;
            w[k] = A.weights && kept ? A.weights[t * A.slots + k0 + k] : 1.f;
            // a dropped slot reads row 0 and takes nothing from it
            v[k] = load_once<V>(ys + (kept ? row[k] : 0) * A.ld_in);
        }
#pragma unroll
        for (int k = 0; k < KC; ++k)
#pragma unroll
            for (int q = 0; q < V; ++q) acc[q] = row[k] >= 0 ? fmaf(w[k], (float)v[k].v[q], acc[q]) : acc[q];
    }
    store_vec<V>((T*)A.out + t * A.ld_out + at, acc);
}

// G threads of a 256-thread workgroup per token; the dot products of KC
// slots are carried along one pass over the row.  16384 tokens x 4 rows of
// 2048 bf16: 105 us, 5.7 TB/s.
template <int V, class T, int KC, int G>
__global__ __launch_bounds__(256) void lx_combine_grad(MoveArgs A)
{
    __shared__ float s_dot[256 / kWave][KC];
    const int part = (int)threadIdx.x % G;
    const int64_t t = group_id<256>() * (256 / G) + (int)threadIdx.x / G;
    const bool live = t < A.tokens;
    const int lane = lane_id(), w = (int)threadIdx.x / kWave;
    const T* dy = (const T*)A.dy + (live ? t : 0) * A.ld_dy;
    const T* ys = (const T*)A.in;
    T* dys = (T*)A.out;
    for (int64_t k0 = 0; k0 < A.slots; k0 += KC) {
        int row[KC];
        float weight[KC], dot[KC];
#pragma unroll
        for (int k = 0; k < KC; ++k) row[k] = -1;
        if (live) slot_rows<KC>(A, t, k0, row);
#pragma unroll
        for (int k = 0; k < KC; ++k) {
            weight[k] = row[k] >= 0 && A.weights ? A.weights[t * A.slots + k0 + k] : 0.f;
            dot[k] = 0.f;
        }
        if (live) {
            for (int col = part; col < A.groups; col += G) {
                const int64_t at = group_col<V>(A, col);
                const int again = (int)((int64_t)col * V - at);  // values that another thread has too
                Pack<T, V> v[KC];
                float d[V];
                load_vec<V>(dy + at, d);
                if (A.dw) {
#pragma unroll
                    for (int k = 0; k < KC; ++k)
                        v[k] = load_once<V>(ys + (row[k] >= 0 ? row[k] : 0) * A.ld_in + at);
                }
                if (dys) {
#pragma unroll
                    for (int k = 0; k < KC; ++k) {
                        if (row[k] < 0) continue;
                        float o[V];
#pragma unroll
                        for (int q = 0; q < V; ++q) o[q] = weight[k] * d[q];
                        store_vec_once<V>(dys + row[k] * A.ld_out + at, o);
                    }
                }
                if (A.dw) {
#pragma unroll
                    for (int k = 0; k < KC; ++k)
#pragma unroll
                        for (int q = 0; q < V; ++q)
                            dot[k] = row[k] >= 0 && q >= again ? fmaf(d[q], (float)v[k].v[q], dot[k]) : dot[k];
                }
            }
        }
        if (A.dw) {
#pragma unroll
            for (int k = 0; k < KC; ++k) {
#pragma unroll
                for (int m = 1; m < kWave; m <<= 1) dot[k] += __shfl_xor(dot[k], m);
            }
            if (G > kWave) {
                if (lane == 0) {
#pragma unroll
                    for (int k = 0; k < KC; ++k) s_dot[w][k] = dot[k];
                }
                __syncthreads();
                if ((int)threadIdx.x < KC && live && k0 + (int)threadIdx.x < A.slots) {
                    float sum = 0.f;
#pragma unroll
                    for (int i = 0; i < 256 / kWave; ++i) sum += s_dot[i][threadIdx.x];
                    A.dw[t * A.slots + k0 + threadIdx.x] = sum;
                }
                __syncthreads();
            } else if (lane == 0 && live) {
#pragma unroll
                for (int k = 0; k < KC; ++k)
                    if (k0 + k < A.slots) A.dw[t * A.slots + k0 + k] = dot[k];
            }
        }
    }
    if (dys && live) {
        const int64_t kept = A.offsets[A.experts];
        for (int col = part; col < A.groups; col += G) zero_tail<V>(A, dys + group_col<V>(A, col), A.ld_out, kept, t);
    }
}

template <int BITS>
hipError_t place_launch(const RouteArgs& a, hipStream_t s)
{
    const size_t lds = (size_t)(kRouteWaves + 1) * a.experts * 4;
    if (a.n <= kRouteSingle) {
        LX_LAUNCH("route", s, (lx_route_place<BITS, true><<<1, kRouteThreads, lds, s>>>(a)));
        return hipSuccess;
    }
    LX_LAUNCH("route_place", s, (lx_route_place<BITS, false><<<(unsigned)a.tiles, kRouteThreads, lds, s>>>(a)));
    return hipSuccess;
}

template <int V, class T, int KC>
hipError_t move_launch(MoveKind kind, MoveArgs a, hipStream_t s)
{
    a.groups = (int)((a.width + V - 1) / V);
    const int64_t blocks = (a.tokens * a.groups + 255) / 256;
    switch (kind) {
        case kMoveDispatch:
            LX_LAUNCH("dispatch", s, (lx_dispatch<V, T, KC><<<grid_of<256>(blocks), 256, 0, s>>>(a)));
            return hipSuccess;
        case kMoveCombine:
            LX_LAUNCH("combine", s, (lx_combine<V, T, KC><<<grid_of<256>(blocks), 256, 0, s>>>(a)));
            return hipSuccess;
        case kMoveCombineGrad:
            // A wave per token while a row is at most two loads per lane, a
            // workgroup above.  bf16, wave against workgroup, us by groups of
            // a row (64, 128, 192, 256): 16384 tokens x 4 rows 28/56, 51/64,
            // 80/81, 115/100; 2048 x 2 5.1/7.1, 6.6/8.5, 8.3/9.5, 10.1/10.3;
            // 64 x 8 5.8/5.5, 7.5/5.7, 9.1/5.9, 10.6/6.2.
            if (a.groups <= 2 * kWave)
                LX_LAUNCH("combine_grad", s,
                          (lx_combine_grad<V, T, KC, 64><<<grid_of<256>((a.tokens + 3) / 4), 256, 0, s>>>(a)));
            else
                LX_LAUNCH("combine_grad", s,
                          (lx_combine_grad<V, T, KC, 256><<<grid_of<256>(a.tokens), 256, 0, s>>>(a)));
            return hipSuccess;
    }
    return hipErrorInvalidValue;
}

template <int V, class T>
hipError_t move_slots(MoveKind kind, const MoveArgs& a, hipStream_t s)
{
    // the smallest chunk that holds the token's slots: rows in flight that
    // are not there cost registers
    return a.slots <= 2 ? move_launch<V, T, 2>(kind, a, s)
                        : a.slots <= 4 ? move_launch<V, T, 4>(kind, a, s) : move_launch<V, T, 8>(kind, a, s);
}

template <class T>
hipError_t move_type(MoveKind kind, const MoveArgs& a, hipStream_t s)
{
    constexpr int V = 16 / (int)sizeof(T);
    return a.width >= V ? move_slots<V, T>(kind, a, s) : move_slots<1, T>(kind, a, s);
}

}  // namespace

hipError_t route_launch(const RouteArgs& a, hipStream_t s)
{
    if (a.n > kRouteSingle) {
        LX_LAUNCH("route_count", s,
                  (lx_route_count<<<(unsigned)a.tiles, kRouteThreads, (size_t)a.experts * 4, s>>>(a)));
        LX_LAUNCH("route_scan", s, (lx_route_scan<<<(unsigned)((a.experts + kCols - 1) / kCols), kColThreads, 0, s>>>(a)));
    }
    return a.experts <= 16 ? place_launch<4>(a, s) : a.experts <= 256 ? place_launch<8>(a, s) : place_launch<12>(a, s);
}

hipError_t move_rows_launch(MoveKind kind, int dtype, const MoveArgs& a, hipStream_t s)
{
    if (a.tokens <= 0) return hipSuccess;
    switch (dtype) {
        case 0: return move_type<float>(kind, a, s);
        case 1: return move_type<bf16_t>(kind, a, s);
        case 2: return move_type<f16_t>(kind, a, s);
        default: return hipErrorInvalidValue;
    }
}

}  // namespace lx

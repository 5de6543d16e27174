// Gated linear recurrence over packed sequences (gfx950): see lx_recur.h for
// the mathematics, the tile layout and how tiles hand their states on.
//
// One pass: x and g are read once and y is written once, bound by memory.
// 65536 x 2048 bf16 with a decay per channel: 148 us, 5.4 TB/s (three passes,
// tile maps, carries, rows: 289 the call); packed 32768 x 4096 bf16 with a decay
// per 64 channels: 119 us, 4.6 TB/s.  Few tiles are bound by a tile's latency, some
// 10 us: load, compose, hand over, write.
#include "lx_recur.h"

namespace lx {

namespace {

// Rows of y (and final states) of one thread from the state entering it.
template <int CARE, class Th, class T, int V>
__device__ __forceinline__ void write_rows(const RecurArgs& A, const RecurRows* R, const Th& th, float (&h)[V])
{
    const RowAt<T, V> y = th.template at<T, V>(A.y, A.ldy);
#pragma unroll
    for (int j = 0; j < Th::L; ++j) {
        float a[Th::D];
        const bool cut = th.template decays<CARE>(R, j, a);
        th.template step<CARE>(A, R, j, a, cut, h);
        if (care_rows(CARE) ? j < th.rows : th.in) store_vec_as<V>(y.row(j), h, A.stream);
        if (th.template special<CARE>(j) && A.final && th.in) {
            const int q = R->last[th.r0 + j];
            if (q >= 0) store_vec<V>(A.final + (int64_t)q * A.width + th.col(), h);
        }
    }
}

template <class T, class TG, int V, int L, bool SH>
__global__ __launch_bounds__((RecurLayout<V, L>::kThreads)) void lx_recur_pass(RecurArgs A)
{
    using Th = RecurThread<T, TG, V, L, SH>;
    using Lay = RecurLayout<V, L>;
    __shared__ RecurRows rows;
    __shared__ RecurGroups<V, L, SH> groups;
    __shared__ float sh[Lay::kGroups][kRecurCols];
    const int ct = channel_tile(A, (uint32_t)group_id<Lay::kThreads>());
    const int64_t tile = next_tile(A, ct);
    if (past_tiles(A, tile)) return;
    const int mark = tile_mark(A, tile);
    Th th;
    th.load(A, tile, ct);
    const RecurRows* R = uniform(recur_rows<Lay::kThreads>(A, tile * kRecurTile, mark, rows)) ? &rows : nullptr;
    float r[Th::D], h[V];
    int care = th.find_odd(A, R);
#pragma unroll
    for (int d = 0; d < Th::D; ++d) r[d] = 0.f;
#pragma unroll
    for (int v = 0; v < V; ++v) h[v] = 0.f;
    // kCareBoth is rare: its code lies behind the others'
    if (care == kCareNone) {
        if (!th.template compose<kCareNone>(A, R, r, h)) care = kCareRoot;
    } else if (care == kCareRows) {
        if (!th.template compose<kCareRows>(A, R, r, h)) care = kCareBoth;
    }
    if (care == kCareRoot) th.template compose<kCareRoot>(A, R, r, h);
    if (__builtin_expect(care == kCareBoth, 0)) th.template compose<kCareBoth>(A, R, r, h);
    groups.put(th.group, th.lane, care, r);
#pragma unroll
    for (int v = 0; v < V; ++v) sh[th.group][th.lane * V + v] = h[v];
    __syncthreads();
    if (threadIdx.x < kRecurCols) {
        const uint32_t waves = groups.rooted();
        float e = 0.f;
        if (A.tiles > 1) {
            float ah;
            const float ar = groups.template compose<false>(waves, sh, ah);
            e = pass_state(A, tile, ct, ar, ah, R && R->start[0] != -1, tile == A.tiles - 1);
        }
        groups.template enter<false>(waves, sh, e);
    }
    __syncthreads();
#pragma unroll
    for (int v = 0; v < V; ++v) h[v] = sh[th.group][th.lane * V + v];
    if (care == kCareNone) write_rows<kCareNone, Th, T>(A, R, th, h);
    else if (care == kCareRoot) write_rows<kCareRoot, Th, T>(A, R, th, h);
    else if (care == kCareRows) write_rows<kCareRows, Th, T>(A, R, th, h);
    else if (__builtin_expect(care == kCareBoth, 0)) write_rows<kCareBoth, Th, T>(A, R, th, h);
}

// Blocks [0, fill): 16 bytes of all ones per thread over the published
// words, the tickets and the marks; the rest: a sequence each, in turn.
__global__ __launch_bounds__(256) void lx_recur_begin(RecurArgs A, int64_t maps16, int64_t states16, unsigned fill,
                                                      const float* __restrict__ from, float* __restrict__ to)
{
    if (blockIdx.x < fill) {
        const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
        const uint4 ones = make_uint4(~0u, ~0u, ~0u, ~0u);
        if (i < maps16) reinterpret_cast<uint4*>(A.maps)[i] = ones;
        else if (i - maps16 < states16) reinterpret_cast<uint4*>(A.states)[i - maps16] = ones;
        if (i < A.cols) A.tickets[i * kRecurTicketPitch] = 0;
        if (A.offsets && i < A.tiles) {
            const int64_t t0 = i * kRecurTile, end = t0 + kRecurTile;
            int64_t lo = 0, hi = A.seqs + 1;  // the first offset at or past t0
            while (lo < hi) {
                const int64_t mid = (lo + hi) / 2;
                if ((int64_t)A.offsets[mid] < t0) lo = mid + 1;
                else hi = mid;
            }
            const bool plain = end <= A.n && lo > 0 && lo <= A.seqs && (int64_t)A.offsets[lo] > end;
            A.marks[i] = plain ? -1 : (int)lo;
        }
        return;
    }
    for (int64_t q = blockIdx.x - fill; q < A.seqs; q += gridDim.x - fill) {
        if (A.offsets && A.offsets[q + 1] > A.offsets[q]) continue;
        for (int c = threadIdx.x; c < A.width; c += 256) to[q * A.width + c] = from ? from[q * A.width + c] : 0.f;
    }
}

template <class T, class TG, int V, int L, bool SH>
hipError_t recur_go(const RecurArgs& a, hipStream_t s)
{
    LX_LAUNCH("recur", s,
              (lx_recur_pass<T, TG, V, L, SH>
               <<<grid_of<RecurLayout<V, L>::kThreads>(a.tiles * a.cols), RecurLayout<V, L>::kThreads, 0, s>>>(a)));
    return hipSuccess;
}

template <class T, class TG>
hipError_t recur_type(const RecurArgs& a, hipStream_t s)
{
    const bool sh = a.per > 1;
    const bool wide = recur_wide(a);
    if (wide && recur_few(a)) return sh ? recur_go<T, TG, 4, 4, true>(a, s) : recur_go<T, TG, 4, 4, false>(a, s);
    if (wide) return sh ? recur_go<T, TG, 4, 16, true>(a, s) : recur_go<T, TG, 4, 16, false>(a, s);
    return recur_go<T, TG, 1, 16, true>(a, s);
}

// Bound by its launch: 256 requests of 4096 channels move 13 MB in 4.2 us.
// One token for each request: state[slot] = e^g state[slot] + x, y = the new state.
template <class T, class TG, int V>
__global__ __launch_bounds__(256) void lx_recur_step(RecurStepArgs A)
{
    const int64_t i0 = group_id<256>() * 256;
    const int64_t b0 = i0 / A.groups;
    const uint32_t rest = (uint32_t)(i0 - b0 * A.groups) + threadIdx.x;
    const uint32_t more = rest / (uint32_t)A.groups;
    const int64_t b = b0 + more;
    if (b >= A.n) return;
    const int col = (int)(rest - more * (uint32_t)A.groups) * V;
    const int64_t slot = A.slots ? (int64_t)A.slots[b] : b;
    float h[V];
#pragma unroll
    for (int v = 0; v < V; ++v) h[v] = 0.f;
    if (slot >= 0 && slot < A.pool) {
        float* st = A.state + slot * A.width + col;
        float x[V], a[V];
        load_vec<V>(st, h);
        load_vec<V>((const T*)A.x + b * A.ldx + col, x);
        const TG* g = (const TG*)A.g + b * A.ldg;
        if (A.per == 1) {
            load_vec<V>(g + col, a);
        } else {
            const float one = (float)g[col / A.per];
#pragma unroll
            for (int v = 0; v < V; ++v) a[v] = one;
        }
#pragma unroll
        for (int v = 0; v < V; ++v) h[v] = step_of(root_of(a[v]), h[v], x[v]);
        store_vec<V>(st, h);
    }
    store_vec<V>((T*)A.y + b * A.ldy + col, h);
}

template <class T, class TG>
hipError_t step_type(RecurStepArgs a, hipStream_t s)
{
    // no two threads may share a channel here: each steps its state once
    const bool wide = a.width % 4 == 0 && (a.per == 1 || a.per % 4 == 0);
    const int v = wide ? 4 : 1;
    a.groups = a.width / v;
    const int64_t blocks = (a.n * a.groups + 255) / 256;
    if (wide)
        LX_LAUNCH("recur_step", s, (lx_recur_step<T, TG, 4><<<grid_of<256>(blocks), 256, 0, s>>>(a)));
    else
        LX_LAUNCH("recur_step", s, (lx_recur_step<T, TG, 1><<<grid_of<256>(blocks), 256, 0, s>>>(a)));
    return hipSuccess;
}

}  // namespace

hipError_t recur_begin(const RecurArgs& a, const float* from, float* to, hipStream_t s)
{
    const int64_t words = a.tiles > 1 ? (a.tiles - 1) * a.cols * kRecurCols : 0;
    const int64_t maps16 = words / 2, states16 = words / 4;
    const unsigned fill = (unsigned)((maps16 + states16 + 255) / 256);
    // n * width <= 2^38 keeps both together below 2^23 workgroups
    const unsigned each = to && (a.offsets || a.n == 0) ? (unsigned)(a.seqs < 65536 ? a.seqs : 65536) : 0;
    if (fill + each > 0)
        LX_LAUNCH("recur_begin", s, (lx_recur_begin<<<fill + each, 256, 0, s>>>(a, maps16, states16, fill, from, to)));
    return hipSuccess;
}

#define LX_BY_TYPE(call, a)                                                           \
    switch (dtype) {                                                                  \
        case 0: return call<float, float>(a, s);                                      \
        case 1: return gtype ? call<bf16_t, bf16_t>(a, s) : call<bf16_t, float>(a, s); \
        case 2: return gtype ? call<f16_t, f16_t>(a, s) : call<f16_t, float>(a, s);    \
        default: return hipErrorInvalidValue;                                         \
    }

hipError_t recur_launch(const RecurArgs& a, int dtype, int gtype, hipStream_t s)
{
    const hipError_t e = recur_begin(a, a.h0, a.final, s);
    if (e != hipSuccess || a.n == 0) return e;
    LX_BY_TYPE(recur_type, a)
}

hipError_t recur_step_launch(const RecurStepArgs& a, int dtype, int gtype, hipStream_t s)
{
    LX_BY_TYPE(step_type, a)
}

}  // namespace lx

// Gated linear recurrence over packed sequences (gfx950): see lx_recur.h for
// the mathematics and the tile layout.
//
// Reduce-then-scan: every tile's composed map, then the states between tiles
// (one thread per channel), then every tile's rows from its entering state.
// No workgroup waits for another and the combine order is fixed, so results
// repeat bit for bit.
#include "lx_recur.h"

namespace lx {

namespace {

// Composes the row groups of a tile.  In: this thread's map, h -> A h + H
// over its rows.  LDS: sa[groups][kRecurCols / V * D], sh[groups][kRecurCols].
template <class T, class TG, int V, bool SH>
__global__ __launch_bounds__(kRecurThreads) void lx_recur_reduce(RecurArgs A)
{
    using Th = RecurThread<T, TG, V, SH>;
    using Lay = RecurLayout<V>;
    __shared__ RecurRows R;
    __shared__ float sa[Lay::kGroups][Lay::kLanes * Th::D];
    __shared__ float sh[Lay::kGroups][kRecurCols];
    const int64_t tile = blockIdx.x / (unsigned)A.cols;
    const int ct = (int)(blockIdx.x % (unsigned)A.cols);
    Th th;
    th.load(A, tile, ct);
    recur_rows(A, tile * kRecurTile, R);
    th.decays();
    if (R.any) th.special(A, R);
    float m[Th::D], h[V];
#pragma unroll
    for (int d = 0; d < Th::D; ++d) m[d] = 1.f;
#pragma unroll
    for (int v = 0; v < V; ++v) h[v] = 0.f;
#pragma unroll
    for (int j = 0; j < Th::L; ++j) {
#pragma unroll
        for (int v = 0; v < V; ++v) h[v] = step_of(th.a[j][SH ? 0 : v], h[v], th.x[j][v]);
#pragma unroll
        for (int d = 0; d < Th::D; ++d) m[d] *= th.a[j][d];
    }
#pragma unroll
    for (int d = 0; d < Th::D; ++d) sa[th.group][th.lane * Th::D + d] = m[d];
#pragma unroll
    for (int v = 0; v < V; ++v) sh[th.group][th.lane * V + v] = h[v];
    __syncthreads();
    if (threadIdx.x < kRecurCols) {
        const int c = threadIdx.x;
        float am = 1.f, ah = 0.f;
#pragma unroll
        for (int i = 0; i < Lay::kGroups; ++i) {
            const float a = sa[i][SH ? c / V : c];
            ah = step_of(a, ah, sh[i][c]);
            am *= a;
        }
        A.maps[(tile * A.cols + ct) * kRecurCols + c] = make_float2(am, ah);
    }
}

// states[t] = state after tile t (in the order of the pass): one thread per channel.
__global__ __launch_bounds__(kRecurCols) void lx_recur_carry(RecurArgs A)
{
    const int64_t ld = (int64_t)A.cols * kRecurCols;
    const int64_t c = (int64_t)blockIdx.x * kRecurCols + threadIdx.x;
    float h = 0.f;
    int64_t t = 0;
    constexpr int U = 16;
    for (; t + U < A.tiles; t += U) {
        float2 m[U];
#pragma unroll
        for (int i = 0; i < U; ++i) m[i] = A.maps[(t + i) * ld + c];
#pragma unroll
        for (int i = 0; i < U; ++i) {
            h = step_of(m[i].x, h, m[i].y);
            A.states[(t + i) * ld + c] = h;
        }
    }
    for (; t < A.tiles - 1; ++t) {
        const float2 m = A.maps[t * ld + c];
        h = step_of(m.x, h, m.y);
        A.states[t * ld + c] = h;
    }
}

template <class T, class TG, int V, bool SH>
__global__ __launch_bounds__(kRecurThreads) void lx_recur_apply(RecurArgs A)
{
    using Th = RecurThread<T, TG, V, SH>;
    using Lay = RecurLayout<V>;
    __shared__ RecurRows R;
    __shared__ float sa[Lay::kGroups][Lay::kLanes * Th::D];
    __shared__ float sh[Lay::kGroups][kRecurCols];
    const int64_t tile = blockIdx.x / (unsigned)A.cols;
    const int ct = (int)(blockIdx.x % (unsigned)A.cols);
    Th th;
    th.load(A, tile, ct);
    recur_rows(A, tile * kRecurTile, R);
    th.decays();
    if (R.any) th.special(A, R);
    float m[Th::D], h[V];
#pragma unroll
    for (int d = 0; d < Th::D; ++d) m[d] = 1.f;
#pragma unroll
    for (int v = 0; v < V; ++v) h[v] = 0.f;
#pragma unroll
    for (int j = 0; j < Th::L; ++j) {
#pragma unroll
        for (int v = 0; v < V; ++v) h[v] = step_of(th.a[j][SH ? 0 : v], h[v], th.x[j][v]);
#pragma unroll
        for (int d = 0; d < Th::D; ++d) m[d] *= th.a[j][d];
    }
#pragma unroll
    for (int d = 0; d < Th::D; ++d) sa[th.group][th.lane * Th::D + d] = m[d];
#pragma unroll
    for (int v = 0; v < V; ++v) sh[th.group][th.lane * V + v] = h[v];
    __syncthreads();
    if (threadIdx.x < kRecurCols) {
        const int c = threadIdx.x;
        float e = tile > 0 ? A.states[((tile - 1) * A.cols + ct) * kRecurCols + c] : 0.f;
#pragma unroll
        for (int i = 0; i < Lay::kGroups; ++i) {
            const float next = step_of(sa[i][SH ? c / V : c], e, sh[i][c]);
            sh[i][c] = e;  // state entering group i
            e = next;
        }
    }
    __syncthreads();
#pragma unroll
    for (int v = 0; v < V; ++v) h[v] = sh[th.group][th.lane * V + v];
#pragma unroll
    for (int j = 0; j < Th::L; ++j) {
#pragma unroll
        for (int v = 0; v < V; ++v) th.x[j][v] = h[v] = step_of(th.a[j][SH ? 0 : v], h[v], th.x[j][v]);
    }
    store_rows<V, Th::L, T>(A.y, A.ldy, th.row0, A.n, th.col, th.in, th.x);
    if (R.any && A.final && th.in) {
#pragma unroll
        for (int j = 0; j < Th::L; ++j) {
            const int q = R.last[th.r0 + j];
            if (q >= 0) store_vec<V>(A.final + (int64_t)q * A.width + th.col, th.x[j]);
        }
    }
}

__global__ __launch_bounds__(256) void lx_recur_empty(RecurArgs A, const float* __restrict__ from, float* __restrict__ to)
{
    const int64_t q = blockIdx.x;
    if (A.offsets && A.offsets[q + 1] > A.offsets[q]) return;
    for (int c = threadIdx.x; c < A.width; c += 256) to[q * A.width + c] = from ? from[q * A.width + c] : 0.f;
}

template <class T, class TG, int V, bool SH>
hipError_t recur_go(const RecurArgs& a, hipStream_t s)
{
    const unsigned blocks = (unsigned)(a.tiles * a.cols);
    if (a.tiles > 1) {
        const unsigned part = (unsigned)((a.tiles - 1) * a.cols);
        LX_LAUNCH("recur_reduce", s, (lx_recur_reduce<T, TG, V, SH><<<part, kRecurThreads, 0, s>>>(a)));
        LX_LAUNCH("recur_carry", s, (lx_recur_carry<<<(unsigned)a.cols, kRecurCols, 0, s>>>(a)));
    }
    LX_LAUNCH("recur", s, (lx_recur_apply<T, TG, V, SH><<<blocks, kRecurThreads, 0, s>>>(a)));
    return hipSuccess;
}

template <class T, class TG>
hipError_t recur_type(const RecurArgs& a, hipStream_t s)
{
    const bool sh = a.per > 1;
    // four channels at a time where rows are aligned for it and a decay
    // serves one channel or whole groups of four
    const bool wide = vec_ok(a.x, a.ldx, a.width, sizeof(T), 4) && vec_ok(a.y, a.ldy, a.width, sizeof(T), 4) &&
                      vec_ok(a.h0, a.width, a.width, 4, 4) && vec_ok(a.final, a.width, a.width, 4, 4) &&
                      (sh ? a.per % 4 == 0 : vec_ok(a.g, a.ldg, a.width, sizeof(TG), 4));
    if (wide) return sh ? recur_go<T, TG, 4, true>(a, s) : recur_go<T, TG, 4, false>(a, s);
    return recur_go<T, TG, 1, true>(a, s);
}

// One token for each request: state[slot] = e^g state[slot] + x, y = the new state.
template <class T, class TG, int V>
__global__ __launch_bounds__(256) void lx_recur_step(RecurStepArgs A)
{
    const int64_t i0 = (int64_t)blockIdx.x * 256;
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
        for (int v = 0; v < V; ++v) {
            const float d = decay_of(a[v]);
            h[v] = d == 0.f ? x[v] : fmaf(d, h[v], x[v]);
        }
        store_vec<V>(st, h);
    }
    store_vec<V>((T*)A.y + b * A.ldy + col, h);
}

template <class T, class TG>
hipError_t step_type(RecurStepArgs a, hipStream_t s)
{
    const bool wide = vec_ok(a.x, a.ldx, a.width, sizeof(T), 4) && vec_ok(a.y, a.ldy, a.width, sizeof(T), 4) &&
                      vec_ok(a.state, a.width, a.width, 4, 4) &&
                      (a.per > 1 ? a.per % 4 == 0 : vec_ok(a.g, a.ldg, a.width, sizeof(TG), 4));
    const int v = wide ? 4 : 1;
    a.groups = a.width / v;
    const int64_t blocks = (a.n * a.groups + 255) / 256;
    if (blocks > 0x7FFFFFFFll) return hipErrorInvalidValue;
    if (wide)
        LX_LAUNCH("recur_step", s, (lx_recur_step<T, TG, 4><<<(unsigned)blocks, 256, 0, s>>>(a)));
    else
        LX_LAUNCH("recur_step", s, (lx_recur_step<T, TG, 1><<<(unsigned)blocks, 256, 0, s>>>(a)));
    return hipSuccess;
}

}  // namespace

hipError_t recur_carry_launch(const RecurArgs& a, hipStream_t s)
{
    LX_LAUNCH("recur_carry", s, (lx_recur_carry<<<(unsigned)a.cols, kRecurCols, 0, s>>>(a)));
    return hipSuccess;
}

hipError_t recur_empty_launch(const RecurArgs& a, const float* from, float* to, hipStream_t s)
{
    LX_LAUNCH("recur_empty", s, (lx_recur_empty<<<(unsigned)a.seqs, 256, 0, s>>>(a, from, to)));
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
    LX_BY_TYPE(recur_type, a)
}

hipError_t recur_step_launch(const RecurStepArgs& a, int dtype, int gtype, hipStream_t s)
{
    LX_BY_TYPE(step_type, a)
}

}  // namespace lx

// Backward pass of the gated recurrence (gfx950).
//
// With u_t = dL/dh_t and w_t the gradient that reaches h_{t-1},
//     u_t = dy_t + w_{t+1},   w_t = a_t u_t,
//     dx_t = u_t,   dg_t = w_t h_{t-1},   dh0 = w of the first row,
// where w past the last row of a sequence is dfinal: the same kind of scan,
// towards earlier rows, with the decay of the row itself.  dg of a decay that
// serves several channels is the sum over them.  The states h_{t-1} are made
// again in float32 from x and the saved state between row tiles (1/128 of
// x's values), which reads no more than a saved y would and loses nothing to
// y's rounding.  Where a_t is 0 the state was forgotten and w_t and dg_t are 0.
#include "lx_recur.h"

namespace lx {

hipError_t recur_carry_launch(const RecurArgs& a, hipStream_t s);

namespace {

// dy plus dfinal on last rows; 0 on rows of no sequence.
template <class Th, int V>
__device__ __forceinline__ void special_dy(const RecurArgs& A, const RecurRows& R, const Th& th, float (&dy)[Th::L][V])
{
#pragma unroll
    for (int j = 0; j < Th::L; ++j) {
        if (R.start[th.r0 + j] == -2) {
#pragma unroll
            for (int v = 0; v < V; ++v) dy[j][v] = 0.f;
        }
        const int q = R.last[th.r0 + j];
        if (q >= 0 && A.dfinal && th.in) {
            float d[V];
            load_vec<V>(A.dfinal + (int64_t)q * A.width + th.col, d);
#pragma unroll
            for (int v = 0; v < V; ++v) dy[j][v] += d[v];
        }
    }
}

// The first row of a sequence passes nothing to the row before it; rows
// of no sequence have no decay.
template <class T, class TG, int V, bool SH>
__global__ __launch_bounds__(kRecurThreads) void lx_recur_grad_reduce(RecurArgs A)
{
    using Th = RecurThread<T, TG, V, SH>;
    using Lay = RecurLayout<V>;
    __shared__ RecurRows R;
    __shared__ float sa[Lay::kGroups][Lay::kLanes * Th::D];
    __shared__ float sw[Lay::kGroups][kRecurCols];
    const int64_t back = blockIdx.x / (unsigned)A.cols;  // tiles before this one in the pass
    const int64_t tile = A.tiles - 1 - back;
    const int ct = (int)(blockIdx.x % (unsigned)A.cols);
    Th th;
    th.load(A, tile, ct);
    load_rows<V, Th::L, T>(A.dy, A.lddy, th.row0, A.n, th.col, th.in, th.x);
    recur_rows(A, tile * kRecurTile, R);
    th.decays();
    if (R.any) {
        special_dy<Th, V>(A, R, th, th.x);
#pragma unroll
        for (int j = 0; j < Th::L; ++j)
            if (R.start[th.r0 + j] != -1)
#pragma unroll
                for (int d = 0; d < Th::D; ++d) th.a[j][d] = 0.f;
    }
    float m[Th::D], w[V];
#pragma unroll
    for (int d = 0; d < Th::D; ++d) m[d] = 1.f;
#pragma unroll
    for (int v = 0; v < V; ++v) w[v] = 0.f;
#pragma unroll
    for (int j = Th::L - 1; j >= 0; --j) {
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const float a = th.a[j][SH ? 0 : v];
            w[v] = a == 0.f ? 0.f : a * (th.x[j][v] + w[v]);
        }
#pragma unroll
        for (int d = 0; d < Th::D; ++d) m[d] *= th.a[j][d];
    }
#pragma unroll
    for (int d = 0; d < Th::D; ++d) sa[th.group][th.lane * Th::D + d] = m[d];
#pragma unroll
    for (int v = 0; v < V; ++v) sw[th.group][th.lane * V + v] = w[v];
    __syncthreads();
    if (threadIdx.x < kRecurCols) {
        const int c = threadIdx.x;
        float am = 1.f, aw = 0.f;
#pragma unroll
        for (int i = Lay::kGroups - 1; i >= 0; --i) {
            const float a = sa[i][SH ? c / V : c];
            aw = step_of(a, aw, sw[i][c]);
            am *= a;
        }
        A.maps[(back * A.cols + ct) * kRecurCols + c] = make_float2(am, aw);
    }
}

template <class T, class TG, int V, bool SH>
__global__ __launch_bounds__(kRecurThreads) void lx_recur_grad_apply(RecurArgs A)
{
    using Th = RecurThread<T, TG, V, SH>;
    using Lay = RecurLayout<V>;
    constexpr int L = Th::L;
    __shared__ RecurRows R;
    __shared__ float sa[Lay::kGroups][Lay::kLanes * Th::D];
    __shared__ float sh[Lay::kGroups][kRecurCols];
    __shared__ float sw[Lay::kGroups][kRecurCols];
    const int64_t back = blockIdx.x / (unsigned)A.cols;
    const int64_t tile = A.tiles - 1 - back;
    const int ct = (int)(blockIdx.x % (unsigned)A.cols);
    Th th;
    float dy[L][V];
    th.load(A, tile, ct);
    load_rows<V, L, T>(A.dy, A.lddy, th.row0, A.n, th.col, th.in, dy);
    recur_rows(A, tile * kRecurTile, R);
    th.decays();
    if (R.any) {
        special_dy<Th, V>(A, R, th, dy);
        th.special(A, R);
    }
    float m[Th::D], h[V], w[V];
#pragma unroll
    for (int d = 0; d < Th::D; ++d) m[d] = 1.f;
#pragma unroll
    for (int v = 0; v < V; ++v) h[v] = w[v] = 0.f;
#pragma unroll
    for (int j = 0; j < L; ++j) {
#pragma unroll
        for (int v = 0; v < V; ++v) h[v] = step_of(th.a[j][SH ? 0 : v], h[v], th.x[j][v]);
#pragma unroll
        for (int d = 0; d < Th::D; ++d) m[d] *= th.a[j][d];
    }
#pragma unroll
    for (int j = L - 1; j >= 0; --j)
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const float a = th.a[j][SH ? 0 : v];
            w[v] = a == 0.f ? 0.f : a * (dy[j][v] + w[v]);
        }
#pragma unroll
    for (int d = 0; d < Th::D; ++d) sa[th.group][th.lane * Th::D + d] = m[d];
#pragma unroll
    for (int v = 0; v < V; ++v) {
        sh[th.group][th.lane * V + v] = h[v];
        sw[th.group][th.lane * V + v] = w[v];
    }
    __syncthreads();
    if (threadIdx.x < kRecurCols) {
        const int c = threadIdx.x;
        float e = tile > 0 ? A.states_in[((tile - 1) * A.cols + ct) * kRecurCols + c] : 0.f;
#pragma unroll
        for (int i = 0; i < Lay::kGroups; ++i) {
            const float next = step_of(sa[i][SH ? c / V : c], e, sh[i][c]);
            sh[i][c] = e;  // state entering group i
            e = next;
        }
        float b = back > 0 ? A.states[((back - 1) * A.cols + ct) * kRecurCols + c] : 0.f;
#pragma unroll
        for (int i = Lay::kGroups - 1; i >= 0; --i) {
            const float next = step_of(sa[i][SH ? c / V : c], b, sw[i][c]);
            sw[i][c] = b;  // gradient entering group i from the rows after it
            b = next;
        }
    }
    __syncthreads();
#pragma unroll
    for (int v = 0; v < V; ++v) {
        h[v] = sh[th.group][th.lane * V + v];
        w[v] = sw[th.group][th.lane * V + v];
    }
    // x[j] becomes the state before row j
#pragma unroll
    for (int j = 0; j < L; ++j)
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const float before = h[v];
            h[v] = step_of(th.a[j][SH ? 0 : v], h[v], th.x[j][v]);
            th.x[j][v] = before;
        }
    // dy[j] becomes u = dx, x[j] the products w h of dg
#pragma unroll
    for (int j = L - 1; j >= 0; --j) {
        const int q = R.any ? R.start[th.r0 + j] : -1;
        if (q >= 0) {
            // the decay of a first row acts on h0 alone
            float g[Th::D], h0[V];
#pragma unroll
            for (int d = 0; d < Th::D; ++d) g[d] = 0.f;
#pragma unroll
            for (int v = 0; v < V; ++v) h0[v] = 0.f;
            if (th.in)
                load_vec<Th::D>((const TG*)A.g + (th.row0 + j) * A.ldg + (SH ? th.col / A.per : th.col), g);
            if (A.h0 && th.in) load_vec<V>(A.h0 + (int64_t)q * A.width + th.col, h0);
            float out[V];
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const float a = decay_of(g[SH ? 0 : v]);
                const float u = dy[j][v] + w[v];
                out[v] = a == 0.f ? 0.f : a * u;
                dy[j][v] = u;
                th.x[j][v] = a == 0.f ? 0.f : out[v] * h0[v];
                w[v] = 0.f;
            }
            if (A.dh0 && th.in) store_vec<V>(A.dh0 + (int64_t)q * A.width + th.col, out);
        } else {
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const float a = th.a[j][SH ? 0 : v];
                const float u = dy[j][v] + w[v];
                w[v] = a == 0.f ? 0.f : a * u;
                dy[j][v] = u;
                th.x[j][v] = a == 0.f ? 0.f : w[v] * th.x[j][v];
            }
        }
    }
    if (A.dx) store_rows<V, L, T>(A.dx, A.lddx, th.row0, A.n, th.col, th.in, dy);
    if (!A.dg) return;
    if (!SH || A.per == 1) {
        store_rows<V, L, TG>(A.dg, A.lddg, th.row0, A.n, th.col, th.in, th.x);
        return;
    }
    // sum over the channels of each decay within this tile: the lanes of a
    // row that share one are neighbours; the first of them gets the sum
    const int head = th.in ? (int)(th.col / A.per) : -1;
    const bool first = th.in && (th.lane == 0 || (int)((th.col - V) / A.per) != head);
    const bool inside = recur_heads_inside(A.width, A.per);
#pragma unroll
    for (int j = 0; j < L; ++j) {
        float sum = 0.f;
#pragma unroll
        for (int v = 0; v < V; ++v) sum += th.x[j][v];
#pragma unroll
        for (int d = 1; d < Lay::kLanes; d <<= 1) {
            const float o = __shfl_down(sum, d, Lay::kLanes);
            const int oh = __shfl_down(head, d, Lay::kLanes);
            if (th.lane + d < Lay::kLanes && oh == head) sum += o;
        }
        const int64_t row = th.row0 + j;
        if (first && row < A.n) {
            if (inside)
                ((TG*)A.dg)[row * A.lddg + head] = (TG)sum;
            else
                A.part[row * (A.cols + A.heads) + ct + head] = sum;
        }
    }
}

// Sums of decays whose channels span several channel tiles: a tile and a
// decay that meet have slot tile + decay of the row's partial sums, which
// no other pair of that row has.
template <class TG>
__global__ __launch_bounds__(256) void lx_recur_grad_heads(RecurArgs A)
{
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    const int64_t row = i / A.heads;
    if (row >= A.n) return;
    const int head = (int)(i - row * A.heads);
    const int first = (int)((int64_t)head * A.per / kRecurCols);
    const int last = (int)(((int64_t)(head + 1) * A.per - 1) / kRecurCols);
    const float* p = A.part + row * (A.cols + A.heads) + head;
    float sum = 0.f;
    for (int c = first; c <= last; ++c) sum += p[c];
    ((TG*)A.dg)[row * A.lddg + head] = (TG)sum;
}

template <class T, class TG, int V, bool SH>
hipError_t grad_go(const RecurArgs& a, hipStream_t s)
{
    const unsigned blocks = (unsigned)(a.tiles * a.cols);
    if (a.tiles > 1) {
        const unsigned part = (unsigned)((a.tiles - 1) * a.cols);
        LX_LAUNCH("recur_grad_reduce", s, (lx_recur_grad_reduce<T, TG, V, SH><<<part, kRecurThreads, 0, s>>>(a)));
        const hipError_t e = recur_carry_launch(a, s);
        if (e != hipSuccess) return e;
    }
    LX_LAUNCH("recur_grad", s, (lx_recur_grad_apply<T, TG, V, SH><<<blocks, kRecurThreads, 0, s>>>(a)));
    if (a.dg && a.per > 1 && !recur_heads_inside(a.width, a.per))
        LX_LAUNCH("recur_grad_heads", s,
                  (lx_recur_grad_heads<TG><<<(unsigned)((a.n * a.heads + 255) / 256), 256, 0, s>>>(a)));
    return hipSuccess;
}

template <class T, class TG>
hipError_t grad_type(const RecurArgs& a, hipStream_t s)
{
    const bool sh = a.per > 1;
    const bool wide = vec_ok(a.x, a.ldx, a.width, sizeof(T), 4) && vec_ok(a.dy, a.lddy, a.width, sizeof(T), 4) &&
                      vec_ok(a.dx, a.lddx, a.width, sizeof(T), 4) && vec_ok(a.h0, a.width, a.width, 4, 4) &&
                      vec_ok(a.dfinal, a.width, a.width, 4, 4) && vec_ok(a.dh0, a.width, a.width, 4, 4) &&
                      (sh ? a.per % 4 == 0
                          : vec_ok(a.g, a.ldg, a.width, sizeof(TG), 4) && vec_ok(a.dg, a.lddg, a.width, sizeof(TG), 4));
    if (wide) return sh ? grad_go<T, TG, 4, true>(a, s) : grad_go<T, TG, 4, false>(a, s);
    return grad_go<T, TG, 1, true>(a, s);
}

}  // namespace

hipError_t recur_grad_launch(const RecurArgs& a, int dtype, int gtype, hipStream_t s)
{
    switch (dtype) {
        case 0: return grad_type<float, float>(a, s);
        case 1: return gtype ? grad_type<bf16_t, bf16_t>(a, s) : grad_type<bf16_t, float>(a, s);
        case 2: return gtype ? grad_type<f16_t, f16_t>(a, s) : grad_type<f16_t, float>(a, s);
        default: return hipErrorInvalidValue;
    }
}

}  // namespace lx

// Backward pass of the gated recurrence (gfx950).
//
// With u_t = dL/dh_t and w_t the gradient that reaches h_{t-1},
//     u_t = dy_t + w_{t+1},   w_t = a_t u_t,
//     dx_t = u_t,   dg_t = w_t h_{t-1},   dh0 = w of the first row,
// where w past the last row of a sequence is dfinal: the same kind of scan,
// towards earlier rows, with the decay of the row itself.  dg of a decay that
// serves several channels is the sum over them.  The states h_{t-1} are made
// again in float32 from x and the saved states between row tiles (1/256 of
// x's values), which reads no more than a saved y would and loses nothing to
// y's rounding.  Packed 32768 x 4096 bf16 with a decay per 64 channels: 230
// us (214 to 247 between launches), 3.6 TB/s of x, dy and dx, bound by what a
// tile waits for (loads 3 us, hand-over 3, writing 4 of 12, three workgroups
// per CU) and by dg, whose 4-byte values 256 bytes apart cost 18 % more bytes
// than they are; a decay per channel: 281 us, 4.8 TB/s.  Where a_t is 0 the state was forgotten and w_t and dg_t are 0.
#include "lx_recur.h"

namespace lx {

namespace {

constexpr int kSumPitch = kRecurCols / 4 + 1;  // sums of four channels per row, rows on different banks

// dy of row j, plus dfinal on a last row; 0 on a row of no sequence.
template <int CARE, class Th, class T, int V>
__device__ __forceinline__ void row_dy(const RecurArgs& A, const RecurRows* R, const Th& th,
                                       const RowPack<T, V, Th::L>& dy, int j, float (&d)[V])
{
    dy.get(j, d);
    if (!th.template special<CARE>(j)) return;
    if (R->start[th.r0 + j] == -2) {
#pragma unroll
        for (int v = 0; v < V; ++v) d[v] = 0.f;
    }
    const int q = R->last[th.r0 + j];
    if (q >= 0 && A.dfinal && th.in) {
        float f[V];
        load_vec<V>(A.dfinal + (int64_t)q * A.width + th.col(), f);
#pragma unroll
        for (int v = 0; v < V; ++v) d[v] += f[v];
    }
}

// Both maps of the thread's rows: the state after them, h -> r (r h) + H, and
// the gradient before them, w -> r (r w) + W.  In row order W is the sum of
// dy_j times the product of the decays up to row j, so one sweep gives both.
// False if the wave has to take care and did not.
template <int CARE, class Th, class T, int V>
__device__ __forceinline__ bool compose_both(const RecurArgs& A, const RecurRows* R, const Th& th,
                                             const RowPack<T, V, Th::L>& dy, float (&r)[Th::D], float (&H)[V], float (&W)[V])
{
    RecurProducts<care_root(CARE), Th::D, Th::L> m;
#pragma unroll
    for (int v = 0; v < V; ++v) H[v] = W[v] = 0.f;
#pragma unroll
    for (int j = 0; j < Th::L; ++j) {
        float a[Th::D], d[V];
        const bool cut = th.template decays<CARE>(R, j, a);
        th.template step<CARE>(A, R, j, a, cut, H);
        row_dy<CARE, Th, T, V>(A, R, th, dy, j, d);
        m.row(a, cut);
#pragma unroll
        for (int v = 0; v < V; ++v) W[v] = m.add(Th::D == 1 ? 0 : v, d[v], W[v]);
        settle(W);
    }
    return m.whole(r);
}

// dg of one row from a product per channel, one channel per lane: the lanes
// of a decay are neighbours and the first of them gets their sum.
template <class TG>
__device__ __forceinline__ void head_sum(const RecurArgs& A, int64_t row, bool here, int ct, int lane, float sum)
{
    const int col = ct * kRecurCols + lane;
    const int head = col < A.width ? col / A.per : -1;
#pragma unroll
    for (int d = 1; d < kWave; d <<= 1) {
        const float o = __shfl_down(sum, d);
        const int oh = __shfl_down(head, d);
        if (lane + d < kWave && oh == head) sum += o;
    }
    if (!here || (lane > 0 && col % A.per != 0)) return;
    if (recur_heads_inside(A.width, A.per)) ((TG*)A.dg)[row * A.lddg + head] = (TG)sum;
    else A.part[row * (A.cols + A.heads) + ct + head] = sum;
}

// dx, dg and dh0 of the thread's rows from the state h entering them and the
// gradient w from the rows after them.
template <int CARE, class T, class TG, int V, int L, bool SH>
__device__ __forceinline__ void write_grads(const RecurArgs& A, const RecurRows* R,
                                            const RecurThread<T, TG, V, L, SH>& th, const RowPack<T, V, L>& dy,
                                            int ct, float (&h)[V], float (&w)[V], float (*s_sum)[kSumPitch])
{
    using Th = RecurThread<T, TG, V, L, SH>;
    constexpr int D = Th::D;
    float before[L][V];  // state before each row
#pragma unroll
    for (int j = 0; j < L; ++j) {
        float a[D];
        __builtin_amdgcn_sched_barrier(0);
        const bool cut = th.template decays<CARE>(R, j, a);
#pragma unroll
        for (int v = 0; v < V; ++v) before[j][v] = h[v];
        th.template step<CARE>(A, R, j, a, cut, h);
    }
    const bool own = V == 1 ? A.per == 1 : !SH;  // a decay for each channel
    const RowAt<T, V> dx = th.template at<T, V>(A.dx, A.lddx);
    const RowAt<TG, V> dg = th.template at<TG, V>(A.dg, A.lddg);
#pragma unroll
    for (int j = L - 1; j >= 0; --j) {
        const bool here = care_rows(CARE) ? j < th.rows : th.in;
        float a[D], u[V], p[V];
        __builtin_amdgcn_sched_barrier(0);
        const bool cut = th.template decays<CARE>(R, j, a);
        row_dy<CARE, Th, T, V>(A, R, th, dy, j, u);
        const int q = th.template special<CARE>(j) ? R->start[th.r0 + j] : -1;
        if (q >= 0) {
            // the decay of a first row acts on h0 alone
            float g[D], h0[V], out[V];
            th.g.get(j, g);
#pragma unroll
            for (int v = 0; v < V; ++v) h0[v] = 0.f;
            if (A.h0 && th.in) load_vec<V>(A.h0 + (int64_t)q * A.width + th.col(), h0);
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const float av = root_of(g[SH ? 0 : v]);
                u[v] += w[v];
                out[v] = decayed(av, u[v]);
                p[v] = av == 0.f ? 0.f : out[v] * h0[v];
                w[v] = 0.f;
            }
            if (A.dh0 && th.in) store_vec<V>(A.dh0 + (int64_t)q * A.width + th.col(), out);
        } else {
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const float av = a[SH ? 0 : v];
                u[v] += w[v];
                w[v] = care_root(CARE) ? decayed(av, u[v]) : cut ? 0.f : av * u[v];
                p[v] = cut || (care_root(CARE) && av == 0.f) ? 0.f : w[v] * before[j][v];
            }
        }
        if (CARE) settle(w);
        if (A.dx && here) store_vec_as<V>(dx.row(j), u, A.stream);
        if (own) {
            if (A.dg && here) store_vec_as<V>(dg.row(j), p, A.stream);
        } else if (V > 1) {
            float sum = 0.f;
#pragma unroll
            for (int v = 0; v < V; ++v) sum += p[v];
            s_sum[th.r0 + j][th.lane] = sum;
        } else if (A.dg) {
            head_sum<TG>(A, th.wave_row + th.lane_row + j, here, ct, th.lane, p[0]);
        }
    }
}

// dg of a tile from s_sum[row][lane], sums over V channels each, V dividing
// the channels of a decay.  All threads; s_sum is complete.
template <class TG, int V, int THREADS, int PITCH>
__device__ __forceinline__ void tile_sums(const RecurArgs& A, int64_t tile, int ct, const float (*s_sum)[PITCH])
{
    const int c0 = ct * kRecurCols;
    const int c1 = c0 + kRecurCols < A.width ? c0 + kRecurCols : A.width;
    const int first = c0 / A.per, count = (c1 - 1) / A.per - first + 1;
    const bool inside = recur_heads_inside(A.width, A.per);
    for (int i = threadIdx.x; i < kRecurTile * count; i += THREADS) {
        const int r = i / count, head = first + i - r * count;
        const int64_t row = tile * kRecurTile + r;
        if (row >= A.n) return;
        int a = head * A.per - c0, b = a + A.per;
        a = a < 0 ? 0 : a / V;
        b = b > c1 - c0 ? (c1 - c0) / V : b / V;
        float sum = 0.f;
        for (; a < b; ++a) sum += s_sum[r][a];
        if (inside) ((TG*)A.dg)[row * A.lddg + head] = (TG)sum;
        else A.part[row * (A.cols + A.heads) + ct + head] = sum;
    }
}

// Rows of a thread and waves per SIMD to compile for.  What counts is bytes
// in flight per CU: half rows with shared decays take 16 rows per thread,
// three workgroups of 256 threads (calls of 4 x 8192 x 4096: 189 us, 8 rows
// 209); the others 8 rows, two workgroups of 512, also where that spills a
// few registers (bf16 rows with float32 decays of their own 326 us, without
// 411; shared float32 297, 368).  float32 rows with decays of their own would
// spill too many (560 us, without 540).
template <class T, bool SH>
constexpr int kGradRows = sizeof(T) == 2 && SH ? 16 : 8;
template <class T, bool SH>
constexpr int kGradWaves = !SH ? (sizeof(T) == 4 ? 2 : 4) : (sizeof(T) == 2 ? 3 : 4);

template <class T, class TG, int V, int L, bool SH>
__global__ __launch_bounds__((RecurLayout<V, L>::kThreads)) __attribute__((
    amdgpu_waves_per_eu((kGradWaves<T, SH>)))) void lx_recur_grad_pass(RecurArgs A)
{
    using Th = RecurThread<T, TG, V, L, SH>;
    using Lay = RecurLayout<V, L>;
    __shared__ RecurRows rows;
    __shared__ RecurGroups<V, L, SH> groups;
    __shared__ float sh[Lay::kGroups][kRecurCols];
    __shared__ float sw[Lay::kGroups][kRecurCols];
    constexpr bool kSums = SH && V > 1;
    __shared__ float s_sum[kSums ? kRecurTile : 1][kSumPitch];
    const int ct = channel_tile(A, (uint32_t)group_id<Lay::kThreads>());
    const int64_t back = next_tile(A, ct);  // tiles before this one in the pass: from the last rows on
    if (past_tiles(A, back)) return;
    const int64_t tile = A.tiles - 1 - back;
    const int mark = tile_mark(A, tile);
    Th th;
    RowPack<T, V, L> dy;
    th.load(A, tile, ct);
    if (th.gone(A)) dy.clear();
    else dy.load(th.template at<T, V>(A.dy, A.lddy), th.whole, th.last, A.stream);
    const RecurRows* R = uniform(recur_rows<Lay::kThreads>(A, tile * kRecurTile, mark, rows)) ? &rows : nullptr;
    float r[Th::D], h[V], w[V];
    int care = th.find_odd(A, R);
#pragma unroll
    for (int d = 0; d < Th::D; ++d) r[d] = 0.f;
#pragma unroll
    for (int v = 0; v < V; ++v) h[v] = w[v] = 0.f;
    // kCareBoth is rare: its code lies behind the others' (float32, shared
    // decays, 8192 x 4096, both directions 169 -> 163 us)
    if (care == kCareNone) {
        if (!compose_both<kCareNone, Th, T, V>(A, R, th, dy, r, h, w)) care = kCareRoot;
    } else if (care == kCareRows) {
        if (!compose_both<kCareRows, Th, T, V>(A, R, th, dy, r, h, w)) care = kCareBoth;
    }
    if (care == kCareRoot) compose_both<kCareRoot, Th, T, V>(A, R, th, dy, r, h, w);
    if (__builtin_expect(care == kCareBoth, 0)) compose_both<kCareBoth, Th, T, V>(A, R, th, dy, r, h, w);
    groups.put(th.group, th.lane, care, r);
#pragma unroll
    for (int v = 0; v < V; ++v) {
        sh[th.group][th.lane * V + v] = h[v];
        sw[th.group][th.lane * V + v] = w[v];
    }
    __syncthreads();
    // one wave carries the gradient, another the state
    if (threadIdx.x < kWave) {
        const uint32_t waves = groups.rooted();
        // nothing comes back into a tile whose last row ends a sequence or has none
        const bool fresh = R && (R->last[kRecurTile - 1] != -1 || R->start[kRecurTile - 1] == -2);
        float b = 0.f;
        if (A.tiles > 1) {
            float aw;
            const float ar = groups.template compose<true>(waves, sw, aw);
            b = pass_state(A, back, ct, ar, aw, fresh, back == A.tiles - 1);
        }
        groups.template enter<true>(waves, sw, b);
    } else if (threadIdx.x < 2 * kWave) {
        const float e = tile > 0 ? A.states_in[((tile - 1) * A.cols + ct) * kRecurCols + lane_id()] : 0.f;
        groups.template enter<false>(groups.rooted(), sh, e);
    }
    __syncthreads();
#pragma unroll
    for (int v = 0; v < V; ++v) {
        h[v] = sh[th.group][th.lane * V + v];
        w[v] = sw[th.group][th.lane * V + v];
    }
    if (care == kCareNone) write_grads<kCareNone>(A, R, th, dy, ct, h, w, s_sum);
    else if (care == kCareRoot) write_grads<kCareRoot>(A, R, th, dy, ct, h, w, s_sum);
    else if (care == kCareRows) write_grads<kCareRows>(A, R, th, dy, ct, h, w, s_sum);
    else if (__builtin_expect(care == kCareBoth, 0)) write_grads<kCareBoth>(A, R, th, dy, ct, h, w, s_sum);
    if (kSums && A.dg) {
        __syncthreads();
        tile_sums<TG, V, Lay::kThreads, kSumPitch>(A, tile, ct, s_sum);
    }
}

// Sums of decays whose channels span several channel tiles: a tile and a
// decay that meet have slot tile + decay of the row's partial sums, which
// no other pair of that row has.
template <class TG>
__global__ __launch_bounds__(256) void lx_recur_grad_heads(RecurArgs A)
{
    const int64_t i = group_id<256>() * 256 + threadIdx.x;
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

template <class T, class TG, int V, int L, bool SH>
hipError_t grad_go(const RecurArgs& a, hipStream_t s)
{
    LX_LAUNCH("recur_grad", s,
              (lx_recur_grad_pass<T, TG, V, L, SH>
               <<<grid_of<RecurLayout<V, L>::kThreads>(a.tiles * a.cols), RecurLayout<V, L>::kThreads, 0, s>>>(a)));
    if (a.dg && a.per > 1 && !recur_heads_inside(a.width, a.per))
        LX_LAUNCH("recur_grad_heads", s,
                  (lx_recur_grad_heads<TG><<<grid_of<256>((a.n * a.heads + 255) / 256), 256, 0, s>>>(a)));
    return hipSuccess;
}

template <class T, class TG>
hipError_t grad_type(const RecurArgs& a, hipStream_t s)
{
    const bool sh = a.per > 1;
    const bool wide = recur_wide(a);
    if (wide && recur_few(a)) return sh ? grad_go<T, TG, 4, 4, true>(a, s) : grad_go<T, TG, 4, 4, false>(a, s);
    if (wide)
        return sh ? grad_go<T, TG, 4, kGradRows<T, true>, true>(a, s)
                  : grad_go<T, TG, 4, kGradRows<T, false>, false>(a, s);
    return grad_go<T, TG, 1, 16, true>(a, s);
}

}  // namespace

hipError_t recur_grad_launch(const RecurArgs& a, int dtype, int gtype, hipStream_t s)
{
    const hipError_t e = recur_begin(a, a.dfinal, a.dh0, s);
    if (e != hipSuccess || a.n == 0) return e;
    switch (dtype) {
        case 0: return grad_type<float, float>(a, s);
        case 1: return gtype ? grad_type<bf16_t, bf16_t>(a, s) : grad_type<bf16_t, float>(a, s);
        case 2: return gtype ? grad_type<f16_t, f16_t>(a, s) : grad_type<f16_t, float>(a, s);
        default: return hipErrorInvalidValue;
    }
}

}  // namespace lx

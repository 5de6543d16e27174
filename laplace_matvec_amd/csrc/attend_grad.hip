// Gradients of the gated matrix memory (gfx950); notation of attend.hip.
//
// With S the state before a chunk, S+ the gradient of the state after it, and
// within the chunk, for j <= i,
//     D_ij = e^{G_i - G_j},  P_ij = scale (q_i . k_j) D_ij,
//     E_ij = scale (dy_i . v_j) D_ij,  W_ij = P_ij (dy_i . v_j),
//     a_i = scale e^{G_i} S dy_i,  b_j = e^{G_63 - G_j} S+ v_j:
//     dq_i = sum_j E_ij k_j + a_i
//     dk_j = sum_i E_ij q_i + b_j
//     dv_j = sum_i P_ij dy_i + e^{G_63 - G_j} S+^T k_j
//     dg_t = sum_{i >= t > j} W_ij + sum_{i >= t} q_i . a_i + sum_{j < t} k_j . b_j + e^{G_63} <S, S+>
// The last line is what passes from rows before t to rows from t on: all of
// it local to the chunk, nothing is summed along the sequence.  The sum over
// pairs is that of W's row sums from t on less that of its column sums.
//
// Two sweeps (attend.hip) leave S and S+ of every chunk in float32; then every
// chunk is on its own.  A workgroup takes a chunk of one query and key head
// and goes through the heads that share it, so their gradients of q and k are
// summed in registers.
#include "lx_attend.h"

namespace lx {

namespace {

constexpr int kGradThreads = 512;

// Sums over the lanes of a group of 16, in all of them.
__device__ __forceinline__ float sum16(float x)
{
#define LX_ROR(n) __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, x), 0x120 + (n), 0xF, 0xF, true))
    x += LX_ROR(8);
    x += LX_ROR(4);
    x += LX_ROR(2);
    x += LX_ROR(1);
#undef LX_ROR
    return x;
}

// Waves 0 to 3 make the rows' side (scores, dq), waves 4 to 7 the columns'
// (dk, dv), sixteen rows of the chunk each; wave w and w + 4 share a SIMD, so
// each has one of either.  What the next head needs is on its way meanwhile.
template <class T, class TG, int DK, int DV>
__global__ __launch_bounds__(kGradThreads) void lx_attend_grad(AttendArgs A)
{
    typedef typename Compute<T>::E E;
    typedef E V4 __attribute__((ext_vector_type(4)));
    constexpr int N = Compute<T>::kTerms;
    constexpr int PK = DK + kPad<E>, PV = DV + kPad<E>, PC = kC + kPad<E>;
    constexpr int NS = DK * DV / 4 / kGradThreads;  // groups of four state values a thread
    __shared__ alignas(16) E s_q[kC * PK];
    __shared__ alignas(16) E s_k[kC * PK];
    __shared__ alignas(16) E s_v[kC * PV];
    __shared__ alignas(16) E s_do[kC * PV];
    __shared__ alignas(16) E s_s[N * DK * PV];  // S
    __shared__ alignas(16) E s_t[N * DK * PV];  // S+
    __shared__ alignas(16) E s_p[kC * PC];
    __shared__ alignas(16) E s_e[kC * PC];
    __shared__ alignas(16) Decays s_d;
    __shared__ float s_row[kC], s_col[4][kC], s_b[kC], s_z[2][8];

    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int side = wave >> 2, w16 = 16 * (wave & 3);
    const int g4 = 4 * (lane >> 4), l16 = lane & 15;
    const int64_t id = group_id<kGradThreads>();
    const int parts = A.heads / A.loop * A.nkb;
    const int64_t unit = id / parts;
    const int part = (int)(id - unit * parts);
    const int h0 = part / A.nkb * A.loop, kb = part % A.nkb;
    const Ragged R{A.offsets, A.seqs, A.n, A.seq_len};
    if (unit >= R.units(kC)) return;
    const RaggedTile t = R.find(unit, kC);
    if (t.rows <= 0) return;
    const int rows = t.rows;
    const int k0 = kb * DK, kcols = A.dk - k0;
    const int rq = A.heads / A.hq, rk = A.heads / A.hk, rv = A.heads / A.hv;
    const int nvb = A.dvp / DV;
    // where results go: the arrays, or planes of partial sums
    auto put = [](float x, float* p, int64_t ldp, void* to, int64_t at, int64_t ld, int row, int col) {
        if (p)
            p[row * ldp + col] = x;
        else
            ((T*)to)[at + row * ld + col] = (T)x;
    };
    auto put_q = [&](float x, int row, int col) {
        float* p = A.part_q ? A.part_q + (h0 % rq / A.loop * A.n + t.row) * ((int64_t)A.hq * A.dk) + h0 / rq * A.dk + k0 : nullptr;
        put(x, p, (int64_t)A.hq * A.dk, A.dq, t.row * A.lddq + h0 / rq * A.dk + k0, A.lddq, row, col);
    };
    auto put_k = [&](float x, int row, int col) {
        float* p = A.part_k ? A.part_k + (h0 % rk / A.loop * A.n + t.row) * ((int64_t)A.hk * A.dk) + h0 / rk * A.dk + k0 : nullptr;
        put(x, p, (int64_t)A.hk * A.dk, A.dkey, t.row * A.lddk + h0 / rk * A.dk + k0, A.lddk, row, col);
    };
    auto put_v = [&](float x, int h, int row, int col) {
        float* p = A.part_v ? A.part_v + ((int64_t)(h % rv * A.nkb + kb) * A.n + t.row) * ((int64_t)A.hv * A.dv) + h / rv * A.dv : nullptr;
        put(x, p, (int64_t)A.hv * A.dv, A.dval, t.row * A.lddv + h / rv * A.dv, A.lddv, row, col);
    };
    auto put_g = [&](float x, int h, int row) {
        if (A.part_g)
            A.part_g[(kb * A.n + t.row + row) * (int64_t)A.heads + h] = x;
        else
            ((TG*)A.dg)[(t.row + row) * A.lddg + h] = (TG)x;
    };
    if (t.group < 0) {
        for (int i = threadIdx.x; i < rows * DK; i += kGradThreads) {
            if (i % DK >= kcols) continue;
            if (A.dq) put_q(0.f, i / DK, i % DK);
            if (A.dkey) put_k(0.f, i / DK, i % DK);
        }
        for (int h = h0; h < h0 + A.loop; ++h) {
            if (A.dval)
                for (int i = threadIdx.x; i < rows * A.dv; i += kGradThreads) put_v(0.f, h, i / A.dv, i % A.dv);
            if (A.dg && (int)threadIdx.x < rows) put_g(0.f, h, threadIdx.x);
        }
        return;
    }

    // The state before the chunk and the gradient of the one after it: an edge
    // of the sequence, or a slot between chunks.
    const bool is_first = t.index == 0, is_last = t.row + t.rows == t.end;
    const int64_t slot = t.first / kC + t.index;
    auto four = [&](const float* edges, const float* slots, bool edge, int64_t at_slot, int h, int v0, int row, int col) {
        f32x4 x = {};
        if (!edge) {
            x = *reinterpret_cast<const f32x4*>(slots + ((at_slot * A.heads + h) * A.dkp + k0 + row) * A.dvp + v0 + col);
        } else if (edges && row < kcols) {
            const float* p = edges + ((t.group * A.heads + h) * A.dk + k0 + row) * (int64_t)A.dv + v0 + col;
#pragma unroll
            for (int r = 0; r < 4; ++r)
                if (v0 + col + r < A.dv) x[r] = p[r];
        }
        return x;
    };
    RowTile<T, DV, kGradThreads> tv, td;
    f32x4 ts[NS], tt[NS];
    float tg = 0.f;
    auto fetch = [&](int h, int vb) {
        const int v0 = vb * DV, vcols = A.dv - v0;
        tv.load((const T*)A.v + t.row * A.ldv + h / rv * A.dv + v0, A.ldv, rows, vcols);
        td.load((const T*)A.dy + t.row * A.lddy + (int64_t)h * A.dv + v0, A.lddy, rows, vcols);
#pragma unroll
        for (int u = 0; u < NS; ++u) {
            const int at = (int)threadIdx.x + u * kGradThreads, row = at / (DV / 4), col = at % (DV / 4) * 4;
            ts[u] = four(A.h0, A.chunk_states, is_first, slot - 1, h, v0, row, col);
            tt[u] = four(A.dfinal, A.chunk_grads, is_last, slot, h, v0, row, col);
        }
        if (wave == 0) tg = lane < rows ? (float)((const TG*)A.g)[(t.row + lane) * A.ldg + h] : 0.f;
    };
    auto put_state = [&](const f32x4& x, E* s, int row, int col) {
        V4 w[N];
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            E e[N];
            split<E, N>(x[r], e);
#pragma unroll
            for (int m = 0; m < N; ++m) w[m][r] = e[m];
        }
#pragma unroll
        for (int m = 0; m < N; ++m) *reinterpret_cast<V4*>(&s[(m * DK + row) * PV + col]) = w[m];
    };
    {
        RowTile<T, DK, kGradThreads> a, b;
        a.load((const T*)A.q + t.row * A.ldq + h0 / rq * A.dk + k0, A.ldq, rows, kcols);
        b.load((const T*)A.k + t.row * A.ldk + h0 / rk * A.dk + k0, A.ldk, rows, kcols);
        fetch(h0, 0);
        a.put(s_q);
        b.put(s_k);
    }
    __syncthreads();
    const int i = w16 + l16;
    // scores, transposed: column i, rows j = 16 jt + g4 + r
    f32x4 score[4] = {};
    if (side == 0) {
#pragma unroll
        for (int jt = 0; jt < 4; ++jt)
            if (16 * jt <= w16)
#pragma unroll
                for (int kk = 0; kk < DK / 32; ++kk)
                    score[jt] = mma(frag_along(s_k + (16 * jt + l16) * PK + 32 * kk + 2 * g4),
                                    frag_along(s_q + i * PK + 32 * kk + 2 * g4), score[jt]);
    }
    // dq, or dk: rows w16 + g4 + r, columns 16 c + l16
    f32x4 acc[DK / 16] = {};
    float dg = 0.f;  // wave 0: row `lane`
    int flip = 0;
    for (int it = 0; it < A.loop * nvb; ++it, flip ^= 1) {
        const int h = h0 + it / nvb, vb = it % nvb;
        const int v0 = vb * DV, vcols = A.dv - v0;
        tv.put(s_v);
        td.put(s_do);
        float z = 0.f;
#pragma unroll
        for (int u = 0; u < NS; ++u) {
            const int at = (int)threadIdx.x + u * kGradThreads, row = at / (DV / 4), col = at % (DV / 4) * 4;
            put_state(ts[u], s_s, row, col);
            put_state(tt[u], s_t, row, col);
#pragma unroll
            for (int r = 0; r < 4; ++r) z += ts[u][r] * tt[u][r];
        }
        z = sum16(z);
        z += __shfl_xor(z, 16);
        z += __shfl_xor(z, 32);
        if (lane == 0) s_z[flip][wave] = z;
        if (wave == 0 && vb == 0) s_d.make(tg);
        __syncthreads();
        if (it + 1 < A.loop * nvb) fetch(h0 + (it + 1) / nvb, (it + 1) % nvb);

        Frag<E> fe[2];
        f32x4 dv[DV / 16];
        if (side == 0) {
            f32x4 u = {};
            const f32x4 into = *reinterpret_cast<const f32x4*>(&s_d.into[w16 + g4]);
#pragma unroll
            for (int c = 0; c < DK / 16; ++c) {
                f32x4 x = {};
#pragma unroll
                for (int kk = 0; kk < DV / 32; ++kk) {
                    const Frag<E> f = frag_along(s_do + i * PV + 32 * kk + 2 * g4);
#pragma unroll
                    for (int m = 0; m < N; ++m)
                        x = mma(f, frag_along(s_s + (m * DK + 16 * c + l16) * PV + 32 * kk + 2 * g4), x);
                }
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    x[r] = into[r] == 0.f ? 0.f : into[r] * A.scale * x[r];
                    u[r] += x[r] * (float)s_q[(w16 + g4 + r) * PK + 16 * c + l16];
                    acc[c][r] += x[r];
                }
            }
            const float hi_i = s_d.hi[i], lo_i = s_d.lo[i];
            const int last_i = s_d.last[i];
            float row_sum = 0.f;
#pragma unroll
            for (int jt = 0; jt < 4; ++jt) {
                V4 p4 = {}, e4 = {};
                f32x4 w = {};
                if (16 * jt <= w16) {
                    f32x4 x = {};
#pragma unroll
                    for (int kk = 0; kk < DV / 32; ++kk)
                        x = mma(frag_along(s_v + (16 * jt + l16) * PV + 32 * kk + 2 * g4),
                                frag_along(s_do + i * PV + 32 * kk + 2 * g4), x);
                    const f32x4 hi = *reinterpret_cast<const f32x4*>(&s_d.hi[16 * jt + g4]);
                    const f32x4 lo = *reinterpret_cast<const f32x4*>(&s_d.lo[16 * jt + g4]);
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        const int j = 16 * jt + g4 + r;
                        const bool on = j <= i && j >= last_i;
                        const float d = A.scale * s_d.between(hi_i, lo_i, hi[r], lo[r]);
                        const float p = on ? score[jt][r] * d : 0.f;
                        p4[r] = (E)p;
                        e4[r] = (E)(on ? x[r] * d : 0.f);
                        w[r] = on && j < i ? p * x[r] : 0.f;
                        row_sum += w[r];
                    }
                }
                *reinterpret_cast<V4*>(&s_p[i * PC + 16 * jt + g4]) = p4;
                *reinterpret_cast<V4*>(&s_e[i * PC + 16 * jt + g4]) = e4;
                f32x4 sums;
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    fe[jt >> 1].v[4 * (jt & 1) + r] = e4[r];
                    sums[r] = sum16(w[r]);
                }
                if (l16 == 0) *reinterpret_cast<f32x4*>(&s_col[wave][16 * jt + g4]) = sums;
            }
            row_sum += __shfl_xor(row_sum, 16);
            row_sum += __shfl_xor(row_sum, 32);
            if (g4 == 0) s_row[i] = row_sum;
#pragma unroll
            for (int r = 0; r < 4; ++r) u[r] = sum16(u[r]);
            // the wave's own rows: no other wave touches them
            if (l16 == 0)
#pragma unroll
                for (int r = 0; r < 4; ++r) s_row[w16 + g4 + r] += u[r];
        } else {
            const f32x4 out = *reinterpret_cast<const f32x4*>(&s_d.out[w16 + g4]);
            f32x4 u = {};
#pragma unroll
            for (int c = 0; c < DK / 16; ++c) {
                f32x4 x = {};
#pragma unroll
                for (int kk = 0; kk < DV / 32; ++kk) {
                    const Frag<E> f = frag_along(s_v + i * PV + 32 * kk + 2 * g4);
#pragma unroll
                    for (int m = 0; m < N; ++m)
                        x = mma(f, frag_along(s_t + (m * DK + 16 * c + l16) * PV + 32 * kk + 2 * g4), x);
                }
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    x[r] = out[r] == 0.f ? 0.f : out[r] * x[r];
                    u[r] += x[r] * (float)s_k[(w16 + g4 + r) * PK + 16 * c + l16];
                    acc[c][r] += x[r];
                }
            }
#pragma unroll
            for (int r = 0; r < 4; ++r) u[r] = sum16(u[r]);
            if (l16 == 0) *reinterpret_cast<f32x4*>(&s_b[w16 + g4]) = u;
            if (A.dval) {
#pragma unroll
                for (int b = 0; b < DV / 16; ++b) {
                    f32x4 x = {};
#pragma unroll
                    for (int kk = 0; kk < DK / 32; ++kk) {
                        const Frag<E> f = frag_along_split(s_k + i * PK + 32 * kk);
#pragma unroll
                        for (int m = 0; m < N; ++m)
                            x = mma(f, frag_across(s_t + (m * DK + 32 * kk) * PV + 16 * b, PV), x);
                    }
#pragma unroll
                    for (int r = 0; r < 4; ++r) dv[b][r] = out[r] == 0.f ? 0.f : out[r] * x[r];
                }
            }
        }
        __syncthreads();
        if (side == 0) {
#pragma unroll
            for (int c = 0; c < DK / 16; ++c)
#pragma unroll
                for (int s = 0; s < 2; ++s)
                    if (32 * s <= w16) acc[c] = mma(fe[s], frag_across(s_k + 32 * s * PK + 16 * c, PK), acc[c]);
        } else {
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                if (32 * s + 16 < w16) continue;
                const Frag<E> f = frag_across(s_e + 32 * s * PC + w16, PC);
#pragma unroll
                for (int c = 0; c < DK / 16; ++c) acc[c] = mma(f, frag_across(s_q + 32 * s * PK + 16 * c, PK), acc[c]);
            }
            if (A.dval) {
#pragma unroll
                for (int s = 0; s < 2; ++s) {
                    if (32 * s + 16 < w16) continue;
                    const Frag<E> f = frag_across(s_p + 32 * s * PC + w16, PC);
#pragma unroll
                    for (int b = 0; b < DV / 16; ++b) dv[b] = mma(f, frag_across(s_do + 32 * s * PV + 16 * b, PV), dv[b]);
                }
#pragma unroll
                for (int b = 0; b < DV / 16; ++b) {
                    const int col = 16 * b + l16;
#pragma unroll
                    for (int r = 0; r < 4; ++r)
                        if (w16 + g4 + r < rows && col < vcols) put_v(dv[b][r], h, w16 + g4 + r, v0 + col);
                }
            }
        }
        __syncthreads();
        if (wave == 0) {
            float from = s_row[lane] - ((s_col[0][lane] + s_col[1][lane]) + (s_col[2][lane] + s_col[3][lane]));
            float to = s_b[lane];
            const float own = to;
#pragma unroll
            for (int d = 1; d < 64; d *= 2) {
                const float above = __shfl_down(from, d), below = __shfl_up(to, d);
                if (lane + d < 64) from += above;
                if (lane >= d) to += below;
            }
            float z = 0.f;
#pragma unroll
            for (int w = 0; w < 8; ++w) z += s_z[flip][w];
            const float whole = s_d.into[kC - 1];
            const float through = whole == 0.f ? 0.f : whole * z;
            // the last cut up to a row is the row itself: its decay has no gradient
            dg = (vb ? dg : 0.f) + (s_d.last[lane] == lane ? 0.f : from + (to - own) + through);
            if (A.dg && vb + 1 == nvb && lane < rows) put_g(dg, h, lane);
        }
    }
#pragma unroll
    for (int c = 0; c < DK / 16; ++c) {
        const int col = 16 * c + l16;
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int row = w16 + g4 + r;
            if (row < rows && col < kcols) {
                if (side == 0 && A.dq) put_q(acc[c][r], row, col);
                if (side == 1 && A.dkey) put_k(acc[c][r], row, col);
            }
        }
    }
}

template <class T, class TG, int DK, int DV>
hipError_t grad_go(const AttendArgs& a, hipStream_t s)
{
    const int64_t groups = Ragged{a.offsets, a.seqs, a.n, a.seq_len}.units(kC) * (a.heads / a.loop) * a.nkb;
    LX_LAUNCH("attend_grad", s, (lx_attend_grad<T, TG, DK, DV><<<grid_of<kGradThreads>(groups), kGradThreads, 0, s>>>(a)));
    return hipSuccess;
}

template <class T, class TG>
hipError_t grad_type(const AttendArgs& a, hipStream_t s)
{
    if constexpr (sizeof(typename Compute<T>::E) == 2) {
        if (a.block_k == 128) return grad_go<T, TG, 128, 64>(a, s);
    }
    return grad_go<T, TG, 64, 64>(a, s);
}

}  // namespace

hipError_t attend_grad_launch(const AttendArgs& a, int dtype, int gtype, hipStream_t s)
{
    hipError_t e = attend_states_launch(a, dtype, gtype, s);
    if (e != hipSuccess || a.n == 0 || (!a.dq && !a.dkey && !a.dval && !a.dg)) return e;
    AttendArgs b = a;
    b.block_k = a.grad_block_k;
    b.nkb = a.dkp / b.block_k;
    switch (dtype) {
        case 0: e = grad_type<float, float>(b, s); break;
        case 1: e = gtype ? grad_type<bf16_t, bf16_t>(b, s) : grad_type<bf16_t, float>(b, s); break;
        case 2: e = gtype ? grad_type<f16_t, f16_t>(b, s) : grad_type<f16_t, float>(b, s); break;
        default: return hipErrorInvalidValue;
    }
    if (e != hipSuccess) return e;
    const int rq = a.heads / a.hq / a.loop, rk = a.heads / a.hk / a.loop, rv = a.heads / a.hv * b.nkb;
    if (a.part_q && a.dq && (e = attend_sum_launch(a.part_q, rq, a.n, (int64_t)a.hq * a.dk, a.dq, a.lddq, dtype, s)) != hipSuccess) return e;
    if (a.part_k && a.dkey && (e = attend_sum_launch(a.part_k, rk, a.n, (int64_t)a.hk * a.dk, a.dkey, a.lddk, dtype, s)) != hipSuccess) return e;
    if (a.part_v && a.dval && (e = attend_sum_launch(a.part_v, rv, a.n, (int64_t)a.hv * a.dv, a.dval, a.lddv, dtype, s)) != hipSuccess) return e;
    if (a.part_g && a.dg) return attend_sum_launch(a.part_g, b.nkb, a.n, a.heads, a.dg, a.lddg, gtype, s);
    return hipSuccess;
}

}  // namespace lx

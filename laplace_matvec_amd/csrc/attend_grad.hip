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
// pairs is that of W's row sums from t on less that of its column sums: what
// stays within the rows from t on cancels, so after a strong decay dg_t is off
// by the rounding of those, not of its own few terms.
//
// Two sweeps (attend.hip) leave S and S+ of every chunk in float32; then every
// chunk is on its own.  A workgroup takes a chunk of one query and key head
// and goes through the heads that share it, so their gradients of q and k are
// summed in registers.  Where several workgroups add to one row (heads that
// share unequally, states of several blocks) each writes a plane and
// lx_attend_sum adds the planes in their order.
//
// 32768 rows, 32 heads of 128 x 64 on 8 query and key heads, bf16: 750 us for
// 1.5 GB (S and S+ 1.1 of them).  Bound by latency: half of the waves' time is
// waiting, at one workgroup of eight waves a CU (157 KB of LDS) and four
// barriers a head; rows padded so that no two lines of a transposing read
// share banks changed nothing.  One workgroup of four waves doing both sides in turn,
// loads where they are used: 1630; addresses worked out per value instead of
// per head 1211 (of eight waves); kept across heads, which spills, 760 (these
// with states in two terms, scores in one and three barriers: 640).  Scores
// go where S was, so they wait in registers until all waves are done with it;
// written at once behind a barrier of their own the whole pass took 1603 us,
// so 1567.
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

// Sums up to each lane.
__device__ __forceinline__ float scan_up(float x)
{
#define LX_DPP(ctrl, rows) __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, x), ctrl, rows, 0xF, false))
    x += LX_DPP(0x111, 0xF);
    x += LX_DPP(0x112, 0xF);
    x += LX_DPP(0x114, 0xF);
    x += LX_DPP(0x118, 0xF);
    x += LX_DPP(0x142, 0xA);
    x += LX_DPP(0x143, 0xC);
#undef LX_DPP
    return x;
}

// Rows of a result, or of a plane of partial sums (float32) where `sums` is there.
template <class T>
struct Out {
    float* sums;
    T* to;
    int64_t ld;
    __device__ __forceinline__ void put(int row, int col, float x) const
    {
        if (sums)
            sums[row * ld + col] = x;
        else
            to[row * ld + col] = (T)x;
    }
    // x[c][r]: rows row0 + r, columns 16 c + col0, as far as they are there
    template <int C>
    __device__ __forceinline__ void put_tiles(int row0, int col0, int rows, int cols, const f32x4 (&x)[C]) const
    {
        if (!sums && rows == kC && cols >= 16 * C) {
            T* p = to + row0 * ld + col0;
#pragma unroll
            for (int r = 0; r < 4; ++r)
#pragma unroll
                for (int c = 0; c < C; ++c) p[r * ld + 16 * c] = (T)x[c][r];
            return;
        }
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            if (row0 + r >= rows) continue;
            if (sums) {
                float* p = sums + (row0 + r) * ld + col0;
#pragma unroll
                for (int c = 0; c < C; ++c)
                    if (16 * c + col0 < cols) p[16 * c] = x[c][r];
            } else {
                T* p = to + (row0 + r) * ld + col0;
#pragma unroll
                for (int c = 0; c < C; ++c)
                    if (16 * c + col0 < cols) p[16 * c] = (T)x[c][r];
            }
        }
    }
};
template <class T>
__device__ __forceinline__ Out<T> out_rows(void* to, int64_t ld, float* sums, int64_t plane, int64_t n, int width,
                                           int64_t row, int col)
{
    if (sums) return {sums + (plane * n + row) * width + col, nullptr, width};
    return {nullptr, (T*)to + row * ld + col, ld};
}

// Waves 0 to 3 make the rows' side (scores, dq), waves 4 to 7 the columns'
// (dk, dv), sixteen rows of the chunk each; wave w and w + 4 share a SIMD, so
// each has one of either.  What the next head needs is on its way meanwhile.
template <class T, class TG, int DK, int DV, bool WHOLE>
__global__ __launch_bounds__(kGradThreads) void lx_attend_grad(AttendArgs A)
{
    typedef typename Compute<T>::E E;
    typedef E V4 __attribute__((ext_vector_type(4)));
    constexpr int N = Compute<T>::kTerms, NP = Compute<T>::kScoreTerms;
    constexpr int NS2 = N < 2 ? N : 2;  // of S+ for dv, which is rounded to T
    constexpr int PK = DK + kPad<E>, PV = DV + kPad<E>, PC = kC + kPad<E>;
    constexpr int NS = DK * DV / 4 / kGradThreads;  // groups of four state values a thread
    __shared__ alignas(16) E s_q[kC * PK];
    __shared__ alignas(16) E s_k[kC * PK];
    __shared__ alignas(16) E s_v[kC * PV];
    __shared__ alignas(16) E s_do[kC * PV];
    // S, transposed; once all waves have used it, P and E in its place
    constexpr int kStates = N * DV * PK, kScores = 2 * NP * kC * PC;
    __shared__ alignas(16) E s_s[kStates > kScores ? kStates : kScores];
    __shared__ alignas(16) E s_t[N * DV * PK];  // S+, transposed
    E *const s_p = s_s, *const s_e = s_s + NP * kC * PC;
    __shared__ alignas(16) Decays s_d;
    __shared__ alignas(16) float s_row[kC], s_col[4][kC], s_a[kC], s_b[kC];
    __shared__ float s_z[2][8];

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
    // This chunk's rows of the results: of the arrays, or of planes of partial
    // sums where several workgroups add to one row.
    const int hq0 = h0 / rq, hk0 = h0 / rk, hv0 = h0 / rv;
    auto out_q = [&] { return out_rows<T>(A.dq, A.lddq, A.part_q, h0 % rq / A.loop, A.n, A.hq * A.dk, t.row, hq0 * A.dk + k0); };
    auto out_k = [&] { return out_rows<T>(A.dkey, A.lddk, A.part_k, h0 % rk / A.loop, A.n, A.hk * A.dk, t.row, hk0 * A.dk + k0); };
    auto out_g = [&] { return out_rows<TG>(A.dg, A.lddg, A.part_g, kb, A.n, A.heads, t.row, h0); };
    if (t.group < 0) {
        const Out<T> oq = out_q(), ok = out_k();
        const Out<TG> og = out_g();
        for (int i = threadIdx.x; i < rows * DK; i += kGradThreads) {
            if (i % DK >= kcols) continue;
            if (A.dq) oq.put(i / DK, i % DK, 0.f);
            if (A.dkey) ok.put(i / DK, i % DK, 0.f);
        }
        for (int h = h0; h < h0 + A.loop; ++h) {
            const Out<T> ov = out_rows<T>(A.dval, A.lddv, A.part_v, h % rv * A.nkb + kb, A.n, A.hv * A.dv, t.row, h / rv * A.dv);
            if (A.dval)
                for (int i = threadIdx.x; i < rows * A.dv; i += kGradThreads) ov.put(i / A.dv, i % A.dv, 0.f);
            if (A.dg && (int)threadIdx.x < rows) og.put(threadIdx.x, h - h0, 0.f);
        }
        return;
    }

    // The state before the chunk and the gradient of the one after it: an edge
    // of the sequence, or a slot between chunks.
    const bool is_first = t.index == 0, is_last = t.row + t.rows == t.end;
    const int64_t slot = t.first / kC + t.index;
    const int64_t size = (int64_t)A.dkp * A.dvp;
    const float* slot_s = A.chunk_states + ((slot - 1) * A.heads + h0) * size + tile_at(k0 / 16, 0, A.dvp);
    const float* slot_t = A.chunk_grads + (slot * A.heads + h0) * size + tile_at(k0 / 16, 0, A.dvp);
    const int64_t edge_at = ((t.group * A.heads + h0) * A.dk + k0) * (int64_t)A.dv;
    // a thread's values: four of tile wave + 8 u of the block, row by row of tiles
    constexpr int kAcross = DV / 16;
    auto state_in = [&](f32x4 (&x)[NS], const float* slots, int hl, int v0) {
        const float* p = slots + hl * size + v0 * 16 + 4 * lane;
#pragma unroll
        for (int u = 0; u < NS; ++u) {
            const int tile = wave + u * (kGradThreads / 64);
            x[u] = *reinterpret_cast<const f32x4*>(p + tile_at(tile / kAcross, tile % kAcross, A.dvp));
        }
    };
    // The same from an edge, where it is used: once or twice in a sequence.
    auto at_edge = [&](const float* edges, int hl, int v0, int row, int col) {
        f32x4 x = {};
        if (edges && v0 + col < A.dv) {
            const float* p = edges + edge_at + hl * ((int64_t)A.dk * A.dv) + v0 + col;
#pragma unroll
            for (int r = 0; r < 4; ++r)
                if (row + r < kcols) x[r] = p[(int64_t)(row + r) * A.dv];
        }
        return x;
    };
    RowTile<T, DV, WHOLE, kGradThreads> tv, td;
    f32x4 ts[NS], tt[NS];
    TG tg = (TG)0.f;
    const T* vp = (const T*)A.v + t.row * A.ldv;
    const T* dp = (const T*)A.dy + t.row * A.lddy + (int64_t)h0 * A.dv;
    const TG* gp = (const TG*)A.g + (t.row + (lane < rows ? lane : rows - 1)) * A.ldg + h0;
    auto fetch = [&](int hl, int hv, int vb) {
        const int v0 = vb * DV, vcols = A.dv - v0;
        tv.load(vp + hv * A.dv + v0, A.ldv, rows, vcols);
        td.load(dp + hl * A.dv + v0, A.lddy, rows, vcols);
        if (!is_first) state_in(ts, slot_s, hl, v0);
        if (!is_last) state_in(tt, slot_t, hl, v0);
        if (wave == 0) tg = gp[hl];
    };
    auto half_of = [](const Frag<E>& f, int h) {
        return h ? __builtin_shufflevector(f.v, f.v, 4, 5, 6, 7) : __builtin_shufflevector(f.v, f.v, 0, 1, 2, 3);
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
        for (int m = 0; m < N; ++m) *reinterpret_cast<V4*>(&s[(m * DV + col) * PK + row]) = w[m];
    };
    {
        RowTile<T, DK, WHOLE, kGradThreads> a, b;
        a.load((const T*)A.q + t.row * A.ldq + hq0 * A.dk + k0, A.ldq, rows, kcols);
        b.load((const T*)A.k + t.row * A.ldk + hk0 * A.dk + k0, A.ldk, rows, kcols);
        fetch(0, hv0, 0);
        a.put(s_q, rows, kcols);
        b.put(s_k, rows, kcols);
    }
    __syncthreads();
    // dq, or dk: rows w16 + g4 + r, columns 16 c + l16
    f32x4 acc[DK / 16] = {};
    float dg = 0.f;  // wave 0: row `lane`
    int flip = 0, vb = 0, hl = 0;  // block of columns; head, from h0 on
    int hv = hv0, in_hv = h0 - hv0 * rv;  // the value head, and which of those that share it
    for (;; flip ^= 1) {
        // Places worked out anew each time: kept for all heads they would take
        // the registers that the next head's values need.
        int here = lane;
        asm volatile("" : "+v"(here));
        const int g4 = 4 * (here >> 4), l16 = here & 15, i = w16 + l16;
        const int v0 = vb * DV, vcols = A.dv - v0;
        const bool ends_head = vb + 1 == nvb;
        const bool more = !(ends_head && hl + 1 == A.loop);
        const int next_hv = ends_head && in_hv + 1 == rv ? hv + 1 : hv;
        tv.put(s_v, rows, vcols);
        td.put(s_do, rows, vcols);
        float z = 0.f;
#pragma unroll
        for (int u = 0; u < NS; ++u) {
            const int tile = wave + u * (kGradThreads / 64);
            const int row = 16 * (tile / kAcross) + g4, col = 16 * (tile % kAcross) + l16;
            const f32x4 x = is_first ? at_edge(A.h0, hl, v0, row, col) : ts[u];
            const f32x4 y = is_last ? at_edge(A.dfinal, hl, v0, row, col) : tt[u];
            put_state(x, s_s, row, col);
            put_state(y, s_t, row, col);
#pragma unroll
            for (int r = 0; r < 4; ++r) z += x[r] * y[r];
        }
        z = sum16(z);
        z += __shfl_xor(z, 16);
        z += __shfl_xor(z, 32);
        if (lane == 0) s_z[flip][wave] = z;
        if (wave == 0 && vb == 0) s_d.make(lane < rows ? (float)tg : 0.f);
        __syncthreads();
        if (more) fetch(ends_head ? hl + 1 : hl, next_hv, ends_head ? 0 : vb + 1);

        Frag<E> fp[NP][2], fe[NP][2];
        f32x4 dv[DV / 16];
        f32x4 u = {};
        if (side == 0) {
            const f32x4 into = *reinterpret_cast<const f32x4*>(&s_d.into[w16 + g4]);
#pragma unroll
            for (int c = 0; c < DK / 16; ++c) {
                f32x4 x = {};
#pragma unroll
                for (int kk = 0; kk < DV / 32; ++kk) {
                    const Frag<E> f = frag_along_split(s_do + i * PV + 32 * kk);
#pragma unroll
                    for (int m = 0; m < N; ++m)
                        x = mma(f, frag_across(s_s + (m * DV + 32 * kk) * PK + 16 * c, PK), x);
                }
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    x[r] = into[r] == 0.f ? 0.f : into[r] * A.scale * x[r];
                    u[r] += x[r] * (float)s_q[(w16 + g4 + r) * PK + 16 * c + l16];
                    acc[c][r] += x[r];
                }
                if ((c & 3) == 3) __builtin_amdgcn_sched_barrier(0);  // not more fragments at a time than registers
            }
#pragma unroll
            for (int r = 0; r < 4; ++r) u[r] = sum16(u[r]);
            if (l16 == 0) *reinterpret_cast<f32x4*>(&s_a[w16 + g4]) = u;
            const float hi_i = s_d.hi[i], lo_i = s_d.lo[i];
            const int last_i = s_d.last[i];
            float row_sum = 0.f;
#pragma unroll
            for (int jt = 0; jt < 4; ++jt) {
                f32x4 w = {}, p = {}, e = {};
                if (16 * jt <= w16) {
                    // scores and dy . v, transposed: column i, rows j = 16 jt + g4 + r.
                    // Scores are made again for every head that shares them:
                    // registers are short.
                    f32x4 x = {}, score = {};
#pragma unroll
                    for (int kk = 0; kk < DK / 32; ++kk)
                        score = mma(frag_along(s_k + (16 * jt + l16) * PK + 32 * kk + 2 * g4),
                                    frag_along(s_q + i * PK + 32 * kk + 2 * g4), score);
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
                        p[r] = on ? score[r] * d : 0.f;
                        e[r] = on ? x[r] * d : 0.f;
                        w[r] = on && j < i ? p[r] * x[r] : 0.f;
                        row_sum += w[r];
                    }
                }
                f32x4 sums;
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    E pt[NP], et[NP];
                    split<E, NP>(p[r], pt);
                    split<E, NP>(e[r], et);
#pragma unroll
                    for (int m = 0; m < NP; ++m) {
                        fp[m][jt >> 1].v[4 * (jt & 1) + r] = pt[m];
                        fe[m][jt >> 1].v[4 * (jt & 1) + r] = et[m];
                    }
                    sums[r] = sum16(w[r]);
                }
                if (l16 == 0) *reinterpret_cast<f32x4*>(&s_col[wave][16 * jt + g4]) = sums;
                __builtin_amdgcn_sched_barrier(0);
            }
            row_sum += __shfl_xor(row_sum, 16);
            row_sum += __shfl_xor(row_sum, 32);
            if (g4 == 0) s_row[i] = row_sum;
        } else {
            const f32x4 out = *reinterpret_cast<const f32x4*>(&s_d.out[w16 + g4]);
#pragma unroll
            for (int c = 0; c < DK / 16; ++c) {
                f32x4 x = {};
#pragma unroll
                for (int kk = 0; kk < DV / 32; ++kk) {
                    const Frag<E> f = frag_along_split(s_v + i * PV + 32 * kk);
#pragma unroll
                    for (int m = 0; m < N; ++m)
                        x = mma(f, frag_across(s_t + (m * DV + 32 * kk) * PK + 16 * c, PK), x);
                }
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    x[r] = out[r] == 0.f ? 0.f : out[r] * x[r];
                    u[r] += x[r] * (float)s_k[(w16 + g4 + r) * PK + 16 * c + l16];
                    acc[c][r] += x[r];
                }
                if ((c & 3) == 3) __builtin_amdgcn_sched_barrier(0);
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
                        const Frag<E> f = frag_along(s_k + i * PK + 32 * kk + 2 * g4);
#pragma unroll
                        for (int m = 0; m < NS2; ++m)
                            x = mma(f, frag_along(s_t + (m * DV + 16 * b + l16) * PK + 32 * kk + 2 * g4), x);
                    }
#pragma unroll
                    for (int r = 0; r < 4; ++r) dv[b][r] = out[r] == 0.f ? 0.f : out[r] * x[r];
                    __builtin_amdgcn_sched_barrier(0);
                }
            }
        }
        __syncthreads();  // S has been used
        if (side == 0) {
#pragma unroll
            for (int m = 0; m < NP; ++m)
#pragma unroll
                for (int jt = 0; jt < 4; ++jt) {
                    const int at = (m * kC + i) * PC + 16 * jt + g4;
                    *reinterpret_cast<V4*>(&s_p[at]) = half_of(fp[m][jt >> 1], jt & 1);
                    *reinterpret_cast<V4*>(&s_e[at]) = half_of(fe[m][jt >> 1], jt & 1);
                }
        }
        __syncthreads();
        if (side == 0) {
#pragma unroll
            for (int c = 0; c < DK / 16; ++c) {
#pragma unroll
                for (int s = 0; s < 2; ++s)
                    if (32 * s <= w16) {
                        const Frag<E> f = frag_across(s_k + 32 * s * PK + 16 * c, PK);
#pragma unroll
                        for (int m = 0; m < NP; ++m) acc[c] = mma(fe[m][s], f, acc[c]);
                    }
                if ((c & 3) == 3) __builtin_amdgcn_sched_barrier(0);
            }
        } else {
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                if (32 * s + 16 < w16) continue;
                Frag<E> f[NP];
#pragma unroll
                for (int m = 0; m < NP; ++m) f[m] = frag_across(s_e + (m * kC + 32 * s) * PC + w16, PC);
#pragma unroll
                for (int c = 0; c < DK / 16; ++c) {
                    const Frag<E> fq = frag_across(s_q + 32 * s * PK + 16 * c, PK);
#pragma unroll
                    for (int m = 0; m < NP; ++m) acc[c] = mma(f[m], fq, acc[c]);
                    if ((c & 3) == 3) __builtin_amdgcn_sched_barrier(0);
                }
            }
            if (A.dval) {
#pragma unroll
                for (int s = 0; s < 2; ++s) {
                    if (32 * s + 16 < w16) continue;
                    Frag<E> f[NP];
#pragma unroll
                    for (int m = 0; m < NP; ++m) f[m] = frag_across(s_p + (m * kC + 32 * s) * PC + w16, PC);
#pragma unroll
                    for (int b = 0; b < DV / 16; ++b) {
                        const Frag<E> fd = frag_across(s_do + 32 * s * PV + 16 * b, PV);
#pragma unroll
                        for (int m = 0; m < NP; ++m) dv[b] = mma(f[m], fd, dv[b]);
                    }
                }
                const Out<T> ov = out_rows<T>(A.dval, A.lddv, A.part_v, in_hv * A.nkb + kb, A.n, A.hv * A.dv, t.row,
                                              hv * A.dv + v0);
                ov.template put_tiles<DV / 16>(w16 + g4, l16, rows, vcols, dv);
            }
        }
        __syncthreads();
        if (wave == 0) {
            float from = (s_row[lane] + s_a[lane]) - ((s_col[0][lane] + s_col[1][lane]) + (s_col[2][lane] + s_col[3][lane]));
            float to = s_b[lane];
            const float own = to;
            to = scan_up(to);
            from = __shfl(scan_up(__shfl(from, 63 - lane)), 63 - lane);  // from each row on
            float z = 0.f;
#pragma unroll
            for (int w = 0; w < 8; ++w) z += s_z[flip][w];
            const float whole = s_d.into[kC - 1];
            const float through = whole == 0.f ? 0.f : whole * z;
            // the last cut up to a row is the row itself: its decay has no gradient
            dg = (vb ? dg : 0.f) + (s_d.last[lane] == lane ? 0.f : from + (to - own) + through);
            if (A.dg && ends_head && lane < rows) out_g().put(lane, hl, dg);
        }
        if (!more) break;
        if (ends_head) {
            vb = 0;
            ++hl;
            in_hv = next_hv == hv ? in_hv + 1 : 0;
            hv = next_hv;
        } else {
            ++vb;
        }
    }
    if (side == 0 ? A.dq != nullptr : A.dkey != nullptr)
        (side == 0 ? out_q() : out_k()).template put_tiles<DK / 16>(w16 + g4, l16, rows, kcols, acc);
}

template <class T, class TG, int DK, int DV>
hipError_t grad_go(const AttendArgs& a, hipStream_t s)
{
    const int64_t groups = Ragged{a.offsets, a.seqs, a.n, a.seq_len}.units(kC) * (a.heads / a.loop) * a.nkb;
    const dim3 grid = grid_of<kGradThreads>(groups);
    if (a.dk % 8 == 0 && a.dv % 8 == 0)
        LX_LAUNCH("attend_grad", s, (lx_attend_grad<T, TG, DK, DV, true><<<grid, kGradThreads, 0, s>>>(a)));
    else
        LX_LAUNCH("attend_grad", s, (lx_attend_grad<T, TG, DK, DV, false><<<grid, kGradThreads, 0, s>>>(a)));
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
    b.nkb = attend_grad_blocks(a);
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

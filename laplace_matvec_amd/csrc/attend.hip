// Gated matrix memory: linear attention with a decay per head and row (gfx950).
//
//     S_t = e^{g_t} S_{t-1} + k_t v_t^T      (dk x dv, float32)
//     y_t = scale S_t^T q_t
//
// In chunks of 64 rows, with G_i the sum of g over the chunk's rows up to i,
//     y_i   = scale (e^{G_i} S^T q_i + sum_{j <= i} e^{G_i - G_j} (q_i . k_j) v_j)
//     S'    = e^{G_63} S + sum_j e^{G_63 - G_j} k_j v_j^T
// so all but the decays is products of matrices.  A workgroup takes one head's
// block of up to 128 x 64 of the state along a segment of a sequence, the
// state in registers in float32.  Segments of one sequence are independent
// but for their first states:
//     sweep kEnd    each segment's last state from a first one of 0
//     scan          the segments' first states, one after the other
//     sweep kOut    the outputs
// A segment is as short as it takes to fill the card (attend_segment); with
// one segment per sequence the first two are left out.
//
// 65536 rows of 16 heads of 128 x 128 bf16 in 518 us; under the profiler, at
// the least, kEnd 156 (keys and values once, 3.4 TB/s), scan 15, kOut 371 (1.07
// GB, 2.9 TB/s); a copy would take 212.  Bound by the latency of a chunk, 11.6
// us in kOut with two workgroups a CU: a third of the waves' time is waiting
// (four barriers), vector instructions (decays, terms) take 47 % of the SIMDs'
// cycles, matrix products 25 %.  Loads of the next chunk are on their way
// meanwhile, which only pays without branches (444 us against 624, with states
// and scores for y in one term).  One block of 128 columns per workgroup shares
// keys and scores: 518 us against 624 with 64.  In the backward pass kStore
// leaves 16 KB to 64 KB a chunk and head, as many bytes as the rows themselves
// or more: 165 to 185 us for 564 MB.
#include "lx_attend.h"

namespace lx {

namespace {

enum SweepMode { kEnd, kOut, kStore };

// REV runs the segments backwards with queries and output gradients in place
// of keys and values: the gradient of the states.
template <class T, class TG, int DK, int DV, int MODE, bool REV, bool WHOLE>
__global__ __launch_bounds__(kAttendThreads, MODE == kOut && DK == 128 && sizeof(typename Compute<T>::E) == 4 ? 1 : 2) void lx_attend_sweep(AttendArgs A)
{
    typedef typename Compute<T>::E E;
    constexpr int NU = sizeof(E) == 2 ? 3 : 1;  // terms of a row times its decay: all of its bits
    constexpr int TB = DV / 16;
    constexpr int PK = DK + kPad<E>, PV = DV + kPad<E>;
    constexpr int TA = DK / 64;  // 16-row tiles of the state per wave
    // Terms of scores and of the state in y.  Two planes of a state of 128 x
    // 128 leave no room for a second workgroup on the CU: the second plane then
    // shares its place with keys and values, which come after it.
    constexpr int NY = sizeof(E) == 2 ? 2 : 1;
    constexpr bool kShare = MODE == kOut && NY == 2 && DK == 128 && DV == 128;
    __shared__ alignas(16) E s_kv[kC * PK + kC * PV];
    __shared__ alignas(16) E s_s[MODE == kOut ? (kShare ? 1 : NY) * DV * PK : 1];  // the state, transposed
    static_assert(!kShare || DV * PK <= kC * PK + kC * PV, "room for a plane");
    E *const s_k = s_kv, *const s_v = s_kv + kC * PK;
    auto plane = [&](int m) { return kShare && m ? s_kv : s_s + m * (DV * PK); };
    __shared__ alignas(16) Decays s_d;
    __shared__ alignas(16) float s_f[kC];
    __shared__ int s_odd[4];
    __shared__ unsigned long long s_rows[DV];

    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int g4 = 4 * (lane >> 4), l16 = lane & 15;
    const int64_t id = group_id<kAttendThreads>();
    const int parts = A.heads * A.nkb * A.nvb;
    const int64_t unit = id / parts;
    const int part = (int)(id - unit * parts);
    const int h = part / (A.nkb * A.nvb), kb = part / A.nvb % A.nkb, vb = part % A.nvb;
    const Ragged R{A.offsets, A.seqs, A.n, A.seq_len};
    if (unit >= R.units(A.segment)) return;
    const RaggedTile t = R.find(unit, A.segment);
    if (t.rows <= 0) return;
    const int k0 = kb * DK, v0 = vb * DV;
    const int kcols = A.dk - k0, vcols = A.dv - v0;  // how many are there
    if (t.group < 0) {
        if (MODE != kOut) return;
        for (int64_t i = threadIdx.x; i < (int64_t)t.rows * DV; i += kAttendThreads) {
            const int64_t row = t.row + i / DV;
            const int c = (int)(i % DV);
            if (c >= vcols) continue;
            if (A.part)
                A.part[(kb * A.n + row) * ((int64_t)A.heads * A.dv) + h * A.dv + v0 + c] = 0.f;
            else
                ((T*)A.y)[row * A.ldy + h * A.dv + v0 + c] = (T)0.f;
        }
        return;
    }
    const bool is_first = t.index == 0, is_last = t.row + t.rows == t.end;
    if (MODE == kEnd && (REV ? is_first : is_last)) return;

    // the state: rows dk 16 (wave TA + a) + g4 + r, columns 16 b + l16
    f32x4 acc[TA][TB];
    // slot i of a sequence: the state between its segments i and i + 1 (the
    // gradient there); before and past the sequence they are the edges
    const int64_t slot = t.first / A.segment + t.index + (MODE == kEnd ? 0 : -1) + (REV ? (MODE == kEnd ? -1 : 1) : 0);
    float* seg_state = A.seg_states + (slot * A.heads + h) * ((int64_t)A.dkp * A.dvp) + tile_at(kb * (DK / 16), vb * TB, A.dvp) + 4 * lane;
    const float* edge = REV ? A.dfinal : A.h0;  // [seqs][heads][dk][dv]
    const bool at_edge = REV ? is_last : is_first;
    const int64_t edge_at = ((t.group * A.heads + h) * A.dk + k0) * (int64_t)A.dv + v0;
#pragma unroll
    for (int a = 0; a < TA; ++a)
#pragma unroll
        for (int b = 0; b < TB; ++b) {
            acc[a][b] = f32x4{};
            if (MODE == kEnd) continue;
            if (!at_edge) {
                acc[a][b] = *reinterpret_cast<const f32x4*>(seg_state + tile_at(wave * TA + a, b, A.dvp));
            } else if (edge) {
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const int row = 16 * (wave * TA + a) + g4 + r, col = 16 * b + l16;
                    if (row < kcols && col < vcols) acc[a][b][r] = edge[edge_at + (int64_t)row * A.dv + col];
                }
            }
        }

    const int64_t ldk = REV ? A.ldq : A.ldk, ldv = REV ? A.lddy : A.ldv;
    const T* kp = (const T*)(REV ? A.q : A.k) + h / (A.heads / (REV ? A.hq : A.hk)) * A.dk + k0;
    const T* vp = (const T*)(REV ? A.dy : A.v) + (REV ? h : h / (A.heads / A.hv)) * A.dv + v0;
    const T* qp = (const T*)A.q + h / (A.heads / A.hq) * A.dk + k0;
    const TG* gp = (const TG*)A.g + h;

    const int chunks = (t.rows + kC - 1) / kC;
    RowTile<T, DK, WHOLE> tk;
    RowTile<T, DV, WHOLE> tv;
    Pack<T, 8> tq[DK / 32];
    TG tg = (TG)0.f;
    auto fetch_q = [&](int ci) {
        const int c = REV ? chunks - 1 - ci : ci;
        const int64_t row = t.row + (int64_t)c * kC;
        const int rows = t.rows - c * kC < kC ? t.rows - c * kC : kC;
        const int i = 16 * wave + l16;
#pragma unroll
        for (int kk = 0; kk < DK / 32; ++kk)
            if (WHOLE) {
                const int at = i < rows ? i : rows - 1, col = 32 * kk + 2 * g4;
                tq[kk] = load8_whole(qp + (row + at) * A.ldq + (col < kcols ? col : kcols - 8));
            } else {
                tq[kk] = load8(qp + (row + i) * A.ldq + 32 * kk + 2 * g4, i < rows ? kcols - 32 * kk - 2 * g4 : 0);
            }
    };
    auto fetch = [&](int ci) {
        const int c = REV ? chunks - 1 - ci : ci;
        const int64_t row = t.row + (int64_t)c * kC;
        const int rows = t.rows - c * kC < kC ? t.rows - c * kC : kC;
        tk.load(kp + row * ldk, ldk, rows, kcols);
        tv.load(vp + row * ldv, ldv, rows, vcols);
        if (MODE == kOut && (!kShare || ci == 0)) fetch_q(ci);
        if (wave == 0) tg = gp[(row + (lane < rows ? lane : rows - 1)) * A.ldg];
    };
    fetch(0);
    float decay = 1.f;  // of the segment
    for (int ci = 0; ci < chunks; ++ci) {
        const int c = REV ? chunks - 1 - ci : ci;
        const int64_t row = t.row + (int64_t)c * kC;
        const int rows = t.rows - c * kC < kC ? t.rows - c * kC : kC;
        // Places worked out anew for each chunk where registers are short.
        int here = lane;
        if (kShare) asm volatile("" : "+v"(here));
        const int g4 = 4 * (here >> 4), l16 = here & 15;
        if (wave == 0) {
            s_d.make(lane < rows ? (float)tg : 0.f);
            s_f[lane] = REV ? s_d.into[lane] * A.scale : s_d.out[lane];
        }
        auto put_rows = [&] {
            tk.put(s_k, rows, kcols);
            tv.put(s_v, rows, vcols);
            const bool odd = __any(tv.odd());
            if (lane == 0) s_odd[wave] = odd;
        };
        if (!kShare) put_rows();
        Frag<E> fq[DK / 32];
        // what the wave's rows see of columns 16 b .. of the state
        auto see = [&](int b) {
            f32x4 o = {};
#pragma unroll
            for (int m = 0; m < NY; ++m)
#pragma unroll
                for (int kk = 0; kk < DK / 32; ++kk)
                    o = mma(fq[kk], frag_along(plane(m) + (16 * b + l16) * PK + 32 * kk + 2 * g4), o);
            return o;
        };
        f32x4 seen[kShare ? TB : 1];
        if (MODE == kOut) {
#pragma unroll
            for (int kk = 0; kk < DK / 32; ++kk) fq[kk] = to_frag<E>(tq[kk]);
            typedef E V4 __attribute__((ext_vector_type(4)));
#pragma unroll
            for (int a = 0; a < TA; ++a)
#pragma unroll
                for (int b = 0; b < TB; ++b) {
                    V4 w[NY];
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        E e[NY];
                        split<E, NY>(acc[a][b][r], e);
#pragma unroll
                        for (int m = 0; m < NY; ++m) w[m][r] = e[m];
                    }
#pragma unroll
                    for (int m = 0; m < NY; ++m)
                        *reinterpret_cast<V4*>(&plane(m)[(16 * b + l16) * PK + 16 * (wave * TA + a) + g4]) = w[m];
                }
        }
        if constexpr (kShare) {
            __syncthreads();
#pragma unroll
            for (int b = 0; b < TB; ++b) {
                seen[b] = see(b);
                if (b & 1) __builtin_amdgcn_sched_barrier(0);
            }
            __syncthreads();
            put_rows();
        }
        __syncthreads();
        // 0 times inf or NaN is not 0: rows that do not see such a value of v
        // must not multiply it.  It becomes 0 and a bit of its column, and what
        // does see it gets NaN.
        const bool odd = (s_odd[0] | s_odd[1] | s_odd[2] | s_odd[3]) != 0;
        if (odd) {
            if (threadIdx.x < DV) s_rows[threadIdx.x] = 0;
            __syncthreads();
            for (int i = threadIdx.x; i < kC * DV; i += kAttendThreads) {
                E* p = s_v + i / DV * PV + i % DV;
                if (!finite(*p)) {
                    atomicOr(&s_rows[i % DV], 1ull << (i / DV));
                    *p = (E)0.f;
                }
            }
            __syncthreads();
        }
        if (ci + 1 < chunks) fetch(ci + 1);
        const float whole = s_d.into[kC - 1];
        if (MODE == kEnd) decay = whole == 0.f ? 0.f : decay * whole;  // also after NaN
        if (MODE == kStore) {
            // slots between chunks, likewise
            const int64_t between = t.first / kC + (row - t.first) / kC - (REV ? 0 : 1);
            float* to = (REV ? A.chunk_grads : A.chunk_states) + (between * A.heads + h) * ((int64_t)A.dkp * A.dvp) +
                        tile_at(kb * (DK / 16) + wave * TA, vb * TB, A.dvp) + 4 * lane;
            if (REV ? row + kC < t.end : row > t.first) {
#pragma unroll
                for (int a = 0; a < TA; ++a)
#pragma unroll
                    for (int b = 0; b < TB; ++b)
                        *reinterpret_cast<f32x4*>(to + tile_at(a, b, A.dvp)) = acc[a][b];
            }
        }
        if (MODE == kOut) {
            const int i = 16 * wave + l16;
            const float hi_i = s_d.hi[i], lo_i = s_d.lo[i];
            const int last_i = s_d.last[i];
            Frag<E> fp[NY][2];
#pragma unroll
            for (int jt = 0; jt < 4; ++jt) {
                f32x4 p = {};
                if (jt <= wave) {
#pragma unroll
                    for (int kk = 0; kk < DK / 32; ++kk)
                        p = mma(frag_along(s_k + (16 * jt + l16) * PK + 32 * kk + 2 * g4), fq[kk], p);
                    const f32x4 hi = *reinterpret_cast<const f32x4*>(&s_d.hi[16 * jt + g4]);
                    const f32x4 lo = *reinterpret_cast<const f32x4*>(&s_d.lo[16 * jt + g4]);
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        const int j = 16 * jt + g4 + r;
                        const float x = p[r] * A.scale * s_d.between(hi_i, lo_i, hi[r], lo[r]);
                        p[r] = j <= i && j >= last_i ? x : 0.f;
                    }
                }
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    E e[NY];
                    split<E, NY>(p[r], e);
#pragma unroll
                    for (int m = 0; m < NY; ++m) fp[m][jt >> 1].v[4 * (jt & 1) + r] = e[m];
                }
                if (kShare) __builtin_amdgcn_sched_barrier(0);  // not more fragments at a time than registers
            }
            if (kShare && ci + 1 < chunks) fetch_q(ci + 1);  // in place of these, which are done with
            const f32x4 into = *reinterpret_cast<const f32x4*>(&s_d.into[16 * wave + g4]);
            T* yp = (T*)A.y + (row + 16 * wave + g4) * A.ldy + h * A.dv + v0 + l16;
#pragma unroll
            for (int b = 0; b < TB; ++b) {
                f32x4 o;
                if constexpr (kShare) o = seen[b];
                else o = see(b);
#pragma unroll
                for (int r = 0; r < 4; ++r) o[r] = into[r] == 0.f ? 0.f : o[r] * (into[r] * A.scale);
#pragma unroll
                for (int s = 0; s < 2; ++s)
                    if (2 * s <= wave) {
                        const Frag<E> f = frag_across(s_v + 32 * s * PV + 16 * b, PV);
#pragma unroll
                        for (int m = 0; m < NY; ++m) o = mma(fp[m][s], f, o);
                    }
                const int col = 16 * b + l16;
                if (odd) {
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        const int at = 16 * wave + g4 + r, from = s_d.last[at];
                        const unsigned long long seen = (2ull << at) - (1ull << (from < 0 ? 0 : from));
                        if (s_rows[col] & seen) o[r] = __builtin_nanf("");
                    }
                }
                if (rows == kC && vcols >= DV && !A.part) {
#pragma unroll
                    for (int r = 0; r < 4; ++r) yp[r * A.ldy + 16 * b] = (T)o[r];
                } else {
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        const int at = 16 * wave + g4 + r;
                        if (at < rows && col < vcols) {
                            if (A.part)
                                A.part[(kb * A.n + row + at) * ((int64_t)A.heads * A.dv) + h * A.dv + v0 + col] = o[r];
                            else
                                yp[r * A.ldy + 16 * b] = (T)o[r];
                        }
                    }
                }
            }
        }
        // S' = whole S + sum_j f_j k_j v_j^T
#pragma unroll
        for (int a = 0; a < TA; ++a)
#pragma unroll
            for (int b = 0; b < TB; ++b)
#pragma unroll
                for (int r = 0; r < 4; ++r) acc[a][b][r] = whole == 0.f ? 0.f : whole * acc[a][b][r];
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            Frag<E> fv[TB];
#pragma unroll
            for (int b = 0; b < TB; ++b) fv[b] = frag_across(s_v + 32 * s * PV + 16 * b, PV);
            const f32x4 f0 = *reinterpret_cast<const f32x4*>(&s_f[32 * s + g4]);
            const f32x4 f1 = *reinterpret_cast<const f32x4*>(&s_f[32 * s + 16 + g4]);
#pragma unroll
            for (int a = 0; a < TA; ++a) {
                const Frag<E> fk = frag_across(s_k + 32 * s * PK + 16 * (wave * TA + a), PK);
                Frag<E> fs[NU];
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float f = i < 4 ? f0[i] : f1[i - 4];
                    E e[NU];
                    split<E, NU>(f == 0.f ? 0.f : f * (float)fk.v[i], e);
#pragma unroll
                    for (int m = 0; m < NU; ++m) fs[m].v[i] = e[m];
                }
#pragma unroll
                for (int b = 0; b < TB; ++b)
#pragma unroll
                    for (int m = 0; m < NU; ++m) acc[a][b] = mma(fs[m], fv[b], acc[a][b]);
            }
        }
        if (odd) {
            const int from = s_d.last[kC - 1];
            const unsigned long long seen = REV ? s_d.sees_before() : 0ull - (1ull << (from < 0 ? 0 : from));
#pragma unroll
            for (int b = 0; b < TB; ++b)
                if (s_rows[16 * b + l16] & seen)
#pragma unroll
                    for (int a = 0; a < TA; ++a) acc[a][b] = f32x4{} + __builtin_nanf("");
        }
        __syncthreads();
    }
    if (MODE == kEnd && threadIdx.x == 0 && kb == 0 && vb == 0) A.seg_decays[slot * A.heads + h] = decay;
    float* end = MODE == kOut ? A.final : A.dh0;
    const bool write_edge = MODE != kEnd && end && (REV ? is_first : MODE == kOut && is_last);
    if (MODE == kEnd) {
#pragma unroll
        for (int a = 0; a < TA; ++a)
#pragma unroll
            for (int b = 0; b < TB; ++b)
                *reinterpret_cast<f32x4*>(seg_state + tile_at(wave * TA + a, b, A.dvp)) = acc[a][b];
    } else if (write_edge) {
#pragma unroll
        for (int a = 0; a < TA; ++a)
#pragma unroll
            for (int b = 0; b < TB; ++b)
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const int rr = 16 * (wave * TA + a) + g4 + r, col = 16 * b + l16;
                    if (rr < kcols && col < vcols) end[edge_at + (int64_t)rr * A.dv + col] = acc[a][b][r];
                }
    }
}

// States between the segments of a sequence (their gradients if REV), in
// place of what each segment alone makes of a state of 0.
template <bool REV>
__global__ __launch_bounds__(256) void lx_attend_scan(AttendArgs A)
{
    const int64_t block = (int64_t)A.dkp * A.dvp;
    const int64_t i = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4;  // of [heads][dkp][dvp]
    if (i >= A.heads * block) return;
    const int h = (int)(i / block), tile = (int)(i % block >> 8), lane = (int)(i & 255) >> 2;
    const int row = 16 * (tile / (A.dvp >> 4)) + 4 * (lane >> 4), col = 16 * (tile % (A.dvp >> 4)) + (lane & 15);
    const Ragged R{A.offsets, A.seqs, A.n, A.seq_len};
    const float* edge = REV ? A.dfinal : A.h0;
    for (int64_t q = blockIdx.y; q < A.seqs; q += gridDim.y) {
        const int64_t first = R.bound(q + 1), end = R.bound(q + 2);
        if (end - first <= A.segment) continue;
        const int64_t count = (end - first + A.segment - 1) / A.segment - 1;
        f32x4 s = {};
        if (edge && col < A.dv)
#pragma unroll
            for (int r = 0; r < 4; ++r)
                if (row + r < A.dk) s[r] = edge[((q * A.heads + h) * A.dk + row + r) * (int64_t)A.dv + col];
        // a slot is loaded while the one before it is worked out
        const int64_t slot0 = first / A.segment + (REV ? count - 1 : 0), step = REV ? -1 : 1;
        f32x4* p = reinterpret_cast<f32x4*>(A.seg_states + slot0 * A.heads * block + i);
        const float* d = A.seg_decays + slot0 * A.heads + h;
        f32x4 own = *p;
        float decay = *d;
        for (int64_t c = 0; c < count; ++c) {
            f32x4* at = p;
            const f32x4 x = own;
            const float a = decay;
            if (c + 1 < count) {
                p += step * A.heads * block / 4;
                d += step * A.heads;
                own = *p;
                decay = *d;
            }
#pragma unroll
            for (int r = 0; r < 4; ++r) s[r] = a == 0.f ? x[r] : a * s[r] + x[r];
            *at = s;
        }
    }
}

// States of sequences without rows stay.
__global__ __launch_bounds__(256) void lx_attend_empty(AttendArgs A, const float* from, float* to)
{
    const Ragged R{A.offsets, A.seqs, A.n, A.seq_len};
    const int64_t size = (int64_t)A.heads * A.dk * A.dv;
    for (int64_t q = blockIdx.y; q < A.seqs; q += gridDim.y) {
        if (R.bound(q + 2) > R.bound(q + 1)) continue;
        for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < size; i += (int64_t)gridDim.x * 256)
            to[q * size + i] = from ? from[q * size + i] : 0.f;
    }
}

// to[n][hx * d] = sum over `planes` of part[plane][n][hx * d], in their order.
template <class T>
__global__ __launch_bounds__(256) void lx_attend_sum(const float* part, int planes, int64_t n, int64_t width, T* to,
                                                     int64_t ld)
{
    const int64_t size = n * width;
    for (int64_t i = group_id<256>() * 256 + threadIdx.x; i < size; i += (int64_t)gridDim.x * gridDim.y * 256) {
        float s = part[i];
        for (int p = 1; p < planes; ++p) s += part[p * size + i];
        to[i / width * ld + i % width] = (T)s;
    }
}

// One token for each request.  A thread has V neighbouring columns of every
// 256 / (columns / V) -th row of a head's state, which is read and written
// once: 256 requests of 16 heads of 128 x 128, 537 MB, in 106 us, 5.1 TB/s.  A
// few requests take the launch (3 of 8 heads of 64 x 64: 5.4 us of kernel).
template <class T, class TG, int V>
__global__ __launch_bounds__(256) void lx_attend_step(AttendStepArgs A)
{
    __shared__ float s_sum[256 * V];
    const int64_t id = group_id<256>();
    const int64_t b = id / A.heads;
    if (b >= A.n) return;
    const int h = (int)(id - b * A.heads);
    const int64_t slot = A.slots ? (int64_t)A.slots[b] : b;
    T* y = (T*)A.y + b * A.ldy + (int64_t)h * A.dv;
    const T* v = (const T*)A.v + b * A.ldv + h / (A.heads / A.hv) * A.dv;
    const bool has = slot >= 0 && slot < A.pool;
    const T* q = (const T*)A.q + b * A.ldq + h / (A.heads / A.hq) * A.dk;
    const T* k = (const T*)A.k + b * A.ldk + h / (A.heads / A.hk) * A.dk;
    const float g = has ? (float)((const TG*)A.g)[b * A.ldg + h] : 0.f;
    const float a = is_cut(g) ? 0.f : exp2_whole((double)g * kLog2e);
    float* state = A.state + (has ? slot * A.heads + h : 0) * (int64_t)A.dk * A.dv;
    // column groups of the row, at most 64 at a time
    const int groups = (A.dv + V - 1) / V;
    const int wide = groups < 64 ? groups : 64;
    const int lines = 256 / wide;
    const int line = threadIdx.x / wide, at = threadIdx.x % wide;
    for (int c0 = 0; c0 < groups; c0 += wide) {
        const int col = (c0 + at) * V;
        const bool here = line < lines && col < A.dv;
        float sum[V] = {};
        if (here && has) {
            float vv[V];
            load_vec<V>(v + col, vv);
            for (int r = line; r < A.dk; r += lines) {
                float* p = state + (int64_t)r * A.dv + col;
                float s[V];
                load_vec<V>(p, s);
                const float kr = (float)k[r], qr = (float)q[r];
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    s[i] = (a == 0.f ? 0.f : a * s[i]) + kr * vv[i];
                    sum[i] += qr * s[i];
                }
                store_vec<V>(p, s);
            }
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < V; ++i) s_sum[threadIdx.x * V + i] = sum[i];
        __syncthreads();
        for (int c = threadIdx.x; c < wide * V; c += 256) {
            float s = 0.f;
            for (int l = 0; l < lines; ++l) s += s_sum[l * wide * V + c];
            if (c0 * V + c < A.dv) y[c0 * V + c] = (T)(s * A.scale);
        }
    }
}

template <class T, class TG, int DK, int DV, int MODE, bool REV>
hipError_t sweep_launch(const AttendArgs& a, const char* label, hipStream_t s)
{
    const int64_t groups = Ragged{a.offsets, a.seqs, a.n, a.seq_len}.units(a.segment) * a.heads * a.nkb * a.nvb;
    const dim3 grid = grid_of<kAttendThreads>(groups);
    if (a.dk % 8 == 0 && a.dv % 8 == 0)
        LX_LAUNCH(label, s, (lx_attend_sweep<T, TG, DK, DV, MODE, REV, true><<<grid, kAttendThreads, 0, s>>>(a)));
    else
        LX_LAUNCH(label, s, (lx_attend_sweep<T, TG, DK, DV, MODE, REV, false><<<grid, kAttendThreads, 0, s>>>(a)));
    return hipSuccess;
}

// With 16-bit products two blocks of columns in one workgroup, which share
// its keys, queries and scores.
template <class T, class TG, int DK, int MODE, bool REV>
hipError_t sweep_go(AttendArgs a, const char* label, hipStream_t s)
{
    if constexpr (sizeof(typename Compute<T>::E) == 2) {
        if (a.nvb % 2 == 0) {
            a.nvb /= 2;
            return sweep_launch<T, TG, DK, 128, MODE, REV>(a, label, s);
        }
    }
    return sweep_launch<T, TG, DK, 64, MODE, REV>(a, label, s);
}

template <bool REV>
hipError_t scan_go(const AttendArgs& a, hipStream_t s)
{
    const int64_t groups = ((int64_t)a.heads * a.dkp * a.dvp + 1023) / 1024;
    const unsigned seqs = (unsigned)(a.seqs < 1024 ? a.seqs : 1024);
    LX_LAUNCH("attend_scan", s, (lx_attend_scan<REV><<<dim3((unsigned)groups, seqs), 256, 0, s>>>(a)));
    return hipSuccess;
}

hipError_t empty_go(const AttendArgs& a, const float* from, float* to, hipStream_t s)
{
    if (!to || (!a.offsets && a.n > 0)) return hipSuccess;
    const int64_t size = ((int64_t)a.heads * a.dk * a.dv + 1023) / 1024;
    const dim3 grid((unsigned)(size < 256 ? size : 256), (unsigned)(a.seqs < 1024 ? a.seqs : 1024));
    LX_LAUNCH("attend_empty", s, (lx_attend_empty<<<grid, 256, 0, s>>>(a, from, to)));
    return hipSuccess;
}

template <class T, class TG, int DK>
hipError_t forward_dk(const AttendArgs& a, hipStream_t s)
{
    hipError_t e = empty_go(a, a.h0, a.final, s);
    if (e != hipSuccess || a.n == 0) return e;
    if (attend_may_split(a)) {
        if ((e = sweep_go<T, TG, DK, kEnd, false>(a, "attend_end", s)) != hipSuccess) return e;
        if ((e = scan_go<false>(a, s)) != hipSuccess) return e;
    }
    if ((e = sweep_go<T, TG, DK, kOut, false>(a, "attend_out", s)) != hipSuccess) return e;
    if (a.part) return attend_sum_launch(a.part, a.nkb, a.n, (int64_t)a.heads * a.dv, a.y, a.ldy, (int)(sizeof(T) == 4 ? 0 : __is_same(T, bf16_t) ? 1 : 2), s);
    return hipSuccess;
}

template <class T, class TG, int DK>
hipError_t states_dk(const AttendArgs& a, hipStream_t s)
{
    hipError_t e = empty_go(a, a.dfinal, a.dh0, s);
    if (e != hipSuccess || a.n == 0) return e;
    if ((e = sweep_go<T, TG, DK, kStore, false>(a, "attend_states", s)) != hipSuccess) return e;
    AttendArgs b = a;
    b.seg_states = a.seg_grads;
    if (attend_may_split(a)) {
        if ((e = sweep_go<T, TG, DK, kEnd, true>(b, "attend_end_back", s)) != hipSuccess) return e;
        if ((e = scan_go<true>(b, s)) != hipSuccess) return e;
    }
    return sweep_go<T, TG, DK, kStore, true>(b, "attend_states_back", s);
}

template <class T, class TG>
hipError_t step_go(const AttendStepArgs& a, hipStream_t s)
{
    const int64_t groups = a.n * a.heads;
    if (a.dv % 4 == 0)
        LX_LAUNCH("attend_step", s, (lx_attend_step<T, TG, 4><<<grid_of<256>(groups), 256, 0, s>>>(a)));
    else
        LX_LAUNCH("attend_step", s, (lx_attend_step<T, TG, 1><<<grid_of<256>(groups), 256, 0, s>>>(a)));
    return hipSuccess;
}

}  // namespace

hipError_t attend_sum_launch(const float* part, int planes, int64_t n, int64_t width, void* to, int64_t ld, int dtype,
                             hipStream_t s)
{
    const int64_t want = (n * width + 255) / 256;
    const dim3 grid((unsigned)(want < 65536 ? want : 65536));
    switch (dtype) {
        case 0: LX_LAUNCH("attend_sum", s, (lx_attend_sum<float><<<grid, 256, 0, s>>>(part, planes, n, width, (float*)to, ld))); break;
        case 1: LX_LAUNCH("attend_sum", s, (lx_attend_sum<bf16_t><<<grid, 256, 0, s>>>(part, planes, n, width, (bf16_t*)to, ld))); break;
        case 2: LX_LAUNCH("attend_sum", s, (lx_attend_sum<f16_t><<<grid, 256, 0, s>>>(part, planes, n, width, (f16_t*)to, ld))); break;
        default: return hipErrorInvalidValue;
    }
    return hipSuccess;
}

#define LX_BY_DK(call, a, T, TG) return a.block_k == 64 ? call<T, TG, 64>(a, s) : call<T, TG, 128>(a, s)
#define LX_BY_TYPE(call, a)                                                                  \
    switch (dtype) {                                                                         \
        case 0: LX_BY_DK(call, a, float, float);                                             \
        case 1: if (gtype) LX_BY_DK(call, a, bf16_t, bf16_t); else LX_BY_DK(call, a, bf16_t, float); \
        case 2: if (gtype) LX_BY_DK(call, a, f16_t, f16_t); else LX_BY_DK(call, a, f16_t, float);    \
        default: return hipErrorInvalidValue;                                                \
    }

hipError_t attend_launch(const AttendArgs& a, int dtype, int gtype, hipStream_t s) { LX_BY_TYPE(forward_dk, a) }

hipError_t attend_states_launch(const AttendArgs& a, int dtype, int gtype, hipStream_t s) { LX_BY_TYPE(states_dk, a) }

hipError_t attend_step_launch(const AttendStepArgs& a, int dtype, int gtype, hipStream_t s)
{
    switch (dtype) {
        case 0: return step_go<float, float>(a, s);
        case 1: return gtype ? step_go<bf16_t, bf16_t>(a, s) : step_go<bf16_t, float>(a, s);
        case 2: return gtype ? step_go<f16_t, f16_t>(a, s) : step_go<f16_t, float>(a, s);
        default: return hipErrorInvalidValue;
    }
}

}  // namespace lx

// Device parts shared by the gated recurrence and its backward pass.
//
// Along the rows (tokens) of one sequence, for every channel,
//     h_t = a_t h_{t-1} + x_t,   a_t = exp(g_t),
// the causal half of the operator's scan with its decays given per token: an
// affine map per row, composed along rows.  Rows are cut into tiles of
// kRecurTile rows by kRecurCols channels, one workgroup each.  A thread has V
// neighbouring channels of L consecutive rows in registers, as stored (half
// types stay packed, so more rows are in flight per register); the threads of
// a row group cover the tile's channels, the row groups its rows.
// A decay of exactly zero forgets the state, whatever it held (inf and NaN
// too): 0 * h is never formed.  The first row of a sequence is such a row,
// with a h0 added to x, so one form serves packed and single sequences.
// States, decays and sums are float32.
#pragma once
#include "lx_device.h"
#include "lx_internal.h"
#include "lx_types.h"

namespace lx {

template <int V, int L>
struct RecurLayout {
    static constexpr int kLanes = kRecurCols / V;         // threads per row
    static constexpr int kGroups = kRecurTile / L;        // row groups
    static constexpr int kThreads = kLanes * kGroups;
};

// Products of decays leave float32's range where the states that they act on
// do not: e^-112 times 1e30 is no 0, an infinite state stays infinite under
// any decay but 0, e^100 times 1e-20 is no infinity and 0 times any growth is
// 0.  So a product that may is held as its square root r and applied as
// r (r h).  Below 2^-298 r is kRootLeast: r (r h) is 0 for any finite h, but
// inf and NaN stay.  Above 2^256 it is kRootMost, which makes any h above
// 2^-127 infinite.  Such a product stays there, as a state would that it acted
// on.  0 forgets.
// A wave whose decays are ordinary has its plain products: roots for all cost
// precision (4 sequences of 2048 float32 rows, relative error of y 1.6e-6 ->
// 1.9e-6, final states of 777 short rows 5.6e-7 -> 9.2e-7).  A product with an
// exponent of its own, in two words, cost up to 15 % of a pass.
constexpr float kRootLeast = 0x1p-149f, kRootMost = 0x1.fffffep127f;

// Root of a decay e^g, which below the smallest float32 is 0 and from 2^256 on
// infinite.
__device__ __forceinline__ float root_of(float g)
{
    const float p = g * (0.5f * 1.44269504088896341f);
    return p <= -75.f ? 0.f : __builtin_amdgcn_exp2f(p);
}

// r h, 0 where r is 0, whatever h is
__device__ __forceinline__ float half_decayed(float r, float h) { return r == 0.f ? 0.f : r * h; }
__device__ __forceinline__ float decayed(float r, float h) { return r * half_decayed(r, h); }
// a h + x from the root of a
__device__ __forceinline__ float step_of(float r, float h, float x) { return fmaf(r, half_decayed(r, h), x); }

// a h + x for an ordinary product of decays or 0
__device__ __forceinline__ float ordinary_step(float a, float h, float x) { return a == 0.f ? x : fmaf(a, h, x); }

__device__ __forceinline__ float root_within(float r) { return r < kRootLeast ? kRootLeast : r > kRootMost ? kRootMost : r; }

// The root of a product of decays, from their roots, row by row.
struct RowsProduct {
    float m = 1.f;
    bool zero = false;

    __device__ __forceinline__ void times(float r)
    {
        zero |= r == 0.f;
        m *= r;
    }
    __device__ __forceinline__ float root() const { return zero ? 0.f : root_within(m); }
};
// The same from products over some rows, ordinary ones as they are or roots,
// as m 2^e.  A root that left its range stays out.
struct GroupsProduct {
    float m = 1.f, least = 1.f, most = 1.f;
    int e = 0;

    __device__ __forceinline__ void ordinary(float a)
    {
        least = fminf(least, a);
        m *= __builtin_amdgcn_frexp_mantf(a);
        e += __builtin_amdgcn_frexp_expf(a);
    }
    __device__ __forceinline__ void root(float r)
    {
        least = fminf(least, r);
        most = fmaxf(most, r);
        const float f = __builtin_amdgcn_frexp_mantf(r);
        m *= f * f;
        e += 2 * __builtin_amdgcn_frexp_expf(r) + __builtin_amdgcn_frexp_expf(m);
        m = __builtin_amdgcn_frexp_mantf(m);
    }
    __device__ __forceinline__ float root() const
    {
        const float r = root_within(ldexpf(__builtin_amdgcn_sqrtf(e & 1 ? 2.f * m : m), e >> 1));
        return least == 0.f ? 0.f : least == kRootLeast ? kRootLeast : most == kRootMost ? kRootMost : r;
    }
};

// A condition that is the same in every lane, as a scalar: a branch on it is
// then one for the whole wave, and neither side keeps the other's registers.
__device__ __forceinline__ bool uniform(bool c) { return __builtin_amdgcn_readfirstlane((int)c) != 0; }

// What is special about a tile's rows.
struct RecurRows {
    int start[kRecurTile];  // sequence whose first row this is; -1: none; -2: a row of no sequence
    int last[kRecurTile];   // sequence whose last row this is; -1: none
    uint64_t odd[kRecurTile / kWave];  // bit per row: either of them is not -1
};

// Packed sequences: the first offset at or past a tile's first row, or -1 if
// the tile has no special rows.  Made for all tiles before the pass (a search
// in the pass would wait behind its row loads); a single tile starts at 0.
__device__ __forceinline__ int tile_mark(const RecurArgs& A, int64_t tile)
{
    return !A.offsets || A.tiles <= 1 ? 0 : A.marks[tile];
}

// Whether the tile of rows [t0, t0 + kRecurTile) has special rows; then R
// says which.  All threads; has barriers only if it returns true.
// `mark` is the tile's of tile_mark().
template <int THREADS>
__device__ __forceinline__ bool recur_rows(const RecurArgs& A, int64_t t0, int mark, RecurRows& R)
{
    static_assert(THREADS >= kRecurTile, "a thread per row");
    const int64_t end = t0 + kRecurTile;
    if (A.offsets) {
        if (mark < 0) return false;
    } else {
        const int64_t at = A.seqs == 1 ? t0 : t0 % A.seq_len;
        if (end <= A.n && at != 0 && at + kRecurTile < A.seq_len) return false;
    }
    const int tid = threadIdx.x;
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
    if (A.offsets) {
        // one wave: the offsets in [t0, end], 64 at a time
        for (int64_t q0 = mark; tid < kWave && q0 <= A.seqs; q0 += kWave) {
            const int64_t q = q0 + tid;
            const int64_t o = q <= A.seqs ? (int64_t)A.offsets[q] : end + 1;
            if (o >= t0 && o <= end) {
                // the last of several equal offsets starts the one sequence that is not empty
                if (q < A.seqs && o < end && (int64_t)A.offsets[q + 1] > o) R.start[o - t0] = (int)q;
                if (q > 0 && o > t0 && (int64_t)A.offsets[q - 1] < o) R.last[o - 1 - t0] = (int)(q - 1);
            }
            if (__ballot(o > end)) break;
        }
        __syncthreads();
    }
    if (tid < kRecurTile) {
        const uint64_t odd = __ballot(R.start[tid] != -1 || R.last[tid] != -1);
        if (tid % kWave == 0) R.odd[tid / kWave] = odd;
    }
    __syncthreads();
    return true;
}

// Where a thread's rows of one array are: a base that is the same for the
// wave (row j is j pitches further, in scalar registers) and a 32-bit offset
// of the lane, so that an address takes one vector register for all rows.
// A wave spans at most 64 rows of one array; a pitch of at most 2^24 values
// (kRecurMaxPitch, see recur_pitch) keeps the offset within 32 bits.
template <class T, int V>
struct RowAt {
    char* base;
    int64_t pitch;  // bytes
    uint32_t off;

    // wave_row: the wave's first row; lane_row: the lane's, from there; col:
    // the lane's
    __host__ __device__ __forceinline__ RowAt(const void* p, int64_t ld, int64_t wave_row, int lane_row, int col)
        : base((char*)p + wave_row * ld * (int64_t)sizeof(T)),
          pitch(ld * (int64_t)sizeof(T)),
          off(((uint32_t)lane_row * (uint32_t)ld + (uint32_t)col) * (uint32_t)sizeof(T))
    {
    }
    __device__ __forceinline__ T* row(int j) const
    {
        int64_t o = j * pitch;
        asm volatile("" : "+s"(o));  // stays in scalar registers, apart from the lane's offset
        return reinterpret_cast<T*>(base + o + off);
    }
    __host__ __device__ __forceinline__ T* any_row(int64_t j) const { return reinterpret_cast<T*>(base + j * pitch + off); }
};

// L rows of V channels of one array as stored (a vector of 16-bit values
// would be taken apart into a register for each).
template <class T, int V, int L>
struct RowPack {
    static constexpr int kBytes = V * (int)sizeof(T);
    typedef MemOf<T, V> Mem;
    typedef typename Words<kBytes == 2 ? 4 : kBytes>::T Reg;  // a register tuple as it is loaded
    Reg w[L];

    // whole: all of the tile's rows are there; else the last one (`last`
    // from the thread's first, perhaps before it) stands for those past it
    __device__ __forceinline__ void load(const RowAt<T, V>& at, bool whole, int64_t last, bool once)
    {
        if (whole && once) {
#pragma unroll
            for (int j = 0; j < L; ++j) w[j] = __builtin_nontemporal_load(reinterpret_cast<const Mem*>(at.row(j)));
        } else if (whole) {
#pragma unroll
            for (int j = 0; j < L; ++j) w[j] = *reinterpret_cast<const Mem*>(at.row(j));
        } else {
#pragma unroll
            for (int j = 0; j < L; ++j) w[j] = *reinterpret_cast<const Mem*>(at.any_row(j < last ? j : last));
        }
    }
    __device__ __forceinline__ void clear()
    {
#pragma unroll
        for (int j = 0; j < L; ++j) w[j] = Reg(0);
    }
    // Row j in float32.  The copy hides that every call gives the same: the
    // compiler would hold all converted values (and all exponentials) in
    // registers from their first use to their last instead of the rows.
    __device__ __forceinline__ void get(int j, float (&out)[V]) const
    {
        Reg t = w[j];
        asm volatile("" : "+v"(t));
#pragma unroll
        for (int v = 0; v < V; ++v) {
            uint32_t q;
            if constexpr (kBytes <= 4) q = t;
            else q = t[v * (int)sizeof(T) / 4];
            if constexpr (sizeof(T) == 4) {
                out[v] = __uint_as_float(q);
            } else if constexpr (__is_same(T, bf16_t)) {
                out[v] = __uint_as_float(v & 1 ? q & 0xFFFF0000u : q << 16);
            } else {
                out[v] = (float)__builtin_bit_cast(f16_t, (uint16_t)(v & 1 ? q >> 16 : q));
            }
        }
    }
};

// Has these values worked out here, not where they are used.
template <int N>
__device__ __forceinline__ void settle(float (&v)[N])
{
#pragma unroll
    for (int i = 0; i < N; ++i) asm volatile("" : "+v"(v[i]));
}

// How a wave goes through its rows: kCareNone if its decays and their
// products are ordinary float32 values, which shows when they are composed;
// kCareRows if it has special rows too: first rows take h0 in and forget
// what came before, rows of no sequence are 0; kCareRoot and kCareBoth, the
// same with roots, if a decay is 0 or a product out of range.  kCareGone: all
// of the wave's rows are past the last one, nothing is read or written.
enum { kCareNone = 0, kCareRows = 1, kCareRoot = 2, kCareBoth = 3, kCareGone = 4 };
constexpr bool care_rows(int care) { return care == kCareRows || care == kCareBoth; }
constexpr bool care_root(int care) { return care == kCareRoot || care == kCareBoth; }

// Products of a thread's decays, row by row; `cut`: the row forgets what came
// before.  The wave needs roots unless every product of neighbouring rows'
// decays (cuts apart) was an ordinary value: with no decay above 4 none of at
// most 16 exceeds 2^32, and if that of all is at least 2^-94, no part of it is
// below 2^-126.  (A decay of NaN makes the product NaN.)
template <bool ROOT, int D, int L>
struct RecurProducts {
    static_assert(L <= 16, "2^-94 and 4 hold for 16 rows");
    float m[D], most = 0.f;
    bool zero = false;

    __device__ __forceinline__ RecurProducts()
    {
#pragma unroll
        for (int d = 0; d < D; ++d) m[d] = 1.f;
    }
    __device__ __forceinline__ void row(const float (&a)[D], bool cut)
    {
#pragma unroll
        for (int d = 0; d < D; ++d) {
            const float f = cut ? 1.f : a[d];
            m[d] *= f;
            most = fmaxf(most, f);
        }
        zero |= cut;
        settle(m);
        asm volatile("" : "+v"(most));
    }
    // W + (product so far) x
    __device__ __forceinline__ float add(int d, float x, float W) const { return zero ? W : fmaf(m[d], x, W); }
    // The whole products; false if they are of no use.
    __device__ __forceinline__ bool whole(float (&r)[D]) const
    {
        bool out = !(most <= 4.f);
#pragma unroll
        for (int d = 0; d < D; ++d) {
            out |= !(m[d] >= 0x1p-94f);
            r[d] = zero ? 0.f : m[d];
        }
        return !uniform(__any(out));
    }
};
// From roots, which are 0 where they cut.
template <int D, int L>
struct RecurProducts<true, D, L> {
    RowsProduct p[D];

    __device__ __forceinline__ void row(const float (&a)[D], bool)
    {
#pragma unroll
        for (int d = 0; d < D; ++d) {
            p[d].times(a[d]);
            asm volatile("" : "+v"(p[d].m));
        }
    }
    __device__ __forceinline__ float add(int d, float x, float W) const { return step_of(p[d].root(), x, W); }
    __device__ __forceinline__ bool whole(float (&r)[D]) const
    {
#pragma unroll
        for (int d = 0; d < D; ++d) r[d] = p[d].root();
        return true;
    }
};

// A thread's rows of x and g.  SH: one decay serves the V channels.
template <class T, class TG, int V, int LL, bool SH>
struct RecurThread {
    static constexpr int L = LL;
    static constexpr int D = SH ? 1 : V;
    RowPack<T, V, L> x;
    RowPack<TG, D, L> g;
    int64_t wave_row;     // the wave's first row
    int tile_col;         // the tile's first channel
    int first_col;        // the thread's
    int lane_row;         // the thread's first row, from the wave's
    int r0;               // the same, from the tile's
    int lane, group;      // thread of the row, row group
    int rows;             // of the thread's L: those that exist and are inside the width
    bool in;              // channels inside the width
    bool whole;           // all rows of the tile exist
    int64_t last;         // the array's last row, from the thread's first
    uint32_t odd;         // special rows

    __device__ __forceinline__ void load(const RecurArgs& A, int64_t tile, int ct)
    {
        using Lay = RecurLayout<V, L>;
        const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x / kWave);
        const int wave_r0 = wave * (kWave / Lay::kLanes) * L;
        lane = (int)threadIdx.x % Lay::kLanes;
        group = (int)threadIdx.x / Lay::kLanes;
        lane_row = lane_id() / Lay::kLanes * L;
        r0 = wave_r0 + lane_row;
        wave_row = tile * kRecurTile + wave_r0;
        tile_col = ct * kRecurCols;
        // the last group of a row that V does not divide takes the row's last
        // V channels: what two groups have is worked out twice, alike, and
        // written twice; lanes past the width do the same and write nothing
        const int c = tile_col + lane * V;
        in = c < A.width;
        first_col = c < A.width - V ? c : A.width - V;
        whole = (tile + 1) * kRecurTile <= A.n;
        last = A.n - 1 - wave_row - lane_row;
        rows = !in || last < 0 ? 0 : (last < L - 1 ? (int)last + 1 : L);
        if (gone(A)) {
            x.clear();
            g.clear();
            return;
        }
        x.load(at<T, V>(A.x, A.ldx), whole, last, A.stream);
        g.load(gate_at<TG>(A, A.g, A.ldg), whole, last, A.stream && !SH);  // a shared decay is read by many tiles
    }
    __device__ __forceinline__ bool gone(const RecurArgs& A) const { return wave_row >= A.n; }
    __device__ __forceinline__ int col() const { return first_col; }
    template <class U, int N>
    __device__ __forceinline__ RowAt<U, N> at(const void* p, int64_t ld) const
    {
        return RowAt<U, N>(p, ld, wave_row, lane_row, col());
    }
    // g or dg
    template <class U>
    __device__ __forceinline__ RowAt<U, D> gate_at(const RecurArgs& A, const void* p, int64_t ld) const
    {
        return RowAt<U, D>(p, ld, wave_row, lane_row, SH ? col() / A.per : col());
    }
    // The thread's special rows, a bit each; the care its wave takes, as far as known.
    __device__ __forceinline__ int find_odd(const RecurArgs& A, const RecurRows* R)
    {
        static_assert(L <= 32 && kWave % L == 0, "a thread's rows lie in one word");
        odd = R ? (uint32_t)(R->odd[r0 / kWave] >> (r0 % kWave)) & (uint32_t)((1ull << L) - 1) : 0u;
        return gone(A) ? kCareGone : uniform(__any(odd != 0)) ? kCareRows : kCareNone;
    }
    template <int CARE>
    __device__ __forceinline__ bool special(int j) const
    {
        return care_rows(CARE) && (odd >> j & 1u);
    }
    // Row j: its decays or their roots, and h -> a h + x.
    // Returns whether the row forgets what came before; a root is 0 then.
    template <int CARE>
    __device__ __forceinline__ bool decays(const RecurRows* R, int j, float (&a)[D]) const
    {
        const bool cut = special<CARE>(j) && R->start[r0 + j] != -1;
        g.get(j, a);
#pragma unroll
        for (int d = 0; d < D; ++d) {
            if (care_root(CARE)) a[d] = cut ? 0.f : root_of(a[d]);
            else a[d] = __builtin_amdgcn_exp2f(a[d] * 1.44269504088896341f);
        }
        return cut;
    }
    template <int CARE>
    __device__ __forceinline__ void step(const RecurArgs& A, const RecurRows* R, int j, const float (&a)[D], bool cut,
                                         float (&h)[V]) const
    {
        float t[V];
        x.get(j, t);
        if (special<CARE>(j)) {
            const int q = R->start[r0 + j];
            if (q == -2) {
#pragma unroll
                for (int v = 0; v < V; ++v) t[v] = 0.f;
            } else if (q >= 0 && A.h0 && in) {
                float h0[V], b[D];
                load_vec<V>(A.h0 + (int64_t)q * A.width + col(), h0);
                g.get(j, b);
#pragma unroll
                for (int v = 0; v < V; ++v) t[v] = step_of(root_of(b[SH ? 0 : v]), h0[v], t[v]);
            }
        }
#pragma unroll
        for (int v = 0; v < V; ++v) {
            if (care_root(CARE)) h[v] = step_of(a[SH ? 0 : v], h[v], t[v]);
            else h[v] = cut ? t[v] : fmaf(a[SH ? 0 : v], h[v], t[v]);
        }
        settle(h);
    }
    // Composed map of the thread's rows: h -> r h + H, from roots
    // h -> r (r h) + H.  False if the wave needs roots and had none.
    template <int CARE>
    __device__ __forceinline__ bool compose(const RecurArgs& A, const RecurRows* R, float (&r)[D], float (&H)[V]) const
    {
        RecurProducts<care_root(CARE), D, L> m;
#pragma unroll
        for (int v = 0; v < V; ++v) H[v] = 0.f;
#pragma unroll
        for (int j = 0; j < L; ++j) {
            float a[D];
            const bool cut = decays<CARE>(R, j, a);
            step<CARE>(A, R, j, a, cut, H);
            m.row(a, cut);
        }
        return m.whole(r);
    }
};

// The decays of a tile's row groups: ordinary products, or roots from waves
// that took them.
template <int V, int L, bool SH>
struct RecurGroups {
    using Lay = RecurLayout<V, L>;
    static constexpr int kWaves = Lay::kThreads / kWave;
    static constexpr int kOf = Lay::kGroups / kWaves;  // groups of a wave
    static constexpr int kDecays = Lay::kLanes * (SH ? 1 : V);
    static constexpr int kRun = 4;  // groups whose loads are in flight together, with roots among them
    static_assert(kRun % kOf == 0 && Lay::kGroups % kRun == 0, "whole waves");
    float a[Lay::kGroups][kDecays];
    int roots[kWaves];

    template <int D>
    __device__ __forceinline__ void put(int group, int lane, int care, const float (&r)[D])
    {
#pragma unroll
        for (int d = 0; d < D; ++d) a[group][lane * D + d] = r[d];
        if (lane_id() == 0) roots[threadIdx.x / kWave] = care_root(care);
    }
    // A bit for each wave that took roots.
    __device__ __forceinline__ uint32_t rooted() const
    {
        return (uint32_t)__ballot(lane_id() < kWaves && roots[lane_id() % kWaves] != 0);
    }
    // Goes through the groups in row order, or (BACK) against it, with a
    // group's number, decay and what s has of it, for ordinary decays and for
    // roots.  One wave, a channel per lane.  A tile without roots has a loop
    // of its own: one form for both made every group wait longer (packed
    // training 333 -> 339 us).
    template <bool BACK, class Ordinary, class Root>
    __device__ __forceinline__ void each(uint32_t waves, const float (*s)[kRecurCols], Ordinary ordinary, Root root) const
    {
        const int c = lane_id(), d = SH ? c / V : c;
        if (waves == 0) {
#pragma unroll 8
            for (int k = 0; k < Lay::kGroups; ++k) {
                const int i = BACK ? Lay::kGroups - 1 - k : k;
                ordinary(i, a[i][d], s[i][c]);
            }
            return;
        }
#pragma unroll 1
        for (int k0 = 0; k0 < Lay::kGroups; k0 += kRun) {
            float r[kRun], x[kRun];
#pragma unroll
            for (int k = 0; k < kRun; ++k) {
                const int i = BACK ? Lay::kGroups - 1 - k0 - k : k0 + k;
                r[k] = a[i][d];
                x[k] = s[i][c];
            }
#pragma unroll
            for (int k = 0; k < kRun; k += kOf) {
                const int i = BACK ? Lay::kGroups - 1 - k0 - k : k0 + k;
                if (waves >> (i / kOf) & 1u) {
#pragma unroll
                    for (int j = 0; j < kOf; ++j) root(BACK ? i - j : i + j, r[k + j], x[k + j]);
                } else {
#pragma unroll
                    for (int j = 0; j < kOf; ++j) ordinary(BACK ? i - j : i + j, r[k + j], x[k + j]);
                }
            }
        }
    }
    // Composes the groups' maps; s: what they add, h: what the tile's adds.
    // Returns the root of its decay.
    template <bool BACK>
    __device__ __forceinline__ float compose(uint32_t waves, const float (*s)[kRecurCols], float& h) const
    {
        GroupsProduct all;
        h = 0.f;
        each<BACK>(
            waves, s,
            [&](int, float a, float x) {
                h = ordinary_step(a, h, x);
                all.ordinary(a);
            },
            [&](int, float r, float x) {
                h = step_of(r, h, x);
                all.root(r);
            });
        return all.root();
    }
    // The state that enters the tile -> in s those that enter its groups.
    template <bool BACK>
    __device__ __forceinline__ void enter(uint32_t waves, float (*s)[kRecurCols], float h) const
    {
        each<BACK>(
            waves, s,
            [&](int i, float a, float x) {
                s[i][lane_id()] = h;
                h = ordinary_step(a, h, x);
            },
            [&](int i, float r, float x) {
                s[i][lane_id()] = h;
                h = step_of(r, h, x);
            });
    }
};

// ---- between tiles -------------------------------------------------------
//
// One pass over the data: a workgroup takes the next row tile of its channel
// tile (in ticket order, so those before it have been taken too and their
// workgroups run), composes its rows' maps, publishes the tile's map
// h -> r (r h) + H, finds the state that enters it and publishes the state that
// leaves it.  Words say by themselves whether they have been written: all
// ones, a NaN that is never stored (NaNs are stored as 0x7fc00000), means
// not yet.  They are moved by relaxed agent-scope atomics, which bypass the
// per-die caches, and nothing else is read across workgroups.
//
// The entering state is the last published state before the tile, carried
// on through the published maps of the tiles between, in row order: the
// very operations by which those tiles make their own states, so the result
// does not depend on where a look-back finds a state.
constexpr uint64_t kNoMap = ~(uint64_t)0;
constexpr uint32_t kNoState = ~(uint32_t)0;

__device__ __forceinline__ uint32_t state_bits(float h) { return h == h ? __float_as_uint(h) : 0x7fc00000u; }
__device__ __forceinline__ uint64_t map_bits(float r, float h)
{
    return (uint64_t)state_bits(h) << 32 | __float_as_uint(r);
}

// State entering `tile` (> 0) for this lane's channel; maps and states point
// at the channel's words of tile 0, ld words between tiles.  All 64 lanes.
__device__ __forceinline__ float look_back(const uint64_t* maps, const uint32_t* states, int64_t ld, int64_t tile)
{
    constexpr int W = 4;  // tiles read at once
    int64_t from = tile - W, known = -1;
    float h = 0.f;
    for (;;) {
        const int64_t w0 = known >= 0 ? known + 1 : (from > 0 ? from : 0);
        uint32_t s[W];
        uint64_t m[W];
#pragma unroll
        for (int q = 0; q < W; ++q) {
            s[q] = kNoState;
            m[q] = kNoMap;
            if (w0 + q < tile) {
                s[q] = ld_agent(states + (w0 + q) * ld);
                m[q] = ld_agent(maps + (w0 + q) * ld);
            }
        }
        const int64_t before = known;
#pragma unroll
        for (int q = 0; q < W; ++q) {
            if (__all(s[q] != kNoState)) {
                known = w0 + q;
                h = __uint_as_float(s[q]);
            } else if (known >= 0 && known == w0 + q - 1 && __all(m[q] != kNoMap)) {
                known = w0 + q;
                h = step_of(__uint_as_float((uint32_t)m[q]), h, __uint_as_float((uint32_t)(m[q] >> 32)));
            }
        }
        if (known == tile - 1) return h;
        if (known == before) {
            if (known < 0 && w0 > 0) from = w0 - W;  // nothing here yet: further back
            else __builtin_amdgcn_s_sleep(1);
        }
    }
}

// The tile's map (r, h) of this lane's channel -> the state entering it.
// `fresh`: nothing enters (its first row starts a sequence or has none);
// `last`: no tile follows.  One whole wave.
__device__ __forceinline__ float pass_state(const RecurArgs& A, int64_t tile, int ct, float r, float h, bool fresh,
                                            bool last)
{
    const int64_t ld = (int64_t)A.cols * kRecurCols;
    const int64_t c = (int64_t)ct * kRecurCols + lane_id();
    const bool cut = __all(r == 0.f);  // the leaving state does not depend on the entering one
    if (!last) {
        if (cut) st_agent(A.states + tile * ld + c, state_bits(h));
        else st_agent(A.maps + tile * ld + c, map_bits(r, h));
    }
    float in = 0.f;
    if (!fresh && tile > 0) in = look_back(A.maps + c, A.states + c, ld, tile);
    if (!last && !cut) st_agent(A.states + tile * ld + c, state_bits(step_of(r, in, h)));
    return in;
}

// Workgroup b's channel tile.  Workgroup b runs on die b % 8; taken as they
// come, each die would keep to every eighth tile's 128 bytes of a row, which
// use a quarter of its L2's channels.  One tile further in each round of the
// channels spreads every die over all of them.
__device__ __forceinline__ int channel_tile(const RecurArgs& A, uint32_t b)
{
    const uint32_t cols = (uint32_t)A.cols, round = b / cols;
    return (int)((b - round * cols + round) % cols);
}

// The workgroup's row tile in the order of the pass: the next of its channel
// tile (a counter for each: one for all made the first of 1280 workgroups
// wait up to 10 us for their turns).  All threads; has a barrier.
__device__ __forceinline__ uint32_t next_tile(const RecurArgs& A, int ct)
{
    __shared__ uint32_t s_ticket;
    if (A.tiles <= 1) return 0;
    if (threadIdx.x == 0) s_ticket = atomicAdd(A.tickets + (int64_t)ct * kRecurTicketPitch, 1u);
    __syncthreads();
    return (uint32_t)__builtin_amdgcn_readfirstlane((int)s_ticket);
}

// Whether all tiles of the channel tile were taken: only a grid of several
// rows has workgroups too many.  (Asked at the start instead, all workgroups
// waited for the sizes: 8192 x 4096 bf16 forward 51.3 -> 52.9 us.)
__device__ __forceinline__ bool past_tiles(const RecurArgs& A, int64_t tile) { return tile >= A.tiles; }

// Four channels per thread, unless a decay serves some other number of them.
inline bool recur_wide(const RecurArgs& a) { return a.width >= 4 && (a.per == 1 || a.per % 4 == 0); }

// With no more than a workgroup per CU the pass is bound by one tile's
// latency: 1024 threads of 4 rows instead of 256 of 16 (or 512 of 8, see
// kGradRows), whose straight code is two to four times as long to fetch.
// Calls in a graph, us, 1024 threads against the others, forward and backward:
//                         128 workgroups        256                   512                   1024
//   bf16, own decays      14.8/15.8 17.8/17.4   15.8/16.7 19.3/18.8   19.4/20.5 30.6/22.9   32.7/27.8 52.5/43.6
//   bf16, shared          13.5/14.2 16.6/20.7   14.6/15.4 18.0/22.3   17.1/18.0 27.0/25.8   28.8/23.4 45.9/39.9
//   float32, own decays   15.6/16.2 18.8/18.7   19.0/19.5 22.1/21.7   31.7/25.0 37.6/37.0   53.4/45.1 68.6/66.7
//   float32, shared       14.4/14.7 17.5/18.3   16.4/16.3 19.7/20.6   26.2/20.2 31.9/25.2   43.2/30.1 54.6/41.0
// Up to 256 it is faster or within 3 %, at 512 in two forms, at 1024 in none.
inline bool recur_few(const RecurArgs& a) { return a.tiles * a.cols <= 256; }

// Clears what a pass publishes and marks the tiles (with more than one tile),
// and gives sequences without rows their result: to[q] = from[q], or 0
// without `from`.
hipError_t recur_begin(const RecurArgs& a, const float* from, float* to, hipStream_t s);

}  // namespace lx

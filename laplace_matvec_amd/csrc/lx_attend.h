// Shared parts of the gated matrix memory's kernels (gfx950).
#pragma once
#include "lx_device.h"
#include "lx_internal.h"
#include "lx_mma.h"
#include "lx_ragged.h"

namespace lx {

constexpr int kAttendThreads = 256;
constexpr int kC = kAttendChunk;  // rows of a chunk: one per lane

// What products are made in for storage type T: bfloat16 rows as they are,
// other types as float32 (float16's range is too small for states and
// scores).  What is made here goes into bfloat16 products rounded, in as many
// terms as its results need:
//     scores, states for y         2   y is off by its own rounding, 0.0017; by
//                                      0.0024 with one term.  65536 rows of 16
//                                      heads of 128 x 128 518 us against 471,
//                                      packed training 1459 against 1425
//     scores and their gradients   2   dq, dk and dv likewise; 0.0019 with one
//                                      term.  Packed training 1612 us against
//                                      1561
//     states for gradients         3   dg is float32: off by 1e-7 to 4e-7,
//                                      which is what float32 products give;
//                                      2.6e-6 with two terms.  1612 against
//                                      1558
//     rows times decays (states)   3   final states and dh0 are float32: off by
//                                      2e-7 of themselves, 1.6e-6 with two terms
template <class T>
struct Compute { typedef float E; static constexpr int kTerms = 1, kScoreTerms = 1; };
template <>
struct Compute<bf16_t> { typedef bf16_t E; static constexpr int kTerms = 3, kScoreTerms = 2; };

// Values of padding at the end of an LDS row of E: 16 bytes.
template <class E>
constexpr int kPad = 16 / (int)sizeof(E);

// States between chunks and segments are kept as their results lie in
// registers, so that a wave moves a tile of 16 x 16 in one piece: tile (kt, vt)
// of a head's [dkp][dvp] is 64 lanes of four values, rows 16 kt + 4 (lane /
// 16) + r, column 16 vt + lane % 16.
__device__ __forceinline__ int64_t tile_at(int kt, int vt, int dvp) { return ((int64_t)kt * (dvp >> 4) + vt) * 256; }

// 8 neighbours from p on, of which `count` are there (0 past them).
template <class T>
__device__ __forceinline__ Pack<T, 8> load8(const T* p, int64_t count)
{
    Pack<T, 8> r;
    if (count >= 8) {
        if constexpr (sizeof(T) == 2) {
            r = load_pack<8>(p);
        } else {
            const Pack<T, 4> a = load_pack<4>(p), b = load_pack<4>(p + 4);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                r.v[i] = a.v[i];
                r.v[4 + i] = b.v[i];
            }
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) r.v[i] = i < count ? p[i] : (T)0.f;
    }
    return r;
}

template <class E, class T>
__device__ __forceinline__ Frag<E> to_frag(const Pack<T, 8>& p)
{
    Frag<E> f;
#pragma unroll
    for (int i = 0; i < 8; ++i) f.v[i] = (E)p.v[i];
    return f;
}

template <class E, class T>
__device__ __forceinline__ void put8(E* s, const Pack<T, 8>& p)
{
    *reinterpret_cast<typename Frag<E>::V*>(s) = to_frag<E>(p).v;
}

__device__ __forceinline__ bool finite(float x) { return (__builtin_bit_cast(uint32_t, x) & 0x7F800000u) != 0x7F800000u; }
__device__ __forceinline__ bool finite(bf16_t x) { return (__builtin_bit_cast(uint16_t, x) & 0x7F80u) != 0x7F80u; }

// 8 neighbours from p on, all there.
template <class T>
__device__ __forceinline__ Pack<T, 8> load8_whole(const T* p)
{
    if constexpr (sizeof(T) == 2) {
        return load_pack<8>(p);
    } else {
        Pack<T, 8> r;
        const Pack<T, 4> a = load_pack<4>(p), b = load_pack<4>(p + 4);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            r.v[i] = a.v[i];
            r.v[4 + i] = b.v[i];
        }
        return r;
    }
}

// A tile of kC rows x W columns on its way from memory to LDS.  WHOLE: rows
// are whole groups of 8 values.  Then what is not there is read from what is,
// and cleared on its way to LDS: loads without branches, which would have to
// wait for their values where the paths meet again.
template <class T, int W, bool WHOLE, int THREADS = kAttendThreads>
struct RowTile {
    static constexpr int kVecs = kC * W / 8 / THREADS;
    Pack<T, 8> r[kVecs];

    // p: first row and column; rows and cols: how many are there, at least one
    __device__ __forceinline__ void load(const T* p, int64_t ld, int rows, int cols)
    {
#pragma unroll
        for (int j = 0; j < kVecs; ++j) {
            const int i = (int)threadIdx.x + j * THREADS;
            int row = i / (W / 8), col = i % (W / 8) * 8;
            if (WHOLE) {
                row = row < rows ? row : rows - 1;
                col = col < cols ? col : cols - 8;
                r[j] = load8_whole(p + row * ld + col);
            } else {
                r[j] = load8(p + row * ld + col, row < rows ? cols - col : 0);
            }
        }
    }
    template <class E>
    __device__ __forceinline__ void put(E* s, int rows, int cols) const
    {
        constexpr int kPitch = W + kPad<E>;
        if (WHOLE && (rows < kC || cols < W)) {
#pragma unroll
            for (int j = 0; j < kVecs; ++j) {
                const int i = (int)threadIdx.x + j * THREADS;
                const int row = i / (W / 8), col = i % (W / 8) * 8;
                put8(s + row * kPitch + col, row < rows && col < cols ? r[j] : Pack<T, 8>{});
            }
        } else {
#pragma unroll
            for (int j = 0; j < kVecs; ++j) {
                const int i = (int)threadIdx.x + j * THREADS;
                put8(s + i / (W / 8) * kPitch + i % (W / 8) * 8, r[j]);
            }
        }
    }
    // Whether any of the values is inf or NaN: its exponent is all ones, and
    // one more carries into the sign.
    __device__ __forceinline__ bool odd() const
    {
        constexpr uint32_t kExp = sizeof(T) == 4 ? 0x7F800000u : sizeof(T) == 2 && __is_same(T, f16_t) ? 0x7C007C00u : 0x7F807F80u;
        constexpr uint32_t kOne = sizeof(T) == 4 ? 0x00800000u : __is_same(T, f16_t) ? 0x04000400u : 0x00800080u;
        constexpr uint32_t kSign = sizeof(T) == 4 ? 0x80000000u : 0x80008000u;
        uint32_t any = 0;
#pragma unroll
        for (int j = 0; j < kVecs; ++j) {
            typedef uint32_t Bits __attribute__((ext_vector_type(2 * sizeof(T))));
            const Bits w = __builtin_bit_cast(Bits, r[j]);
#pragma unroll
            for (int i = 0; i < 2 * (int)sizeof(T); ++i) any |= (w[i] & kExp) + kOne;
        }
        return any & kSign;
    }
};

constexpr double kLog2e = 1.4426950408889634074;

// 2^x: from x in two floats, as one is off by 2^-24 of x, and also where it is
// below the smallest normal number, which v_exp_f32 makes 0.
__device__ __forceinline__ float exp2_whole(double x)
{
    const float hi = (float)x, lo = (float)(x - (double)hi);
    const bool deep = hi < -126.f;
    const float e = __builtin_amdgcn_exp2f(deep ? hi + 64.f : hi) * __builtin_fmaf(lo, 0.69314718f, 1.f);
    return e * (deep ? 0x1p-64f : 1.f);
}

// The logarithm of a decay that is 0 in float32: e^g <= 2^-150.
__device__ __forceinline__ bool is_cut(float g) { return g < -103.97208f; }

// Decays of a chunk, worked out by one wave with a row per lane.  Sums of the
// logarithms are float64, handed on in two floats, so that a difference of two
// is as good after thousands of strong decays as at the start.  A decay that
// is 0 in float32 cuts: rows before it are gone for the rows from it on.  One
// that is NaN, or infinite in float32, is left out of the sums too, which would
// carry it past the next cut: the sums from it up to there are set to NaN.
// Products of decays are float32 numbers, subnormal ones included, as those of
// the single-token form are.
struct Decays {
    float hi[kC], lo[kC];  // half the sums of log2 of the decays up to each row, cuts left out
    float into[kC];        // what a row sees of the state before the chunk
    float out[kC];         // what the state after the chunk holds of a row
    int last[kC];          // the last cut up to each row, -1 for none

    __device__ __forceinline__ void make(float g)
    {
        const int lane = threadIdx.x & 63;
        const bool cut = is_cut(g);
        const bool bad = !(g < 88.72284f);  // e^g >= 2^128, or NaN
        const uint64_t cuts = __ballot(cut), bads = __ballot(bad);
        double sum = cut || bad ? 0.0 : (double)g * kLog2e;
        sum += dpp_move<0x111>(sum, 0.0);
        sum += dpp_move<0x112>(sum, 0.0);
        sum += dpp_move<0x114>(sum, 0.0);
        sum += dpp_move<0x118>(sum, 0.0);
        sum += dpp_move<0x142, 0xA>(sum, 0.0);
        sum += dpp_move<0x143, 0xC>(sum, 0.0);
        const uint64_t upto = (2ull << lane) - 1, mine = cuts & upto;
        if (bads & upto && (bads & upto) > mine) sum = __builtin_nan("");  // the last bad one lies past the last cut
        const double total = __shfl(sum, 63);
        hi[lane] = (float)(0.5 * sum);
        lo[lane] = (float)(0.5 * sum - (double)(float)(0.5 * sum));
        last[lane] = mine ? 63 - __builtin_clzll(mine) : -1;
        into[lane] = mine ? 0.f : exp2_whole(sum);
        // a cut after this row takes it away; its own does not
        out[lane] = (cuts >> lane) > 1 ? 0.f : exp2_whole(total - sum);
    }
    // rows that see the state before the chunk, a bit each
    __device__ __forceinline__ unsigned long long sees_before() const
    {
        return __ballot(last[threadIdx.x & 63] < 0);
    }
    // exp of the decays after row j up to row i >= j: the square of the root
    __device__ __forceinline__ float between(float hi_i, float lo_i, float hi_j, float lo_j) const
    {
        const float root = __builtin_amdgcn_exp2f((hi_i - hi_j) + (lo_i - lo_j));
        return root * root;
    }
};

// x in terms: each the rounding of what the ones before it leave.
template <class E, int N>
__device__ __forceinline__ void split(float x, E (&t)[N])
{
#pragma unroll
    for (int m = 0; m < N; ++m) {
        t[m] = (E)x;
        if (m + 1 < N) x -= (float)t[m];
    }
}

}  // namespace lx

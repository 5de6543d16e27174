// Products of rows with their experts' matrices (gfx950).
//
// Rows come sorted by expert (laplex_route, laplex_dispatch); expert e has
// the rows offsets[e] <= r < offsets[e + 1], any number of them:
//     y_r   = W_e x_r                  rows: n x out, contraction in
//     dx_r  = W_e^T dy_r               rows: n x in, contraction out
//     dW_e  = sum over r of dy_r x_r^T  out x in for each expert, contraction its rows
// Row tiles of one expert are numbered in closed form, first tile
// offsets[e] / BM + e, so a workgroup finds its expert by a search in the
// offsets and no list of tiles is made; what the numbering leaves over (less
// than one tile per expert) ends at once.
#include "lx_device.h"
#include "lx_internal.h"
#include "lx_mma.h"
#include "lx_ragged.h"

namespace lx {

namespace {

// ---- any layout, alignment and size --------------------------------------

constexpr int kAnyThreads = 256;
constexpr int kAnyK = 32;

// One operand tile of ROWS rows x kAnyK values of the contraction: in
// registers on the way, and in LDS with the contraction along rows.
// ALONG: the contraction runs along memory, else the operand's rows do.
template <class T, int ROWS, bool ALONG>
struct AnyTile {
    static constexpr int kV = 16 / sizeof(T);
    static constexpr int kVecs = ROWS * kAnyK / kV / kAnyThreads;
    static constexpr int kPitch = kAnyK + 16 / (int)sizeof(T);
    Pack<T, kV> r[kVecs];

    // rows and k: how many are there from p on
    __device__ __forceinline__ void load(const T* p, int64_t ld, int64_t rows, int64_t k)
    {
#pragma unroll
        for (int j = 0; j < kVecs; ++j) {
            const int i = (int)threadIdx.x + j * kAnyThreads;
            constexpr int kPer = (ALONG ? kAnyK : ROWS) / kV;  // vectors of a line of memory
            const int line = i / kPer, at = i % kPer * kV;
            const int64_t lines = ALONG ? rows : k, along = (ALONG ? k : rows) - at;
            const T* q = p + line * ld + at;
            if (line < lines && along >= kV) {
                r[j] = load_pack<kV>(q);
            } else {
#pragma unroll
                for (int v = 0; v < kV; ++v) r[j].v[v] = line < lines && v < along ? q[v] : (T)0.f;
            }
        }
    }
    __device__ __forceinline__ void put(T* s) const
    {
#pragma unroll
        for (int j = 0; j < kVecs; ++j) {
            const int i = (int)threadIdx.x + j * kAnyThreads;
            constexpr int kPer = (ALONG ? kAnyK : ROWS) / kV;
            const int line = i / kPer, at = i % kPer * kV;
            if (ALONG) {
                *reinterpret_cast<Pack<T, kV>*>(s + line * kPitch + at) = r[j];
            } else {
#pragma unroll
                for (int v = 0; v < kV; ++v) s[(at + v) * kPitch + line] = r[j].v[v];
            }
        }
    }
};

// C tile of (32 WM) x (32 WN), four waves in two rows and two columns.
template <class T, int WM, int WN, bool AALONG, bool BALONG>
__device__ __forceinline__ void any_tile(const T* a, int64_t lda, int64_t rows, const T* b, int64_t ldb, int64_t cols,
                                         int64_t k, T* c, int64_t ldc)
{
    typedef AnyTile<T, 32 * WM, AALONG> TA;
    typedef AnyTile<T, 32 * WN, BALONG> TB;
    __shared__ alignas(16) T s_a[32 * WM * TA::kPitch], s_b[32 * WN * TB::kPitch];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int m0 = (wave >> 1) * 16 * WM, n0 = (wave & 1) * 16 * WN;
    f32x4 acc[WM][WN] = {};
    TA ta;
    TB tb;
    ta.load(a, lda, rows, k);
    tb.load(b, ldb, cols, k);
    for (int64_t k0 = 0; k0 < k; k0 += kAnyK) {
        __syncthreads();
        ta.put(s_a);
        tb.put(s_b);
        __syncthreads();
        if (k0 + kAnyK < k) {
            ta.load(AALONG ? a + (k0 + kAnyK) : a + (k0 + kAnyK) * lda, lda, rows, k - k0 - kAnyK);
            tb.load(BALONG ? b + (k0 + kAnyK) : b + (k0 + kAnyK) * ldb, ldb, cols, k - k0 - kAnyK);
        }
        Frag<T> fa[WM], fb[WN];
#pragma unroll
        for (int i = 0; i < WM; ++i) fa[i] = frag_along(s_a + (m0 + 16 * i + (lane & 15)) * TA::kPitch + 8 * (lane >> 4));
#pragma unroll
        for (int i = 0; i < WN; ++i) fb[i] = frag_along(s_b + (n0 + 16 * i + (lane & 15)) * TB::kPitch + 8 * (lane >> 4));
#pragma unroll
        for (int i = 0; i < WM; ++i)
#pragma unroll
            for (int j = 0; j < WN; ++j) acc[i][j] = mma(fa[i], fb[j], acc[i][j]);
    }
#pragma unroll
    for (int i = 0; i < WM; ++i)
#pragma unroll
        for (int j = 0; j < WN; ++j)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int m = m0 + 16 * i + 4 * (lane >> 4) + r, n = n0 + 16 * j + (lane & 15);
                if (m < rows && n < cols) c[m * ldc + n] = (T)acc[i][j][r];
            }
}

// y = W x for each row (BALONG: the contraction runs along W's rows).
template <class T, int WM, int WN, bool BALONG>
__global__ __launch_bounds__(kAnyThreads) void lx_experts_any(ExpertsArgs A)
{
    constexpr int BM = 32 * WM, BN = 32 * WN;
    const int64_t id = group_id<kAnyThreads>();
    const int64_t unit = id / A.col_tiles;
    const int64_t c0 = (id - unit * A.col_tiles) * BN;
    const Ragged R{A.offsets, A.experts, A.n, 0};
    if (unit >= R.units(BM)) return;
    const RaggedTile t = R.find(unit, BM);
    if (t.rows <= 0) return;
    const int64_t cols = A.out - c0 < BN ? A.out - c0 : BN;
    T* y = (T*)A.y + t.row * A.ldy + c0;
    if (t.group < 0) {
        for (int i = threadIdx.x; i < t.rows * BN; i += kAnyThreads)
            if (i % BN < cols) y[(int64_t)(i / BN) * A.ldy + i % BN] = (T)0.f;
        return;
    }
    const T* w = (const T*)A.w + t.group * A.pitch_w + (BALONG ? c0 * A.ldw : c0);
    any_tile<T, WM, WN, true, BALONG>((const T*)A.x + t.row * A.ldx, A.ldx, t.rows, w, A.ldw, cols, A.in, y, A.ldy);
}

// dW_e = sum over its rows of dy x^T.
template <class T, int WM, int WN>
__global__ __launch_bounds__(kAnyThreads) void lx_experts_any_grad(ExpertsArgs A)
{
    constexpr int BM = 32 * WM, BN = 32 * WN;
    const int64_t id = group_id<kAnyThreads>();
    const int64_t e = id / (A.row_tiles * A.col_tiles);
    if (e >= A.experts) return;
    const int64_t rest = id - e * A.row_tiles * A.col_tiles;
    const int64_t m0 = rest / A.col_tiles * BM, c0 = rest % A.col_tiles * BN;
    const Ragged R{A.offsets, A.experts, A.n, 0};
    const int64_t first = R.bound(e + 1), end = R.bound(e + 2);
    any_tile<T, WM, WN, false, false>((const T*)A.y + first * A.ldy + m0, A.ldy, A.out - m0 < BM ? A.out - m0 : BM,
                                      (const T*)A.x + first * A.ldx + c0, A.ldx, A.in - c0 < BN ? A.in - c0 : BN,
                                      end > first ? end - first : 0, (T*)A.dw + e * A.pitch_w + m0 * A.ldw + c0,
                                      A.ldw);
}

template <class T>
hipError_t any_go(ExpertsArgs a, hipStream_t s)
{
    constexpr int B = 64;
    a.col_tiles = (a.out + B - 1) / B;
    const int64_t groups = Ragged{a.offsets, a.experts, a.n, 0}.units(B) * a.col_tiles;
    if (a.transpose)
        LX_LAUNCH("experts", s, (lx_experts_any<T, 2, 2, false><<<grid_of<kAnyThreads>(groups), kAnyThreads, 0, s>>>(a)));
    else
        LX_LAUNCH("experts", s, (lx_experts_any<T, 2, 2, true><<<grid_of<kAnyThreads>(groups), kAnyThreads, 0, s>>>(a)));
    return hipSuccess;
}

template <class T>
hipError_t any_grad_go(ExpertsArgs a, hipStream_t s)
{
    constexpr int B = 64;
    a.row_tiles = (a.out + B - 1) / B;
    a.col_tiles = (a.in + B - 1) / B;
    const int64_t groups = a.experts * a.row_tiles * a.col_tiles;
    LX_LAUNCH("experts_grad", s, (lx_experts_any_grad<T, 2, 2><<<grid_of<kAnyThreads>(groups), kAnyThreads, 0, s>>>(a)));
    return hipSuccess;
}

}  // namespace

hipError_t experts_launch(const ExpertsArgs& a, int dtype, hipStream_t s)
{
    switch (dtype) {
        case 0: return any_go<float>(a, s);
        case 1: return any_go<bf16_t>(a, s);
        case 2: return any_go<f16_t>(a, s);
        default: return hipErrorInvalidValue;
    }
}

hipError_t experts_grad_launch(const ExpertsArgs& a, int dtype, hipStream_t s)
{
    switch (dtype) {
        case 0: return any_grad_go<float>(a, s);
        case 1: return any_grad_go<bf16_t>(a, s);
        case 2: return any_grad_go<f16_t>(a, s);
        default: return hipErrorInvalidValue;
    }
}

}  // namespace lx

// Products of rows with their experts' matrices (gfx950).
//
// Rows come sorted by expert (laplex_route, laplex_dispatch); expert e has
// the rows offsets[e] <= r < offsets[e + 1], any number of them:
//     y_r   = W_e x_r                  rows: n x out, contraction in
//     dx_r  = W_e^T dy_r               rows: n x in, contraction out
//     dW_e  = sum over r of dy_r x_r^T  out x in for each expert, contraction its rows
// A workgroup finds its expert by a search in the offsets (lx_ragged.h), so
// no list of tiles is made and nothing is launched before.
//
// Three families of kernels:
//   lx_experts_tile   16-bit values, tiles of 256 x 256, 128 x 128 or 64 x 64
//     through LDS.  Bound by issue and waits within a step: the matrix units
//     are busy for 56 % of the cycles (at 1.7 GHz, below the full clock), a
//     third of the waves' time is waiting, and about one scalar instruction is
//     issued for each matrix instruction.  8 x 4096 rows, 4096 x 4096 bf16:
//     905 to 945 us, 1.16 to 1.21 PFLOP/s; a library product
//     of all rows with one matrix 700 (steps of 1.6 us a tile against 1.3: 85 %
//     busy at 1.5 GHz, a third of the scalar and two thirds of the vector
//     instructions; it
//     reads a third less LDS with four waves of 128 x 128, which lost here, 890
//     against 850 in one matrix, and waits less).  Also tried for one matrix
//     of 32768 x 4096 x 4096: matrix instructions of 32 x 32 x 16 980, four
//     steps of 32 in LDS 1000, two workgroups of 128 x 256 a CU 1030, one half
//     of the waves multiplying while the other reads LDS 845 to 860, the same
//     as all of them together.
//   lx_experts_few    a few rows: bound by memory, 64 x 2048 x 2048 read for
//     one row each in 92 us, 5.8 TB/s; 4 rows of 16 experts 5.7 us of kernel.
//   lx_experts_any    float32, any layout: 4096 x 512 x 769 in 8 experts 49 us,
//     66 TFLOP/s of the 154 of a large library product: short of workgroups
//     and of LDS reads ahead of their products.
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

// ---- 16-bit values, tiles by LDS ------------------------------------------

constexpr int kK = 64;  // contraction of a step

// How a product's operands lie in memory and LDS.  ALONG: lines are rows of
// the operand, kK values of the contraction in 8 vectors of 16 bytes; vector c
// of line r lies at c ^ (r % 8), so that eight lanes that read one vector of
// eight lines each use all banks.  Else lines are steps of the contraction
// with ROWS of the operand's rows next to each other; pairs of vectors are
// exchanged so that the 16 lines of a transposing read spread over the banks.
template <int ROWS, bool ALONG>
struct Lines {
    static constexpr int kVecs = ALONG ? kK / 8 : ROWS / 8;  // of a line
    static constexpr int kCount = ALONG ? ROWS : kK;
    static constexpr int kValues = ROWS * kK;
    static __device__ __forceinline__ int swap(int line)
    {
        return ALONG ? line & 7 : (((line & 3) | ((line >> 1) & 4)) << 1) & (kVecs - 1);
    }
    // Zeros from contraction `left` on.
    template <class T>
    static __device__ __forceinline__ void blank(T* p, int left, int threads)
    {
        for (int i = threadIdx.x; i < kValues / 8; i += threads) {
            const int line = i / kVecs;
            if (ALONG ? 8 * ((i % kVecs) ^ swap(line)) >= left : line >= left) *reinterpret_cast<Pack<T, 8>*>(p + 8 * i) = Pack<T, 8>{};
        }
    }
    // 16 rows from row0 on, contraction 32 s .. 32 s + 31 in the order 8 g + i
    template <class T>
    static __device__ __forceinline__ Frag<T> read(const T* p, int row0, int s)
    {
        const int lane = threadIdx.x & 63;
        Frag<T> f;
        if constexpr (ALONG) {
            const int r = row0 + (lane & 15);
            f = frag_along(p + r * kK + ((4 * s + (lane >> 4)) ^ swap(r)) * 8);
        } else {
            typedef short S4 __attribute__((ext_vector_type(4)));
            typedef __attribute__((address_space(3))) S4* At;
            union { S4 h[2]; typename Frag<T>::V v; } u;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int line = 32 * s + 8 * (lane >> 4) + 4 * i + ((lane & 15) >> 2);
                const int at = row0 + 4 * (lane & 3);
                u.h[i] = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                    (At)(const_cast<T*>(p) + line * ROWS + (((at >> 3) ^ swap(line)) << 3) + (at & 7)));
            }
            f.v = u.v;
        }
        return f;
    }
};

// 16 bytes a lane from base + off to LDS, lane after lane from s on.  By hand
// because the compiler, which cannot tell the two tiles apart, would wait for
// every such load before the next read of LDS; tile_product waits for them
// itself before it hands a tile over.  No register is written; m0, which holds
// the place in LDS, is an operand, so the compiler sets it and knows of it.  A
// scalar register that a vector instruction wrote may not be read here for
// five cycles, and m0 not for one: the wait covers both.
__device__ __forceinline__ void to_lds(const void* base, uint32_t off, void* s)
{
    const uint32_t at = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) void*)s;
    asm volatile("s_nop 4\n\tglobal_load_lds_dwordx4 %0, %1" : : "v"(off), "s"(base), "{m0}"(at) : "memory");
}

// What a thread moves of a tile: kVecs vectors of 16 bytes a step, straight to
// LDS (DMA: 16-byte aligned lines; lines and vectors that are not there are
// read from the last ones that are) or by registers (any alignment, 0 for
// what is not there).
template <class T, int ROWS, bool ALONG, int THREADS, bool DMA>
struct Mover {
    typedef Lines<ROWS, ALONG> L;
    static constexpr int kVecs = ROWS * kK / 8 / THREADS;
    static_assert(kVecs * THREADS * 8 == ROWS * kK, "whole vectors for every thread");
    // vectors of wave w, j-th: 64 from here on
    static __device__ __forceinline__ int first(int j)
    {
        return (__builtin_amdgcn_readfirstlane(threadIdx.x >> 6) * kVecs + j) * 64;
    }
    const T* base;    // first row, first step
    int64_t ld;
    int rows;         // rows that are there
    uint32_t line[kVecs], at[kVecs];  // values from base to the line and within it
    Pack<T, 8> r[DMA ? 1 : kVecs];

    __device__ __forceinline__ void init(const T* p, int64_t pitch, int there)
    {
        base = (const T*)(uintptr_t)uniform((int64_t)(uintptr_t)p);
        ld = pitch;
        rows = there;
#pragma unroll
        for (int j = 0; j < kVecs; ++j) {
            const int i = first(j) + (threadIdx.x & 63);
            const int l = i / L::kVecs, v = (i % L::kVecs) ^ L::swap(l);
            if (DMA) {
                line[j] = (uint32_t)(ALONG ? (l < rows ? l : rows - 1) : l) * (uint32_t)ld;
                at[j] = 8 * v;
                if (!ALONG && (int)at[j] > rows - 8) at[j] = rows - 8;
            } else {
                line[j] = l;
                at[j] = 8 * v;
            }
        }
    }
    // Vector j of the step whose contraction starts at k0, of k in all.
    __device__ __forceinline__ void load(int j, int64_t k0, int64_t k, T* s)
    {
        const T* p = base + (ALONG ? k0 : k0 * ld);
        if constexpr (DMA) {
            const int64_t left = k - k0;
            uint32_t off;
            if (ALONG) {
                const uint32_t most = left < kK ? (uint32_t)left - 8 : kK;
                off = line[j] + (at[j] < most ? at[j] : most);
            } else {
                const uint32_t most = (uint32_t)(left < kK ? left - 1 : kK) * (uint32_t)ld;
                off = (line[j] < most ? line[j] : most) + at[j];
            }
            to_lds(p, off * (uint32_t)sizeof(T), s + first(j) * 8);
        } else {
            const int64_t left = k - k0;
            const int64_t lines = ALONG ? rows : left, along = (ALONG ? left : rows) - at[j];
            const T* q = p + line[j] * ld + at[j];
            if (line[j] < lines && along >= 8) {
                r[j] = load_pack<8>(q);
            } else {
#pragma unroll
                for (int v = 0; v < 8; ++v) r[j].v[v] = line[j] < lines && v < along ? q[v] : (T)0.f;
            }
        }
    }
    __device__ __forceinline__ void put(T* s) const
    {
        if constexpr (!DMA) {
#pragma unroll
            for (int j = 0; j < kVecs; ++j)
                *reinterpret_cast<Pack<T, 8>*>(s + (first(j) + (threadIdx.x & 63)) * 8) = r[j];
        }
    }
};

// Shapes of a tile: BM rows by BN columns, WM x WN waves.
template <int BM_, int BN_, int WM_, int WN_>
struct Shape {
    static constexpr int BM = BM_, BN = BN_, WM = WM_, WN = WN_;
    static constexpr int kThreads = 64 * WM * WN, TM = BM / WM / 16, TN = BN / WN / 16;
    // Workgroups that stay for several tiles: one on each of the 256 CUs,
    // which saves the wait for a tile's first values.  Where the contraction k
    // is short the results' way to memory is the bound, and tiles that end at
    // any time do better (gradient of 128 matrices of 1536 x 2048: 30 rows each
    // 289 us against 267, 200 rows 210 against 213).  Smaller shapes overlap
    // by themselves, and what staying costs in registers costs more.
    static constexpr bool kMayStay = BM >= 256;
    static bool stays(int64_t tiles, int64_t k) { return kMayStay && tiles > 256 && k >= 192; }
    // A wave's place.  Waves w and w + 4 share a SIMD: of 2 x 4 waves they get
    // different halves both ways, so that half a tile keeps all SIMDs at work.
    static __device__ __forceinline__ int row_of(int w) { return WM == 2 && WN == 4 ? (w ^ (w >> 2)) & 1 : w / WN; }
    static __device__ __forceinline__ int col_of(int w) { return WM == 2 && WN == 4 ? w >> 1 : w % WN; }
};

// One tile c [rows][cols] = a b^T of a launch's work.
template <class T>
struct Work {
    const T *a, *b;
    T* c;
    int rows, cols;
    int64_t k;
};

// The tiles that `next` gives, one after the other.  Two steps in LDS: while
// one is multiplied, the next one is on its way, across the end of a tile
// too; a barrier a step.  The order within a step is fixed by hand: fragments
// are read two ahead of the products that use them, loads go out among the
// first products.
template <class T, class S, bool AALONG, bool BALONG, bool DMA, bool STAYS, class Next>
__device__ __forceinline__ void tile_products(int64_t lda, int64_t ldb, int64_t ldc, Next next_work)
{
    typedef Lines<S::BM, AALONG> LA;
    typedef Lines<S::BN, BALONG> LB;
    constexpr int TM = S::TM, TN = S::TN;
    constexpr int kTile = LA::kValues + LB::kValues;
    __shared__ alignas(1024) T s_tiles[2 * kTile];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int m0 = S::row_of(wave) * 16 * TM, n0 = S::col_of(wave) * 16 * TN;
    Mover<T, S::BM, AALONG, S::kThreads, DMA> ma;
    Mover<T, S::BN, BALONG, S::kThreads, DMA> mb;
    constexpr int VA = decltype(ma)::kVecs, VB = decltype(mb)::kVecs;
    auto load = [&](int q, int64_t k0, int64_t k, T* to) {
        if (q < VA) ma.load(q, k0, k, to);
        else if (q < VA + VB) mb.load(q - VA, k0, k, to + LA::kValues);
    };
    auto put = [&](T* to) {
        ma.put(to);
        mb.put(to + LA::kValues);
    };

    Work<T> w;
    if (!next_work(w)) return;
    T* now = s_tiles;
    T* next = s_tiles + kTile;
    ma.init(w.a, lda, w.rows);
    mb.init(w.b, ldb, w.cols);
#pragma unroll
    for (int q = 0; q < VA + VB; ++q) load(q, 0, w.k, now);
    put(now);
    for (;;) {
        const bool on = m0 < w.rows && n0 < w.cols;  // whether any of the wave's results are there
        f32x4 acc[TM][TN] = {};
        Work<T> then;
        const bool goes_on = STAYS && next_work(then);
        bool more = true;  // whether anything is loaded during a step
        for (int64_t k0 = 0; k0 < w.k; k0 += kK) {
            int64_t k1 = k0 + kK, k = w.k;  // the next step
            if (k1 >= w.k) {
                more = goes_on;
                if (more) {
                    ma.init(then.a, lda, then.rows);
                    mb.init(then.b, ldb, then.cols);
                    k1 = 0;
                    k = then.k;
                }
            }
            // this step's values are there and everyone is done with the other ones
            __builtin_amdgcn_s_waitcnt(0x0f70);  // vmcnt(0)
            __syncthreads();
            if (DMA && w.k - k0 < kK) {  // past the end of the contraction: other rows' values, or whatever else
                LA::blank(now, (int)(w.k - k0), S::kThreads);
                LB::blank(now + LA::kValues, (int)(w.k - k0), S::kThreads);
                __syncthreads();
            }
            if (on) {
                const T *sa = now, *sb = now + LA::kValues;
                Frag<T> fa[2][TM], fb[2][TN];
#pragma unroll
                for (int j = 0; j < TN; ++j) fb[0][j] = LB::read(sb, n0 + 16 * j, 0);
                fa[0][0] = LA::read(sa, m0, 0);
                fa[0][1] = LA::read(sa, m0 + 16, 0);
#pragma unroll
                for (int s = 0; s < 2; ++s)
#pragma unroll
                    for (int i = 0; i < TM; ++i) {
                        __builtin_amdgcn_sched_barrier(0);
                        if (i + 2 < TM) {
                            fa[s][i + 2] = LA::read(sa, m0 + 16 * (i + 2), s);
                        } else if (s == 0) {
                            fa[1][i + 2 - TM] = LA::read(sa, m0 + 16 * (i + 2 - TM), 1);
#pragma unroll
                            for (int j = 0; j < TN; ++j)
                                if ((j < TN / 2) == (i == TM - 2)) fb[1][j] = LB::read(sb, n0 + 16 * j, 1);
                        }
                        constexpr int kEach = TM >= 8 ? 2 : VA + VB;
                        if (s == 0 && i * kEach < VA + VB && more) {
#pragma unroll
                            for (int q = 0; q < kEach; ++q) load(i * kEach + q, k1, k, next);
                        }
#pragma unroll
                        for (int j = 0; j < TN; ++j) acc[i][j] = mma(fb[s][j], fa[s][i], acc[i][j]);
                    }
                __builtin_amdgcn_sched_barrier(0);
            } else if (more) {
#pragma unroll
                for (int q = 0; q < VA + VB; ++q) load(q, k1, k, next);
            }
            if (more) put(next);
            T* t = now;
            now = next;
            next = t;
        }
        if (on) {
            // a lane holds row l % 16 and four neighbouring columns of each tile
#pragma unroll
            for (int i = 0; i < TM; ++i) {
                const int m = m0 + 16 * i + (lane & 15);
                if (m >= w.rows) continue;
#pragma unroll
                for (int j = 0; j < TN; ++j) {
                    const int n = n0 + 16 * j + 4 * (lane >> 4);
                    T* p = w.c + m * ldc + n;
                    const float v[4] = {acc[i][j][0], acc[i][j][1], acc[i][j][2], acc[i][j][3]};
                    if (n + 4 <= w.cols) {
                        store_vec<4>(p, v);
                    } else {
#pragma unroll
                        for (int r = 0; r < 4; ++r)
                            if (n + r < w.cols) p[r] = (T)v[r];
                    }
                }
            }
        }
        if (!more) return;
        w = then;
    }
}

// Zeros for rows x (at most W) cols.
template <int W, int THREADS, class T>
__device__ __forceinline__ void zero_tile(T* p, int64_t ld, int64_t rows, int64_t cols)
{
    for (int64_t i = threadIdx.x; i < rows * W; i += THREADS)
        if (i % W < cols) p[i / W * ld + i % W] = (T)0.f;
}

constexpr int kBand = 8;  // row tiles of a band: its tiles go column by column

// Place `at` among rows x cols tiles.
struct Place {
    int64_t row, col;
};
__device__ __forceinline__ Place in_bands(int64_t at, int64_t rows, int64_t cols)
{
    const int64_t band = at / (kBand * cols), in_band = at - band * kBand * cols;
    const int64_t high = rows - band * kBand < kBand ? rows - band * kBand : kBand;
    return {band * kBand + in_band % high, in_band / high};
}

// Workgroups go round the eight dies in turn, so each die takes a run of
// tiles, which share operands in its cache.  Where there are more tiles than
// workgroups, a workgroup takes every gridDim-th.
template <class T, class S, bool BALONG, bool DMA, bool STAYS>
__global__ __launch_bounds__(S::kThreads, 2) void lx_experts_tile(ExpertsArgs A)
{
    const Ragged R{A.offsets, A.experts, A.n, 0};
    const int64_t id = group_id<S::kThreads>(), die = id & 7;
    int64_t turn = id >> 3;
    const Ragged::Dense d = R.dense(S::BM);
    const int64_t rows = d.inside + d.outside, run = (rows * A.col_tiles + 7) / 8;
    tile_products<T, S, true, BALONG, DMA, STAYS>(A.ldx, A.ldw, A.ldy, [&](Work<T>& w) {
        for (;; turn += A.groups >> 3) {
            const int64_t at = die * run + turn;
            if (turn >= run || at >= rows * A.col_tiles) return false;
            const Place p = in_bands(at, rows, A.col_tiles);
            const RaggedTile t = p.row < d.inside ? R.dense_tile(d, (int)p.row, S::BM)
                                                  : R.outside_tile((int)p.row - d.inside, S::BM);
            if (t.rows <= 0) continue;
            const int64_t c0 = p.col * S::BN;
            w.rows = t.rows;
            w.cols = A.out - c0 < S::BN ? (int)(A.out - c0) : S::BN;
            w.c = (T*)A.y + t.row * A.ldy + c0;
            if (t.group < 0) {
                zero_tile<S::BN, S::kThreads>(w.c, A.ldy, w.rows, w.cols);
                continue;
            }
            w.a = (const T*)A.x + t.row * A.ldx;
            w.b = (const T*)A.w + t.group * A.pitch_w + (BALONG ? c0 * A.ldw : c0);
            w.k = A.in;
            turn += A.groups >> 3;
            return true;
        }
    });
}

template <class T, class S, bool DMA, bool STAYS>
__global__ __launch_bounds__(S::kThreads, 2) void lx_experts_tile_grad(ExpertsArgs A)
{
    const int64_t each = A.row_tiles * A.col_tiles, run = (A.experts * each + 7) / 8;
    const int64_t id = group_id<S::kThreads>(), die = id & 7;
    int64_t turn = id >> 3;
    const Ragged R{A.offsets, A.experts, A.n, 0};
    tile_products<T, S, false, false, DMA, STAYS>(A.ldy, A.ldx, A.ldw, [&](Work<T>& w) {
        for (;; turn += A.groups >> 3) {
            const int64_t at = die * run + turn;
            if (turn >= run || at >= A.experts * each) return false;
            const int64_t e = at / each;
            const Place p = in_bands(at - e * each, A.row_tiles, A.col_tiles);
            const int64_t r0 = p.row * S::BM, c0 = p.col * S::BN;
            const int64_t first = uniform(R.bound(e + 1)), end = uniform(R.bound(e + 2));
            w.rows = A.out - r0 < S::BM ? (int)(A.out - r0) : S::BM;
            w.cols = A.in - c0 < S::BN ? (int)(A.in - c0) : S::BN;
            w.c = (T*)A.dw + e * A.pitch_w + r0 * A.ldw + c0;
            if (end <= first) {  // no rows
                zero_tile<S::BN, S::kThreads>(w.c, A.ldw, w.rows, w.cols);
                continue;
            }
            w.a = (const T*)A.y + first * A.ldy + r0;
            w.b = (const T*)A.x + first * A.ldx + c0;
            w.k = end - first;
            turn += A.groups >> 3;
            return true;
        }
    });
}

// 8 neighbours from p on, of which `left` are there (0 past them).
template <class T>
__device__ __forceinline__ Pack<T, 8> load_some(const T* p, int64_t left)
{
    Pack<T, 8> r;
    if (left >= 8) return load_pack<8>(p);
#pragma unroll
    for (int i = 0; i < 8; ++i) r.v[i] = i < left ? p[i] : (T)0.f;
    return r;
}

// ---- a few rows: the contraction in eight parts ----------------------------

// 16 rows by 16 columns, each wave an eighth of the contraction, four steps of
// it in flight, so that a call is little more than one way to memory.
constexpr int kFewWaves = 8, kFewThreads = 64 * kFewWaves;
template <class T>
__global__ __launch_bounds__(kFewThreads) void lx_experts_few(ExpertsArgs A)
{
    __shared__ f32x4 s_part[kFewWaves][64];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t id = group_id<kFewThreads>();
    const int64_t unit = id / A.col_tiles, c0 = (id - unit * A.col_tiles) * 16;
    const Ragged R{A.offsets, A.experts, A.n, 0};
    if (unit >= R.units(16)) return;
    const RaggedTile t = R.find(unit, 16);
    if (t.rows <= 0) return;
    const int64_t cols = A.out - c0 < 16 ? A.out - c0 : 16;
    T* y = (T*)A.y + t.row * A.ldy + c0;
    f32x4 sum = {};
    if (t.group >= 0) {
        const int l = lane & 15;
        // rows and columns that are not there: the last ones' values, not stored
        const T* x = (const T*)A.x + (t.row + (l < t.rows ? l : t.rows - 1)) * A.ldx;
        const T* w = (const T*)A.w + t.group * A.pitch_w + (c0 + (l < cols ? l : cols - 1)) * A.ldw;
        const int64_t steps = (A.in + 31) / 32, each = (steps + kFewWaves - 1) / kFewWaves;
        const int64_t from = wave * each, to = from + each < steps ? from + each : steps;
        for (int64_t s = from; s < to; s += 4) {
            Frag<T> fx[4], fw[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int64_t k = (s + i) * 32 + 8 * (lane >> 4), left = s + i < to ? A.in - k : 0;
                fw[i].v = __builtin_bit_cast(typename Frag<T>::V, load_some(w + k, left));
                fx[i].v = __builtin_bit_cast(typename Frag<T>::V, load_some(x + k, left));
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) sum = mma(fw[i], fx[i], sum);
        }
    }
    s_part[wave][lane] = sum;
    __syncthreads();
    if (threadIdx.x < 256) {  // value r of lane l: row l % 16, column 4 (l / 16) + r
        const int m = threadIdx.x >> 4, n = threadIdx.x & 15, l = m + 16 * (n >> 2);
        float v = 0.f;
#pragma unroll
        for (int i = 0; i < kFewWaves; ++i) v += s_part[i][l][n & 3];
        if (m < t.rows && n < cols) y[m * A.ldy + n] = (T)v;
    }
}

template <class T>
hipError_t few_go(ExpertsArgs a, hipStream_t s)
{
    a.col_tiles = (a.out + 15) / 16;
    const int64_t groups = Ragged{a.offsets, a.experts, a.n, 0}.units(16) * a.col_tiles;
    LX_LAUNCH("experts", s, (lx_experts_few<T><<<grid_of<kFewThreads>(groups), kFewThreads, 0, s>>>(a)));
    return hipSuccess;
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

bool lines16(const void* p, int64_t ld) { return (uintptr_t)p % 16 == 0 && ld % 8 == 0 && ld <= 1 << 22; }

template <class T, class S, bool BALONG, bool DMA>
hipError_t tile_layout_go(ExpertsArgs a, hipStream_t s)
{
    a.col_tiles = (a.out + S::BN - 1) / S::BN;
    a.groups = (Ragged{a.offsets, a.experts, a.n, 0}.units(S::BM) * a.col_tiles + 7) / 8 * 8;
    if constexpr (S::kMayStay && DMA) {
        if (S::stays(a.groups, a.in)) {
            a.groups = 256;
            LX_LAUNCH("experts", s, (lx_experts_tile<T, S, BALONG, DMA, true><<<256, S::kThreads, 0, s>>>(a)));
            return hipSuccess;
        }
    }
    LX_LAUNCH("experts", s,
              (lx_experts_tile<T, S, BALONG, DMA, false><<<grid_of<S::kThreads>(a.groups), S::kThreads, 0, s>>>(a)));
    return hipSuccess;
}

template <class T, class S>
hipError_t tile_go(const ExpertsArgs& a, bool dma, hipStream_t s)
{
    if (a.transpose) return dma ? tile_layout_go<T, S, false, true>(a, s) : tile_layout_go<T, S, false, false>(a, s);
    return dma ? tile_layout_go<T, S, true, true>(a, s) : tile_layout_go<T, S, true, false>(a, s);
}

template <class T, class S, bool DMA>
hipError_t tile_grad_layout_go(ExpertsArgs a, hipStream_t s)
{
    a.row_tiles = (a.out + S::BM - 1) / S::BM;
    a.col_tiles = (a.in + S::BN - 1) / S::BN;
    a.groups = (a.experts * a.row_tiles * a.col_tiles + 7) / 8 * 8;
    if constexpr (S::kMayStay && DMA) {
        if (S::stays(a.groups, a.n / a.experts)) {
            a.groups = 256;
            LX_LAUNCH("experts_grad", s, (lx_experts_tile_grad<T, S, DMA, true><<<256, S::kThreads, 0, s>>>(a)));
            return hipSuccess;
        }
    }
    LX_LAUNCH("experts_grad", s,
              (lx_experts_tile_grad<T, S, DMA, false><<<grid_of<S::kThreads>(a.groups), S::kThreads, 0, s>>>(a)));
    return hipSuccess;
}

template <class T, class S>
hipError_t tile_grad_go(const ExpertsArgs& a, bool dma, hipStream_t s)
{
    return dma ? tile_grad_layout_go<T, S, true>(a, s) : tile_grad_layout_go<T, S, false>(a, s);
}

typedef Shape<256, 256, 2, 4> Large;
typedef Shape<128, 128, 2, 2> Middle;
typedef Shape<64, 64, 2, 2> Little;

// Tiles that a launch of shape S has work for, at most.
template <class S>
int64_t tiles_of(const ExpertsArgs& a)
{
    const int64_t rows = a.n / S::BM + (a.n < a.experts ? a.n : a.experts);
    return rows * ((a.out + S::BN - 1) / S::BN);
}

template <class T>
hipError_t tiles_go(const ExpertsArgs& a, hipStream_t s)
{
    const bool dma = a.in % 8 == 0 && (!a.transpose || a.out % 8 == 0) && lines16(a.x, a.ldx) && lines16(a.w, a.ldw) &&
                     a.pitch_w % 8 == 0;
    // Rows of an expert.  us for 64 experts of 2048 x 2048, with each shape:
    //   rows     few  Little  Middle  Large
    //      1      92     126     130    130
    //      8     127     127     130    130
    //     16     161     128     130    132
    //    100     779     167     146    151
    //    192    1389     248     188    169
    //   1024            966     669    526
    // Fewer experts need smaller tiles to fill the card: 8 of them, rows 192:
    // Little 27.7, Middle 29.6, Large 51.7; 400: 55, 37, 57; 1024: 115, 75, 66;
    // rows 8: few 18.7, Little 21.6.  An expert with more than 16 rows is read
    // twice by `few`: 512 rows unevenly on 128 experts 151, Little 143.
    // The host knows the average only.  Where a router sends all rows to one
    // expert, the shape is that of the even case, and the call takes longer than
    // the shape for one expert would, but no longer than the even case: 128
    // experts of 2048 x 2048, 256 rows 72 (one expert 16, even 193), 4096 rows
    // 64 (39, 214), 16384 rows 152 (127, 255); the farthest, two rows an expert
    // on average in 4096 experts of 512 x 1024, 479 (18, 1090).
    const int64_t each = a.n / a.experts;
    if (!a.transpose && (each <= 2 || (each <= 8 && tiles_of<Little>(a) < 512))) return few_go<T>(a, s);
    if (each > 160 && tiles_of<Large>(a) >= 224) return tile_go<T, Large>(a, dma, s);
    if (each > 40 && tiles_of<Middle>(a) >= 256) return tile_go<T, Middle>(a, dma, s);
    return tile_go<T, Little>(a, dma, s);
}

template <class T>
hipError_t tiles_grad_go(const ExpertsArgs& a, hipStream_t s)
{
    const bool dma = a.in % 8 == 0 && a.out % 8 == 0 && lines16(a.x, a.ldx) && lines16(a.y, a.ldy);
    const double tiles = (double)a.experts * (double)a.out * (double)a.in / 65536.0;
    if (tiles >= 256.0) return tile_grad_go<T, Large>(a, dma, s);
    return tile_grad_go<T, Middle>(a, dma, s);
}

}  // namespace

hipError_t experts_launch(const ExpertsArgs& a, int dtype, hipStream_t s)
{
    switch (dtype) {
        case 0: return any_go<float>(a, s);
        case 1: return tiles_go<bf16_t>(a, s);
        case 2: return tiles_go<f16_t>(a, s);
        default: return hipErrorInvalidValue;
    }
}

hipError_t experts_grad_launch(const ExpertsArgs& a, int dtype, hipStream_t s)
{
    switch (dtype) {
        case 0: return any_grad_go<float>(a, s);
        case 1: return tiles_grad_go<bf16_t>(a, s);
        case 2: return tiles_grad_go<f16_t>(a, s);
        default: return hipErrorInvalidValue;
    }
}

}  // namespace lx

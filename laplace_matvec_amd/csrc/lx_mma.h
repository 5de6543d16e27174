// Matrix fragments of one wave (gfx950): products of 16 x 16 tiles with a
// contraction of 32 in float32 sums.
//
// A lane of group g = lane / 16 and row (column) r = lane % 16 holds 8 values
// of the contraction.  Which 8 does not matter as long as both operands agree;
// two orders are used:
//     along rows   8 g + i                        8 neighbours, one 16-byte load
//     across rows  4 g + i, 16 + 4 g + i (i < 4)  what a transposing LDS read
//                  gives, and what two 16 x 16 results side by side hold
// A result holds column lane % 16 and rows 4 g + i.
//
// 16-bit values go through v_mfma_f32_16x16x32 (16 cycles), float32 through
// eight v_mfma_f32_16x16x4 (32 cycles each), value i of each lane at a time.
#pragma once
#include "lx_types.h"

namespace lx {

typedef float f32x4 __attribute__((ext_vector_type(4)));

template <class E>
struct Frag {
    typedef E V __attribute__((ext_vector_type(8)));
    V v;
};

__device__ __forceinline__ f32x4 mma(const Frag<bf16_t>& a, const Frag<bf16_t>& b, f32x4 c)
{
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a.v, b.v, c, 0, 0, 0);
}
__device__ __forceinline__ f32x4 mma(const Frag<f16_t>& a, const Frag<f16_t>& b, f32x4 c)
{
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(a.v, b.v, c, 0, 0, 0);
}
__device__ __forceinline__ f32x4 mma(const Frag<float>& a, const Frag<float>& b, f32x4 c)
{
#pragma unroll
    for (int i = 0; i < 8; ++i) c = __builtin_amdgcn_mfma_f32_16x16x4f32(a.v[i], b.v[i], c, 0, 0, 0);
    return c;
}

// 8 neighbours from p on (LDS, 16-byte aligned): rows of the operand, contraction along them.
template <class E>
__device__ __forceinline__ Frag<E> frag_along(const E* p)
{
    Frag<E> f;
    f.v = *reinterpret_cast<const typename Frag<E>::V*>(p);
    return f;
}

// Contraction across rows of an LDS array: p is its first value, row pitch ld
// (8-byte aligned rows).  The operand's row is column lane % 16 from p on.
template <class E>
__device__ __forceinline__ Frag<E> frag_across(const E* p, int ld)
{
    const int lane = threadIdx.x & 63;
    Frag<E> f;
    if constexpr (sizeof(E) == 2) {
        // lane l of a group of 16 points at row l / 4, columns 4 (l % 4) .. + 3
        // of a 4 x 16 block and receives column l of it
        typedef short S4 __attribute__((ext_vector_type(4)));
        typedef __attribute__((address_space(3))) S4* At;
        const E* q = p + (4 * (lane >> 4) + ((lane & 15) >> 2)) * ld + 4 * (lane & 3);
        union { S4 s[2]; typename Frag<E>::V v; } u;
        u.s[0] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((At)(const_cast<E*>(q)));
        u.s[1] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((At)(const_cast<E*>(q + 16 * ld)));
        f.v = u.v;
    } else {
        const E* q = p + 4 * (lane >> 4) * ld + (lane & 15);
#pragma unroll
        for (int i = 0; i < 8; ++i) f.v[i] = q[(i < 4 ? i : i + 12) * ld];
    }
    return f;
}

// Contraction along rows in the order of frag_across: p is the row's first value.
template <class E>
__device__ __forceinline__ Frag<E> frag_along_split(const E* p)
{
    typedef E V4 __attribute__((ext_vector_type(4)));
    const int g = (threadIdx.x & 63) >> 4;
    union { V4 h[2]; typename Frag<E>::V v; } u;
    u.h[0] = *reinterpret_cast<const V4*>(p + 4 * g);
    u.h[1] = *reinterpret_cast<const V4*>(p + 16 + 4 * g);
    Frag<E> f;
    f.v = u.v;
    return f;
}

}  // namespace lx

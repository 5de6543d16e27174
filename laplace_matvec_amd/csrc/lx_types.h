// Storage types of the token operators (gfx950): float32, bfloat16 and
// float16 arrays moved in groups of V neighbouring values, arithmetic in
// float32.  Conversions round to nearest even (v_cvt_pk_bf16_f32 and
// v_cvt_f16_f32), once, at the store.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

namespace lx {

typedef __bf16 bf16_t;
typedef _Float16 f16_t;

template <class T, int V>
struct alignas(sizeof(T) * V) Pack {
    T v[V];
};

// What N bytes are moved as.
template <int N>
struct Words;
template <>
struct Words<2> { typedef uint16_t T; };
template <>
struct Words<4> { typedef uint32_t T; };
template <>
struct Words<8> { typedef uint32_t T __attribute__((ext_vector_type(2))); };
template <>
struct Words<16> { typedef uint32_t T __attribute__((ext_vector_type(4))); };

// Moves that leave the caches to others (non-temporal), for data that is not
// used again before it would have left them anyway.
template <class P>
__device__ __forceinline__ P load_once(const P* p)
{
    typedef typename Words<(int)sizeof(P)>::T W;
    return __builtin_bit_cast(P, __builtin_nontemporal_load(reinterpret_cast<const W*>(p)));
}
template <class P>
__device__ __forceinline__ void store_once(P* p, const P& v)
{
    typedef typename Words<(int)sizeof(P)>::T W;
    __builtin_nontemporal_store(__builtin_bit_cast(W, v), reinterpret_cast<W*>(p));
}

template <int V, class T>
__device__ __forceinline__ void load_vec(const T* p, float (&out)[V])
{
    const Pack<T, V> q = *reinterpret_cast<const Pack<T, V>*>(p);
#pragma unroll
    for (int i = 0; i < V; ++i) out[i] = (float)q.v[i];
}

template <int V, class T>
__device__ __forceinline__ Pack<T, V> round_vec(const float (&in)[V])
{
    Pack<T, V> q;
#pragma unroll
    for (int i = 0; i < V; ++i) q.v[i] = (T)in[i];
    return q;
}

template <int V, class T>
__device__ __forceinline__ void store_vec(T* p, const float (&in)[V])
{
    *reinterpret_cast<Pack<T, V>*>(p) = round_vec<V, T>(in);
}

template <int V, class T>
__device__ __forceinline__ void store_vec_once(T* p, const float (&in)[V])
{
    store_once(reinterpret_cast<Pack<T, V>*>(p), round_vec<V, T>(in));
}

// Whether rows of `width` values of `size` bytes, `ld` values apart from p
// on, can be moved in groups of v values.
inline bool vec_ok(const void* p, int64_t ld, int64_t width, size_t size, int v)
{
    return p == nullptr || (width % v == 0 && ld % v == 0 && (uintptr_t)p % (size * (size_t)v) == 0);
}

}  // namespace lx

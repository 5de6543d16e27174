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

// What N bytes are moved as, in a register and in memory: there only as
// aligned as their values of A bytes (the hardware takes any address).
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
template <int N, int A>
struct Mem {
    typedef typename Words<N>::T T __attribute__((aligned(A)));
};
template <class T, int V>
using MemOf = typename Mem<(int)sizeof(T) * V, (int)sizeof(T)>::T;

// V neighbouring values from p on.  The `once` forms leave the caches to
// others (non-temporal), for data that is not used again before it would
// have left them anyway.
template <int V, class T>
__device__ __forceinline__ Pack<T, V> load_pack(const T* p)
{
    const typename Words<(int)sizeof(T) * V>::T w = *reinterpret_cast<const MemOf<T, V>*>(p);
    return __builtin_bit_cast(Pack<T, V>, w);
}
template <int V, class T>
__device__ __forceinline__ Pack<T, V> load_once(const T* p)
{
    const typename Words<(int)sizeof(T) * V>::T w = __builtin_nontemporal_load(reinterpret_cast<const MemOf<T, V>*>(p));
    return __builtin_bit_cast(Pack<T, V>, w);
}
template <int V, class T>
__device__ __forceinline__ void store_pack(T* p, const Pack<T, V>& v)
{
    *reinterpret_cast<MemOf<T, V>*>(p) = __builtin_bit_cast(typename Words<(int)sizeof(T) * V>::T, v);
}
template <int V, class T>
__device__ __forceinline__ void store_once(T* p, const Pack<T, V>& v)
{
    __builtin_nontemporal_store(__builtin_bit_cast(typename Words<(int)sizeof(T) * V>::T, v),
                                reinterpret_cast<MemOf<T, V>*>(p));
}

template <int V, class T>
__device__ __forceinline__ void load_vec(const T* p, float (&out)[V])
{
    const Pack<T, V> q = load_pack<V>(p);
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
    store_pack<V>(p, round_vec<V, T>(in));
}

template <int V, class T>
__device__ __forceinline__ void store_vec_once(T* p, const float (&in)[V])
{
    store_once<V>(p, round_vec<V, T>(in));
}

// Either, as `once` says.  The empty statements keep the two stores apart:
// the compiler would make one of them and drop the hint.
template <int V, class T>
__device__ __forceinline__ void store_vec_as(T* p, const float (&in)[V], bool once)
{
    const Pack<T, V> q = round_vec<V, T>(in);
    if (once) {
        asm volatile("");
        store_once<V>(p, q);
        asm volatile("");
    } else {
        store_pack<V>(p, q);
    }
}

}  // namespace lx

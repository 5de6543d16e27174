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

template <int V, class T>
__device__ __forceinline__ void load_vec(const T* p, float (&out)[V])
{
    const Pack<T, V> q = *reinterpret_cast<const Pack<T, V>*>(p);
#pragma unroll
    for (int i = 0; i < V; ++i) out[i] = (float)q.v[i];
}

template <int V, class T>
__device__ __forceinline__ void store_vec(T* p, const float (&in)[V])
{
    Pack<T, V> q;
#pragma unroll
    for (int i = 0; i < V; ++i) q.v[i] = (T)in[i];
    *reinterpret_cast<Pack<T, V>*>(p) = q;
}

// Whether rows of `width` values of `size` bytes, `ld` values apart from p
// on, can be moved in groups of v values.
inline bool vec_ok(const void* p, int64_t ld, int64_t width, size_t size, int v)
{
    return p == nullptr || (width % v == 0 && ld % v == 0 && (uintptr_t)p % (size * (size_t)v) == 0);
}

}  // namespace lx

// Vector loads and stores of the training-head kernels: K elements of a
// storage type as fp32 values. The addresses need only the alignment of one
// element: gfx950's global loads and stores take any such address (unaligned
// access mode, which the HSA runtime sets), and a wave's consecutive 16-byte
// pieces then touch one cache line more than aligned ones.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

namespace im2win {

template <typename T, int K>
struct __attribute__((packed, aligned(sizeof(T)))) Pack {
    T v[K];
};

template <int K, typename T>
__device__ __forceinline__ void load_vec(const T *p, float (&f)[K])
{
    const Pack<T, K> q = *reinterpret_cast<const Pack<T, K> *>(p);
#pragma unroll
    for (int e = 0; e < K; ++e) f[e] = static_cast<float>(q.v[e]);
}

template <int K, typename T>
__device__ __forceinline__ void store_vec(T *p, const float (&f)[K])
{
    Pack<T, K> q;
#pragma unroll
    for (int e = 0; e < K; ++e) q.v[e] = static_cast<T>(f[e]);
    *reinterpret_cast<Pack<T, K> *>(p) = q;
}

// the first n elements (0 <= n); the others read as 0 and are not touched
template <int K, typename T>
__device__ __forceinline__ void load_some(const T *p, int n, float (&f)[K])
{
    if (n >= K) {
        load_vec<K>(p, f);
    } else {
#pragma unroll
        for (int e = 0; e < K; ++e) f[e] = e < n ? static_cast<float>(p[e]) : 0.f;
    }
}

template <int K, typename T>
__device__ __forceinline__ void store_some(T *p, int n, const float (&f)[K])
{
    if (n >= K) {
        store_vec<K>(p, f);
    } else {
#pragma unroll
        for (int e = 0; e < K; ++e)
            if (e < n) p[e] = static_cast<T>(f[e]);
    }
}

}  // namespace im2win

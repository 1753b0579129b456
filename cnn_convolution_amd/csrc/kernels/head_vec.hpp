// Vector loads and stores of the training-head kernels: K elements of a
// storage type, as fp32 values or as stored (Raw). The addresses need only the
// alignment of one element: gfx950's global loads and stores take any such
// address (unaligned access mode, which the HSA runtime sets), and a wave's
// consecutive 16-byte pieces then touch one cache line more than aligned ones.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>
#include <type_traits>

namespace im2win {

// K elements as stored, two half-precision ones to a dword
template <typename T, int K>
struct Raw {
    static constexpr int ND = K * int(sizeof(T)) / 4;
    uint32_t d[ND];
};

template <typename T, int K>
__device__ __forceinline__ Raw<T, K> load_raw(const T *p)
{
    constexpr int ND = Raw<T, K>::ND, W = ND < 4 ? ND : 4;
    typedef uint32_t vec __attribute__((ext_vector_type(W), aligned(sizeof(T))));
    Raw<T, K> r;
#pragma unroll
    for (int i = 0; i < ND; i += W) {
        const vec v = *reinterpret_cast<const vec *>(reinterpret_cast<const char *>(p) + i * 4);
#pragma unroll
        for (int e = 0; e < W; ++e) r.d[i + e] = v[e];
    }
    return r;
}

template <typename T, int K>
__device__ __forceinline__ float element(const Raw<T, K> &r, int e)
{
    if constexpr (sizeof(T) == 4) return __uint_as_float(r.d[e]);
    const uint32_t u = r.d[e / 2];
    if constexpr (std::is_same<T, __bf16>::value) return __uint_as_float(e & 1 ? u & 0xFFFF0000u : u << 16);
    return static_cast<float>(__builtin_bit_cast(_Float16, uint16_t(e & 1 ? u >> 16 : u)));
}

// all elements kept (mask ~0) or cleared (mask 0): as a mask, for a choice between
// values may become a branch
template <typename T, int K>
__device__ __forceinline__ void keep_if(Raw<T, K> &r, uint32_t mask)
{
#pragma unroll
    for (int i = 0; i < Raw<T, K>::ND; ++i) r.d[i] &= mask;
}

// r moved down by s elements (s >= 0), zeros moving in
template <typename T, int K>
__device__ __forceinline__ void shift_down(Raw<T, K> &r, int s)
{
    constexpr int ND = Raw<T, K>::ND;
    const int ds = sizeof(T) == 2 ? s >> 1 : s;
#pragma unroll
    for (int b = 1; b < ND; b <<= 1)
#pragma unroll
        for (int i = 0; i < ND; ++i) r.d[i] = ds & b ? (i + b < ND ? r.d[i + b] : 0u) : r.d[i];
    if constexpr (sizeof(T) == 2) {
#pragma unroll
        for (int i = 0; i < ND; ++i) {
            const uint32_t up = i + 1 < ND ? r.d[i + 1] : 0u;
            r.d[i] = s & 1 ? (r.d[i] >> 16 | up << 16) : r.d[i];
        }
    }
#pragma unroll
    for (int i = 0; i < ND; ++i) r.d[i] = s >= K ? 0u : r.d[i];
}

// Elements c .. c + K - 1 of a row of `count` >= K elements, zeros past its end,
// without a branch (a branch around a load makes the wave wait for it there): the
// last K elements of the row are read instead and moved down. EXACT: count is a
// multiple of K and what lies past the end is not used, so nothing is moved.
template <typename T, int K, bool EXACT>
__device__ __forceinline__ Raw<T, K> load_row(const T *row, int64_t c, int64_t count)
{
    const int64_t at = c < count - K ? c : count - K;
    Raw<T, K> r = load_raw<T, K>(row + at);
    if constexpr (!EXACT) shift_down(r, int(c - at < K ? c - at : K));
    return r;
}

template <int K, typename T>
__device__ __forceinline__ void load_vec(const T *p, float (&f)[K])
{
    const Raw<T, K> r = load_raw<T, K>(p);
#pragma unroll
    for (int e = 0; e < K; ++e) f[e] = element(r, e);
}

template <typename T, int K>
__device__ __forceinline__ Raw<T, K> to_raw(const float (&f)[K])
{
    Raw<T, K> r;
    if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int e = 0; e < K; ++e) r.d[e] = __float_as_uint(f[e]);
    } else {
        typedef T pair __attribute__((ext_vector_type(2)));
#pragma unroll
        for (int e = 0; e < K; e += 2)
            r.d[e / 2] = __builtin_bit_cast(uint32_t, pair{static_cast<T>(f[e]), static_cast<T>(f[e + 1])});
    }
    return r;
}

template <typename T, int K>
__device__ __forceinline__ void store_raw(T *p, const Raw<T, K> &r)
{
    constexpr int ND = Raw<T, K>::ND, W = ND < 4 ? ND : 4;
    typedef uint32_t vec __attribute__((ext_vector_type(W), aligned(sizeof(T))));
#pragma unroll
    for (int i = 0; i < ND; i += W) {
        vec v;
#pragma unroll
        for (int e = 0; e < W; ++e) v[e] = r.d[i + e];
        *reinterpret_cast<vec *>(reinterpret_cast<char *>(p) + i * 4) = v;
    }
}

// Waits for the loads of r. Loads and stores return in order, and behind a
// branch the compiler cannot count the stores: a wait for loads that come
// before such stores would wait for the stores too, so prefetched loads are
// waited for ahead of them. (The values become opaque to the compiler here.)
template <typename T, int K>
__device__ __forceinline__ void arrive(Raw<T, K> &r)
{
#pragma unroll
    for (int i = 0; i < Raw<T, K>::ND; ++i) asm volatile("" : "+v"(r.d[i]));
}

template <int K, typename T>
__device__ __forceinline__ void store_vec(T *p, const float (&f)[K])
{
    store_raw(p, to_raw<T, K>(f));
}

// the first n elements (0 <= n); the others read as 0 and are not touched
template <int K, typename T>
__device__ __forceinline__ void load_some(const T *p, int64_t n, float (&f)[K])
{
    if (n >= K) {
        load_vec<K>(p, f);
    } else {
#pragma unroll
        for (int e = 0; e < K; ++e) f[e] = e < n ? static_cast<float>(p[e]) : 0.f;
    }
}

template <typename T, int K>
__device__ __forceinline__ void store_some_raw(T *p, int64_t n, const Raw<T, K> &r)
{
    if (n >= K) {
        store_raw(p, r);
    } else {
#pragma unroll
        for (int e = 0; e < K; ++e) {
            if (e >= n) break;
            if constexpr (sizeof(T) == 4)
                p[e] = __uint_as_float(r.d[e]);
            else
                reinterpret_cast<uint16_t *>(p)[e] = uint16_t(e & 1 ? r.d[e / 2] >> 16 : r.d[e / 2]);
        }
    }
}

template <int K, typename T>
__device__ __forceinline__ void store_some(T *p, int64_t n, const float (&f)[K])
{
    store_some_raw(p, n, to_raw<T, K>(f));
}

// sum over the L lanes (a power of two up to 64) of an aligned group: within 16
// lanes by data-parallel moves (lane pairs, pairs of pairs, mirrored halves),
// then between rows of 16 and halves of 32 by lane swaps
template <int L>
__device__ __forceinline__ float lane_sum(float v)
{
    auto dpp = [](float x, auto ctrl) {
        return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(x), decltype(ctrl)::value, 0xF, 0xF, true));
    };
    using std::integral_constant;
    if constexpr (L >= 2) v += dpp(v, integral_constant<int, 0xB1>{});    // quad_perm 1,0,3,2
    if constexpr (L >= 4) v += dpp(v, integral_constant<int, 0x4E>{});    // quad_perm 2,3,0,1
    if constexpr (L >= 8) v += dpp(v, integral_constant<int, 0x141>{});   // row_half_mirror
    if constexpr (L >= 16) v += dpp(v, integral_constant<int, 0x140>{});  // row_mirror
    if constexpr (L >= 32) {
        const auto p = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
        v = __uint_as_float(p[0]) + __uint_as_float(p[1]);
    }
    if constexpr (L >= 64) {
        const auto p = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
        v = __uint_as_float(p[0]) + __uint_as_float(p[1]);
    }
    return v;
}

}  // namespace im2win

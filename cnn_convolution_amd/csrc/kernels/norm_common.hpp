// Shared by the layer-norm kernels: type dispatch, dropout of a run of
// elements, and the second step of the weight-gradient reduction.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

#include "../head_launch.hpp"
#include "head_vec.hpp"
#include "philox.hpp"

namespace im2win {

template <typename T>
struct TypeTag {
    using type = T;
};

// f(TypeTag<type of x>, TypeTag<type of y>)
template <typename F>
hipError_t with_norm_types(int dtype, int y_dtype, F f)
{
    if (dtype == 0 && y_dtype == 0) return f(TypeTag<float>{}, TypeTag<float>{});
    if (dtype == 0 && y_dtype == 1) return f(TypeTag<float>{}, TypeTag<_Float16>{});
    if (dtype == 0 && y_dtype == 2) return f(TypeTag<float>{}, TypeTag<__bf16>{});
    if (dtype == 1 && y_dtype == 1) return f(TypeTag<_Float16>{}, TypeTag<_Float16>{});
    if (dtype == 2 && y_dtype == 2) return f(TypeTag<__bf16>{}, TypeTag<__bf16>{});
    return hipErrorInvalidValue;
}

// dropout of elements first .. first + K - 1
template <int K>
__device__ __forceinline__ void drop_run(int64_t first, const DropSpec &d, float (&f)[K])
{
    if constexpr (K == 8) {
        if ((first & 7) == 0) {
            drop_block(uint64_t(first) >> 3, d, f);
            return;
        }
    }
    const uint32_t keep = keep_run<K>(first, d);
#pragma unroll
    for (int e = 0; e < K; ++e) f[e] = (keep >> e) & 1 ? f[e] * d.scale : 0.f;
}

// dweight, dbias from the blocks' partial sums [rows][2][C], in a fixed order
hipError_t launch_norm_reduce(const float *partial, int64_t rows, int C, float *dweight, float *dbias,
                              hipStream_t s);

}  // namespace im2win

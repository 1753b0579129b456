// Dropout from a counter-based generator: y = keep ? x * scale : 0, one
// counter block per 8 elements (im2win_head.h). Bound by HBM: every element is
// read and written once, the mask is arithmetic. A thread takes whole blocks of
// 8 elements, a grid's width apart: 16-byte accesses for half precision, and a
// Philox block costs 199 cycles of a SIMD per 64 of them, half of what its memory
// traffic takes. 2^27 bf16 elements in 99 us, 5.4 TB/s.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstdint>

#include "../head_launch.hpp"
#include "head_vec.hpp"
#include "philox.hpp"

namespace im2win {
namespace {

template <typename T>
__global__ __launch_bounds__(256) void dropout_kernel(const T *x, T *y, int64_t n, const DropSpec d)
{
    const int64_t blocks = (n + 7) >> 3, step = int64_t(gridDim.x) * 256;
    for (int64_t b = int64_t(blockIdx.x) * 256 + threadIdx.x; b < blocks; b += step) {
        const int m = int(min(int64_t(8), n - b * 8));
        float f[8];
        load_some<8>(x + b * 8, m, f);
        drop_block(uint64_t(b), d, f);
        store_some<8>(y + b * 8, m, f);
    }
}

}  // namespace

hipError_t launch_dropout(const void *x, void *y, int64_t n, int dtype, const DropSpec &d, hipStream_t s)
{
    const int64_t blocks = (n + 7) / 8;
    const dim3 grid(unsigned(std::min<int64_t>((blocks + 255) / 256, 256 * 16)));
    if (dtype == 0)
        hipLaunchKernelGGL((dropout_kernel<float>), grid, dim3(256), 0, s, static_cast<const float *>(x),
                           static_cast<float *>(y), n, d);
    else if (dtype == 1)
        hipLaunchKernelGGL((dropout_kernel<_Float16>), grid, dim3(256), 0, s,
                           static_cast<const _Float16 *>(x), static_cast<_Float16 *>(y), n, d);
    else
        hipLaunchKernelGGL((dropout_kernel<__bf16>), grid, dim3(256), 0, s, static_cast<const __bf16 *>(x),
                           static_cast<__bf16 *>(y), n, d);
    return hipGetLastError();
}

}  // namespace im2win

// Softmax cross entropy of a linear classifier, logits x w^T formed tile by
// tile and never stored: forward (loss, lse) and backward (dx, dw).
//
// Forward: each 64 classes x 64 rows tile of logits is reduced in its
// workgroup to one (maximum, sum of exponentials around it) per row; a second
// kernel joins a row's partials in a fixed order. Backward: pieces of the
// classes; a piece's G = S * grad * (exp(l - lse) - [target]) goes to the
// workspace in the type of x (S a power of two that places the largest |grad|
// near the top of fp16's range, 1 for the other types), then dx += G w and
// dw = G^T x.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstdint>

#include "../head_launch.hpp"
#include "lds_dma.hpp"

namespace im2win {
namespace {

constexpr int TM = 64, TN = 64, BK = 32, kThreads = 256;

template <typename T>
__device__ __forceinline__ floatx4_t mfma_k32(const T *a, const T *b, floatx4_t c)
{
    // a, b: 8 consecutive K values of this lane's row (lane group g: K 8g ..)
    if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int e = 0; e < 8; ++e) c = __builtin_amdgcn_mfma_f32_16x16x4f32(a[e], b[e], c, 0, 0, 0);
        return c;
    } else {
        return mfma16x16x32<std::is_same<T, __bf16>::value>(*reinterpret_cast<const uint4 *>(a),
                                                            *reinterpret_cast<const uint4 *>(b), c);
    }
}

struct Operand {
    const void *p;
    int64_t row, k;          // strides in elements
    int64_t rows;
};

// acc[i][j]: 16x16 blocks of the workgroup's 64 x 64 tile; wave w holds rows
// m 32*(w%2) + 16i + 4*(lane/16) + v, columns 32*(w/2) + 16j + lane%16
template <typename T>
__device__ __forceinline__ void tile_product(const Operand &A, const Operand &B, int64_t K, int64_t m0,
                                             int64_t n0, floatx4_t (&acc)[2][2])
{
    __shared__ __align__(16) T sa[TM][BK + 16 / sizeof(T)], sb[TN][BK + 16 / sizeof(T)];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int ar = (wave & 1) * 32 + (lane & 15), br = (wave >> 1) * 32 + (lane & 15), kk = (lane >> 4) * 8;
    const T *ap = static_cast<const T *>(A.p), *bp = static_cast<const T *>(B.p);
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j) acc[i][j] = floatx4_t{0.f, 0.f, 0.f, 0.f};
    for (int64_t k0 = 0; k0 < K; k0 += BK) {
        __syncthreads();
        for (int i = threadIdx.x; i < TM * BK; i += kThreads) {
            // consecutive threads along the operand's contiguous index
            const int r = A.k == 1 ? i / BK : i % TM, k = A.k == 1 ? i % BK : i / TM;
            const bool ok = m0 + r < A.rows && k0 + k < K;
            sa[r][k] = ok ? ap[(m0 + r) * A.row + (k0 + k) * A.k] : T(0.f);
        }
        for (int i = threadIdx.x; i < TN * BK; i += kThreads) {
            const int r = B.k == 1 ? i / BK : i % TN, k = B.k == 1 ? i % BK : i / TN;
            const bool ok = n0 + r < B.rows && k0 + k < K;
            sb[r][k] = ok ? bp[(n0 + r) * B.row + (k0 + k) * B.k] : T(0.f);
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int j = 0; j < 2; ++j) acc[i][j] = mfma_k32<T>(&sa[ar + 16 * i][kk], &sb[br + 16 * j][kk], acc[i][j]);
    }
}

__device__ __forceinline__ bool valid_target(int64_t t, int64_t V) { return t >= 0 && t < V; }

// partial (maximum, sum) of each row over this tile's classes; the target's
// logit goes to a.loss
template <typename T>
__global__ __launch_bounds__(kThreads) void xent_loss_kernel(const XentArgs a, float2 *partial)
{
    __shared__ float2 red[2][TN];
    const int64_t m0 = int64_t(blockIdx.x) * TM, n0 = int64_t(blockIdx.y) * TN;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    floatx4_t acc[2][2];
    tile_product<T>(Operand{a.w, a.ldw, 1, a.V}, Operand{a.x, a.ldx, 1, a.N}, a.D, m0, n0, acc);
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        const int col = (wave >> 1) * 32 + 16 * j + (lane & 15);
        const int64_t row = n0 + col;
        const int64_t t = row < a.N ? a.target[row] : -1;
        float m = -__builtin_inff(), s = 0.f;
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int v = 0; v < 4; ++v) {
                const int64_t cls = m0 + (wave & 1) * 32 + 16 * i + (lane >> 4) * 4 + v;
                if (cls < a.V) {
                    m = fmaxf(m, acc[i][j][v]);
                    if (cls == t) a.loss[row] = acc[i][j][v];
                }
            }
        m = fmaxf(m, __shfl_xor(m, 16, 64));
        m = fmaxf(m, __shfl_xor(m, 32, 64));
        const float mm = m == -__builtin_inff() ? 0.f : m;
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int v = 0; v < 4; ++v)
                if (m0 + (wave & 1) * 32 + 16 * i + (lane >> 4) * 4 + v < a.V) s += __expf(acc[i][j][v] - mm);
        s += __shfl_xor(s, 16, 64);
        s += __shfl_xor(s, 32, 64);
        if (lane < 16) red[wave & 1][col] = float2{m, s};
    }
    __syncthreads();
    if (threadIdx.x < TN && n0 + threadIdx.x < a.N) {
        const float2 p = red[0][threadIdx.x], q = red[1][threadIdx.x];
        const float m = fmaxf(p.x, q.x), mm = m == -__builtin_inff() ? 0.f : m;
        partial[blockIdx.x * a.N + n0 + threadIdx.x] =
            float2{m, p.y * __expf(p.x - mm) + q.y * __expf(q.x - mm)};
    }
}

// one wave per row: lse over the tiles' partials, then the loss
__global__ __launch_bounds__(256) void xent_join_kernel(const XentArgs a, const float2 *partial, int tiles)
{
    const int64_t row = int64_t(blockIdx.x) * 4 + (threadIdx.x >> 6);
    const int lane = threadIdx.x & 63;
    if (row >= a.N) return;
    float m = -__builtin_inff(), s = 0.f;
    for (int t = lane; t < tiles; t += 64) m = fmaxf(m, partial[t * a.N + row].x);
    for (int k = 1; k < 64; k <<= 1) m = fmaxf(m, __shfl_xor(m, k, 64));
    const float mm = m == -__builtin_inff() ? 0.f : m;
    for (int t = lane; t < tiles; t += 64) {
        const float2 p = partial[t * a.N + row];
        s += p.y * __expf(p.x - mm);
    }
    for (int k = 1; k < 64; k <<= 1) s += __shfl_xor(s, k, 64);
    if (lane == 0) {
        const float lse = mm + logf(s);
        const bool ok = valid_target(a.target[row], a.V);
        a.loss[row] = ok ? lse - a.loss[row] : 0.f;
        a.lse[row] = ok ? lse : 0.f;
    }
}

// S: the power of two with S * max |grad| in [2^14, 2^15]
__global__ __launch_bounds__(1024) void xent_scale_kernel(const float *grad, int64_t N, float *scale)
{
    __shared__ float red[16];
    float m = 0.f;
    for (int64_t i = threadIdx.x; i < N; i += 1024) m = fmaxf(m, fabsf(grad[i]));
    for (int k = 1; k < 64; k <<= 1) m = fmaxf(m, __shfl_xor(m, k, 64));
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = m;
    __syncthreads();
    if (threadIdx.x == 0) {
        for (int w = 1; w < 16; ++w) m = fmaxf(m, red[w]);
        int e = 0;
        const bool ok = m > 0.f && m < __builtin_inff();
        if (ok) (void)frexpf(m, &e);
        e = max(-100, min(100, 15 - e));
        scale[0] = ok ? ldexpf(1.f, e) : 1.f;
        scale[1] = ok ? ldexpf(1.f, -e) : 1.f;
    }
}

// x with the masked rows cleared
template <typename T>
__global__ __launch_bounds__(256) void xent_rows_kernel(const XentArgs a, T *xs)
{
    const int64_t row = blockIdx.x;
    const bool ok = valid_target(a.target[row], a.V);
    const T *x = static_cast<const T *>(a.x) + row * a.ldx;
    for (int64_t d = threadIdx.x; d < a.D; d += 256) xs[row * a.D + d] = ok ? x[d] : T(0.f);
}

// G of classes v0 .. v0 + P - 1 into g [N][P]
template <typename T>
__global__ __launch_bounds__(kThreads) void xent_g_kernel(const XentArgs a, int64_t v0, int64_t P, T *g,
                                                          const float *scale)
{
    const int64_t m0 = int64_t(blockIdx.x) * TM, n0 = int64_t(blockIdx.y) * TN;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    floatx4_t acc[2][2];
    tile_product<T>(Operand{static_cast<const T *>(a.w) + v0 * a.ldw, a.ldw, 1, P}, Operand{a.x, a.ldx, 1, a.N},
                    a.D, m0, n0, acc);
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        const int64_t row = n0 + (wave >> 1) * 32 + 16 * j + (lane & 15);
        if (row >= a.N) continue;
        const int64_t t = a.target[row];
        const bool ok = valid_target(t, a.V);
        const float lse = a.lse[row], gs = a.grad[row] * scale[0];
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int v = 0; v < 4; ++v) {
                const int64_t m = m0 + (wave & 1) * 32 + 16 * i + (lane >> 4) * 4 + v;
                if (m >= P) continue;
                const float q = expf(acc[i][j][v] - lse) - (v0 + m == t ? 1.f : 0.f);
                g[row * P + m] = T(ok ? gs * q : 0.f);
            }
    }
}

// dx += G w for one piece into fp32 sums [N][D]
template <typename T>
__global__ __launch_bounds__(kThreads) void xent_dx_kernel(const XentArgs a, int64_t v0, int64_t P, const T *g,
                                                           float *sum)
{
    const int64_t m0 = int64_t(blockIdx.x) * TM, n0 = int64_t(blockIdx.y) * TN;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    floatx4_t acc[2][2];
    tile_product<T>(Operand{static_cast<const T *>(a.w) + v0 * a.ldw, 1, a.ldw, a.D}, Operand{g, P, 1, a.N}, P, m0,
                    n0, acc);
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        const int64_t row = n0 + (wave >> 1) * 32 + 16 * j + (lane & 15);
        if (row >= a.N) continue;
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int v = 0; v < 4; ++v) {
                const int64_t m = m0 + (wave & 1) * 32 + 16 * i + (lane >> 4) * 4 + v;
                if (m < a.D) sum[row * a.D + m] = acc[i][j][v] + (v0 ? sum[row * a.D + m] : 0.f);
            }
    }
}

template <typename T>
__global__ __launch_bounds__(256) void xent_dx_out_kernel(const float *sum, int64_t n, const float *scale, T *dx)
{
    const int64_t i = int64_t(blockIdx.x) * 256 + threadIdx.x;
    if (i < n) dx[i] = T(sum[i] * scale[1]);
}

// dw of one piece = G^T x
template <typename T>
__global__ __launch_bounds__(kThreads) void xent_dw_kernel(const XentArgs a, int64_t v0, int64_t P, const T *g,
                                                           const T *xs, const float *scale)
{
    const int64_t m0 = int64_t(blockIdx.x) * TM, n0 = int64_t(blockIdx.y) * TN;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    floatx4_t acc[2][2];
    tile_product<T>(Operand{xs, 1, a.D, a.D}, Operand{g, 1, P, P}, a.N, m0, n0, acc);
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        const int64_t cls = n0 + (wave >> 1) * 32 + 16 * j + (lane & 15);
        if (cls >= P) continue;
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int v = 0; v < 4; ++v) {
                const int64_t m = m0 + (wave & 1) * 32 + 16 * i + (lane >> 4) * 4 + v;
                if (m < a.D) static_cast<T *>(a.dw)[(v0 + cls) * a.D + m] = T(acc[i][j][v] * scale[1]);
            }
    }
}

template <typename T>
__global__ __launch_bounds__(256) void xent_zero_kernel(T *p, int64_t n)
{
    const int64_t i = int64_t(blockIdx.x) * 256 + threadIdx.x;
    if (i < n) p[i] = T(0.f);
}

int64_t round_up(int64_t v, int64_t m) { return (v + m - 1) / m * m; }
int64_t elem(int dtype) { return dtype == 0 ? 4 : 2; }
unsigned tiles(int64_t n, int t) { return unsigned((n + t - 1) / t); }

constexpr int64_t kPieceBytes = int64_t(128) << 20;   // of G
int64_t piece_classes(int64_t N, int64_t V, int dtype)
{
    return std::min(round_up(V, TM), std::max<int64_t>(TM, kPieceBytes / (N * elem(dtype)) / TM * TM));
}

template <typename F>
hipError_t with_type(int dtype, F f)
{
    if (dtype == 0) return f(float{});
    if (dtype == 1) return f(_Float16{});
    return f(__bf16{});
}

}  // namespace

int64_t xent_fwd_ws_bytes(int64_t N, int64_t V, int64_t D, int64_t ldx, int64_t ldw, int dtype)
{
    return round_up(int64_t(tiles(V, TM)) * N * 8, 256);
}

int64_t xent_bwd_ws_bytes(int64_t N, int64_t V, int64_t D, int64_t ldx, int64_t ldw, int dtype)
{
    if (N == 0) return 0;
    return 256 + round_up(N * D * elem(dtype), 256) + round_up(N * D * 4, 256) +
           round_up(N * piece_classes(N, V, dtype) * elem(dtype), 256);
}

hipError_t launch_xent_fwd(const XentArgs &a, hipStream_t s)
{
    if (a.N == 0) return hipSuccess;
    float2 *partial = static_cast<float2 *>(a.ws);
    const dim3 grid(tiles(a.V, TM), tiles(a.N, TN));
    return with_type(a.dtype, [&](auto t) {
        using T = decltype(t);
        hipLaunchKernelGGL((xent_loss_kernel<T>), grid, dim3(kThreads), 0, s, a, partial);
        hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
        hipLaunchKernelGGL(xent_join_kernel, dim3(tiles(a.N, 4)), dim3(256), 0, s, a, partial, int(grid.x));
        return hipGetLastError();
    });
}

hipError_t launch_xent_bwd(const XentArgs &a, hipStream_t s)
{
    return with_type(a.dtype, [&](auto tt) {
        using T = decltype(tt);
        if (a.N == 0) {
            const int64_t n = a.V * a.D;
            hipLaunchKernelGGL((xent_zero_kernel<T>), dim3(tiles(n, 256)), dim3(256), 0, s, static_cast<T *>(a.dw),
                               n);
            return hipGetLastError();
        }
        char *p = static_cast<char *>(a.ws);
        float *scale = reinterpret_cast<float *>(p);
        p += 256;
        T *xs = reinterpret_cast<T *>(p);
        p += round_up(a.N * a.D * int64_t(sizeof(T)), 256);
        float *sum = reinterpret_cast<float *>(p);
        p += round_up(a.N * a.D * 4, 256);
        T *g = reinterpret_cast<T *>(p);
        hipLaunchKernelGGL(xent_scale_kernel, dim3(1), dim3(1024), 0, s, a.grad, a.N, scale);
        hipLaunchKernelGGL((xent_rows_kernel<T>), dim3(unsigned(a.N)), dim3(256), 0, s, a, xs);
        const int64_t step = piece_classes(a.N, a.V, a.dtype);
        for (int64_t v0 = 0; v0 < a.V; v0 += step) {
            const int64_t P = std::min(step, a.V - v0);
            hipLaunchKernelGGL((xent_g_kernel<T>), dim3(tiles(P, TM), tiles(a.N, TN)), dim3(kThreads), 0, s, a, v0,
                               P, g, scale);
            hipLaunchKernelGGL((xent_dx_kernel<T>), dim3(tiles(a.D, TM), tiles(a.N, TN)), dim3(kThreads), 0, s, a,
                               v0, P, g, sum);
            hipLaunchKernelGGL((xent_dw_kernel<T>), dim3(tiles(a.D, TM), tiles(P, TN)), dim3(kThreads), 0, s, a, v0,
                               P, g, xs, scale);
        }
        hipLaunchKernelGGL((xent_dx_out_kernel<T>), dim3(tiles(a.N * a.D, 256)), dim3(256), 0, s, sum, a.N * a.D,
                           scale, static_cast<T *>(a.dx));
        return hipGetLastError();
    });
}

}  // namespace im2win

// Philox4x32-10 (Salmon, Moraes, Dror, Shaw, "Parallel random numbers: as easy
// as 1, 2, 3", SC 2011): ten rounds of two 32 x 32 -> 64 bit products over a
// 128-bit counter. A block gives eight 16-bit numbers, one per element: with 32
// bits per element the products (quarter rate on the vector ALUs) would be
// what a half-precision dropout waits for.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

#include "../head_launch.hpp"

namespace im2win {

// a ^ b ^ c as one gfx950 instruction (two take a quarter more time over the
// ten rounds: 264 against 199 cycles of a SIMD per 64 blocks)
__device__ __forceinline__ uint32_t xor3(uint32_t a, uint32_t b, uint32_t c)
{
    return __builtin_amdgcn_bitop3_b32(a, b, c, 0x96);
}

// counter (block, high), 64 bits each
__device__ __forceinline__ uint4 philox(uint64_t block, uint64_t high, uint64_t seed)
{
    uint32_t c0 = uint32_t(block), c1 = uint32_t(block >> 32), c2 = uint32_t(high), c3 = uint32_t(high >> 32);
    uint32_t k0 = uint32_t(seed), k1 = uint32_t(seed >> 32);
#pragma unroll
    for (int r = 0; r < 10; ++r) {
        const uint64_t a = uint64_t(c0) * 0xD2511F53u, b = uint64_t(c2) * 0xCD9E8D57u;
        c0 = xor3(uint32_t(b >> 32), c1, k0);
        c1 = uint32_t(b);
        c2 = xor3(uint32_t(a >> 32), c3, k1);
        c3 = uint32_t(a);
        k0 += 0x9E3779B9u;
        k1 += 0xBB67AE85u;
    }
    return uint4{c0, c1, c2, c3};
}

// bit j: element j of the block is kept
__device__ __forceinline__ uint32_t keep_bits(uint64_t block, const DropSpec &d)
{
    const uint4 w = philox(d.offset + block, 0, d.seed);
    const uint32_t v[4] = {w.x, w.y, w.z, w.w};
    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        m |= uint32_t((v[j] & 0xFFFFu) >= d.threshold) << (2 * j);
        m |= uint32_t((v[j] >> 16) >= d.threshold) << (2 * j + 1);
    }
    return m;
}

// a whole block: f = kept ? f * scale : 0
__device__ __forceinline__ void drop_block(uint64_t block, const DropSpec &d, float (&f)[8])
{
    const uint4 w = philox(d.offset + block, 0, d.seed);
    const uint32_t v[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        f[2 * j] = (v[j] & 0xFFFFu) >= d.threshold ? f[2 * j] * d.scale : 0.f;
        f[2 * j + 1] = (v[j] >> 16) >= d.threshold ? f[2 * j + 1] * d.scale : 0.f;
    }
}

// bit j: element first + j is kept, j < K (K <= 8); the run may cross into
// the next block
template <int K>
__device__ __forceinline__ uint32_t keep_run(int64_t first, const DropSpec &d)
{
    const uint32_t s = uint32_t(first) & 7;
    uint32_t m = keep_bits(uint64_t(first) >> 3, d) >> s;
    if (s + K > 8) m |= keep_bits((uint64_t(first) >> 3) + 1, d) << (8 - s);
    return m;
}

}  // namespace im2win

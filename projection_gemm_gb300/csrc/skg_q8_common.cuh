// skg_q8_common.cuh -- device code shared by the 8-bit path's kernels.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "skg_q8_internal.h"

namespace skg {

__device__ __forceinline__ float bf16_to_f32(uint16_t b) { return __uint_as_float(static_cast<uint32_t>(b) << 16); }

__device__ __forceinline__ uint16_t f32_to_bf16(float v) { return __bfloat16_as_ushort(__float2bfloat16_rn(v)); }

// silu(g) = g / (1 + exp(-g)), from exp(-|g|) so that neither side overflows
// (at g = -89 exp(-g) has left fp32 while the quotient has not).  The fast
// exponential, off by up to 2 + |g| units in the last place: of 67 million gated
// values 5.8e-7 get another integer than in 64 bits, with expf 5.7e-7, in plain
// 32-bit operations 4.2e-7; expf takes 8 to 30% longer.
__device__ __forceinline__ float silu(float g)
{
    const float e = __expf(-fabsf(g));
    return g * __fdividef(g < 0.0f ? e : 1.0f, 1.0f + e);
}

// silu(g) x far below 0, where exp(g) nears or leaves the end of fp32's range, 1 +
// exp(g) is 1, and x may be large: by quarters of the exponential, each in range.
constexpr float kFarGate = -80.0f;

__device__ __forceinline__ float far_gated(float g, float x)
{
    const float e = __expf(0.25f * g);
    return x * e * e * g * e * e;
}

// Four int8 of a word as four fp16: with the sign bit flipped a byte b is
// b + 128 in 0..255; as the low byte of fp16 0x6400 it reads 1024 + b + 128,
// exactly, and 1152 is taken off again.
__device__ __forceinline__ void widen4(uint32_t w, uint32_t &lo, uint32_t &hi)
{
    const uint32_t t = w ^ 0x80808080u;
    const __half2 off = __halves2half2(__ushort_as_half(0x6480), __ushort_as_half(0x6480));
    uint32_t a = __byte_perm(t, 0x64646464u, 0x4140), b = __byte_perm(t, 0x64646464u, 0x4342);
    const __half2 x = __hsub2(*reinterpret_cast<__half2 *>(&a), off);
    const __half2 y = __hsub2(*reinterpret_cast<__half2 *>(&b), off);
    lo = *reinterpret_cast<const uint32_t *>(&x);
    hi = *reinterpret_cast<const uint32_t *>(&y);
}

// One output from its exact integer sum: the same four fp32 operations in the
// same order in every kernel (no contraction), so that they agree bit for bit.
__device__ __forceinline__ float q8_scaled(int sum, float xs, float ws)
{
    return __fmul_rn(__fmul_rn(__int2float_rn(sum), xs), ws);
}

__device__ __forceinline__ void q8_store(const Q8LinearParams &p, int m, int n, int sum, float xs, float ws)
{
    const size_t o = static_cast<size_t>(m) * p.N + n;
    float v = q8_scaled(sum, xs, ws);
    if (p.epilogue == SKG_EPI_FP32) {
        static_cast<float *>(p.y)[o] = v;
        return;
    }
    if (p.epilogue == SKG_EPI_BF16_RESIDUAL)
        v = __fadd_rn(v, bf16_to_f32(p.res[o]));
    static_cast<uint16_t *>(p.y)[o] = f32_to_bf16(v);
}

} // namespace skg

// skg_q8_rows.cu -- rows of bf16 turned into rows of 8-bit integers with one
// scale each: the norm with the residual's addition, and the quantiser of an
// activation (plain, or gated by silu).
//
//   norm:      h = x + residual;  v = h / sqrt(mean(h^2) + eps) * gamma
//   quantiser: v = x, or silu(gate) * x with silu(g) = g / (1 + exp(-g))
//   both:      scale = max|v| / 127;  q = v * 127 / max|v|, half to even
//
// Everything is fp32 until the stores; h and y are each rounded once to bf16,
// and the norm continues from the unrounded h.
#include "skg_q8_common.cuh"
#include "skg_q8_internal.h"

namespace skg {
namespace {

constexpr int kRowThreads = 256;

// Sum or maximum over the block; every thread gets the result.
template <bool MAX>
__device__ __forceinline__ float block_reduce(float v, float *sh)
{
#pragma unroll
    for (int o = 16; o; o >>= 1) {
        const float u = __shfl_xor_sync(0xFFFFFFFFu, v, o);
        v = MAX ? fmaxf(v, u) : v + u;
    }
    __syncthreads();
    if ((threadIdx.x & 31) == 0)
        sh[threadIdx.x >> 5] = v;
    __syncthreads();
    v = sh[0];
#pragma unroll
    for (int w = 1; w < kRowThreads / 32; ++w)
        v = MAX ? fmaxf(v, sh[w]) : v + sh[w];
    return v;
}

// A row's scale and the factor that takes a value to its integer.  A row of
// zeros has scale 0 and integers 0.  A row with a value that is not finite
// has scale NaN and integers 0, so that whatever it multiplies is NaN; amax
// cannot say so by itself (fmaxf drops NaN), hence `finite`.  Below 1e-30 the
// quotient 127 / amax would leave fp32's range: both are raised by 2^100,
// which is exact.
struct RowScale {
    float scale, up, factor;
};

__device__ __forceinline__ RowScale row_scale(float amax, bool finite)
{
    RowScale r;
    r.up = amax < 1e-30f ? 0x1p100f : 1.0f;
    r.factor = amax > 0.0f && finite ? 127.0f / (amax * r.up) : 0.0f;
    r.scale = finite ? amax / 127.0f : __int_as_float(0x7FC00000);
    return r;
}

__device__ __forceinline__ int8_t to_q8(float v, const RowScale &r, bool finite)
{
    return finite ? static_cast<int8_t>(__float2int_rn((v * r.up) * r.factor)) : static_cast<int8_t>(0);
}

template <bool NORM>
__device__ __forceinline__ float row_value(const Q8RowParams &p, size_t row, int k, float rms)
{
    const float a = bf16_to_f32(p.x[row * p.ldx + k]);
    if (NORM) {
        const float h = p.second ? a + bf16_to_f32(p.second[row * p.ld2 + k]) : a;
        return h * rms * (p.gamma ? bf16_to_f32(p.gamma[k]) : 1.0f);
    }
    if (!p.second)
        return a;
    return silu(bf16_to_f32(p.second[row * p.ld2 + k])) * a;
}

__device__ __forceinline__ float sum_of_squares(const Q8RowParams &p, size_t row, float unit, float *sh)
{
    float s = 0.0f;
    for (int k = threadIdx.x; k < p.K; k += kRowThreads) {
        float h = bf16_to_f32(p.x[row * p.ldx + k]);
        if (p.second)
            h += bf16_to_f32(p.second[row * p.ld2 + k]);
        h *= unit;
        s += h * h;
    }
    return block_reduce<false>(s, sh);
}

template <bool NORM>
__global__ void __launch_bounds__(kRowThreads) q8_rows_kernel(const Q8RowParams p)
{
    __shared__ float sh[kRowThreads / 32];
    const size_t row = blockIdx.x;
    float rms = 1.0f;
    if (NORM) {
        float s = sum_of_squares(p, row, 1.0f, sh);
        rms = rsqrtf(s / static_cast<float>(p.K) + p.eps);
        if (!(s <= 3.402823466e38f)) {
            // squares beyond fp32's range: the same with h taken 2^70 smaller
            // (where h itself is not finite, so is this sum, and the row)
            s = sum_of_squares(p, row, 0x1p-70f, sh);
            rms = rsqrtf(s / static_cast<float>(p.K) + p.eps * 0x1p-140f) * 0x1p-70f;
        }
    }
    float amax = 0.0f;
    int bad = 0;
    for (int k = threadIdx.x; k < p.K; k += kRowThreads) {
        const float v = row_value<NORM>(p, row, k, rms);
        bad |= !(fabsf(v) <= 3.402823466e38f);
        amax = fmaxf(amax, fabsf(v));
    }
    amax = block_reduce<true>(amax, sh);
    const bool finite = !__syncthreads_or(bad);
    const RowScale r = row_scale(amax, finite);
    for (int k = threadIdx.x; k < p.K; k += kRowThreads) {
        const float v = row_value<NORM>(p, row, k, rms);
        if (NORM && p.h)
            p.h[row * p.ldh + k] = f32_to_bf16(bf16_to_f32(p.x[row * p.ldx + k]) + bf16_to_f32(p.second[row * p.ld2 + k]));
        if (NORM && p.y)
            p.y[row * p.K + k] = f32_to_bf16(v);
        p.q[row * p.K + k] = to_q8(v, r, finite);
    }
    if (threadIdx.x == 0)
        p.scale[row] = r.scale;
}

} // namespace

cudaError_t launch_q8_norm(const Q8RowParams &p, cudaStream_t s)
{
    q8_rows_kernel<true><<<p.M, kRowThreads, 0, s>>>(p);
    return cudaGetLastError();
}

cudaError_t launch_q8_quantize(const Q8RowParams &p, cudaStream_t s)
{
    q8_rows_kernel<false><<<p.M, kRowThreads, 0, s>>>(p);
    return cudaGetLastError();
}

} // namespace skg

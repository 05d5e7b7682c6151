// skg_q8_gemv.cu -- the 8-bit projection on the integer units: each warp
// computes one output channel for up to MT tokens, four products at a time
// (dp4a: int8 x int8 into int32, exact).
#include "skg_q8_common.cuh"
#include "skg_q8_internal.h"

namespace skg {
namespace {

constexpr int kQ8GemvThreads = 256;

__device__ __forceinline__ int dot16(const uint4 &a, const uint4 &b, int acc)
{
    acc = __dp4a(static_cast<int>(a.x), static_cast<int>(b.x), acc);
    acc = __dp4a(static_cast<int>(a.y), static_cast<int>(b.y), acc);
    acc = __dp4a(static_cast<int>(a.z), static_cast<int>(b.z), acc);
    return __dp4a(static_cast<int>(a.w), static_cast<int>(b.w), acc);
}

template <int MT>
__global__ void __launch_bounds__(kQ8GemvThreads) q8_gemv_kernel(const Q8LinearParams p)
{
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int n = blockIdx.x * (kQ8GemvThreads / 32) + warp;
    const int m0 = blockIdx.y * MT;
    if (n >= p.N)
        return;
    const int nv = p.K / 16;
    const uint4 *w = reinterpret_cast<const uint4 *>(p.W + static_cast<size_t>(n) * p.K);
    int acc[MT] = {};
    for (int v = lane; v < nv; v += 32) {
        const uint4 wv = __ldg(w + v);
#pragma unroll
        for (int i = 0; i < MT; ++i)
            if (m0 + i < p.M) {
                const uint4 *x = reinterpret_cast<const uint4 *>(p.x + static_cast<size_t>(m0 + i) * p.K);
                acc[i] = dot16(wv, __ldg(x + v), acc[i]);
            }
    }
#pragma unroll
    for (int i = 0; i < MT; ++i) {
        const int sum = __reduce_add_sync(0xFFFFFFFFu, acc[i]);
        if (lane == i && m0 + i < p.M) {
            q8_store(p, m0 + i, n, sum, p.x_scale[m0 + i], p.w_scale[n]);
        }
    }
}

} // namespace

cudaError_t launch_q8_gemv(const Q8LinearParams &p, cudaStream_t s)
{
    constexpr int rows = kQ8GemvThreads / 32;
    const unsigned gx = static_cast<unsigned>((p.N + rows - 1) / rows);
    if (p.M == 1)
        q8_gemv_kernel<1><<<dim3(gx, 1), kQ8GemvThreads, 0, s>>>(p);
    else
        q8_gemv_kernel<8><<<dim3(gx, static_cast<unsigned>((p.M + 7) / 8)), kQ8GemvThreads, 0, s>>>(p);
    return cudaGetLastError();
}

} // namespace skg

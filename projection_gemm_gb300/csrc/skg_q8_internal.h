// skg_q8_internal.h -- shared between the host ABI of the 8-bit path
// (skg_q8_api.cu) and its kernels.  Not part of the public ABI.
#pragma once

#include <cstddef>
#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>

#include "skg.h"

namespace skg {

// One launch over the rows of a norm (gamma, eps) or a quantiser (gate).
// Row strides are in elements.
struct Q8RowParams {
    const uint16_t *x;        // bf16 [M, K], row stride ldx
    const uint16_t *second;   // residual (norm) or gate (quantiser), or null
    const uint16_t *gamma;    // norm: bf16 [K], or null for ones
    uint16_t *h;              // norm: bf16 x + residual, or null
    uint16_t *y;              // norm: bf16 normalised rows, or null
    int8_t *q;                // [M, K] dense
    float *scale;             // [M]
    size_t ldx, ld2, ldh;
    int M, K;
    float eps;
};

// y[m, n] = x_scale[m] * w_scale[n] * sum_k x[m, k] W[n, k] (+ residual).
struct Q8LinearParams {
    const int8_t *x;          // [M, K]
    const float *x_scale;     // [M]
    const int8_t *W;          // [N, K]
    const float *w_scale;     // [N]
    const uint16_t *res;      // bf16 [M, N] or null
    void *y;                  // [M, N] bf16 or fp32
    int M, N, K, epilogue;
};

// The split kernel's launch: clusters of `split` CTAs, one tile of 128 channels
// x m_tile tokens each, K cut over the cluster in units of 128.
struct Q8SplitParams {
    Q8LinearParams g;
    int *carry;               // [grid][carried][m_tile][128] int32
    int carried;              // accumulations a CTA puts away: those of 1024 k beyond 2048
    unsigned *err;
    int nkb, m_tiles, split, static_w;
    int vec4;                 // N a multiple of 4, w_scale, residual and y aligned for four channels at a time
    unsigned long long timeout_ns;
};

// The wide kernel's launch: tiles of 2 x 128 channels x m_tile tokens, one per
// cluster of `split` pairs of CTAs at a time, each pair with its part of K.
constexpr int kQ8WideMaxSplit = 4;         // 8 CTAs, the portable cluster size
struct Q8WideParams {
    Q8LinearParams g;
    unsigned *err;
    int nkb, n_pairs, m_tiles, tiles, band, split, static_w;
    int vec4;                 // as in Q8SplitParams
    unsigned long long timeout_ns;
};

struct Q8TcShape {
    int m_tile, ctas_per_sm, smem_bytes, threads, stages;
};

Q8TcShape q8_split_shape(int m_tile);
Q8TcShape q8_wide_shape();
cudaError_t launch_q8_split(const CUtensorMap &tmW, const CUtensorMap &tmX, const Q8SplitParams &p, int m_tile, int grid,
                            cudaStream_t s);
cudaError_t launch_q8_wide(const CUtensorMap &tmW, const CUtensorMap &tmX, const Q8WideParams &p, int grid,
                           cudaStream_t s);

cudaError_t launch_q8_norm(const Q8RowParams &p, cudaStream_t s);
cudaError_t launch_q8_quantize(const Q8RowParams &p, cudaStream_t s);

// The streaming kernel's launch: CTAs of 16 x groups channels.
struct Q8StreamShape {
    int groups, warps, ctas_per_sm;
};

Q8StreamShape q8_stream_shape(int M, int N, int num_sms);
cudaError_t launch_q8_stream(const Q8LinearParams &p, const Q8StreamShape &shape, bool static_w, cudaStream_t s);

} // namespace skg

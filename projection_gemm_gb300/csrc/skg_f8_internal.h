// skg_f8_internal.h -- shared between the host ABI of the 8-bit floating point
// path (skg_f8_api.cu) and its kernels.  Not part of the public ABI.
#pragma once

#include <cstddef>
#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>

#include "skg.h"

namespace skg {

constexpr int kF8Block = 128;              // values that share a scale: of a row, and channels of a weight
constexpr int kF8MaxExperts = 1024;

// Rows of bf16 to e4m3, a scale for each block of 128 of a row.
struct F8RowParams {
    const uint16_t *x;        // bf16 [x_rows, K], row stride ldx
    const uint16_t *gate;     // as x, row stride ldg, or null
    const int *rows;          // [M]: the row of x that each row is of, or null
    uint8_t *q;               // e4m3 [M, K] dense
    float *scale;             // [M, kb]
    size_t ldx, ldg;
    int M, K, kb, x_rows;
};

// A weight of bf16 to e4m3, a scale for each block of 128 x 128.
struct F8WeightParams {
    const uint16_t *W;        // bf16 [E, N, K]
    uint8_t *q;
    float *scale;             // [E, nb, kb]
    int E, N, K, nb, kb;
};

cudaError_t launch_f8_quantize(const F8RowParams &p, cudaStream_t s);
cudaError_t launch_f8_quantize_weights(const F8WeightParams &p, cudaStream_t s);

// y[m, n] = sum_b xs[m, b] ws[e, n / 128, b] sum_(k in b) x[m, k] W[e, n, k]
// (+ residual), e the expert whose rows m is among (0 without experts).
struct F8LinearParams {
    const float *x_scale;     // [M, nkb]
    const float *w_scale;     // [E, nb, nkb]
    const uint16_t *res;      // bf16 [M, N] or null
    void *y;                  // [M, N] bf16 or fp32
    const int *offsets;       // [experts + 1], or null
    unsigned *err;
    int M, N, K, epilogue, experts;
    int nkb, nb;
    int m_tiles, n_tiles;     // m_tiles: without experts
    int x_box, w_box;         // rows of x and of W that a copy takes: see f8_window
    int split, static_w;
    int vec4;                 // N a multiple of 4, residual and y aligned for four channels at a time
    int vec;                  // the same for 16 bytes of sums, or of bf16 where no residual is added
    unsigned long long timeout_ns;
};

struct F8TcShape {
    int m_tile, ctas_per_sm, smem_bytes, threads, stages;
};

constexpr int kF8SplitMax = 8;             // CTAs of a cluster that share a tile's K
F8TcShape f8_split_shape(int m_tile, int experts);
constexpr int kF8WideMaxSplit = 4;         // the same of the wide kernel, whose tiles of 256 tokens take two CTAs for one
F8TcShape f8_wide_shape(int m_tile, int experts);
cudaError_t launch_f8_split(const CUtensorMap &tmW, const CUtensorMap &tmX, const F8LinearParams &p, int m_tile, int grid,
                            cudaStream_t s);
cudaError_t launch_f8_wide(const CUtensorMap &tmW, const CUtensorMap &tmX, const F8LinearParams &p, int m_tile, int grid,
                           cudaStream_t s);

} // namespace skg

// skg_q8_tc_common.cuh -- device code shared by the 8-bit path's tcgen05 kernels:
// widening, the epilogue's reading of accumulators and its stores.  Included inside namespace skg's anonymous namespace.
#pragma once

constexpr int kQ8BlockK = 128;                       // k of one unit: 128 bytes of a W row
constexpr int kExactBlocks = 1024 / kQ8BlockK;       // units summed by the MMA from a fresh accumulator
constexpr int kWidenSets = 2;                        // sets of 4 warps (a set covers the 128 TMEM lanes)
constexpr int kWidenWarps = 4 * kWidenSets;
constexpr uint32_t kQ8WBytes = kTileN * kQ8BlockK;   // 16 KB

__device__ __forceinline__ void q8_fail(unsigned *err, volatile int *abort, unsigned bit)
{
    *abort = 1;
    if (err)
        atomicOr(err, bit);
}

__device__ __forceinline__ void widen16(const uint4 &v, uint32_t *r)
{
    widen4(v.x, r[0], r[1]);
    widen4(v.y, r[2], r[3]);
    widen4(v.z, r[4], r[5]);
    widen4(v.w, r[6], r[7]);
}

// CHUNKS 16-byte pieces, from `first` on, of W row `row` of a unit (a tile of
// 128-byte rows, 128-byte swizzle) as fp16 into this thread's TMEM lane: 8
// columns a piece.
template <int CHUNKS>
__device__ __forceinline__ void widen_row(const uint8_t *tile, int row, int first, uint32_t taddr)
{
    const uint8_t *src = tile + row * kQ8BlockK;
#pragma unroll
    for (int i = 0; i < CHUNKS / 2; ++i) {
        uint32_t r[16];
#pragma unroll
        for (int h = 0; h < 2; ++h)
            widen16(*reinterpret_cast<const uint4 *>(src + (((first + 2 * i + h) ^ (row & 7)) << 4)), r + 8 * h);
        tmem_st_x16(taddr + 16 * i, r);
    }
}

// NC outputs (tokens m0...) of one channel n from their sums, 4 at a time so
// that their loads are in flight together and few registers hold them.
template <int EPI, int NC>
__device__ __forceinline__ void store_columns_as(const Q8LinearParams &g, int m0, int n, const int (&acc)[NC])
{
    const int valid = g.M - m0;
    const float ws = __ldcg(g.w_scale + n);
    const float *xsp = g.x_scale + m0;
    size_t at = static_cast<size_t>(m0) * g.N + n;
#pragma unroll
    for (int c0 = 0; c0 < NC; c0 += 4) {
        float v[4];
#pragma unroll
        for (int c = 0; c < 4; ++c)
            v[c] = c0 + c < valid ? q8_scaled(acc[c0 + c], __ldcg(xsp + c0 + c), ws) : 0.0f;
        if (EPI == SKG_EPI_BF16_RESIDUAL) {
            const uint16_t *r = g.res + at;
            uint16_t b[4];
#pragma unroll
            for (int c = 0; c < 4; ++c, r += g.N)
                b[c] = c0 + c < valid ? __ldcg(r) : 0;
#pragma unroll
            for (int c = 0; c < 4; ++c)
                v[c] = __fadd_rn(v[c], bf16_to_f32(b[c]));
        }
#pragma unroll
        for (int c = 0; c < 4; ++c, at += g.N) {
            if (c0 + c < valid) {
                if (EPI == SKG_EPI_FP32)
                    static_cast<float *>(g.y)[at] = v[c];
                else
                    static_cast<uint16_t *>(g.y)[at] = f32_to_bf16(v[c]);
            }
        }
    }
}

template <int NC>
__device__ __forceinline__ void store_columns(const Q8LinearParams &g, int m0, int n, const int (&acc)[NC])
{
    if (n >= g.N || m0 >= g.M)
        return;
    if (g.epilogue == SKG_EPI_FP32)
        store_columns_as<SKG_EPI_FP32>(g, m0, n, acc);
    else if (g.epilogue == SKG_EPI_BF16_RESIDUAL)
        store_columns_as<SKG_EPI_BF16_RESIDUAL>(g, m0, n, acc);
    else
        store_columns_as<SKG_EPI_BF16>(g, m0, n, acc);
}

// NC accumulator columns of this thread's TMEM lane as integers (they are
// integers of at most 2^24 in fp32: the conversion is exact).
template <int NC>
__device__ __forceinline__ void load_sums(uint32_t taddr, int (&v)[NC])
{
    uint32_t r[NC / 8][8];
#pragma unroll
    for (int i = 0; i < NC / 8; ++i)
        tmem_ld_x8(taddr + 8 * i, r[i]);
    tmem_wait_ld();
#pragma unroll
    for (int c = 0; c < NC; ++c) {
        asm volatile("" : "+r"(r[c >> 3][c & 7]));
        v[c] = __float2int_rn(__uint_as_float(r[c >> 3][c & 7]));
    }
}

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
//
// What bounds it is HBM for many rows and latency for few.  A row is read once:
// its values stay in registers (up to 32 a thread) through the sum of squares
// and the maximum, with one block barrier each, and what a thread loads is all
// in flight together.  Rows that are not 16-byte aligned (any odd length) are
// still read in 16-byte blocks, shifted into place; rows longer than 16384 take
// three passes over memory.
//
// Measured, with the bytes that have to move (6.70 TB/s copy peak): norm with
// residual 8192 x 7168 61.2 us (6.72 TB/s), 4096 x 2048 8.2 us (from the L2), 1 x
// 7168 2.5 us; gated quantiser 4096 x 16384 56.8 us (5.9 TB/s: exp, the quotient
// and the conversions issue in 64% of the cycles); quantiser 8192 x 7168 30-35
// us; rows of odd length cost twice the instructions: norm 8191 x 7169 121 us
// (3.4 TB/s), quantiser 1023 x 5001 5.1 us; norm 2048 x 20000, three passes, 109.
#include <algorithm>

#include "skg_internal.h"
#include "skg_ptx.cuh"
#include "skg_q8_common.cuh"
#include "skg_q8_internal.h"

namespace skg {
namespace {

constexpr int kWarpRows = 8;              // rows of a CTA where a warp takes a row
constexpr int kMaxRow = 16384;            // longest row held in registers
constexpr int kLongThreads = 1024;

// A row's scale and the factor that takes a value to its integer, from the bits
// of max|v| (|NaN| > infinity > every finite value, as integers).  A row of
// zeros has scale 0 and integers 0.  A row with a value that is not finite has
// scale NaN and integers 0, so that whatever it multiplies is NaN.  Below 1e-30
// the quotient 127 / max would leave fp32's range: both are raised by 2^100,
// which is exact.
//
// The quotient is rounded up.  In a row of bf16 the only values that lie half way
// between two integers, whatever the maximum, are those of half the maximum: 63.5,
// which goes to 64, as does anything above it.  (254 v / max is an odd integer
// only where 127 divides that integer or max's significand, and then max is 127
// or 254 times a power of two and the quotient exact.)  Rounded to nearest, the
// quotient is below 127 / max half of the time, and such a value goes to 63: 0.07%
// of the elements of normal rows.  Every other value is further from half way
// than the quotient's rounding takes it.  (The quotient to nearest, raised by a
// unit where its product with the maximum falls short: __fdiv_ru does the same
// and costs a warp-bound row kernel 3 to 10%, 131072 x 256 24.9 and 27.6 us.)
struct RowScale {
    float scale, up, factor;
    bool finite;
};

__device__ __forceinline__ float quotient_up(float a, float b)
{
    const float f = a / b;
    return fmaf(f, b, -a) < 0.0f ? __uint_as_float(__float_as_uint(f) + 1) : f;
}

__device__ __forceinline__ RowScale row_scale(uint32_t max_bits)
{
    RowScale r;
    const float amax = __uint_as_float(max_bits);
    r.finite = max_bits < 0x7F800000u;
    r.up = amax < 1e-30f ? 0x1p100f : 1.0f;
    r.factor = amax > 0.0f && r.finite ? quotient_up(127.0f, amax * r.up) : 0.0f;
    r.scale = r.finite ? amax / 127.0f : __int_as_float(0x7FC00000);
    return r;
}

// v * factor rounded to the nearest integer, half to even, as the low byte of
// the fp32 sum with 1.5 * 2^23, which is rounded at the units.
__device__ __forceinline__ uint32_t to_q8(float v, const RowScale &r)
{
    return __float_as_uint(fmaf(v, r.factor, 12582912.0f));
}

// max(m, |v|), NaN where either is.
__device__ __forceinline__ float max_nan(float m, float v)
{
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(m), "f"(fabsf(v)));
    return r;
}

__device__ __forceinline__ uint32_t abs_bits(float v) { return __float_as_uint(v) & 0x7FFFFFFFu; }

// The norm's factor, 1 / sqrt(mean(h^2) + eps), is had from the sum of squares in
// fp32.  Where that has left, or is about to leave, the range in which fp32 holds
// the sum and the mean to their precision (`plain` is false), it is taken again with
// h scaled by a power of two:
//   sum > 2^100: by 2^-80.  The largest h are below 2^48 then, and no row's sum
//     (K < 2^31) overflows; the mean was above 2^69, so it stays above 2^-91.  The
//     factor, scaled back, is 2^-128 at the least.
//   mean + eps < 2^-100: by 2^90, exactly, and the norm goes on from the scaled h.
//     All of h was below 2^-34, so the sum stays below 2^111; bf16's smallest
//     value becomes 2^-43.
// A value that is not finite makes the sum infinite or NaN, and the row's maximum
// NaN.  A row of zeros with eps = 0 is 0 / 0.
struct RowNorm {
    float mean, n, eps;
    bool plain, large;

    __device__ __forceinline__ RowNorm(float sum, int K, float e) : n(static_cast<float>(K)), eps(e)
    {
        mean = sum / n + e;
        large = !(sum <= 0x1p100f);
        plain = !large && mean >= 0x1p-100f;
    }

    __device__ __forceinline__ float unit() const { return large ? 0x1p-80f : 0x1p90f; }
    __device__ __forceinline__ float factor() const { return rsqrtf(mean); }

    // From the sum with h scaled by unit(): the factor of h itself if large, else of the scaled h.
    __device__ __forceinline__ float scaled_factor(float sum) const
    {
        return rsqrtf(sum / n + eps * unit() * unit()) * (large ? unit() : 1.0f);
    }
};

// ------------------------------------------------------------ rows in registers
// Eight elements as loaded.  (Not by the read-only path: the kernel may have
// started before its inputs were written.)
struct Raw8 {
    uint32_t w[4];
};

__device__ __forceinline__ void load_block(const uint16_t *p, uint32_t *w)
{
    asm volatile("ld.global.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]) : "l"(p));
}

__device__ __forceinline__ float value(const Raw8 &r, int i)
{
    return i & 1 ? bf16hi(r.w[i >> 1]) : bf16lo(r.w[i >> 1]);
}

// The larger of two bf16 in each half of a word, as unsigned integers: of negative
// gates the lowest.
__device__ __forceinline__ uint32_t lowest_gate(uint32_t m, const Raw8 &r)
{
#pragma unroll
    for (int i = 0; i < 4; ++i)
        m = __vmaxu2(m, r.w[i]);
    return m;
}

__device__ __forceinline__ bool far_gate(uint32_t m)
{
    constexpr uint32_t kFarBits = 0xC2A0;            // kFarGate
    return (m & 0xFFFF) > kFarBits || (m >> 16) > kFarBits;
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi)
{
    return f32_to_bf16(lo) | static_cast<uint32_t>(f32_to_bf16(hi)) << 16;
}

// A row of bf16 read 8 elements at a time.  ANY: from an address of any
// alignment, by the two 16-byte blocks around the eight elements; where those
// reach beyond the row (near its ends), element by element.
template <bool ANY>
struct RowLoad {
    uint32_t w[ANY ? 8 : 4];
    int d = 0;               // the eight elements begin at element d of w

    __device__ __forceinline__ void load(const uint16_t *row, int e, int K)
    {
#pragma unroll
        for (int i = 0; i < (ANY ? 8 : 4); ++i)
            w[i] = 0;
        if constexpr (!ANY) {
            if (e < K)
                load_block(row + e, w);
        } else {
            d = phase(row, e);
            if (e - d >= 0 && e - d + (d ? 16 : 8) <= K) {
                load_block(row + (e - d), w);
                if (d)
                    load_block(row + (e - d) + 8, w + 4);
            } else if (e + 8 > 0 && e < K) {
                d = 0;
                uint16_t h[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    h[i] = 0;
                    if (e + i >= 0 && e + i < K)
                        asm volatile("ld.global.u16 %0, [%1];" : "=h"(h[i]) : "l"(row + e + i));
                }
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    w[i] = h[2 * i] | static_cast<uint32_t>(h[2 * i + 1]) << 16;
            }
        }
    }

    // Elements by which row + e lies beyond a 16-byte boundary.
    static __device__ __forceinline__ int phase(const uint16_t *row, int e)
    {
        return static_cast<int>((reinterpret_cast<uintptr_t>(row) >> 1) + static_cast<unsigned>(e)) & 7;
    }

    __device__ __forceinline__ Raw8 get() const
    {
        Raw8 r;
        if constexpr (!ANY) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                r.w[i] = w[i];
        } else {
            uint32_t u[6], t[5];
#pragma unroll
            for (int i = 0; i < 6; ++i)
                u[i] = d & 4 ? w[i + 2] : w[i];
#pragma unroll
            for (int i = 0; i < 5; ++i)
                t[i] = d & 2 ? u[i + 1] : u[i];
#pragma unroll
            for (int i = 0; i < 4; ++i)
                r.w[i] = d & 1 ? __funnelshift_r(t[i], t[i + 1], 16) : t[i];
        }
        return r;
    }
};

// Eight values as bf16 at element e of a row; ANY: those inside the row, in the
// widest pieces the address allows.
template <bool ANY>
__device__ __forceinline__ void store_bf16(uint16_t *row, int e, int K, const float *v)
{
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        w[i] = pack_bf16(v[2 * i], v[2 * i + 1]);
    const int d = ANY ? RowLoad<true>::phase(row, e) : 0;
    if (ANY && (e < 0 || e + 8 > K || d & 1)) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (e + i >= 0 && e + i < K)
                row[e + i] = static_cast<uint16_t>(w[i >> 1] >> (16 * (i & 1)));
    } else if (ANY && d) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            *reinterpret_cast<uint32_t *>(row + e + 2 * i) = w[i];
    } else if (e < K) {
        *reinterpret_cast<uint4 *>(row + e) = make_uint4(w[0], w[1], w[2], w[3]);
    }
}

// Eight values as integers at element e of a row; row + e is 8-byte aligned.
template <bool ANY>
__device__ __forceinline__ void store_q8(int8_t *row, int e, int K, const float *v, const RowScale &r)
{
    uint32_t w[2];
#pragma unroll
    for (int i = 0; i < 2; ++i)
        w[i] = __byte_perm(__byte_perm(to_q8(v[4 * i], r), to_q8(v[4 * i + 1], r), 0x0040),
                           __byte_perm(to_q8(v[4 * i + 2], r), to_q8(v[4 * i + 3], r), 0x0040), 0x5410);
    if (ANY && (e < 0 || e + 8 > K)) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (e + i >= 0 && e + i < K)
                row[e + i] = static_cast<int8_t>(w[i >> 2] >> (8 * (i & 3)));
    } else if (e < K) {
        *reinterpret_cast<uint2 *>(row + e) = make_uint2(w[0], w[1]);
    }
}

// Sum and maximum over a row's threads: a warp (WARP), or the block, in a
// buffer of one value a warp (each used for one reduction of the kernel).
template <bool WARP>
__device__ __forceinline__ float row_sum(float v, float *buf)
{
#pragma unroll
    for (int o = 16; o; o >>= 1)
        v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    if constexpr (!WARP) {
        if ((threadIdx.x & 31) == 0)
            buf[threadIdx.x >> 5] = v;
        __syncthreads();
        const int lane = threadIdx.x & 31;
        v = lane < static_cast<int>(blockDim.x >> 5) ? buf[lane] : 0.0f;
#pragma unroll
        for (int o = 16; o; o >>= 1)
            v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    }
    return v;
}

template <bool WARP>
__device__ __forceinline__ uint32_t row_max(uint32_t v, uint32_t *buf)
{
    v = __reduce_max_sync(0xFFFFFFFFu, v);
    if constexpr (!WARP) {
        if ((threadIdx.x & 31) == 0)
            buf[threadIdx.x >> 5] = v;
        __syncthreads();
        const int lane = threadIdx.x & 31;
        v = __reduce_max_sync(0xFFFFFFFFu, lane < static_cast<int>(blockDim.x >> 5) ? buf[lane] : 0u);
    }
    return v;
}

// VALUES a thread.  ANY: tensors of any alignment; the eights then lie where
// the row of q is 8-byte aligned, so the first and the last may stick out.
template <bool NORM, bool ANY, int VALUES, bool WARP>
__global__ void __launch_bounds__(WARP ? 32 * kWarpRows : (VALUES == 8 ? 1024 : kMaxRow / VALUES), WARP ? 2 : VALUES / 16 + (VALUES == 8))
q8_rows_kernel(const Q8RowParams p)
{
    constexpr int NV = VALUES / 8;
    __shared__ float sums[2][32];
    __shared__ uint32_t maxima[32];
    pdl_wait();
    pdl_launch_dependents();
    const size_t row = WARP ? static_cast<size_t>(blockIdx.x) * kWarpRows + (threadIdx.x >> 5) : blockIdx.x;
    if (WARP && row >= static_cast<size_t>(p.M))
        return;
    const int t = WARP ? threadIdx.x & 31 : threadIdx.x, T = WARP ? 32 : blockDim.x;
    const uint16_t *x = p.x + row * p.ldx, *second = p.second ? p.second + row * p.ld2 : nullptr;
    int8_t *q = p.q + row * p.K;
    const int first = ANY ? t * 8 - static_cast<int>(reinterpret_cast<uintptr_t>(q) & 7) : t * 8;
    const int step = T * 8;

    float v[NV][8];
    {
        RowLoad<ANY> a[NV], w[NV];
        uint32_t far = 0;
#pragma unroll
        for (int j = 0; j < NV; ++j)
            a[j].load(x, first + j * step, p.K);
        if (second) {
#pragma unroll
            for (int j = 0; j < NV; ++j)
                w[j].load(second, first + j * step, p.K);
        }
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const Raw8 xa = a[j].get();
#pragma unroll
            for (int c = 0; c < 8; ++c)
                v[j][c] = value(xa, c);
            if (second) {
                const Raw8 xw = w[j].get();
#pragma unroll
                for (int c = 0; c < 8; ++c)
                    v[j][c] = NORM ? v[j][c] + value(xw, c) : silu(value(xw, c)) * v[j][c];
                if constexpr (!NORM && WARP) {
                    if (far_gate(lowest_gate(0, xw))) {
#pragma unroll
                        for (int c = 0; c < 8; ++c)
                            v[j][c] = value(xw, c) < kFarGate ? far_gated(value(xw, c), value(xa, c)) : v[j][c];
                    }
                } else if (!NORM) {
                    far = lowest_gate(far, xw);
                }
            }
        }
        if (!NORM && !WARP && far_gate(far)) {       // rare: fetched again
#pragma unroll
            for (int j = 0; j < NV; ++j) {
                RowLoad<ANY> b;
                b.load(x, first + j * step, p.K);
                const Raw8 xa = b.get();
                b.load(second, first + j * step, p.K);
                const Raw8 xw = b.get();
#pragma unroll
                for (int c = 0; c < 8; ++c)
                    v[j][c] = value(xw, c) < kFarGate ? far_gated(value(xw, c), value(xa, c)) : v[j][c];
            }
        }
    }
    if constexpr (NORM) {
        RowLoad<ANY> w[NV];
        if (p.h) {
#pragma unroll
            for (int j = 0; j < NV; ++j)
                store_bf16<ANY>(p.h + row * p.ldh, first + j * step, p.K, v[j]);
        }
        if (p.gamma) {                   // on its way during the sum; after h's stores, whose registers it takes
#pragma unroll
            for (int j = 0; j < NV; ++j)
                w[j].load(p.gamma, first + j * step, p.K);
        }
        auto sum_of_squares = [&](float unit, float *buf) {
            float s = 0.0f;
#pragma unroll
            for (int j = 0; j < NV; ++j)
#pragma unroll
                for (int c = 0; c < 8; ++c)
                    s = fmaf(v[j][c] * unit, v[j][c] * unit, s);
            return row_sum<WARP>(s, buf);
        };
        const RowNorm norm(sum_of_squares(1.0f, sums[0]), p.K, p.eps);
        float rms = norm.factor();
        if (!norm.plain) {
            if (!norm.large) {
#pragma unroll
                for (int j = 0; j < NV; ++j)
#pragma unroll
                    for (int c = 0; c < 8; ++c)
                        v[j][c] *= norm.unit();
            }
            rms = norm.scaled_factor(sum_of_squares(norm.large ? norm.unit() : 1.0f, sums[1]));
        }
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const Raw8 g = w[j].get();
#pragma unroll
            for (int c = 0; c < 8; ++c)
                v[j][c] = p.gamma ? v[j][c] * rms * value(g, c) : v[j][c] * rms;
        }
        if (p.y) {
#pragma unroll
            for (int j = 0; j < NV; ++j)
                store_bf16<ANY>(p.y + row * p.K, first + j * step, p.K, v[j]);
        }
    }
    float m = 0.0f;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const int e = first + j * step;
        // (what lies beyond the row holds 0 * rms, which is NaN where that factor is infinite)
        if (!ANY ? e < p.K : e >= 0 && e + 8 <= p.K) {
#pragma unroll
            for (int c = 0; c < 8; ++c)
                m = max_nan(m, v[j][c]);
        } else if (ANY) {
#pragma unroll
            for (int c = 0; c < 8; ++c)
                m = e + c >= 0 && e + c < p.K ? max_nan(m, v[j][c]) : m;
        }
    }
    const RowScale r = row_scale(row_max<WARP>(abs_bits(m), maxima));
    if (r.up != 1.0f || !r.finite) {
#pragma unroll
        for (int j = 0; j < NV; ++j)
#pragma unroll
            for (int c = 0; c < 8; ++c)
                v[j][c] = r.finite ? v[j][c] * r.up : 0.0f;
    }
#pragma unroll
    for (int j = 0; j < NV; ++j)
        store_q8<ANY>(q, first + j * step, p.K, v[j], r);
    if (t == 0)
        p.scale[row] = r.scale;
}

// ------------------------------------------------------------------ longer rows
// (K up to 2^31 - 1: the index passes it.)
// EDGE: the norm goes on from the scaled sum, and the gate has values below kFarGate.
template <bool EDGE>
__device__ __forceinline__ float long_sum(const Q8RowParams &p, size_t row, unsigned k)
{
    const float a = bf16_to_f32(p.x[row * p.ldx + k]);
    const float h = p.second ? a + bf16_to_f32(p.second[row * p.ld2 + k]) : a;
    return EDGE ? h * 0x1p90f : h;
}

template <bool NORM, bool EDGE>
__device__ __forceinline__ float long_value(const Q8RowParams &p, size_t row, unsigned k, float rms, float &gate)
{
    if (NORM) {
        const float h = long_sum<EDGE>(p, row, k);
        return p.gamma ? h * rms * bf16_to_f32(p.gamma[k]) : h * rms;
    }
    const float a = bf16_to_f32(p.x[row * p.ldx + k]);
    if (!p.second)
        return a;
    gate = bf16_to_f32(p.second[row * p.ld2 + k]);
    return EDGE && gate < kFarGate ? far_gated(gate, a) : silu(gate) * a;
}

// The maximum and the integers of a row.
template <bool NORM, bool EDGE>
__device__ __forceinline__ void long_row(const Q8RowParams &p, size_t row, float rms, uint32_t *maxima)
{
    uint32_t m = 0;
    float gate = 0.0f, lowest = 0.0f;
    for (unsigned k = threadIdx.x; k < static_cast<unsigned>(p.K); k += kLongThreads) {
        m = max(m, abs_bits(long_value<NORM, EDGE>(p, row, k, rms, gate)));
        lowest = fminf(lowest, gate);
    }
    if constexpr (!NORM && !EDGE) {
        if (__syncthreads_or(lowest < kFarGate)) {
            long_row<false, true>(p, row, rms, maxima);
            return;
        }
    }
    const RowScale r = row_scale(row_max<false>(m, maxima));
    for (unsigned k = threadIdx.x; k < static_cast<unsigned>(p.K); k += kLongThreads) {
        const float v = long_value<NORM, EDGE>(p, row, k, rms, gate);
        if (NORM && p.h)                 // may be the residual itself: read by this thread, above
            p.h[row * p.ldh + k] = f32_to_bf16(long_sum<false>(p, row, k));
        if (NORM && p.y)
            p.y[row * p.K + k] = f32_to_bf16(v);
        p.q[row * p.K + k] = static_cast<int8_t>(to_q8(r.finite ? v * r.up : 0.0f, r));
    }
    if (threadIdx.x == 0)
        p.scale[row] = r.scale;
}

template <bool NORM>
__global__ void __launch_bounds__(kLongThreads) q8_long_rows_kernel(const Q8RowParams p)
{
    __shared__ float sums[2][32];
    __shared__ uint32_t maxima[32];
    pdl_wait();
    pdl_launch_dependents();
    const size_t row = blockIdx.x;
    float rms = 1.0f;
    if (NORM) {
        auto sum_of_squares = [&](float unit, float *buf) {
            float s = 0.0f;
            for (unsigned k = threadIdx.x; k < static_cast<unsigned>(p.K); k += kLongThreads) {
                const float h = long_sum<false>(p, row, k) * unit;
                s = fmaf(h, h, s);
            }
            return row_sum<false>(s, buf);
        };
        const RowNorm norm(sum_of_squares(1.0f, sums[0]), p.K, p.eps);
        rms = norm.factor();
        if (!norm.plain) {
            rms = norm.scaled_factor(sum_of_squares(norm.unit(), sums[1]));
            if (!norm.large) {
                long_row<true, true>(p, row, rms, maxima);
                return;
            }
        }
    }
    long_row<NORM, false>(p, row, rms, maxima);
}

template <class... A>
cudaError_t launch(void (*kernel)(A...), unsigned grid, unsigned threads, const Q8RowParams &p, cudaStream_t s)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(threads);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, p);
}

// Threads and values a thread for rows of K.  A warp a row up to 1024 (1017
// where the eights may stick out).  Beyond, few rows want many threads
// (latency); many rows want as many values a thread as registers allow (32, or
// 16 where every eight takes two blocks): fewer warps at each barrier, more
// bytes in flight.  At 8192 x 7168 the norm with residual takes 63 us at 32, 92
// at 16 and 83 at 8.
template <bool NORM, bool ANY>
cudaError_t launch_rows_as(const Q8RowParams &p, cudaStream_t s)
{
    const int eights = (p.K + (ANY ? 7 : 0) + 7) / 8;
    auto threads = [&](int values) { return static_cast<unsigned>((eights + 4 * values - 1) / (4 * values) * 32); };
    if (eights <= 128) {
        const unsigned grid = (static_cast<unsigned>(p.M) + kWarpRows - 1) / kWarpRows;
        if (eights <= 32)
            return launch(q8_rows_kernel<NORM, ANY, 8, true>, grid, 32 * kWarpRows, p, s);
        if (eights <= 64)
            return launch(q8_rows_kernel<NORM, ANY, 16, true>, grid, 32 * kWarpRows, p, s);
        return launch(q8_rows_kernel<NORM, ANY, 32, true>, grid, 32 * kWarpRows, p, s);
    }
    const bool few = p.M <= 2 * 152;     // two rows for each of a GB300's SMs
    if (few && eights <= 1024)
        return launch(q8_rows_kernel<NORM, ANY, 8, false>, p.M, threads(8), p, s);
    if constexpr (!ANY) {
        if (!few)
            return launch(q8_rows_kernel<NORM, false, 32, false>, p.M, threads(32), p, s);
    }
    return launch(q8_rows_kernel<NORM, ANY, 16, false>, p.M, threads(16), p, s);
}

bool multiple(const void *ptr, size_t bytes) { return reinterpret_cast<uintptr_t>(ptr) % bytes == 0; }

template <bool NORM>
cudaError_t launch_rows(const Q8RowParams &p, cudaStream_t s)
{
    // null tensors are aligned
    const bool aligned = p.K % 8 == 0 && p.ldx % 8 == 0 && (!p.second || p.ld2 % 8 == 0) && (!p.h || p.ldh % 8 == 0) &&
                         multiple(p.x, 16) && multiple(p.second, 16) && multiple(p.gamma, 16) && multiple(p.h, 16) &&
                         multiple(p.y, 16) && multiple(p.q, 8);
    if (aligned ? p.K > kMaxRow : p.K > kMaxRow - 7)
        return launch(q8_long_rows_kernel<NORM>, p.M, kLongThreads, p, s);
    return aligned ? launch_rows_as<NORM, false>(p, s) : launch_rows_as<NORM, true>(p, s);
}

} // namespace

cudaError_t launch_q8_norm(const Q8RowParams &p, cudaStream_t s) { return launch_rows<true>(p, s); }

cudaError_t launch_q8_quantize(const Q8RowParams &p, cudaStream_t s) { return launch_rows<false>(p, s); }

} // namespace skg

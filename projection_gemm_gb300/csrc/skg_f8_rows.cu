// skg_f8_rows.cu -- bf16 turned into e4m3 with one fp32 scale for each block of
// 128 values of a row (activations), or of 128 x 128 (weights).
//
//   v = x, or silu(gate) * x;   scale = max|v| / 448;   q = e4m3(v * (448 / max|v|))
//
// v, the quotient and the product are fp32, and the product is rounded once, half
// to even.  A block is read once: its values stay in registers through the
// maximum.  16 lanes take a block of a row, 8 values a lane; a CTA takes a block of a
// weight.  Rows that are not 16-byte aligned are read in 16-byte blocks shifted into
// place, and their numbers stored in aligned words that two lanes fill.
//
// What bounds it is HBM where rows are aligned: 8192 x 7168 30.5 us (5.8 TB/s of 6.71),
// weight 12288 x 7168 48 us (5.5); gated by silu it is nearly instructions (78% of
// the issue slots): 4096 x 16384 61 us (5.5 TB/s).  Instructions elsewhere: 8191 x
// 7169 76 us, weight 5001 x 4113 29 us (89 and 40 with single elements loaded and
// stored), rows of 4096 tokens taken 8 times each 106 us; 512 rows of 7168 4.1 us.
// With 2 or 4 blocks a warp instead of 8, 8192 x 7168 took 44 and 35 us.
#include <algorithm>

#include "skg_f8_internal.h"
#include "skg_internal.h"
#include "skg_ptx.cuh"
#include "skg_q8_common.cuh"

namespace skg {
namespace {

// A block's scale and the factor that takes a value to its e4m3 number, from the
// bits of max|v| (|NaN| > infinity > every finite value, as integers).  A block of
// zeros has scale 0.  One with a value that is not finite has scale NaN and
// numbers 0, so that whatever it multiplies is NaN.  Below 1e-30 the quotient 448 /
// max would leave fp32's range: both are raised by 2^100, which is exact.
struct BlockScale {
    float scale, up, factor;
};

__device__ __forceinline__ BlockScale block_scale(uint32_t max_bits)
{
    BlockScale b;
    const float amax = __uint_as_float(max_bits);
    const bool finite = max_bits < 0x7F800000u;
    b.up = amax < 1e-30f ? 0x1p100f : 1.0f;
    b.factor = amax > 0.0f && finite ? 448.0f / (amax * b.up) : 0.0f;
    b.scale = finite ? amax / 448.0f : __int_as_float(0x7FC00000);
    return b;
}

// Two values as e4m3 numbers, the first in the low byte.  (Beyond 448 by a
// rounding: 448.)
__device__ __forceinline__ uint32_t two_e4m3(float a, float b)
{
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(b), "f"(a));
    return r;
}

template <int N>
struct Values {
    float v[N];
};

using Eight = Values<8>;

// max|v| as bits, larger than infinity's where a value is NaN.
template <int N>
__device__ __forceinline__ uint32_t max_bits(const Values<N> &e)
{
    float m = 0.0f;
#pragma unroll
    for (int i = 0; i < N; ++i)
        asm("max.NaN.f32 %0, %0, %1;" : "+f"(m) : "f"(fabsf(e.v[i])));
    return __float_as_uint(m) & 0x7FFFFFFFu;
}

template <int N>
__device__ __forceinline__ void scale_values(Values<N> &e, const BlockScale &b)
{
    if (b.up != 1.0f || b.factor == 0.0f) {          // rare
#pragma unroll
        for (int i = 0; i < N; ++i)      // (a factor of 0 does not make a NaN or an infinity 0)
            e.v[i] = b.factor == 0.0f ? 0.0f : e.v[i] * b.up;
    }
#pragma unroll
    for (int i = 0; i < N; ++i)
        e.v[i] *= b.factor;
}

__device__ __forceinline__ uint2 to_e4m3(Eight e, const BlockScale &b)
{
    scale_values(e, b);
    return make_uint2(two_e4m3(e.v[0], e.v[1]) | two_e4m3(e.v[2], e.v[3]) << 16,
                      two_e4m3(e.v[4], e.v[5]) | two_e4m3(e.v[6], e.v[7]) << 16);
}

// silu(g) x.
template <int N>
__device__ __forceinline__ Values<N> gated(const Values<N> &g, const Values<N> &x)
{
    Values<N> v;
    float lowest = g.v[0];
#pragma unroll
    for (int i = 0; i < N; ++i) {
        v.v[i] = silu(g.v[i]) * x.v[i];
        lowest = fminf(lowest, g.v[i]);
    }
    if (lowest < kFarGate) {             // rare
#pragma unroll
        for (int i = 0; i < N; ++i)
            v.v[i] = g.v[i] < kFarGate ? far_gated(g.v[i], x.v[i]) : v.v[i];
    }
    return v;
}

// Eight numbers at element e of a row of K.  ANY: of any alignment; L neighbouring
// lanes have neighbouring eights (all of them call), and a lane stores the aligned 8
// bytes that its eight begins in: the end of the lane's before and the beginning of its
// own.
template <bool ANY, int L>
__device__ __forceinline__ void store8(uint8_t *row, int e, int K, const uint2 &w)
{
    if constexpr (!ANY) {
        if (e < K)
            *reinterpret_cast<uint2 *>(row + e) = w;
    } else {
        const int lane = static_cast<int>(threadIdx.x) & (L - 1);
        const int s = static_cast<int>(reinterpret_cast<uintptr_t>(row) + e) & 7;
        const unsigned long long own = w.x | static_cast<unsigned long long>(w.y) << 32;
        const unsigned long long before = __shfl_up_sync(0xFFFFFFFFu, own, 1, L);
        const unsigned long long both = s ? own << (8 * s) | before >> (64 - 8 * s) : own;
        if ((lane > 0 || s == 0) && e - s + 8 <= K) {
            *reinterpret_cast<unsigned long long *>(row + (e - s)) = both;
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if ((lane > 0 || i >= s) && e - s + i < K)
                    row[e - s + i] = static_cast<uint8_t>(both >> (8 * i));
        }
        if (lane == L - 1) {
#pragma unroll
            for (int i = 1; i < 8; ++i)
                if (i >= 8 - s && e + i < K)
                    row[e + i] = static_cast<uint8_t>(own >> (8 * i));
        }
    }
}

__device__ __forceinline__ Eight widen8(const Raw8 &r)
{
    Eight e;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        e.v[2 * i] = bf16lo(r.w[i]), e.v[2 * i + 1] = bf16hi(r.w[i]);
    return e;
}

// The row of x that a row of q is of: none where its index is out of range.
struct RowSource {
    long long row;
    bool live;
};

__device__ __forceinline__ RowSource row_source(const F8RowParams &p, long long row)
{
    if (!p.rows)
        return {row, true};
    const int r = __ldcg(p.rows + row);
    const bool live = r >= 0 && r < p.x_rows;
    return {live ? r : 0, live};
}

constexpr int kRowWarps = 8;

// A warp takes 2 P blocks of a row, 16 lanes a block, 8 values a lane.
template <bool ANY, bool GATE, int P>
__global__ void __launch_bounds__(32 * kRowWarps) f8_rows_kernel(const F8RowParams p, int groups)
{
    pdl_wait();
    pdl_launch_dependents();
    const long long unit = static_cast<long long>(blockIdx.x) * kRowWarps + (threadIdx.x >> 5);
    const long long row = unit / groups;
    if (row >= p.M)
        return;
    const int b0 = static_cast<int>(unit - row * groups) * 2 * P, lane = threadIdx.x & 31, half = lane >> 4;
    const RowSource from = row_source(p, row);
    const int e0 = (b0 + half) * kF8Block + (lane & 15) * 8;
    const int K = from.live ? p.K : 0;
    RowLoad<ANY> a[P], c[P];
#pragma unroll
    for (int i = 0; i < P; ++i)
        a[i].load(p.x + from.row * p.ldx, e0 + i * 2 * kF8Block, K);
    if (GATE) {
#pragma unroll
        for (int i = 0; i < P; ++i)
            c[i].load(p.gate + from.row * p.ldg, e0 + i * 2 * kF8Block, K);
    }
#pragma unroll
    for (int i = 0; i < P; ++i) {
        Eight v = widen8(a[i].get());
        if (GATE)
            v = gated(widen8(c[i].get()), v);
        uint32_t m = max_bits(v);
#pragma unroll
        for (int o = 8; o; o >>= 1)
            m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
        const BlockScale s = block_scale(m);
        store8<ANY, 32>(p.q + row * p.K, e0 + i * 2 * kF8Block, p.K, to_e4m3(v, s));
        const int b = b0 + 2 * i + half;
        if ((lane & 15) == 0 && b < p.kb)
            p.scale[row * p.kb + b] = s.scale;
    }
}

// A CTA takes a block of 128 x 128: 16 lanes a row, 16 rows at a time.
template <bool ANY>
__global__ void __launch_bounds__(256, 2) f8_weights_kernel(const F8WeightParams p)
{
    __shared__ uint32_t maxima[8];
    pdl_wait();
    pdl_launch_dependents();
    const long long block = blockIdx.x, en = block / p.kb;
    const int b = static_cast<int>(block - en * p.kb), e = static_cast<int>(en / p.nb), nb = static_cast<int>(en - static_cast<long long>(e) * p.nb);
    const int t = threadIdx.x, k = (t & 15) * 8;
    RowLoad<ANY> a[8];
    uint32_t m = 0;
    const int e0 = b * kF8Block + k;
    auto at = [&](int i) {
        return (static_cast<size_t>(e) * p.N + nb * kF8Block + (t >> 4) + 16 * i) * p.K;
    };
    auto inside = [&](int i) { return static_cast<long long>(nb) * kF8Block + (t >> 4) + 16 * i < p.N; };
#pragma unroll
    for (int i = 0; i < 8; ++i)
        a[i].load(p.W + at(i), e0, inside(i) ? p.K : 0);
#pragma unroll
    for (int i = 0; i < 8; ++i)
        m = max(m, max_bits(widen8(a[i].get())));
    m = __reduce_max_sync(0xFFFFFFFFu, m);
    if ((t & 31) == 0)
        maxima[t >> 5] = m;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 8; ++i)
        m = max(m, maxima[i]);
    const BlockScale s = block_scale(m);
#pragma unroll
    for (int i = 0; i < 8; ++i)
        store8<ANY, 16>(p.q + at(i), e0, inside(i) ? p.K : 0, to_e4m3(widen8(a[i].get()), s));
    if (t == 0)
        p.scale[block] = s.scale;
}

template <class P, class... A>
cudaError_t launch(void (*kernel)(P, A...), long long grid, unsigned threads, cudaStream_t s, const P &p, A... a)
{
    if (grid > 0x7FFFFFFFll)
        return cudaErrorInvalidConfiguration;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(grid));
    cfg.blockDim = dim3(threads);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, p, a...);
}

bool multiple(const void *ptr, size_t bytes) { return reinterpret_cast<uintptr_t>(ptr) % bytes == 0; }

template <bool ANY, bool GATE>
cudaError_t launch_rows(const F8RowParams &p, cudaStream_t s)
{
    auto run = [&](auto kernel, int blocks) {
        const int groups = (p.kb + blocks - 1) / blocks;
        return launch(kernel, (static_cast<long long>(p.M) * groups + kRowWarps - 1) / kRowWarps, 32 * kRowWarps, s, p, groups);
    };
    // Many blocks of long rows: more of them a warp, for bytes in flight.
    const bool many = p.kb >= 8 && static_cast<long long>(p.M) * p.kb >= 8 * 16 * 152;
    if (!many)
        return run(f8_rows_kernel<ANY, GATE, 1>, 2);
    return run(f8_rows_kernel<ANY, GATE, 4>, 8);
}

} // namespace

cudaError_t launch_f8_quantize(const F8RowParams &p, cudaStream_t s)
{
    const bool aligned = p.K % 8 == 0 && p.ldx % 8 == 0 && (!p.gate || p.ldg % 8 == 0) && multiple(p.x, 16) &&
                         multiple(p.gate, 16) && multiple(p.q, 8);           // null is aligned
    if (p.gate)
        return aligned ? launch_rows<false, true>(p, s) : launch_rows<true, true>(p, s);
    return aligned ? launch_rows<false, false>(p, s) : launch_rows<true, false>(p, s);
}

cudaError_t launch_f8_quantize_weights(const F8WeightParams &p, cudaStream_t s)
{
    const bool aligned = p.K % 8 == 0 && multiple(p.W, 16) && multiple(p.q, 8);
    const long long grid = static_cast<long long>(p.E) * p.nb * p.kb;
    return aligned ? launch(f8_weights_kernel<false>, grid, 256, s, p) : launch(f8_weights_kernel<true>, grid, 256, s, p);
}

} // namespace skg

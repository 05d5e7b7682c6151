// skg_f8_rows.cu -- bf16 turned into e4m3 with one fp32 scale for each block of
// 128 values of a row (activations), or of 128 x 128 (weights).
//
//   v = x, or silu(gate) * x;   scale = max|v| / 448;   q = e4m3(v * (448 / max|v|))
//
// v, the quotient and the product are fp32, and the product is rounded once, half
// to even.  A block is read once: its values stay in registers through the
// maximum.  8 lanes take a block of a row, 16 values a lane; a CTA takes a block of a
// weight.  Rows that are not aligned are read in 16-byte blocks shifted into place, and
// their numbers stored in aligned words that two lanes fill.
//
// What bounds it is HBM where rows are aligned: 8192 x 7168 29 us (6.1 TB/s of 6.71),
// 65536 x 256 8.1, weight 12288 x 7168 42 us (6.3); gated by silu nearly instructions:
// 4096 x 16384 60 us (5.6 TB/s).  Instructions elsewhere: 8191 x 7169 56 us, gated 4095 x
// 16383 104, weight 5001 x 4113 22.5 us, rows of 4096 tokens taken 8 times each 92 us;
// 512 rows of 7168 take 3.6 us.  (With 16 lanes a block, 8 values a lane, each of which
// works out its block's scale: 30.5, 12, 48; 61; 76, 144, 29, 106.  With single elements
// loaded and stored where rows are not aligned: 89, 176, 40.)
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
// numbers 0, so that whatever it multiplies is NaN.  Below 1.3e-36 the quotient 448 /
// max would leave fp32's range: from 1e-30 down, a margin, both are raised by 2^100,
// which is exact.
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

// 16 values as numbers, 8 to a word.
struct Numbers {
    uint32_t u[4];

    __device__ __forceinline__ unsigned long long eight(int h) const { return u[2 * h] | static_cast<unsigned long long>(u[2 * h + 1]) << 32; }
};

__device__ __forceinline__ Numbers to_e4m3(Values<16> e, const BlockScale &b)
{
    scale_values(e, b);
    Numbers n;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const uint32_t lo = two_e4m3(e.v[8 * i], e.v[8 * i + 1]) | two_e4m3(e.v[8 * i + 2], e.v[8 * i + 3]) << 16;
        const uint32_t hi = two_e4m3(e.v[8 * i + 4], e.v[8 * i + 5]) | two_e4m3(e.v[8 * i + 6], e.v[8 * i + 7]) << 16;
        n.u[2 * i] = lo;
        n.u[2 * i + 1] = hi;
    }
    return n;
}

// silu(g) x, by the fast exponential.  Of 201 million gated normal values 573 get another
// number than in 64 bits, in plain 32-bit operations 588, with expf 555, with expf and
// an IEEE quotient 554: what is left is v's rounding beside a border.  expf takes 4096 x
// 16384 from 60 to 70 us, with the quotient to 80.
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

// 16 numbers at element e of a row of K.  ANY: of any alignment; L neighbouring lanes
// have neighbouring sixteens (all of them call), and a lane stores the two aligned
// words that its eights begin in: the end of what comes before and the beginning of its
// own.
template <bool ANY, int L>
__device__ __forceinline__ void store16(uint8_t *row, int e, int K, const Numbers &n)
{
    if constexpr (!ANY) {
        if (e < K)                       // K is a multiple of 16
            *reinterpret_cast<uint4 *>(row + e) = make_uint4(n.u[0], n.u[1], n.u[2], n.u[3]);
    } else {
        const int lane = static_cast<int>(threadIdx.x) & (L - 1);
        const int s = static_cast<int>(reinterpret_cast<uintptr_t>(row) + e) & 7;
        unsigned long long before = __shfl_up_sync(0xFFFFFFFFu, n.eight(1), 1, L);
#pragma unroll
        for (int h = 0; h < 2; ++h, e += 8) {
            const unsigned long long both = s ? n.eight(h) << (8 * s) | before >> (64 - 8 * s) : n.eight(h);
            const bool first = lane == 0 && h == 0;          // what comes before is not this warp's
            if ((!first || s == 0) && e - s + 8 <= K) {
                *reinterpret_cast<unsigned long long *>(row + (e - s)) = both;
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    if ((!first || i >= s) && e - s + i < K)
                        row[e - s + i] = static_cast<uint8_t>(both >> (8 * i));
            }
            before = n.eight(h);
        }
        if (lane == L - 1) {             // nor what comes after: the end of the last eight
#pragma unroll
            for (int i = 1; i < 8; ++i)
                if (i >= 8 - s && e - 8 + i < K)
                    row[e - 8 + i] = static_cast<uint8_t>(n.eight(1) >> (8 * i));
        }
    }
}

// 16 values of a row from element e on, zeros where it ends.
template <bool ANY>
struct Load16 {
    RowLoad<ANY> a, b;

    __device__ __forceinline__ void load(const uint16_t *row, int e, int K)
    {
        a.load(row, e, K);
        b.load(row, e + 8, K);
    }

    __device__ __forceinline__ Values<16> get() const
    {
        const Raw8 x = a.get(), y = b.get();
        Values<16> v;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v.v[2 * i] = bf16lo(x.w[i]), v.v[2 * i + 1] = bf16hi(x.w[i]);
            v.v[8 + 2 * i] = bf16lo(y.w[i]), v.v[9 + 2 * i] = bf16hi(y.w[i]);
        }
        return v;
    }
};

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

// A warp takes 4 P blocks of a row, 8 lanes a block, 16 values a lane.  SHORT: rows of
// fewer than 4 blocks, whose warps take 4 blocks of neighbouring rows.
constexpr int kLanes = kF8Block / 16;
constexpr int kWarpBlocks = 32 / kLanes;

// (16 blocks a warp take 66 registers if they may, and 105 us instead of 92 for rows that come
// from the L2: three CTAs an SM instead of four.)
template <bool ANY, bool GATE, bool SHORT, int P>
__global__ void __launch_bounds__(32 * kRowWarps, P == 4 ? 4 : 0) f8_rows_kernel(const F8RowParams p, int groups)
{
    constexpr int B = kWarpBlocks;
    pdl_wait();
    pdl_launch_dependents();
    const long long warp = static_cast<long long>(blockIdx.x) * kRowWarps + (threadIdx.x >> 5);
    const int lane = threadIdx.x & 31;
    const long long unit = SHORT ? warp * B + lane / kLanes : warp;
    const long long row = unit / groups;
    // (SHORT: beyond the last row, as on a row of nothing, for the sake of the other lanes)
    const bool beyond = row >= p.M;
    if (!SHORT && beyond)
        return;
    const int b0 = static_cast<int>(unit - row * groups) * (SHORT ? 1 : B * P) + (SHORT ? 0 : lane / kLanes);
    const RowSource from = beyond ? RowSource{0, false} : row_source(p, row);
    const int e0 = b0 * kF8Block + lane % kLanes * 16;
    const int K = from.live ? p.K : 0;
    Load16<ANY> a[P], c[P];
#pragma unroll
    for (int i = 0; i < P; ++i)
        a[i].load(p.x + from.row * p.ldx, e0 + i * B * kF8Block, K);
    if (GATE) {
#pragma unroll
        for (int i = 0; i < P; ++i)
            c[i].load(p.gate + from.row * p.ldg, e0 + i * B * kF8Block, K);
    }
#pragma unroll
    for (int i = 0; i < P; ++i) {
        Values<16> v = a[i].get();
        if (GATE)
            v = gated(c[i].get(), v);
        uint32_t m = max_bits(v);
#pragma unroll
        for (int o = kLanes / 2; o; o >>= 1)
            m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
        const BlockScale s = block_scale(m);
        store16<ANY, SHORT ? kLanes : 32>(p.q + row * p.K, e0 + i * B * kF8Block, beyond ? 0 : p.K, to_e4m3(v, s));
        const int b = b0 + i * B;
        if (lane % kLanes == 0 && b < p.kb && !beyond)
            p.scale[row * p.kb + b] = s.scale;
    }
}

// A CTA takes a block of 128 x 128: 8 lanes a row, 32 rows at a time.
template <bool ANY>
__global__ void __launch_bounds__(256, 3) f8_weights_kernel(const F8WeightParams p)
{
    constexpr int ROWS = 256 / kLanes, P = kF8Block / ROWS;
    __shared__ uint32_t maxima[8];
    pdl_wait();
    pdl_launch_dependents();
    const long long block = blockIdx.x, en = block / p.kb;
    const int b = static_cast<int>(block - en * p.kb), e = static_cast<int>(en / p.nb), nb = static_cast<int>(en - static_cast<long long>(e) * p.nb);
    const int t = threadIdx.x;
    Load16<ANY> a[P];
    uint32_t m = 0;
    const int e0 = b * kF8Block + t % kLanes * 16;
    auto at = [&](int i) { return (static_cast<size_t>(e) * p.N + nb * kF8Block + t / kLanes + ROWS * i) * p.K; };
    auto inside = [&](int i) { return static_cast<long long>(nb) * kF8Block + t / kLanes + ROWS * i < p.N; };
#pragma unroll
    for (int i = 0; i < P; ++i)
        a[i].load(p.W + at(i), e0, inside(i) ? p.K : 0);
#pragma unroll
    for (int i = 0; i < P; ++i)
        m = max(m, max_bits(a[i].get()));
    m = __reduce_max_sync(0xFFFFFFFFu, m);
    if ((t & 31) == 0)
        maxima[t >> 5] = m;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 8; ++i)
        m = max(m, maxima[i]);
    const BlockScale s = block_scale(m);
#pragma unroll
    for (int i = 0; i < P; ++i)
        store16<ANY, kLanes>(p.q + at(i), e0, inside(i) ? p.K : 0, to_e4m3(a[i].get(), s));
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

// Blocks a warp: 4, or for many blocks 8 or 16, for bytes in flight, if rows leave few
// of them over.  Measured with 4, 8, 16: 8192 x 7168 39, 29.5, 28.7 us, gated 4096 x
// 16384 68, 61, 62; of any alignment 8191 x 7169 -, 56, 71, gated 4095 x 16383 104,
// 121, 233.
template <bool ANY, bool GATE>
cudaError_t launch_rows(const F8RowParams &p, cudaStream_t s)
{
    auto run = [&](auto kernel, int groups, long long warps) {
        return launch(kernel, (warps + kRowWarps - 1) / kRowWarps, 32 * kRowWarps, s, p, groups);
    };
    if (p.kb < kWarpBlocks) {
        const long long warps = (static_cast<long long>(p.M) * p.kb + kWarpBlocks - 1) / kWarpBlocks;
        return run(f8_rows_kernel<ANY, GATE, true, 1>, p.kb, warps);
    }
    auto groups = [&](int P) { return (p.kb + kWarpBlocks * P - 1) / (kWarpBlocks * P); };
    auto fits = [&](int P) {
        return static_cast<long long>(p.M) * p.kb >= 8 * 16 * 152 && groups(P) * kWarpBlocks * P <= p.kb + p.kb / 6;
    };
    if constexpr (!ANY && !GATE) {
        if (fits(4))
            return run(f8_rows_kernel<ANY, GATE, false, 4>, groups(4), static_cast<long long>(p.M) * groups(4));
    }
    if constexpr (!ANY || !GATE) {
        if (fits(2))
            return run(f8_rows_kernel<ANY, GATE, false, 2>, groups(2), static_cast<long long>(p.M) * groups(2));
    }
    return run(f8_rows_kernel<ANY, GATE, false, 1>, groups(1), static_cast<long long>(p.M) * groups(1));
}

} // namespace

cudaError_t launch_f8_quantize(const F8RowParams &p, cudaStream_t s)
{
    const bool aligned = p.K % 16 == 0 && p.ldx % 8 == 0 && (!p.gate || p.ldg % 8 == 0) && multiple(p.x, 16) &&
                         multiple(p.gate, 16) && multiple(p.q, 16);           // null is aligned
    if (p.gate)
        return aligned ? launch_rows<false, true>(p, s) : launch_rows<true, true>(p, s);
    return aligned ? launch_rows<false, false>(p, s) : launch_rows<true, false>(p, s);
}

cudaError_t launch_f8_quantize_weights(const F8WeightParams &p, cudaStream_t s)
{
    const bool aligned = p.K % 16 == 0 && multiple(p.W, 16) && multiple(p.q, 16);
    const long long grid = static_cast<long long>(p.E) * p.nb * p.kb;
    return aligned ? launch(f8_weights_kernel<false>, grid, 256, s, p) : launch(f8_weights_kernel<true>, grid, 256, s, p);
}

} // namespace skg

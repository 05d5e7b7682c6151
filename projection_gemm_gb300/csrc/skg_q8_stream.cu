// skg_q8_stream.cu -- the 8-bit projection for few tokens (M <= 16): W streams
// from HBM straight into registers, once.
//
// What bounds it is N K bytes of W.  A CTA owns 16 RG output channels and the
// whole of K, cut over its warps, so the sums meet in shared memory and nothing
// is exchanged between CTAs (a split of K across CTAs costs 6-8 us of partial
// sums and arrivals at these sizes, as long as streaming 40 MB).
//
// The product runs on the warp-level fp16 MMA (m16n8k16: 16 channels x 8 tokens):
// 8-bit integers are exact in fp16, their products and sums of up to 1024
// products in fp32, and every 1024 k the sums move to int32.  Both operands
// come from memory as 16-byte pieces of rows: a sum over k may take k in any
// order, so thread t of a row's four takes bytes 16 t .. 16 t + 15 of 64 and
// feeds them to four MMAs, and x follows the same order.
//
// Measured, back to back with weights from HBM (GB300, 6.70 TB/s copy peak):
// 1 x 12288 x 7168 16.0-16.4 us (5.4 TB/s), 1 x 7168 x 16384 21.0 us (5.6 TB/s),
// 8 x 7168 x 7168 9.9 us (5.2 TB/s), 16 x 7168 x 7168 11.9 us (4.3 TB/s), 1 x
// 1024 x 1024 1.8 us.  Up to 8 tokens HBM and the launch's ends bound it; with 16
// the widening of x weighs as much as that of W (instructions issue in 58% of
// the cycles, the ALU pipe is at 51%).  With the int8 MMA (no widening) 16 tokens
// take 14.0 us at 7168 x 7168.
#include "skg_internal.h"
#include "skg_ptx.cuh"
#include "skg_q8_common.cuh"
#include "skg_q8_internal.h"

namespace skg {
namespace {

constexpr int kStepK = 64;                 // k of one step: 16 bytes for each of a row's 4 threads
constexpr int kFlush = 1024 / kStepK;      // steps summed in fp32

__device__ __forceinline__ void mma_m16n8k16(float (&d)[4], const uint32_t (&a)[4], const uint32_t (&b)[2])
{
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 "
                 "{%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b[0]), "r"(b[1]));
}

// Weights: read once, so not kept in L1 and first out of L2.  Not the
// read-only path: without static weights they may have been written by the
// kernel that this one waits for.
__device__ __forceinline__ uint4 ld_stream(const int8_t *p, uint64_t pol)
{
    uint4 v;
    asm volatile("ld.global.L1::no_allocate.L2::cache_hint.v4.u32 {%0,%1,%2,%3}, [%4], %5;"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p), "l"(pol) : "memory");
    return v;
}

__device__ __forceinline__ uint4 ld_row(const int8_t *p)
{
    uint4 v;
    asm volatile("ld.global.v4.u32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p) : "memory");
    return v;
}

__device__ __forceinline__ uint32_t word(const uint4 &v, int i) { return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w; }

// NT: tiles of 8 tokens; RG: groups of 16 channels; DEPTH: steps in flight a warp.
template <int NT, int RG, int WARPS, int CTAS, int DEPTH>
__global__ void __launch_bounds__(WARPS * 32, CTAS) q8_stream_kernel(const Q8LinearParams p, int static_w)
{
    static_assert(kFlush % DEPTH == 0, "the fp32 sums are moved at whole rounds");
    __shared__ int part[WARPS][RG * 16][NT * 8];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int n0 = static_cast<int>(blockIdx.x) * (16 * RG);
    const int steps = (p.K + kStepK - 1) / kStepK;
    const int s0 = warp * steps / WARPS, s1 = (warp + 1) * steps / WARPS;
    const uint64_t pol = policy_evict_first();
    // rows beyond N and M repeat the last one; their sums are not stored
    const int8_t *wrow[RG][2], *xrow[NT];
#pragma unroll
    for (int r = 0; r < RG; ++r)
#pragma unroll
        for (int h = 0; h < 2; ++h)
            wrow[r][h] = p.W + static_cast<size_t>(min(n0 + r * 16 + h * 8 + g, p.N - 1)) * p.K + 16 * t;
#pragma unroll
    for (int i = 0; i < NT; ++i)
        xrow[i] = p.x + static_cast<size_t>(min(i * 8 + g, p.M - 1)) * p.K + 16 * t;

    uint4 w[DEPTH][RG][2], x[DEPTH][NT];
    const uint4 zero = make_uint4(0, 0, 0, 0);
    auto in_row = [&](int s) { return s < s1 && s * kStepK + 16 * t < p.K; };     // K is a multiple of 16
    auto load_w = [&](int s, int d) {
        const bool in = in_row(s);
#pragma unroll
        for (int r = 0; r < RG; ++r)
#pragma unroll
            for (int h = 0; h < 2; ++h)
                w[d][r][h] = in ? ld_stream(wrow[r][h] + s * kStepK, pol) : zero;
    };
    auto load_x = [&](int s, int d) {
        const bool in = in_row(s);
#pragma unroll
        for (int i = 0; i < NT; ++i)
            x[d][i] = in ? ld_row(xrow[i] + s * kStepK) : zero;
    };
    if (!static_w)
        pdl_wait();
#pragma unroll
    for (int d = 0; d < DEPTH; ++d)
        load_w(s0 + d, d);
    if (static_w)
        pdl_wait();                      // x, scales, residual and y only from here on
    // The next kernel may start once the one before this is done, not sooner: a
    // chain of kernels that all start early fills the SMs with waiting CTAs.
    pdl_launch_dependents();
#pragma unroll
    for (int d = 0; d < DEPTH; ++d)
        load_x(s0 + d, d);

    int sum[RG][NT][4] = {};
    float acc[RG][NT][4] = {};
    auto flush = [&] {
#pragma unroll
        for (int r = 0; r < RG; ++r)
#pragma unroll
            for (int i = 0; i < NT; ++i)
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    sum[r][i][c] += __float2int_rn(acc[r][i][c]);
                    acc[r][i][c] = 0.0f;
                }
    };
    int since = 0;
    for (int s = s0; s < s1; s += DEPTH) {
#pragma unroll
        for (int d = 0; d < DEPTH; ++d) {
            uint4 wc[RG][2], xc[NT];
#pragma unroll
            for (int r = 0; r < RG; ++r)
#pragma unroll
                for (int h = 0; h < 2; ++h)
                    wc[r][h] = w[d][r][h];
#pragma unroll
            for (int i = 0; i < NT; ++i)
                xc[i] = x[d][i];
            load_w(s + d + DEPTH, d);
            load_x(s + d + DEPTH, d);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                uint32_t b[NT][2];
#pragma unroll
                for (int i = 0; i < NT; ++i)
                    widen4(word(xc[i], j), b[i][0], b[i][1]);
#pragma unroll
                for (int r = 0; r < RG; ++r) {
                    uint32_t a[4];
                    widen4(word(wc[r][0], j), a[0], a[2]);
                    widen4(word(wc[r][1], j), a[1], a[3]);
#pragma unroll
                    for (int i = 0; i < NT; ++i)
                        mma_m16n8k16(acc[r][i], a, b[i]);
                }
            }
        }
        since += DEPTH;
        if (since == kFlush) {
            flush();
            since = 0;
        }
    }
    flush();

#pragma unroll
    for (int r = 0; r < RG; ++r)
#pragma unroll
        for (int i = 0; i < NT; ++i)
#pragma unroll
            for (int c = 0; c < 4; ++c)
                part[warp][r * 16 + (c >> 1) * 8 + g][i * 8 + 2 * t + (c & 1)] = sum[r][i][c];
    __syncthreads();
    for (int o = threadIdx.x; o < RG * 16 * NT * 8; o += WARPS * 32) {
        const int m = o / (RG * 16), n = o % (RG * 16);
        if (m < p.M && n0 + n < p.N) {
            int v = 0;
#pragma unroll
            for (int k = 0; k < WARPS; ++k)
                v += part[k][n][m];
            q8_store(p, m, n0 + n, v, __ldcg(p.x_scale + m), __ldcg(p.w_scale + n0 + n));
        }
    }
}

template <int NT, int RG, int WARPS, int CTAS, int DEPTH>
cudaError_t launch_as(const Q8LinearParams &p, bool static_w, cudaStream_t s)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((static_cast<unsigned>(p.N) + 16 * RG - 1) / (16 * RG));      // N up to 2^31 - 1
    cfg.blockDim = dim3(WARPS * 32);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, q8_stream_kernel<NT, RG, WARPS, CTAS, DEPTH>, p, static_w ? 1 : 0);
}

} // namespace

// The launch shape.  What decides is how evenly the CTAs fill the SMs: with
// slots left over, CTAs of the next launch crowd onto some SMs and their share
// of the stream ends late.  So as many warps a CTA, and as few CTAs an SM, as
// hold the grid in one wave (M = 1: N = 2048 16 warps 5.0 us, 8 warps 8.5 us;
// N = 4096 two CTAs of 16 warps 4.2, three of 8 5.5; N = 7168 three of 8 9.6,
// two of 16 11.2).  Beyond one wave of 16-channel CTAs, 32 (M <= 8: N = 12288
// 16.0 us against 17.4).  (With M > 8 such a grid is the split kernel's, but for
// small W: 12288 x 1024 with M = 16 5.9 us, 48 channels a CTA 7.3.)
Q8StreamShape q8_stream_shape(int M, int N, int num_sms)
{
    const long long groups = (static_cast<long long>(N) + 15) / 16;
    const bool two = M > 8;
    if (groups <= num_sms)
        return {1, 16, 1};
    if (groups <= 2ll * num_sms)
        return two ? Q8StreamShape{1, 8, 2} : Q8StreamShape{1, 16, 2};
    if (groups <= 3ll * num_sms)
        return {1, 8, 3};
    return two ? Q8StreamShape{1, 8, 3} : Q8StreamShape{2, 8, 3};
}

cudaError_t launch_q8_stream(const Q8LinearParams &p, const Q8StreamShape &sh, bool static_w, cudaStream_t s)
{
    if (p.M <= 8) {
        if (sh.groups == 2)
            return launch_as<1, 2, 8, 3, 2>(p, static_w, s);
        if (sh.warps == 8)
            return launch_as<1, 1, 8, 3, 2>(p, static_w, s);
        return sh.ctas_per_sm == 1 ? launch_as<1, 1, 16, 1, 1>(p, static_w, s)
                                   : launch_as<1, 1, 16, 2, 1>(p, static_w, s);
    }
    if (sh.warps == 16)
        return launch_as<2, 1, 16, 1, 1>(p, static_w, s);
    return sh.ctas_per_sm == 2 ? launch_as<2, 1, 8, 2, 2>(p, static_w, s) : launch_as<2, 1, 8, 3, 1>(p, static_w, s);
}

} // namespace skg

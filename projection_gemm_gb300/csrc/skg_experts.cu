// skg_experts.cu -- tokens to their experts and back: a stable sort of the
// choices by expert, rows gathered in that order, rows combined with weights, and
// the gradients of both.
//
//   rows[p]  the token of sorted row p;   pos[t, j]  the sorted row of a choice, or -1
//   gather:   out[p] = x[rows[p]]
//   combine:  out[t] = residual[t] + sum_j weight[t, j] y[pos[t, j]]
//   gradients of combine:  grad_y[pos[t, j]] = weight[t, j] grad_out[t],
//                          grad_weight[t, j] = <grad_out[t], y[pos[t, j]]>
//   (of gather: combine without weights)
//
// Sums are fp32 in a fixed order, rounded once, so a call gives the same bits
// each time.
//
// What bounds the rows' kernels is HBM (copy peak 6.71 TB/s).  4096 tokens, 8 choices
// each, rows of 7168: gather 97 us (5.4 TB/s, nearly all of it writes; hints to keep
// x in the L2 change nothing), combination 93 us (6.3; CTAs of 8 warps 110), without
// residual 81, gradients 166 (6.0).  Rows that are not whole blocks of 16 bytes move 4, 2 or 1
// elements a lane: 1001 tokens, 3 choices, rows of 2004, 2002, 2001: gather 4.2, 3.8, 5.0,
// combination 4.6, 5.2, 7.4, gradients 8.3, 8.3, 11.6 us (aligned blocks that two lanes fill
// by shuffles, for rows of any alignment: 9, 12, 35).  The sort is latency: 8 choices 2.1 us,
// 128 3.5, 32768 10.9 (8 CTAs); 524288 141, by the scattered stores of 8 SMs.
#include <algorithm>
#include <cstdint>

#include <cuda.h>
#include <cuda_runtime.h>

#include "skg.h"
#include "skg_f8_internal.h"
#include "skg_internal.h"
#include "skg_ptx.cuh"
#include "skg_q8_common.cuh"

namespace skg {
namespace {

// ---------------------------------------------------------------------- sort
// One cluster.  CTA c takes the c-th part of the choices, its warps a run of that
// each: a warp counts its run by expert, the counts are added up over the warps
// and CTAs before and the experts before, and the warp goes over its run again and
// gives each choice its place.  Lanes with the same expert find each other by
// match_any; all of it is in order, so the sort is stable and nothing is atomic.
constexpr int kSortWarps = 32, kSortCtas = 8;
constexpr int kSortHeld = 4;             // rounds of 32 choices that a warp holds in registers from one pass to the next

struct SortParams {
    const int *expert;        // [n]
    int *offsets, *rows, *pos;
    int n, k, E;
    int warps, run;           // warps that have choices, and how many each (a multiple of 32)
    int ctas;
};

__device__ __forceinline__ int ld_shared_cluster_int(uint32_t addr)
{
    int v;
    asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
    return v;
}

__global__ void __launch_bounds__(32 * kSortWarps) sort_kernel(const SortParams p)
{
    extern __shared__ int hist[];        // [warps][E], then total [E], then base [E]
    __shared__ int warp_sum[kSortWarps];
    int *total = hist + p.warps * p.E, *base = total + p.E;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, cta = blockIdx.x, threads = blockDim.x;
    for (int i = threadIdx.x; i < p.warps * p.E; i += threads)
        hist[i] = 0;
    __syncthreads();
    pdl_wait();
    pdl_launch_dependents();

    const long long begin = (static_cast<long long>(cta) * p.warps + warp) * p.run;
    const int steps = warp < p.warps && begin < p.n ? static_cast<int>(min(static_cast<long long>(p.run), p.n - begin) + 31) / 32 : 0;
    int *mine = hist + warp * p.E;
    auto key_at = [&](int s) {           // -1: no expert
        const long long i = begin + s * 32 + lane;
        const int e = s < steps && i < p.n ? __ldcg(p.expert + i) : -1;
        return e >= 0 && e < p.E ? e : -1;
    };
    auto count = [&](int key, unsigned same) {
        if (key >= 0 && lane == __ffs(same) - 1)
            mine[key] += __popc(same);
        __syncwarp();
    };
    int held[kSortHeld];
    unsigned held_same[kSortHeld];
#pragma unroll
    for (int s = 0; s < kSortHeld; ++s)
        held[s] = key_at(s);
#pragma unroll
    for (int s = 0; s < kSortHeld; ++s) {
        held_same[s] = 0;
        if (s < steps) {
            held_same[s] = __match_any_sync(0xFFFFFFFFu, held[s]);
            count(held[s], held_same[s]);
        }
    }
    int next = key_at(kSortHeld);
    for (int s = kSortHeld; s < steps; ++s) {
        const int key = next;
        next = key_at(s + 1);
        count(key, __match_any_sync(0xFFFFFFFFu, key));
    }
    __syncthreads();
    for (int e = threadIdx.x; e < p.E; e += threads) {
        int sum = 0;
#pragma unroll 8
        for (int w = 0; w < p.warps; ++w) {
            const int c = hist[w * p.E + e];
            hist[w * p.E + e] = sum;
            sum += c;
        }
        total[e] = sum;
    }
    if (p.ctas > 1)
        cluster_sync();
    else
        __syncthreads();
    // the experts' first rows: up to two experts a thread (threads >= E / 2), added up in their order
    int all[2], before[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int e = 2 * threadIdx.x + i;
        all[i] = before[i] = 0;
        if (e < p.E) {
            if (p.ctas == 1) {
                all[i] = total[e];
            } else {
                int v[kSortCtas];
#pragma unroll
                for (int c = 0; c < kSortCtas; ++c)
                    v[c] = ld_shared_cluster_int(map_shared_rank(smem_u32(total + e), c));
#pragma unroll
                for (int c = 0; c < kSortCtas; ++c) {
                    before[i] += c < cta ? v[c] : 0;
                    all[i] += v[c];
                }
            }
        }
    }
    int scan = all[0] + all[1];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xFFFFFFFFu, scan, o);
        scan += lane >= o ? v : 0;
    }
    if (lane == 31)
        warp_sum[warp] = scan;
    __syncthreads();
    const int sum = lane < threads / 32 ? warp_sum[lane] : 0;
    const int lower = __reduce_add_sync(0xFFFFFFFFu, lane < warp ? sum : 0), routed = __reduce_add_sync(0xFFFFFFFFu, sum);
    int start = lower + scan - all[0] - all[1];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int e = 2 * threadIdx.x + i;
        if (e < p.E) {
            base[e] = start + before[i];
            if (cta == 0)
                p.offsets[e] = start;
        }
        start += all[i];
    }
    if (cta == 0 && threadIdx.x == 0)
        p.offsets[p.E] = routed;
    __syncthreads();
    auto put = [&](int s, int key, unsigned same) {
        const int at = key >= 0 ? mine[key] : 0;
        __syncwarp();
        if (key >= 0 && lane == __ffs(same) - 1)
            mine[key] = at + __popc(same);
        const long long i = begin + s * 32 + lane;
        const int place = key >= 0 ? base[key] + at + __popc(same & ((1u << lane) - 1)) : -1;
        if (i < p.n)
            p.pos[i] = place;
        if (key >= 0)
            p.rows[place] = static_cast<int>(i) / p.k;
        __syncwarp();
    };
#pragma unroll
    for (int s = 0; s < kSortHeld; ++s)
        if (s < steps)
            put(s, held[s], held_same[s]);
    next = key_at(kSortHeld);
    for (int s = kSortHeld; s < steps; ++s) {
        const int key = next;
        next = key_at(s + 1);
        put(s, key, __match_any_sync(0xFFFFFFFFu, key));
    }
    for (long long i = routed + static_cast<long long>(cta) * threads + threadIdx.x; i < p.n; i += p.ctas * threads)
        p.rows[i] = -1;
    if (p.ctas > 1)
        cluster_sync();                  // no CTA leaves while a peer reads its totals
}

// ---------------------------------------------------------------- rows moved
__device__ __forceinline__ uint32_t two_bf16(float a, float b)
{
    return f32_to_bf16(a) | static_cast<uint32_t>(f32_to_bf16(b)) << 16;
}

// V elements at a time: as many of 8, 4, 2, 1 as every row's alignment allows.  (The
// loads' "memory" keeps a row's stores behind them where gradients take y's place.)
template <int V>
struct Piece;

template <>
struct Piece<8> {
    uint4 w;
    __device__ __forceinline__ void load(const uint16_t *p)
    {
        asm volatile("ld.global.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(w.x), "=r"(w.y), "=r"(w.z), "=r"(w.w) : "l"(p) : "memory");
    }
    __device__ __forceinline__ void zero() { w = make_uint4(0, 0, 0, 0); }
    __device__ __forceinline__ void store(uint16_t *p) const { __stcs(reinterpret_cast<uint4 *>(p), w); }
    __device__ __forceinline__ void get(float (&v)[8]) const
    {
        v[0] = bf16lo(w.x), v[1] = bf16hi(w.x), v[2] = bf16lo(w.y), v[3] = bf16hi(w.y);
        v[4] = bf16lo(w.z), v[5] = bf16hi(w.z), v[6] = bf16lo(w.w), v[7] = bf16hi(w.w);
    }
    __device__ __forceinline__ void set(const float (&v)[8])
    {
        w = make_uint4(two_bf16(v[0], v[1]), two_bf16(v[2], v[3]), two_bf16(v[4], v[5]), two_bf16(v[6], v[7]));
    }
};

template <>
struct Piece<4> {
    uint2 w;
    __device__ __forceinline__ void load(const uint16_t *p)
    {
        asm volatile("ld.global.v2.u32 {%0,%1}, [%2];" : "=r"(w.x), "=r"(w.y) : "l"(p) : "memory");
    }
    __device__ __forceinline__ void zero() { w = make_uint2(0, 0); }
    __device__ __forceinline__ void store(uint16_t *p) const { __stcs(reinterpret_cast<uint2 *>(p), w); }
    __device__ __forceinline__ void get(float (&v)[4]) const { v[0] = bf16lo(w.x), v[1] = bf16hi(w.x), v[2] = bf16lo(w.y), v[3] = bf16hi(w.y); }
    __device__ __forceinline__ void set(const float (&v)[4]) { w = make_uint2(two_bf16(v[0], v[1]), two_bf16(v[2], v[3])); }
};

template <>
struct Piece<2> {
    uint32_t w;
    __device__ __forceinline__ void load(const uint16_t *p) { asm volatile("ld.global.u32 %0, [%1];" : "=r"(w) : "l"(p) : "memory"); }
    __device__ __forceinline__ void zero() { w = 0; }
    __device__ __forceinline__ void store(uint16_t *p) const { __stcs(reinterpret_cast<uint32_t *>(p), w); }
    __device__ __forceinline__ void get(float (&v)[2]) const { v[0] = bf16lo(w), v[1] = bf16hi(w); }
    __device__ __forceinline__ void set(const float (&v)[2]) { w = two_bf16(v[0], v[1]); }
};

template <>
struct Piece<1> {
    uint16_t w;
    __device__ __forceinline__ void load(const uint16_t *p) { asm volatile("ld.global.u16 %0, [%1];" : "=h"(w) : "l"(p) : "memory"); }
    __device__ __forceinline__ void zero() { w = 0; }
    __device__ __forceinline__ void store(uint16_t *p) const { *p = w; }
    __device__ __forceinline__ void get(float (&v)[1]) const { v[0] = bf16_to_f32(w); }
    __device__ __forceinline__ void set(const float (&v)[1]) { w = f32_to_bf16(v[0]); }
};

struct MoveParams {
    const uint16_t *x;        // gather: [x_rows, N]; combine: y [R, N] -- row stride ldx
    const uint16_t *res;      // combine: [T, N] dense, or null; gradient: grad_out
    const int *index;         // gather: rows [R]; else pos [T, k]
    const float *weight;      // [T, k], or null
    uint16_t *out;            // dense rows of N; gradient: grad_y
    float *grad_weight;
    size_t ldx;
    long long units;          // gather, combine: warps with work
    int rows, x_rows, N, k, groups;
};

constexpr int kGatherWarps = 8, kCombineWarps = 4;
constexpr int kDeep = 8;                 // gather: pieces a lane
constexpr int kMaxN = 1 << 30;           // element indexes of a row, and those just behind it, fit 32 bits

// A warp takes kDeep pieces a lane of one row.
template <int V>
__global__ void __launch_bounds__(32 * kGatherWarps) gather_kernel(const MoveParams p)
{
    pdl_wait();
    pdl_launch_dependents();
    const long long unit = static_cast<long long>(blockIdx.x) * kGatherWarps + (threadIdx.x >> 5);
    if (unit >= p.units)
        return;
    const long long row = unit / p.groups;
    const int n0 = static_cast<int>(unit - row * p.groups) * (32 * V * kDeep) + static_cast<int>(threadIdx.x & 31) * V;
    const int from = __ldcg(p.index + row);
    const bool live = from >= 0 && from < p.x_rows;
    const uint16_t *x = p.x + (live ? from : 0) * p.ldx;
    Piece<V> a[kDeep];
#pragma unroll
    for (int i = 0; i < kDeep; ++i) {
        a[i].zero();
        if (live && n0 + i * 32 * V < p.N)
            a[i].load(x + n0 + i * 32 * V);
    }
#pragma unroll
    for (int i = 0; i < kDeep; ++i)
        if (n0 + i * 32 * V < p.N)
            a[i].store(p.out + row * p.N + n0 + i * 32 * V);
}

constexpr int kBatch = 8;                // choices of a token whose rows are on their way together

// A warp takes PC pieces a lane of one token.
template <int V, int PC>
__global__ void __launch_bounds__(32 * kCombineWarps) combine_kernel(const MoveParams p)
{
    pdl_wait();
    pdl_launch_dependents();
    const long long unit = static_cast<long long>(blockIdx.x) * kCombineWarps + (threadIdx.x >> 5);
    if (unit >= p.units)
        return;
    const long long t = unit / p.groups;
    const int lane = threadIdx.x & 31, n = static_cast<int>(unit - t * p.groups) * (32 * V * PC) + lane * V;
    float acc[PC][V];
#pragma unroll
    for (int i = 0; i < PC; ++i) {
#pragma unroll
        for (int c = 0; c < V; ++c)
            acc[i][c] = 0.0f;
        if (p.res && n + i * 32 * V < p.N) {
            Piece<V> r;
            r.load(p.res + t * p.N + n + i * 32 * V);
            r.get(acc[i]);
        }
    }
    for (int j0 = 0; j0 < p.k; j0 += kBatch) {
        int at = -1;
        float w = 1.0f;
        if (lane < kBatch && j0 + lane < p.k) {
            at = __ldcg(p.index + t * p.k + j0 + lane);
            if (p.weight)
                w = __ldcg(p.weight + t * p.k + j0 + lane);
        }
        Piece<V> y[kBatch][PC];
#pragma unroll
        for (int j = 0; j < kBatch; ++j) {
            const int from = __shfl_sync(0xFFFFFFFFu, at, j);
#pragma unroll
            for (int i = 0; i < PC; ++i)
                if (from >= 0 && from < p.x_rows && n + i * 32 * V < p.N)
                    y[j][i].load(p.x + from * p.ldx + n + i * 32 * V);
        }
#pragma unroll
        for (int j = 0; j < kBatch; ++j) {
            const int from = __shfl_sync(0xFFFFFFFFu, at, j);
            const float wj = __shfl_sync(0xFFFFFFFFu, w, j);
            if (from >= 0 && from < p.x_rows) {
#pragma unroll
                for (int i = 0; i < PC; ++i) {
                    float v[V];
                    y[j][i].get(v);
#pragma unroll
                    for (int c = 0; c < V; ++c)
                        acc[i][c] = fmaf(wj, v[c], acc[i][c]);
                }
            }
        }
    }
#pragma unroll
    for (int i = 0; i < PC; ++i) {
        if (n + i * 32 * V < p.N) {
            Piece<V> r;
            r.set(acc[i]);
            r.store(p.out + t * p.N + n + i * 32 * V);
        }
    }
}

// A CTA takes a token.
constexpr int kGradThreads = 256;

template <int V, int PC>
__global__ void __launch_bounds__(kGradThreads) combine_grad_kernel(const MoveParams p)
{
    __shared__ float sums[kBatch][kGradThreads / 32];
    pdl_wait();
    pdl_launch_dependents();
    const long long t = blockIdx.x;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    for (int j0 = 0; j0 < p.k; j0 += kBatch) {
        int at[kBatch];
        float w[kBatch], dot[kBatch];
#pragma unroll
        for (int j = 0; j < kBatch; ++j) {
            at[j] = j0 + j < p.k ? __ldcg(p.index + t * p.k + j0 + j) : -1;
            at[j] = at[j] < p.x_rows ? at[j] : -1;
            w[j] = at[j] >= 0 ? __ldcg(p.weight + t * p.k + j0 + j) : 0.0f;
            dot[j] = 0.0f;
        }
        for (int n0 = threadIdx.x * V; n0 < p.N; n0 += kGradThreads * V * PC) {
            Piece<V> g[PC], y[kBatch][PC];
#pragma unroll
            for (int i = 0; i < PC; ++i)
                if (n0 + i * kGradThreads * V < p.N)
                    g[i].load(p.res + t * p.N + n0 + i * kGradThreads * V);
#pragma unroll
            for (int j = 0; j < kBatch; ++j)
#pragma unroll
                for (int i = 0; i < PC; ++i)
                    if (at[j] >= 0 && n0 + i * kGradThreads * V < p.N)
                        y[j][i].load(p.x + at[j] * p.ldx + n0 + i * kGradThreads * V);
#pragma unroll
            for (int i = 0; i < PC; ++i) {
                const int n = n0 + i * kGradThreads * V;
                if (n >= p.N)
                    continue;
                float gv[V];
                g[i].get(gv);
#pragma unroll
                for (int j = 0; j < kBatch; ++j) {
                    if (at[j] >= 0) {
                        float v[V], d[V];
                        y[j][i].get(v);
#pragma unroll
                        for (int c = 0; c < V; ++c) {
                            dot[j] = fmaf(gv[c], v[c], dot[j]);
                            d[c] = w[j] * gv[c];
                        }
                        Piece<V> o;
                        o.set(d);
                        o.store(p.out + static_cast<size_t>(at[j]) * p.N + n);
                    }
                }
            }
        }
#pragma unroll
        for (int j = 0; j < kBatch; ++j) {
#pragma unroll
            for (int o = 16; o; o >>= 1)
                dot[j] += __shfl_xor_sync(0xFFFFFFFFu, dot[j], o);
            if (lane == 0)
                sums[j][warp] = dot[j];
        }
        __syncthreads();
        if (threadIdx.x < kBatch && j0 + static_cast<int>(threadIdx.x) < p.k) {
            float s = 0.0f;
#pragma unroll
            for (int i = 0; i < kGradThreads / 32; ++i)
                s += sums[threadIdx.x][i];
            p.grad_weight[t * p.k + j0 + threadIdx.x] = s;
        }
        __syncthreads();
    }
}

template <class P, class... A>
cudaError_t launch(void (*kernel)(P, A...), long long grid, unsigned threads, size_t smem, unsigned cluster, cudaStream_t s,
                   const P &p, A... a)
{
    if (grid > 0x7FFFFFFFll)
        return cudaErrorInvalidConfiguration;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(grid));
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = cluster;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kernel, p, a...);
}

bool aligned(const void *p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }      // null is aligned

skg_status launched(cudaError_t e, const char *who)
{
    return e == cudaSuccess ? SKG_OK
                            : set_error(SKG_ERR_CUDA, "%s: %s (%s)", who, cudaGetErrorName(e), cudaGetErrorString(e));
}

// What the three calls that read pos have in common.
skg_status check_choices(const char *who, int T, int k, int R, int N, const void *pos)
{
    if (T < 0 || k < 1 || R < 0 || N < 1)
        return set_error(SKG_ERR_INVALID_ARG, "%s: T and R must be >= 0, k and N >= 1 (got T=%d, k=%d, R=%d, N=%d)", who, T,
                         k, R, N);
    if (static_cast<long long>(T) * k > 0x7FFFFFFFll || N > kMaxN)
        return set_error(SKG_ERR_UNSUPPORTED, "%s: more than 2^31 - 1 choices or rows longer than 2^30 (T=%d, k=%d, N=%d)",
                         who, T, k, N);
    if (T > 0 && !pos)
        return set_error(SKG_ERR_INVALID_ARG, "%s: pos must be non-NULL", who);
    return SKG_OK;
}

template <int V>
cudaError_t launch_gather(MoveParams &p, cudaStream_t s)
{
    p.groups = static_cast<int>((static_cast<long long>(p.N) + 32 * V * kDeep - 1) / (32 * V * kDeep));
    p.units = static_cast<long long>(p.rows) * p.groups;
    return launch(gather_kernel<V>, (p.units + kGatherWarps - 1) / kGatherWarps, 32 * kGatherWarps, 0, 1, s, p);
}

template <int V, int PC>
cudaError_t launch_combine_rows(MoveParams &p, cudaStream_t s)
{
    p.groups = static_cast<int>((static_cast<long long>(p.N) + 32 * V * PC - 1) / (32 * V * PC));
    p.units = static_cast<long long>(p.rows) * p.groups;
    return launch(combine_kernel<V, PC>, (p.units + kCombineWarps - 1) / kCombineWarps, 32 * kCombineWarps, 0, 1, s, p);
}

// Elements that every row allows to be moved together.
int width(const MoveParams &p)
{
    for (int v = 8; v > 1; v /= 2)
        if (p.N % v == 0 && p.ldx % v == 0 && aligned(p.x, 2 * v) && aligned(p.res, 2 * v) && aligned(p.out, 2 * v))
            return v;
    return 1;
}

} // namespace
} // namespace skg

using namespace skg;

extern "C" {

skg_status skg_experts_sort(int T, int k, int experts, const int *expert, int *offsets, int *rows, int *pos, void *stream)
{
    static const char who[] = "skg_experts_sort";
    if (T < 0 || k < 1 || experts < 1)
        return set_error(SKG_ERR_INVALID_ARG, "%s: T must be >= 0, k and experts >= 1 (got %d, %d, %d)", who, T, k, experts);
    if (experts > kF8MaxExperts || static_cast<long long>(T) * k > (1 << 24))
        return set_error(SKG_ERR_UNSUPPORTED, "%s: at most %d experts and 2^24 choices (got %d and %d x %d)", who,
                         kF8MaxExperts, experts, T, k);
    if (!offsets || (T > 0 && (!expert || !rows || !pos)))
        return set_error(SKG_ERR_INVALID_ARG, "%s: expert, offsets, rows and pos must be non-NULL", who);
    if (!aligned(expert, 4) || !aligned(offsets, 4) || !aligned(rows, 4) || !aligned(pos, 4))
        return set_error(SKG_ERR_ALIGNMENT, "%s: a tensor misses its element alignment", who);
    static int attr_set[kMaxDevices] = {};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess && dev >= kMaxDevices)
        e = cudaErrorInvalidDevice;
    if (e != cudaSuccess)
        return launched(e, who);
    if (__atomic_load_n(&attr_set[dev], __ATOMIC_ACQUIRE) == 0) {
        e = cudaFuncSetAttribute(sort_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 (kSortWarps + 2) * kF8MaxExperts * 4);
        if (e != cudaSuccess)
            return launched(e, who);
        __atomic_store_n(&attr_set[dev], 1, __ATOMIC_RELEASE);
    }
    SortParams p = {expert, offsets, rows, pos, T * k, k, experts, 0, 0, 0};
    p.ctas = p.n > 32 * kSortHeld * kSortWarps ? kSortCtas : 1;
    const int a_cta = (p.n + p.ctas - 1) / p.ctas, held = 32 * kSortHeld;
    p.warps = std::min(kSortWarps, std::max(1, (a_cta + held - 1) / held));
    p.run = (a_cta + 32 * p.warps - 1) / (32 * p.warps) * 32;
    const int threads = std::max(32 * p.warps, (experts + 63) / 64 * 32);   // two experts a thread at the most
    return launched(launch(sort_kernel, p.ctas, threads, static_cast<size_t>(p.warps + 2) * experts * 4, p.ctas,
                           static_cast<cudaStream_t>(stream), p), who);
}

skg_status skg_experts_gather(int R, int T, int N, const void *x, size_t ldx, const int *rows, void *out, void *stream)
{
    static const char who[] = "skg_experts_gather";
    if (R < 0 || T < 0 || N < 1)
        return set_error(SKG_ERR_INVALID_ARG, "%s: R and T must be >= 0, N >= 1 (got %d, %d, %d)", who, R, T, N);
    if (N > kMaxN)
        return set_error(SKG_ERR_UNSUPPORTED, "%s: rows longer than 2^30 (N=%d)", who, N);
    if (R > 0 && ((T > 0 && !x) || !rows || !out))
        return set_error(SKG_ERR_INVALID_ARG, "%s: x, rows and out must be non-NULL", who);
    if (ldx < static_cast<size_t>(N))
        return set_error(SKG_ERR_INVALID_ARG, "%s: row stride %zu of x is below N = %d", who, ldx, N);
    if (!aligned(x, 2) || !aligned(rows, 4) || !aligned(out, 2))
        return set_error(SKG_ERR_ALIGNMENT, "%s: a tensor misses its element alignment", who);
    if (R == 0)
        return SKG_OK;
    MoveParams p = {};
    p.x = static_cast<const uint16_t *>(x);
    p.index = rows;
    p.out = static_cast<uint16_t *>(out);
    p.ldx = ldx;
    p.rows = R;
    p.x_rows = T;
    p.N = N;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const int v = width(p);
    return launched(v == 8 ? launch_gather<8>(p, s) : v == 4 ? launch_gather<4>(p, s) : v == 2 ? launch_gather<2>(p, s)
                                                                                               : launch_gather<1>(p, s), who);
}

skg_status skg_experts_combine(int T, int k, int R, int N, const void *y, size_t ldy, const int *pos, const float *weight,
                               const void *residual, void *out, void *stream)
{
    static const char who[] = "skg_experts_combine";
    const skg_status st = check_choices(who, T, k, R, N, pos);
    if (st != SKG_OK)
        return st;
    if (T > 0 && ((R > 0 && !y) || !out))
        return set_error(SKG_ERR_INVALID_ARG, "%s: y and out must be non-NULL", who);
    if (ldy < static_cast<size_t>(N))
        return set_error(SKG_ERR_INVALID_ARG, "%s: row stride %zu of y is below N = %d", who, ldy, N);
    if (!aligned(y, 2) || !aligned(pos, 4) || !aligned(weight, 4) || !aligned(residual, 2) || !aligned(out, 2))
        return set_error(SKG_ERR_ALIGNMENT, "%s: a tensor misses its element alignment", who);
    if (T == 0)
        return SKG_OK;
    MoveParams p = {};
    p.x = static_cast<const uint16_t *>(y);
    p.res = static_cast<const uint16_t *>(residual);
    p.index = pos;
    p.weight = weight;
    p.out = static_cast<uint16_t *>(out);
    p.ldx = ldy;
    p.rows = T;
    p.x_rows = R;
    p.N = N;
    p.k = k;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const int v = width(p);
    return launched(v == 8   ? launch_combine_rows<8, 1>(p, s)
                    : v == 4 ? launch_combine_rows<4, 2>(p, s)
                    : v == 2 ? launch_combine_rows<2, 4>(p, s)
                             : launch_combine_rows<1, 4>(p, s), who);
}

skg_status skg_experts_combine_grad(int T, int k, int R, int N, const void *grad_out, const void *y, size_t ldy,
                                    const int *pos, const float *weight, void *grad_y, float *grad_weight, void *stream)
{
    static const char who[] = "skg_experts_combine_grad";
    const skg_status st = check_choices(who, T, k, R, N, pos);
    if (st != SKG_OK)
        return st;
    if (T > 0 && (!grad_out || (R > 0 && (!y || !grad_y)) || !weight || !grad_weight))
        return set_error(SKG_ERR_INVALID_ARG, "%s: grad_out, y, weight, grad_y and grad_weight must be non-NULL", who);
    if (ldy < static_cast<size_t>(N))
        return set_error(SKG_ERR_INVALID_ARG, "%s: row stride %zu of y is below N = %d", who, ldy, N);
    if (!aligned(grad_out, 2) || !aligned(y, 2) || !aligned(pos, 4) || !aligned(weight, 4) || !aligned(grad_y, 2) ||
        !aligned(grad_weight, 4))
        return set_error(SKG_ERR_ALIGNMENT, "%s: a tensor misses its element alignment", who);
    if (T == 0)
        return SKG_OK;
    MoveParams p = {};
    p.x = static_cast<const uint16_t *>(y);
    p.res = static_cast<const uint16_t *>(grad_out);
    p.index = pos;
    p.weight = weight;
    p.out = static_cast<uint16_t *>(grad_y);
    p.grad_weight = grad_weight;
    p.ldx = ldy;
    p.rows = T;
    p.x_rows = R;
    p.N = N;
    p.k = k;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const int v = width(p);
    return launched(v == 8   ? launch(combine_grad_kernel<8, 1>, T, kGradThreads, 0, 1, s, p)
                    : v == 4 ? launch(combine_grad_kernel<4, 1>, T, kGradThreads, 0, 1, s, p)
                    : v == 2 ? launch(combine_grad_kernel<2, 2>, T, kGradThreads, 0, 1, s, p)
                             : launch(combine_grad_kernel<1, 2>, T, kGradThreads, 0, 1, s, p), who);
}

} // extern "C"

// skg_f8_wide.cu -- the projection of e4m3 rows by e4m3 weights for many tokens,
// or many of each expert: tcgen05 by pairs of CTAs.
//
//   y[m, n] = sum_b xs[m, b] ws[n / 128, b] sum_(k in block b) x[m, k] W[n, k]
//
// The arithmetic is that of skg_f8_split.cu.  Two CTAs work as one
// (cta_group::2): 256 tokens x 256 channels, each CTA with its 128 rows of x (A),
// half of the rows of W (B) and the accumulator of its tokens, 128 lanes x 256
// columns.  A token a lane makes a unit's scale one number a thread: xs of its
// token times ws of the 128 channels that its warp has.  Two accumulators take
// all of the SM's tensor memory.
//
// What bounds it is the tensor core: a unit of 128 k is 512 cycles of an SM's
// MMAs, in which 8 warps take the 128 x 256 sums of the unit before into
// registers.
//
// Roles of a CTA (one per SM, pairs persistent over tiles):
//   1 + 1     TMA; TMEM and, in the first CTA of the pair, MMA issue for both
//   8 warps   accumulators into registers, and the tile's end: residual,
//             rounding, store, while the next tile's first two units are computed
//
// Every wait is bounded as in skg_f8_split.cu.
#include <algorithm>

#include "skg_f8_internal.h"
#include "skg_internal.h"
#include "skg_ptx.cuh"
#include "skg_q8_common.cuh"

namespace skg {
namespace {

#include "skg_f8_tc_common.cuh"

constexpr int kPair = 2;
constexpr int MT = 256, NT = 256;                    // tokens and channels of a pair's tile
constexpr uint64_t kLandNs = 10000000;               // 10 ms: far longer than any copy takes

struct WideShape {
    static constexpr int kEpiWarps = 8;
    static constexpr int kCols = NT * 4 / kEpiWarps;         // 128: one block of channels
    static_assert(kCols == kF8Block, "one scale of W a thread");
    static constexpr int kMmaWarp = 0, kTmaWarp = 1, kFirstEpi = 2;
    static constexpr int kThreads = 32 * (2 + kEpiWarps);
    static constexpr int kStages = 6;
    static constexpr int kAcc = 2;
    static constexpr uint32_t kTmemCols = 512;
    static constexpr uint32_t kStage = 2 * kF8TileBytes;     // a CTA's x and W of a unit
    static constexpr uint32_t kIdesc = idesc_e4m3_f32(MT, NT);
    static constexpr int kBars = 2 * kStages + 2 * kAcc + 1;
    static constexpr int kSmem = 1024 + kStages * kStage + kBars * 8 + 16;
    static_assert(kSmem + f8_table_bytes(kF8MaxExperts) <= 227 * 1024, "shared memory of a CTA");
};

// 16 outputs (channels n0 ...) of one token.
template <int EPI>
__device__ __forceinline__ void store_row(const F8LinearParams &p, int m, int n0, const float *v)
{
    const size_t o = static_cast<size_t>(m) * p.N + n0;
    if (p.vec4) {
#pragma unroll
        for (int c = 0; c < 16; c += 4) {
            if (n0 + c >= p.N)
                return;
            float4 s = make_float4(v[c], v[c + 1], v[c + 2], v[c + 3]);
            if (EPI == SKG_EPI_FP32) {
                *reinterpret_cast<float4 *>(static_cast<float *>(p.y) + o + c) = s;
                continue;
            }
            if (EPI == SKG_EPI_BF16_RESIDUAL) {
                const uint2 b = __ldcg(reinterpret_cast<const uint2 *>(p.res + o + c));
                s.x += bf16lo(b.x), s.y += bf16hi(b.x), s.z += bf16lo(b.y), s.w += bf16hi(b.y);
            }
            *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(p.y) + o + c) =
                make_uint2(f32_to_bf16(s.x) | static_cast<uint32_t>(f32_to_bf16(s.y)) << 16,
                           f32_to_bf16(s.z) | static_cast<uint32_t>(f32_to_bf16(s.w)) << 16);
        }
        return;
    }
#pragma unroll
    for (int c = 0; c < 16; ++c) {
        if (n0 + c >= p.N)
            return;
        float s = v[c];
        if (EPI == SKG_EPI_FP32) {
            static_cast<float *>(p.y)[o + c] = s;
            continue;
        }
        if (EPI == SKG_EPI_BF16_RESIDUAL)
            s += bf16_to_f32(__ldcg(p.res + o + c));
        static_cast<uint16_t *>(p.y)[o + c] = f32_to_bf16(s);
    }
}

__global__ void __launch_bounds__(WideShape::kThreads, 1)
f8_wide_kernel(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmX, const F8LinearParams p)
{
    using Sh = WideShape;
    constexpr int S = Sh::kStages, NA = Sh::kAcc, NC = Sh::kCols;

    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    uint8_t *sX = smem, *sW = smem + S * kF8TileBytes;
    uint64_t *full = reinterpret_cast<uint64_t *>(smem + S * Sh::kStage);
    uint64_t *empty = full + S;
    uint64_t *afull = empty + S;         // [NA] accumulators
    uint64_t *aempty = afull + NA;       // [NA]
    uint64_t *drain = aempty + NA;       // [1]
    // full and aempty are those of the first CTA, with bytes and arrivals of both;
    // the MMA's commits arrive at both CTAs' empty and afull
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(drain + 1);
    volatile int *flags = reinterpret_cast<volatile int *>(tmem_slot + 1);   // [0] abort
    F8Table table;
    table.row0 = reinterpret_cast<int *>(tmem_slot + 4);
    table.tile0 = table.row0 + p.experts + 1;

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = static_cast<int>(blockIdx.x) % kPair, first = static_cast<int>(blockIdx.x) / kPair;
    const int step = static_cast<int>(gridDim.x) / kPair;
    const int units = p.nkb;

    if (threadIdx.x == 0) {
        tma_prefetch_desc(&tmW);
        tma_prefetch_desc(&tmX);
        for (int i = 0; i < S; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], 1);
        }
        for (int i = 0; i < NA; ++i) {
            mbar_init(&afull[i], 1);
            mbar_init(&aempty[i], kPair * Sh::kEpiWarps);
        }
        mbar_init(drain, 1);
        flags[0] = 0;
        fence_mbar_init();
    }
    if (p.experts) {
        pdl_wait();
        if (warp == Sh::kFirstEpi)
            f8_build_table(p, MT, table);
    }
    __syncthreads();
    const int tiles = f8_tiles(p, table);
    if (first >= tiles)                  // both CTAs of the pair
        return;
    if (warp == Sh::kMmaWarp) {
        tmem_alloc_pair(tmem_slot, Sh::kTmemCols);
        tmem_relinquish_pair();
    }
    tc_fence_before();
    cluster_sync();                      // the peer's barriers exist before anything is sent there
    tc_fence_after();
    constexpr uint32_t tmem_base = 0;    // all 512 columns are this CTA's
    if (warp != Sh::kTmaWarp)            // the bounded waits do not count the previous kernel's time
        pdl_wait();

    if (warp == Sh::kTmaWarp) {
        // -------------------------------------------------------- TMA producer
        const bool leader = elect_one();
        const uint64_t pol = policy_evict_normal();
        const uint32_t full0 = map_shared_rank(smem_u32(full), 0);
        auto load_w = [&](int u, const F8Tile &t, int kb) {
            if (rank == 0)               // for both CTAs' copies, which may be counted before
                mbar_arrive_expect_tx(&full[u % S], kPair * Sh::kStage);
            tma_load_2d_pair(sW + u % S * kF8TileBytes, &tmW, full0 + u % S * 8, kb * kF8Block,
                             t.e * p.N + t.nt * NT + rank * (NT / kPair), pol);
        };
        auto load_x = [&](int u, const F8Tile &t, int kb) {
            tma_load_2d_pair(sX + u % S * kF8TileBytes, &tmX, full0 + u % S * 8, kb * kF8Block, t.m0 + rank * (MT / kPair), pol);
        };
        F8Tile t = f8_tile(p, MT, table, first);
        const int ahead = p.static_w && !p.experts ? min(S, units) : 0;
        if (leader)
            for (int u = 0; u < ahead; ++u)
                load_w(u, t, u);
        pdl_wait();
        if (leader)
            for (int u = 0; u < ahead; ++u)
                load_x(u, t, u);
        bool ok = true;
        int j = 0;
        for (int tile = first; ok && tile < tiles; tile += step) {
            if (tile != first)
                t = f8_tile(p, MT, table, tile);
            for (int kb = 0; kb < units; ++kb, ++j) {
                if (j < ahead)
                    continue;
                ok = __all_sync(0xFFFFFFFFu, mbar_wait_cluster(&empty[j % S], ((j / S) & 1) ^ 1, p.timeout_ns, &flags[0]));
                if (!ok)
                    break;
                if (leader) {
                    load_w(j, t, kb);
                    load_x(j, t, kb);
                }
                __syncwarp();
            }
        }
        if (!ok)
            f8_fail(p.err, &flags[0], kErrTimeoutProducer);
        if (flags[0]) {                  // abort: let every copy land before exit, a few microseconds after its issue
            const uint64_t t0 = globaltimer_ns();    // (the second CTA's are counted in the first)
            while (globaltimer_ns() - t0 < kLandNs) {
            }
        }
    } else if (warp == Sh::kMmaWarp) {
        // ---------------------------------------------------------- MMA issuer
        if (rank == 0) {
            const bool leader = elect_one();
            const uint64_t w0 = smem_desc_kmajor_sw128(smem_u32(sW)), x0 = smem_desc_kmajor_sw128(smem_u32(sX));
            const int total = ((tiles - first + step - 1) / step) * units;
            bool ok = true;
            int sl = 0, phase = 0;
            for (int j = 0; j < total; ++j) {
                const int t = j % NA;
                ok = mbar_wait_cluster(&aempty[t], ((j / NA) & 1) ^ 1, p.timeout_ns, &flags[0]) &&
                     mbar_wait_cluster(&full[sl], phase, p.timeout_ns, &flags[0]);
                ok = __all_sync(0xFFFFFFFFu, ok);
                if (!ok)
                    break;
                tc_fence_after();
                if (leader) {
                    const uint64_t a = x0 + static_cast<uint64_t>(sl * (kF8TileBytes / 16));
                    const uint64_t b = w0 + static_cast<uint64_t>(sl * (kF8TileBytes / 16));
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk)
                        tc_mma_f8_pair(tmem_base + t * NT, a + 2 * kk, b + 2 * kk, Sh::kIdesc, kk > 0);
                    // nobody waits for the last units' slots, and the peer's producer may be gone by then
                    if (j + S < total)
                        tc_commit_pair_multicast(&empty[sl], 3);
                    tc_commit_pair_multicast(&afull[t], 3);
                }
                __syncwarp();
                if (++sl == S) {
                    sl = 0;
                    phase ^= 1;
                }
            }
            if (!ok) {                   // abort: wait for the MMAs already issued before TMEM is freed
                f8_fail(p.err, &flags[0], kErrTimeoutMma);
                if (leader)
                    tc_commit_pair(drain);
                volatile int never = 0;
                mbar_wait(drain, 0, kDefaultTimeoutNs, &never);
            }
        }
    } else {
        // ------------------------------------------------------------ epilogue
        pdl_launch_dependents();         // not sooner: see skg_q8_stream.cu
        const int ew = warp - Sh::kFirstEpi;
        const int row = rank * (MT / kPair) + (warp & 3) * 32 + lane, col0 = (ew >> 2) * NC;
        const uint32_t lane_base = tmem_base + (static_cast<uint32_t>((warp & 3) * 32) << 16) + static_cast<uint32_t>(col0);
        const uint32_t aempty0 = map_shared_rank(smem_u32(aempty), 0);
        constexpr int AHEAD = 4;
        bool ok = true;
        int j = 0;
        for (int tile = first; ok && tile < tiles; tile += step) {
            const F8Tile t = f8_tile(p, MT, table, tile);
            const int m = t.m0 + row, nb = t.nt * (NT / kF8Block) + (ew >> 2);
            const bool live = m < t.m1 && nb < p.nb;
            const float *ws = p.w_scale + (static_cast<size_t>(t.e) * p.nb + nb) * p.nkb;
            const float *xs = p.x_scale + static_cast<size_t>(m) * p.nkb;
            float w[AHEAD], x[AHEAD];
#pragma unroll
            for (int i = 0; i < AHEAD; ++i) {
                w[i] = live && i < units ? __ldcg(ws + i) : 0.0f;
                x[i] = live && i < units ? __ldca(xs + i) : 0.0f;
            }
            float acc[NC];
#pragma unroll
            for (int c = 0; c < NC; ++c)
                acc[c] = 0.0f;
            for (int kb = 0; ok && kb < units; kb += AHEAD) {
#pragma unroll
                for (int i = 0; i < AHEAD; ++i) {
                    if (kb + i >= units)
                        break;
                    const float s = x[i] * w[i];
                    const bool more = live && kb + i + AHEAD < units;
                    w[i] = more ? __ldcg(ws + kb + i + AHEAD) : 0.0f;
                    x[i] = more ? __ldca(xs + kb + i + AHEAD) : 0.0f;
                    const int a = j % NA;
                    ok = __all_sync(0xFFFFFFFFu, mbar_wait_cluster(&afull[a], (j / NA) & 1, p.timeout_ns, &flags[0]));
                    if (!ok)
                        break;
                    tc_fence_after();
#pragma unroll
                    for (int c0 = 0; c0 < NC; c0 += 32) {
                        uint32_t r[2][16];
                        tmem_ld_x16(lane_base + static_cast<uint32_t>(a * NT + c0), r[0]);
                        tmem_ld_x16(lane_base + static_cast<uint32_t>(a * NT + c0 + 16), r[1]);
                        tmem_wait_ld();
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            f8_taken(r[h]);
#pragma unroll
                            for (int c = 0; c < 16; ++c)
                                acc[c0 + 16 * h + c] = fmaf(__uint_as_float(r[h][c]), s, acc[c0 + 16 * h + c]);
                        }
                    }
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0)
                        mbar_arrive_cluster(aempty0 + a * 8);
                    ++j;
                }
            }
            if (!ok)
                break;
            if (live) {
                const int n0 = t.nt * NT + col0;
#pragma unroll
                for (int c = 0; c < NC; c += 16) {
                    if (p.epilogue == SKG_EPI_FP32)
                        store_row<SKG_EPI_FP32>(p, m, n0 + c, acc + c);
                    else if (p.epilogue == SKG_EPI_BF16_RESIDUAL)
                        store_row<SKG_EPI_BF16_RESIDUAL>(p, m, n0 + c, acc + c);
                    else
                        store_row<SKG_EPI_BF16>(p, m, n0 + c, acc + c);
                }
            }
        }
        if (!ok)
            f8_fail(p.err, &flags[0], kErrTimeoutEpilogue);
    }

    __syncwarp();
    tc_fence_before();
    cluster_sync();                      // no CTA leaves while its peer may still send to it
    if (warp == Sh::kMmaWarp) {
        tc_fence_after();
        tmem_dealloc_pair(tmem_base, Sh::kTmemCols);
    }
}

} // namespace

F8TcShape f8_wide_shape(int experts)
{
    return {MT, 1, WideShape::kSmem + f8_table_bytes(experts), WideShape::kThreads, WideShape::kStages};
}

cudaError_t launch_f8_wide(const CUtensorMap &tmW, const CUtensorMap &tmX, const F8LinearParams &p, int grid, cudaStream_t s)
{
    static int attr_set[kMaxDevices] = {};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess)
        return e;
    if (dev >= kMaxDevices)
        return cudaErrorInvalidDevice;
    if (__atomic_load_n(&attr_set[dev], __ATOMIC_ACQUIRE) == 0) {
        e = cudaFuncSetAttribute(f8_wide_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 WideShape::kSmem + f8_table_bytes(kF8MaxExperts));
        if (e != cudaSuccess)
            return e;
        __atomic_store_n(&attr_set[dev], 1, __ATOMIC_RELEASE);
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(grid));
    cfg.blockDim = dim3(WideShape::kThreads);
    cfg.dynamicSmemBytes = WideShape::kSmem + f8_table_bytes(p.experts);
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = kPair;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, f8_wide_kernel, tmW, tmX, p);
}

} // namespace skg

// skg_f8_split.cu -- the projection of e4m3 rows by e4m3 weights for few tokens,
// or few tokens of each expert: tcgen05, with K split over the CTAs of a cluster.
//
//   y[m, n] = sum_b xs[m, b] ws[n / 128, b] sum_(k in block b) x[m, k] W[n, k]
//
// The sum over a block of 128 k is the MMA's (kind::f8f6f4, fp32), from a fresh
// accumulator; the sum over blocks is in fp32 registers, each block scaled by
// xs ws in fp32 as it is added.
//
// What bounds it is W's way from HBM.  Tile: 128 rows of W are the MMA's M (the
// scale of a weight block is then one number), MT tokens its N.  A cluster of S
// CTAs computes a tile, CTA r the r-th part of K; with S = 1 CTAs are persistent
// over tiles.  Two CTAs an SM, with 160 KB of W on its way (128 KB at 64 tokens).  Roles of a CTA:
//   1 + 1     TMA; TMEM and MMA issue
//   4         accumulators into registers, and the tile's end: residual,
//             rounding, store
// With S > 1 the cluster's CTAs leave their sums in their own shared memory and
// each adds up and stores 1/S of the tile's tokens, read from its peers in order
// of their ranks.  No workspace, no counters: runs may overlap as they like.
//
// Measured, weights from HBM (copy peak 6.71 TB/s): 1 x 12288 x 7168 15.5 us (5.7 TB/s
// of weights), 16 x 7168 x 16384 21.4, 64 x 7168 x 16384 23.7 (5.0), 64 x 7168 x 7168
// 13.4; 128 rows of 384 experts, 2048 x 4096, 108 to 123 us (6.2 to 7.1 TB/s); one
// token's 8 experts of 384, 2048 x 4096, 13.9 us, of 64, 1024 x 1024, 5.9 us.  A
// launch's ends take 3 to 5 us (with experts the offsets are read first); between
// them W comes at 6.3 TB/s.  Unsplit, 64 x 7168 x 7168 takes 21 us; 128 tokens a tile, in
// which an epilogue warp needs a scale a column from shared memory, took 1024 x 7168
// x 7168 212 us, where the wide kernel's tiles of 128 take 62.
//
// Every wait is bounded; on expiry a thread records the timeout in the plan's error
// word and raises the CTA's abort flag, and the issuer waits for its MMAs.  The CTA
// goes on to the cluster's barriers; behind them, every role having ended, the producer
// waits for its copies in flight, and the CTA frees its TMEM and returns.
#include <algorithm>

#include "skg_f8_internal.h"
#include "skg_internal.h"
#include "skg_ptx.cuh"
#include "skg_q8_common.cuh"

namespace skg {
namespace {

#include "skg_f8_tc_common.cuh"

template <int MT>
struct SplitShape {
    static constexpr int kEpiWarps = 4;
    static constexpr int kCols = MT * 4 / kEpiWarps;         // accumulator columns of an epilogue thread
    static constexpr int kMmaWarp = 0, kTmaWarp = 1, kFirstEpi = 2;
    static constexpr int kThreads = 32 * (2 + kEpiWarps);
    static constexpr int kStages = MT <= 32 ? 5 : 4;
    static constexpr int kAcc = 4;                           // accumulators in flight
    static constexpr uint32_t kTmemCols = kAcc * MT;
    static_assert(kTmemCols <= 256, "two CTAs share the SM's tensor memory");
    static constexpr uint32_t kXBytes = MT * kF8Block;
    static constexpr uint32_t kStage = kF8TileBytes + kXBytes;
    static_assert(kStages * kStage >= MT * kTileN * 4 && kCols == MT, "the sums take the ring's place");
    static constexpr uint32_t kIdesc = idesc_e4m3_f32(kTileN, MT);
    static constexpr int kBars = 2 * kStages + 2 * kAcc + 1;
    static constexpr int kScales = kEpiWarps * 2 * kCols * 4;        // a unit's scales, by warp, twice
    static constexpr int kSmem = 1024 + kStages * kStage + kScales + kBars * 8 + 16;
    static_assert(2 * (kSmem + f8_table_bytes(kF8MaxExperts) + 1024) <= 228 * 1024, "two CTAs an SM");
};

// The outputs of one channel n from its sums of the tokens from m0 on: those of
// columns lo to hi.
template <int EPI, int NC>
__device__ __forceinline__ void store_columns(const F8LinearParams &p, int m0, int n, int lo, int hi, const float (&acc)[NC])
{
    size_t at = static_cast<size_t>(m0) * p.N + n;
#pragma unroll
    for (int c0 = 0; c0 < NC; c0 += 8, at += static_cast<size_t>(8) * p.N) {
        if (c0 >= hi)
            return;
        uint16_t b[8];
        if (EPI == SKG_EPI_BF16_RESIDUAL) {
            const uint16_t *r = p.res + at;
#pragma unroll
            for (int c = 0; c < 8; ++c, r += p.N)
                b[c] = c0 + c >= lo && c0 + c < hi ? __ldcg(r) : 0;
        }
        size_t o = at;
#pragma unroll
        for (int c = 0; c < 8; ++c, o += p.N) {
            const float v = EPI == SKG_EPI_BF16_RESIDUAL ? acc[c0 + c] + bf16_to_f32(b[c]) : acc[c0 + c];
            if (c0 + c >= lo && c0 + c < hi) {
                if (EPI == SKG_EPI_FP32)
                    static_cast<float *>(p.y)[o] = v;
                else
                    static_cast<uint16_t *>(p.y)[o] = f32_to_bf16(v);
            }
        }
    }
}

template <int MT>
__global__ void __launch_bounds__(SplitShape<MT>::kThreads, 2)
f8_split_kernel(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmX, const F8LinearParams p)
{
    using Sh = SplitShape<MT>;
    constexpr int S = Sh::kStages, NA = Sh::kAcc, NC = Sh::kCols;

    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    uint8_t *sW = smem, *sX = smem + S * kF8TileBytes;
    float *scales = reinterpret_cast<float *>(smem + S * Sh::kStage);
    uint64_t *full = reinterpret_cast<uint64_t *>(smem + S * Sh::kStage + Sh::kScales);
    uint64_t *empty = full + S;
    uint64_t *afull = empty + S;         // [NA] accumulators
    uint64_t *aempty = afull + NA;       // [NA]
    uint64_t *drain = aempty + NA;       // [1]
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(drain + 1);
    volatile int *flags = reinterpret_cast<volatile int *>(tmem_slot + 1);   // [0] abort
    F8Table table;
    table.row0 = reinterpret_cast<int *>(tmem_slot + 4);
    table.tile0 = table.row0 + p.experts + 1;

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = static_cast<int>(blockIdx.x) % p.split, first = static_cast<int>(blockIdx.x) / p.split;
    const int step = static_cast<int>(gridDim.x) / p.split;
    const int kb0 = rank * p.nkb / p.split, units = (rank + 1) * p.nkb / p.split - kb0;

    if (threadIdx.x == 0) {
        tma_prefetch_desc(&tmW);
        tma_prefetch_desc(&tmX);
        for (int i = 0; i < S; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], 1);
        }
        for (int i = 0; i < NA; ++i) {
            mbar_init(&afull[i], 1);
            mbar_init(&aempty[i], Sh::kEpiWarps);
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
    if (first >= tiles)                  // all of the cluster's CTAs
        return;
    uint32_t tmem_base = 0;
    if (warp != Sh::kTmaWarp) {          // the TMA warp needs no TMEM: its first copies leave at once
        if (warp == Sh::kMmaWarp) {
            tmem_alloc(tmem_slot, Sh::kTmemCols);
            tmem_relinquish();
        }
        tc_fence_before();
        asm volatile("bar.sync 2, %0;" :: "n"(Sh::kThreads - 32) : "memory");
        tc_fence_after();
        tmem_base = __shfl_sync(0xFFFFFFFFu, *tmem_slot, 0);
        // Without x there is nothing to do before the previous kernel's end, and the
        // bounded waits do not count its time.
        pdl_wait();
    }

    int issued = 0;                      // units whose copies this thread has issued
    if (warp == Sh::kTmaWarp) {
        // -------------------------------------------------------- TMA producer
        if (lane == 0) {
            // W passes once where one token tile holds all of M
            const uint64_t pol_w = !p.experts && p.m_tiles == 1 ? policy_evict_first() : policy_evict_normal();
            const uint64_t pol_x = policy_evict_last();
            int j = 0;
            auto load_w = [&](int u, const F8Tile &t, int kb) {
                mbar_arrive_expect_tx(&full[u % S], (p.w_box + p.x_box) * kF8Block);
                tma_load_2d(sW + u % S * kF8TileBytes, &tmW, &full[u % S], (kb0 + kb) * kF8Block,
                            f8_w_window(p, t.e, t.nt * kTileN), pol_w);
            };
            auto load_x = [&](int u, const F8Tile &t, int kb) {
                tma_load_2d(sX + u % S * Sh::kXBytes, &tmX, &full[u % S], (kb0 + kb) * kF8Block, f8_x_window(p, t.m0), pol_x);
            };
            F8Tile t = f8_tile(p, MT, table, first);
            // weights may be requested before the wait for the previous kernel
            const int ahead = p.static_w && !p.experts ? min(S, units) : 0;
            for (int u = 0; u < ahead; ++u)
                load_w(u, t, u);
            pdl_wait();
            for (int u = 0; u < ahead; ++u)
                load_x(u, t, u);
            bool ok = true;
            for (int tile = first; ok && tile < tiles; tile += step) {
                if (tile != first)
                    t = f8_tile(p, MT, table, tile);
                for (int kb = 0; kb < units; ++kb, ++j) {
                    if (j < ahead)
                        continue;
                    ok = mbar_wait(&empty[j % S], ((j / S) & 1) ^ 1, p.timeout_ns, &flags[0]);
                    if (!ok)
                        break;
                    load_w(j, t, kb);
                    load_x(j, t, kb);
                }
            }
            if (!ok)
                f8_fail(p.err, &flags[0], kErrTimeoutProducer);
            issued = max(j, ahead);
        }
    } else if (warp == Sh::kMmaWarp) {
        // ---------------------------------------------------------- MMA issuer
        const bool leader = elect_one();
        const uint64_t w0 = smem_desc_kmajor_sw128(smem_u32(sW)), x0 = smem_desc_kmajor_sw128(smem_u32(sX));
        const int total = ((tiles - first + step - 1) / step) * units;
        bool ok = true;
        for (int j = 0; j < total; ++j) {
            const int sl = j % S, t = j % NA;
            ok = mbar_wait(&aempty[t], ((j / NA) & 1) ^ 1, p.timeout_ns, &flags[0]) &&
                 mbar_wait(&full[sl], (j / S) & 1, p.timeout_ns, &flags[0]);
            ok = __all_sync(0xFFFFFFFFu, ok);
            if (!ok)
                break;
            tc_fence_after();
            if (leader) {
                const uint64_t a = w0 + static_cast<uint64_t>(sl * (kF8TileBytes / 16));
                const uint64_t b = x0 + static_cast<uint64_t>(sl * (Sh::kXBytes / 16));
#pragma unroll
                for (int kk = 0; kk < 4; ++kk)
                    tc_mma_f8(tmem_base + t * MT, a + 2 * kk, b + 2 * kk, Sh::kIdesc, kk > 0);
                tc_commit(&empty[sl]);
                tc_commit(&afull[t]);
            }
            __syncwarp();
        }
        if (!ok) {                       // abort: wait for the MMAs already issued before TMEM is freed
            f8_fail(p.err, &flags[0], kErrTimeoutMma);
            if (leader)
                tc_commit(drain);
            volatile int never = 0;
            mbar_wait(drain, 0, kDefaultTimeoutNs, &never);
        }
    } else {
        // ------------------------------------------------------------ epilogue
        // Not sooner (see skg_q8_stream.cu), and after this CTA's TMEM is allocated.
        pdl_launch_dependents();
        const int ew = warp - Sh::kFirstEpi;
        const int row = (warp & 3) * 32 + lane;
        const uint32_t lane_base = tmem_base + (static_cast<uint32_t>((warp & 3) * 32) << 16);
        float *mine = scales + ew * 2 * NC;
        constexpr int CP = (NC + 31) / 32;               // tokens whose scales a lane fetches
        constexpr int AHEAD = 4;                         // units whose scales are on their way
        constexpr int H = NC >= 32 ? 2 : 1;              // 16 columns read at a time, or 32
        bool ok = true;
        int j = 0;
        float w[AHEAD], x[AHEAD][CP];
        const float *ws, *xs;
        F8Tile t;
        int m0, lo, hi;                  // tokens m0 + lo to m0 + hi of the window are the tile's
        auto fetch = [&](int kb, float &wv, float (&xv)[CP]) {
            wv = kb < units ? __ldcg(ws + kb) : 0.0f;
#pragma unroll
            for (int c = 0; c < CP; ++c)
                xv[c] = kb < units && lane + 32 * c >= lo && lane + 32 * c < hi ? __ldca(xs + static_cast<size_t>(32 * c) * p.nkb + kb) : 0.0f;
        };
        // A tile's scales, from its first units' on: of the next tile they are on their
        // way while the outputs of this one are stored.
        auto begin = [&](int tile) {
            t = f8_tile(p, MT, table, tile);
            m0 = f8_x_window(p, t.m0);
            lo = t.m0 - m0;
            hi = min(t.m1, t.m0 + MT) - m0;
            ws = p.w_scale + (static_cast<size_t>(t.e) * p.nb + t.nt) * p.nkb + kb0;
            xs = p.x_scale + static_cast<size_t>(m0 + lane) * p.nkb + kb0;
#pragma unroll
            for (int i = 0; i < AHEAD; ++i)
                fetch(i, w[i], x[i]);
        };
        begin(first);
        for (int tile = first; ok && tile < tiles; tile += step) {
            float acc[NC];
#pragma unroll
            for (int c = 0; c < NC; ++c)
                acc[c] = 0.0f;
            for (int kb = 0; ok && kb < units; kb += AHEAD) {
#pragma unroll
                for (int i = 0; i < AHEAD; ++i) {
                    if (kb + i >= units)
                        break;
                    float *sc = mine + (j & 1) * NC;
#pragma unroll
                    for (int c = 0; c < CP; ++c)
                        if (NC >= 32 || lane < NC)
                            sc[lane + 32 * c] = x[i][c] * w[i];
                    __syncwarp();
                    fetch(kb + i + AHEAD, w[i], x[i]);
                    const int a = j % NA;
                    ok = __all_sync(0xFFFFFFFFu, mbar_wait(&afull[a], (j / NA) & 1, p.timeout_ns, &flags[0]));
                    if (!ok)
                        break;
                    tc_fence_after();
#pragma unroll
                    for (int c0 = 0; c0 < NC; c0 += 16 * H) {
                        uint32_t r[H][16];
#pragma unroll
                        for (int h = 0; h < H; ++h)
                            tmem_ld_x16(lane_base + static_cast<uint32_t>(a * MT + c0 + 16 * h), r[h]);
                        tmem_wait_ld();
#pragma unroll
                        for (int h = 0; h < H; ++h) {
                            f8_taken(r[h]);
#pragma unroll
                            for (int c = 0; c < 16; c += 4) {
                                const int at = c0 + 16 * h + c;
                                const float4 s = *reinterpret_cast<const float4 *>(sc + at);
                                acc[at] = fmaf(__uint_as_float(r[h][c]), s.x, acc[at]);
                                acc[at + 1] = fmaf(__uint_as_float(r[h][c + 1]), s.y, acc[at + 1]);
                                acc[at + 2] = fmaf(__uint_as_float(r[h][c + 2]), s.z, acc[at + 2]);
                                acc[at + 3] = fmaf(__uint_as_float(r[h][c + 3]), s.w, acc[at + 3]);
                            }
                        }
                    }
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0)
                        mbar_arrive(&aempty[a]);
                    ++j;
                }
            }
            if (!ok)
                break;
            if (p.split == 1) {
                const int n = f8_w_window(p, t.e, t.nt * kTileN) - t.e * p.N + row, from = m0, first_c = lo;
                const int end_c = n >= t.nt * kTileN && n < p.N ? hi : 0;
                if (tile + step < tiles)
                    begin(tile + step);
                if (p.epilogue == SKG_EPI_FP32)
                    store_columns<SKG_EPI_FP32>(p, from, n, first_c, end_c, acc);
                else if (p.epilogue == SKG_EPI_BF16_RESIDUAL)
                    store_columns<SKG_EPI_BF16_RESIDUAL>(p, from, n, first_c, end_c, acc);
                else
                    store_columns<SKG_EPI_BF16>(p, from, n, first_c, end_c, acc);
                __syncwarp();
            } else {
                // in the ring's place: the last MMA has read its operands
#pragma unroll
                for (int c = 0; c < NC; ++c)
                    *reinterpret_cast<float *>(smem + f8_sum_at(kTileN, c, row)) = acc[c];
            }
        }
        if (!ok)
            f8_fail(p.err, &flags[0], kErrTimeoutEpilogue);
    }

    __syncwarp();
    tc_fence_before();
    if (p.split > 1) {
        const F8Tile t = f8_tile(p, MT, table, first);
        const int n0[1] = {f8_w_window(p, t.e, t.nt * kTileN) - t.e * p.N}, na[1] = {t.nt * kTileN};
        f8_join<kF8SplitMax, Sh::kThreads, 1>(p, smem_u32(smem), f8_x_window(p, t.m0), t.m0, min(t.m1, t.m0 + MT), n0, na, rank, 0, 1);
    } else {
        __syncthreads();
    }
    // Abort: every copy lands before the CTA exits.  (Looked at here, where no role raises the
    // flag any more; what a join has read meanwhile is of a launch that is reported.)
    if (issued && flags[0]) {
        volatile int never = 0;
        for (int u = max(0, issued - S); u < issued; ++u)
            mbar_wait(&full[u % S], (u / S) & 1, kDefaultTimeoutNs, &never);
    }
    if (warp == Sh::kMmaWarp) {
        tc_fence_after();
        tmem_dealloc(tmem_base, Sh::kTmemCols);
    }
}

template <int MT>
cudaError_t launch_shape(const CUtensorMap &tmW, const CUtensorMap &tmX, const F8LinearParams &p, int grid, cudaStream_t s)
{
    using Sh = SplitShape<MT>;
    static int attr_set[kMaxDevices] = {};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess)
        return e;
    if (dev >= kMaxDevices)
        return cudaErrorInvalidDevice;
    if (__atomic_load_n(&attr_set[dev], __ATOMIC_ACQUIRE) == 0) {
        e = cudaFuncSetAttribute(f8_split_kernel<MT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 Sh::kSmem + f8_table_bytes(kF8MaxExperts));
        if (e == cudaSuccess)
            e = cudaFuncSetAttribute(f8_split_kernel<MT>, cudaFuncAttributePreferredSharedMemoryCarveout,
                                     cudaSharedmemCarveoutMaxShared);
        if (e != cudaSuccess)
            return e;
        __atomic_store_n(&attr_set[dev], 1, __ATOMIC_RELEASE);
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(grid));
    cfg.blockDim = dim3(Sh::kThreads);
    cfg.dynamicSmemBytes = Sh::kSmem + f8_table_bytes(p.experts);
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = static_cast<unsigned>(p.split);
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = p.split > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, f8_split_kernel<MT>, tmW, tmX, p);
}

template <int MT>
F8TcShape shape_of(int experts)
{
    return {MT, 2, SplitShape<MT>::kSmem + f8_table_bytes(experts), SplitShape<MT>::kThreads, SplitShape<MT>::kStages};
}

} // namespace

F8TcShape f8_split_shape(int m_tile, int experts)
{
    return m_tile == 16 ? shape_of<16>(experts) : m_tile == 32 ? shape_of<32>(experts)
                                                                        : shape_of<64>(experts);
}

cudaError_t launch_f8_split(const CUtensorMap &tmW, const CUtensorMap &tmX, const F8LinearParams &p, int m_tile, int grid,
                            cudaStream_t s)
{
    return m_tile == 16   ? launch_shape<16>(tmW, tmX, p, grid, s)
           : m_tile == 32 ? launch_shape<32>(tmW, tmX, p, grid, s)
                          : launch_shape<64>(tmW, tmX, p, grid, s);
}

} // namespace skg

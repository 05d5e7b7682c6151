// skg_q8_split.cu -- the 8-bit projection for a decode batch: tcgen05, with K
// split over the CTAs of a cluster.
//
// sm_103a has no integer kind of tcgen05.mma, and 8-bit integers are exact in
// fp16, as are their products (at most 2^14) and, in fp32, sums of up to 1024
// such products (at most 2^24).  So the integers are widened to fp16 on chip,
// multiplied with kind::f16 from a fresh accumulator every 1024 k, and the
// accumulators are added as int32: the exact integer sum, for any split of K.
//
// Tile (swap-AB): 128 rows of W are the MMA's M, MT tokens its N.  A cluster of
// S CTAs computes one tile; CTA r takes the r-th part of K in units of 128.
// Two CTAs an SM hold 2 x 3 units (MT = 64) in flight.  Roles of a CTA:
//   8 warps   widen W, two sets of 4 on alternate units: a thread reads its W
//             row's 128 bytes from the TMA ring and writes them as fp16 to its
//             TMEM lane (the MMA's A operand)
//   4 or 8    widen x into shared memory (the B operand), two sets as well; every
//             2048 k and at the end, epilogue: accumulators to integers
//   1 + 1     TMA; TMEM and MMA issue
// Sets of warps on alternate units rather than all on each: what a unit costs a
// warp besides the widening (two waits, fences, two arrivals) is as much again
// as half of it, and all 8 on every unit took 31.2 us at 64 x 7168 x 16384.
// The cluster's CTAs then leave their sums in their own shared memory and each
// adds up and stores 1/S of the tile's tokens, read from its peers.  Through
// global memory instead (partial sums, an arrival counter, the last CTA adds
// up) the same step took 6 us at M = 32 and 10 at M = 64: each round trip waits
// 1 to 1.7 us behind the next launch's weights.
//
// Measured, back to back with weights from HBM (6.70 TB/s copy peak): 32 x 7168 x
// 7168 12.7 us (4.1 TB/s), 64 x 7168 x 7168 15.3 us (3.4), 64 x 7168 x 16384 29.0
// us (4.1), 64 x 384 x 7168 6.5 us.  What bounds the deep one: 4.8 us are the
// launch's ends and the join; then a unit takes the SM's two CTAs 0.93 us.
// Without any widening it takes 0.92 with W from HBM, and 0.76 with widening but
// W from the L2, 0.58 with neither (the MMAs: at N = 64 they run at half rate), so
// the memory's latency and the widening bound it together.  A fourth stage for W,
// units requested in pairs, or another start in K for each tile changed nothing
// (28.8, 29.3, 28.2 us).
//
// Every wait is bounded; on expiry a thread records the timeout in the plan's error
// word and raises the CTA's abort flag, and the issuer waits for its MMAs.  The CTA
// goes on to the cluster's barriers; behind them, every role having ended, the producer
// waits for its copies in flight, and the CTA frees its TMEM and returns.
#include <algorithm>

#include "skg_internal.h"
#include "skg_ptx.cuh"
#include "skg_q8_common.cuh"
#include "skg_q8_internal.h"

namespace skg {
namespace {

#include "skg_q8_tc_common.cuh"

template <int MT>
struct SplitShape {
    static constexpr int kEpiWarps = MT / 8;
    static constexpr int kXWarps = kEpiWarps / 2;            // a set that widens x: two, on alternate units
    static constexpr int kCols = MT * 4 / kEpiWarps;         // accumulator columns of an epilogue thread: 32
    static constexpr int kThreads = 32 * (kWidenWarps + kEpiWarps + 2);
    // The MMA warp first: the oldest warp of a scheduler goes before the others
    static constexpr int kMmaWarp = 0, kTmaWarp = 1, kFirstWiden = 2, kFirstEpi = kFirstWiden + kWidenWarps;
    static constexpr int kStages = MT == 32 ? 4 : 3;         // ring of W and int8 x
    static constexpr int kOps = MT == 32 ? 3 : 2;            // widened operand buffers
    static_assert(kStages >= kOps && kOps >= kWidenSets, "the widen warps' waits need this");
    static constexpr uint32_t kRawX = MT * kQ8BlockK;
    static constexpr uint32_t kX16 = MT * kQ8BlockK * 2;     // fp16 x of one unit: two 64-wide halves
    static constexpr uint32_t kTmemCols = 256;
    static_assert(2 * MT + kOps * 64 <= 256, "two CTAs share the SM's tensor memory");
    static constexpr uint32_t kIdesc = idesc_f16_f32(kTileN, MT);
    static constexpr int kBars = 2 * kStages + 2 * kOps + 5;
    static constexpr int kSmem = 1024 + kStages * (kQ8WBytes + kRawX) + kOps * kX16 + kBars * 8 + 16;
    static_assert(kStages * (kQ8WBytes + kRawX) >= MT * kTileN * 4, "the sums take the ring's place");
};

template <int MT>
__global__ void __launch_bounds__(SplitShape<MT>::kThreads, 2)
q8_split_kernel(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmX, const Q8SplitParams p)
{
    using Sh = SplitShape<MT>;
    constexpr int S = Sh::kStages, OPS = Sh::kOps;

    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    uint8_t *sW = smem;
    uint8_t *sXraw = sW + S * kQ8WBytes;
    uint8_t *sX16 = sXraw + S * Sh::kRawX;
    uint64_t *wfull = reinterpret_cast<uint64_t *>(sX16 + OPS * Sh::kX16);
    uint64_t *wempty = wfull + S;
    uint64_t *opfull = wempty + S;
    uint64_t *opempty = opfull + OPS;
    uint64_t *afull = opempty + OPS;     // [2] accumulators
    uint64_t *aempty = afull + 2;        // [2]
    uint64_t *drain = aempty + 2;        // [1]
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(drain + 1);
    volatile int *flags = reinterpret_cast<volatile int *>(tmem_slot + 1);  // [0] abort

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int tile = static_cast<int>(blockIdx.x) / p.split, rank = static_cast<int>(blockIdx.x) % p.split;
    const int n0 = tile / p.m_tiles * kTileN, m0 = tile % p.m_tiles * MT;
    const int kb0 = rank * p.nkb / p.split, blocks = (rank + 1) * p.nkb / p.split - kb0;

    if (threadIdx.x == 0) {
        tma_prefetch_desc(&tmW);
        tma_prefetch_desc(&tmX);
        for (int i = 0; i < S; ++i) {
            mbar_init(&wfull[i], 1);
            mbar_init(&wempty[i], 4 + Sh::kXWarps);
        }
        for (int i = 0; i < OPS; ++i) {
            mbar_init(&opfull[i], 4 + Sh::kXWarps);
            mbar_init(&opempty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&afull[i], 1);
            mbar_init(&aempty[i], Sh::kEpiWarps);
        }
        mbar_init(drain, 1);
        flags[0] = 0;
        fence_mbar_init();
    }
    __syncthreads();
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
        // bounded waits do not count its time.  Scales, residual, workspace and y are
        // touched only from here on.
        pdl_wait();
    }

    int issued = 0;                      // units whose copies this thread has issued
    if (warp == Sh::kTmaWarp) {
        // -------------------------------------------------------- TMA producer
        if (lane == 0) {
            // W passes once where one token tile holds all of M
            const uint64_t pol_w = p.m_tiles == 1 ? policy_evict_first() : policy_evict_normal();
            const uint64_t pol_x = policy_evict_last();
            auto load_w = [&](int j) {
                mbar_arrive_expect_tx(&wfull[j % S], kQ8WBytes + Sh::kRawX);
                tma_load_2d(sW + j % S * kQ8WBytes, &tmW, &wfull[j % S], (kb0 + j) * kQ8BlockK, n0, pol_w);
            };
            auto load_x = [&](int j) {
                tma_load_2d(sXraw + j % S * Sh::kRawX, &tmX, &wfull[j % S], (kb0 + j) * kQ8BlockK, m0, pol_x);
            };
            if (!p.static_w)
                pdl_wait();
            const int first = min(S, blocks);
            for (int j = 0; j < first; ++j)
                load_w(j);
            if (p.static_w)              // weights may be requested before the wait for the previous kernel
                pdl_wait();
            for (int j = 0; j < first; ++j)
                load_x(j);
            int j = first;
            for (; j < blocks; ++j) {
                if (!mbar_wait(&wempty[j % S], ((j / S) & 1) ^ 1, p.timeout_ns, &flags[0])) {
                    q8_fail(p.err, &flags[0], kErrTimeoutProducer);
                    break;
                }
                load_w(j);
                load_x(j);
            }
            issued = j;
        }
    } else if (warp == Sh::kMmaWarp) {
        // ---------------------------------------------------------- MMA issuer
        {
            const bool leader = elect_one();
            const uint64_t x0 = smem_desc_kmajor_sw128(smem_u32(sX16));
            bool ok = true;
            // A round of the operand buffers at a time, unrolled, so that their
            // addresses and descriptors are constants.
            for (int j0 = 0; ok && j0 < blocks; j0 += OPS) {
#pragma unroll
                for (int b = 0; b < OPS; ++b) {
                    const int j = j0 + b, chunk = j / kExactBlocks, in_chunk = j % kExactBlocks, t = chunk & 1;
                    if (!ok || j >= blocks)
                        break;
                    if (in_chunk == 0)
                        ok = mbar_wait(&aempty[t], ((chunk >> 1) & 1) ^ 1, p.timeout_ns, &flags[0]);
                    ok = __all_sync(0xFFFFFFFFu, ok && mbar_wait(&opfull[b], (j / OPS) & 1, p.timeout_ns, &flags[0]));
                    if (!ok)
                        break;
                    tc_fence_after();
                    if (leader) {
                        const uint32_t d = tmem_base + static_cast<uint32_t>(t * MT), a = tmem_base + 2 * MT + b * 64;
                        const uint64_t bx = x0 + static_cast<uint64_t>(b * (Sh::kX16 / 16));
#pragma unroll
                        for (int kk = 0; kk < kQ8BlockK / 16; ++kk)
                            tc_mma_f16_ts(d, a + 8 * kk, bx + (kk >= 4) * (MT * 128 / 16) + 2 * (kk & 3), Sh::kIdesc,
                                          (in_chunk > 0 || kk > 0) ? 1u : 0u);
                        tc_commit(&opempty[b]);
                        if (in_chunk == kExactBlocks - 1 || j + 1 == blocks)
                            tc_commit(&afull[t]);
                    }
                    __syncwarp();
                }
            }
            if (!ok)
                q8_fail(p.err, &flags[0], kErrTimeoutMma);
            if (!ok) {                   // abort: wait for the MMAs already issued before TMEM is freed
                if (leader)
                    tc_commit(drain);
                volatile int never = 0;
                mbar_wait(drain, 0, kDefaultTimeoutNs, &never);
            }
        }
    } else if (warp < Sh::kFirstEpi) {
        // --------------------------------------------------------------- widen
        const int quarter = warp & 3, row = quarter * 32 + lane;
        const uint32_t lane_base = tmem_base + (static_cast<uint32_t>(quarter * 32) << 16) + 2 * MT;
        for (int j = (warp - Sh::kFirstWiden) >> 2; j < blocks; j += kWidenSets) {
            const int sl = j % S, b = j % OPS;
            // The operand buffer first: once the MMA of unit j - OPS is done, unit
            // j - S <= j - OPS has been widened, so the ring slot's barrier is at
            // most one phase behind and its parity says which.  (The warps run
            // apart: by the parity alone, a slot still waiting for unit j - S
            // looks like one that holds unit j.)
            const bool ok = mbar_wait(&opempty[b], ((j / OPS) & 1) ^ 1, p.timeout_ns, &flags[0]) &&
                            mbar_wait(&wfull[sl], (j / S) & 1, p.timeout_ns, &flags[0]);
            if (!__all_sync(0xFFFFFFFFu, ok)) {      // the whole warp goes on, or none of it
                q8_fail(p.err, &flags[0], kErrTimeoutWiden);
                break;
            }
            tc_fence_after();
            widen_row(sW + sl * kQ8WBytes, row, lane_base + b * 64);
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(&opfull[b]);
                mbar_arrive(&wempty[sl]);
            }
        }
    } else {
        // ------------------------------------------- widen x, and the epilogue
        constexpr int NC = Sh::kCols;
        // Not sooner (see skg_q8_stream.cu), and after this CTA's TMEM is allocated: the
        // dependents' CTAs may take the rest of an SM's, and they wait for this one.
        pdl_launch_dependents();
        const int ew = warp - Sh::kFirstEpi;
        const int row = (warp & 3) * 32 + lane;
        const int col0 = (ew >> 2) * NC, valid = p.g.M - m0 - col0;
        const uint32_t lane_base = tmem_base + (static_cast<uint32_t>((warp & 3) * 32) << 16) + static_cast<uint32_t>(col0);
        // The last two accumulations stay in TMEM until the end; earlier ones
        // (K parts of more than 2048) are put into global memory, a slot each,
        // while the MMAs fill the other buffer: registers and shared memory are
        // taken.
        const int chunks = (blocks + kExactBlocks - 1) / kExactBlocks;
        const size_t slot = MT * kTileN;
        int *carry = p.carry + blockIdx.x * p.carried * slot + col0 * kTileN + row;
        int *sums = reinterpret_cast<int *>(smem) + col0 * kTileN + row;
        constexpr int kStep = Sh::kXWarps * 4;           // tokens that a set takes at a time
        static_assert(kStep % 8 == 0, "the swizzle repeats every 8 rows");
        const XPiece piece(ew % Sh::kXWarps * 4, lane, MT);
        bool ok = true;
        int put = 0;                     // accumulations put away
        auto put_away = [&] {
            const int t = put & 1;
            ok = __all_sync(0xFFFFFFFFu, mbar_wait(&afull[t], (put >> 1) & 1, p.timeout_ns, &flags[0]));
            if (!ok)
                return;
            tc_fence_after();
#pragma unroll 1
            for (int c0 = 0; c0 < NC; c0 += 16) {
                int v[16];
                load_sums(lane_base + static_cast<uint32_t>(t * MT + c0), v);
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    if (c0 + i < valid)
                        __stcg(carry + put * slot + (c0 + i) * kTileN, v[i]);
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0)
                mbar_arrive(&aempty[t]);
            ++put;
        };
        for (int u = ew / Sh::kXWarps; u < blocks; u += 2) {
            const int sl = u % S, b = u % OPS;
            // the operand buffer first, as above
            ok = mbar_wait(&opempty[b], ((u / OPS) & 1) ^ 1, p.timeout_ns, &flags[0]) &&
                 mbar_wait(&wfull[sl], (u / S) & 1, p.timeout_ns, &flags[0]);
            ok = __all_sync(0xFFFFFFFFu, ok);
            if (!ok)
                break;
            piece.widen<MT / kStep>(sXraw + sl * Sh::kRawX, sX16 + b * Sh::kX16, kStep);
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(&opfull[b]);
                mbar_arrive(&wempty[sl]);
            }
            // an accumulation is done once the unit two after it has been widened, or nearly
            if (put + 2 < chunks && u >= (put + 1) * kExactBlocks + 2) {
                put_away();
                if (!ok)
                    break;
            }
        }
        while (ok && put + 2 < chunks)
            put_away();
        // The end: what was put away (fetched while the last MMAs run), and the
        // one or two accumulations in TMEM.
        int acc[NC];
#pragma unroll
        for (int i = 0; i < NC; ++i)
            acc[i] = 0;
        for (int k = 0; k < put; ++k) {
            int v[NC];
#pragma unroll
            for (int i = 0; i < NC; ++i)
                v[i] = i < valid ? __ldcg(carry + k * slot + i * kTileN) : 0;
#pragma unroll
            for (int i = 0; i < NC; ++i)
                acc[i] += v[i];
        }
        const int last = chunks - 1;
        const bool pair = chunks > 1;
        ok = ok && (!pair || mbar_wait(&afull[(last - 1) & 1], ((last - 1) >> 1) & 1, p.timeout_ns, &flags[0])) &&
             mbar_wait(&afull[last & 1], (last >> 1) & 1, p.timeout_ns, &flags[0]);
        ok = __all_sync(0xFFFFFFFFu, ok);
        if (!ok)
            q8_fail(p.err, &flags[0], kErrTimeoutEpilogue);
        tc_fence_after();
#pragma unroll
        for (int c0 = 0; c0 < NC && ok; c0 += 8) {
            int v[8];
            load_sums(lane_base + static_cast<uint32_t>((last & 1) * MT + c0), v);
#pragma unroll
            for (int i = 0; i < 8; ++i)
                acc[c0 + i] += v[i];
            if (pair) {
                load_sums(lane_base + static_cast<uint32_t>(((last - 1) & 1) * MT + c0), v);
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    acc[c0 + i] += v[i];
            }
        }
        if (ok && p.split == 1) {
            store_columns(p.g, m0 + col0, n0 + row, load_scales(p.g, m0 + col0, n0 + row), acc);
        } else if (ok) {
            // in the ring's place: the last MMA has read its operands
#pragma unroll
            for (int i = 0; i < NC; ++i)
                sums[i * kTileN] = acc[i];
        }
    }

    __syncwarp();
    tc_fence_before();
    if (p.split > 1) {
        join_and_store<8, Sh::kThreads>(p.g, smem_u32(smem), m0, n0, min(MT, p.g.M - m0), p.split, rank, 1, 0, p.vec4 != 0);
    } else {
        __syncthreads();
    }
    // Abort: every copy lands before the CTA exits.  (Looked at here, where no role raises the
    // flag any more; what a join has read meanwhile is of a launch that is reported.)
    if (issued && flags[0]) {
        volatile int never = 0;
        for (int u = max(0, issued - S); u < issued; ++u)
            mbar_wait(&wfull[u % S], (u / S) & 1, kDefaultTimeoutNs, &never);
    }
    if (warp == Sh::kMmaWarp) {
        tc_fence_after();
        tmem_dealloc(tmem_base, Sh::kTmemCols);
    }
}

template <int MT>
cudaError_t launch_shape(const CUtensorMap &tmW, const CUtensorMap &tmX, const Q8SplitParams &p, int grid, cudaStream_t s)
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
        e = cudaFuncSetAttribute(q8_split_kernel<MT>, cudaFuncAttributeMaxDynamicSharedMemorySize, Sh::kSmem);
        if (e == cudaSuccess)
            e = cudaFuncSetAttribute(q8_split_kernel<MT>, cudaFuncAttributePreferredSharedMemoryCarveout,
                                     cudaSharedmemCarveoutMaxShared);
        if (e != cudaSuccess)
            return e;
        __atomic_store_n(&attr_set[dev], 1, __ATOMIC_RELEASE);
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(grid));
    cfg.blockDim = dim3(Sh::kThreads);
    cfg.dynamicSmemBytes = Sh::kSmem;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = static_cast<unsigned>(p.split);
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = p.split > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, q8_split_kernel<MT>, tmW, tmX, p);
}

template <int MT>
Q8TcShape shape_of()
{
    return {MT, 2, SplitShape<MT>::kSmem, SplitShape<MT>::kThreads, SplitShape<MT>::kStages};
}

} // namespace

Q8TcShape q8_split_shape(int m_tile) { return m_tile == 32 ? shape_of<32>() : shape_of<64>(); }

cudaError_t launch_q8_split(const CUtensorMap &tmW, const CUtensorMap &tmX, const Q8SplitParams &p, int m_tile, int grid,
                            cudaStream_t s)
{
    return m_tile == 32 ? launch_shape<32>(tmW, tmX, p, grid, s) : launch_shape<64>(tmW, tmX, p, grid, s);
}

} // namespace skg

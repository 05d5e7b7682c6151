// skg_q8_wide.cu -- the 8-bit projection for many tokens: tcgen05 over whole
// tiles, by pairs of CTAs.
//
// The arithmetic is that of skg_q8_split.cu: integers widened to fp16 on chip,
// products summed by kind::f16 MMAs from a fresh fp32 accumulator every 1024 k,
// and the accumulators added as int32, so the sums are exact.  What bounds it is
// the tensor core, if its operands can be had in time.  Two CTAs work as one
// (cta_group::2): 256 channels x 128 tokens, each CTA with its 128 rows of W in
// its own TMEM (A) and half of x in its own shared memory (B), so a unit of 128
// k costs a CTA 16 KB of W and 8 of x from the L2 and the MMAs 512 cycles.
//
// Roles of a CTA (one per SM, pairs persistent over tiles):
//   1          TMEM; in the first CTA of the pair, MMA issue for both
//   1          TMA
//   8 warps    widen, two sets of 4 on alternate units: W into TMEM, x into
//              shared memory
//   16         epilogue: accumulators into int32 registers; at a tile's end
//              scales, residual, rounding and the store, while the next tile's
//              MMAs go on in the other accumulator
// The MMA issuer is what the rest is arranged around.  About three MMAs queue up
// behind the one that runs, and one wait on a barrier, even one already past,
// takes as long as one or two of them; so it waits once a unit, for a barrier at
// which everything the unit needs arrives, looks for the next one while half of
// this one is still to issue, and commits once a unit.
//
// Where the tiles leave SMs idle, K is split over the up to 4 pairs of a cluster,
// which leave their sums in shared memory and add them up as the split kernel's
// CTAs do.
//
// Measured, weights from HBM: 4096 x 12288 x 7168 463-500 us (1.44-1.56 PFLOP/s of
// the 1.96 that cuBLAS reaches; it draws 1.34 kW and the clock falls to 1.8 GHz
// if it runs for seconds), 1024 x 7168 x 7168 72 us (1.46), 333 x 5001 x 4112 20.4
// us, 256 x 4096 x 4096 15.3 us (17.4 unsplit), 128 x 7168 x 7168 19.6 us (26.3
// unsplit).  A unit takes 0.39 us, where its MMAs take 0.27.  What bounds it is
// the widening: without that of W 4096 tokens take 368 us, without that of x 424,
// without the epilogue's sums 440.  Instructions issue in 60% of the cycles and
// shared memory moves 87 KB a unit.  Three sets of widening warps (460 us) or 8
// epilogue warps instead of 16 (547: registers spill) are no better; with all 8
// warps on every unit it takes 550.  x widened by a kernel before took 475 us
// where this took 500, but 22.7 for 333 x 5001 x 4112 and a workspace.
//
// Every wait is bounded as in skg_q8_split.cu.
#include "skg_internal.h"
#include "skg_ptx.cuh"
#include "skg_q8_common.cuh"
#include "skg_q8_internal.h"

namespace skg {
namespace {

#include "skg_q8_tc_common.cuh"

constexpr int kPair = 2;                             // CTAs that work as one
constexpr int MT = 128;                              // tokens of a tile: the MMA's N
constexpr int kHalfTokens = MT / kPair;              // of which a CTA holds these

struct WideShape {
    static constexpr int kEpiWarps = 16;
    static constexpr int kCols = MT * 4 / kEpiWarps;         // accumulator columns of an epilogue thread
    static_assert(kCols == 32, "a lane holds the scale of a token");
    static constexpr int kThreads = 32 * (2 + kWidenWarps + kEpiWarps);
    static constexpr int kMmaWarp = 0, kTmaWarp = 1, kFirstWiden = 2, kFirstEpi = kFirstWiden + kWidenWarps;
    static constexpr int kStages = 6;                        // ring of W and int8 x
    static constexpr int kOps = (512 - 2 * MT) / 64;         // widened operand buffers: 4
    static_assert(kStages >= kOps && kOps >= kWidenSets, "the widen warps' waits need this");
    static constexpr uint32_t kRawX = kHalfTokens * kQ8BlockK;
    static constexpr uint32_t kX16 = 2 * kRawX;              // two 64-wide halves
    static constexpr uint32_t kTmemCols = 512;
    static constexpr uint32_t kIdesc = idesc_f16_f32(2 * kTileN, MT);
    static_assert(kStages * kQ8WBytes >= MT * kTileN * 4, "the sums take the ring's place");
    static constexpr int kBars = 2 * kStages + 2 * kOps + 5;
    static constexpr int kSmem = 1024 + kStages * (kQ8WBytes + kRawX) + kOps * kX16 + kBars * 8 + 16;
};

// Tiles (pairs of 128 channels x 128 tokens) in bands of p.band token tiles:
// within a band, token tiles fastest, so that the CTAs of a wave share a
// compact block of x and W in L2.
__device__ __forceinline__ void tile_at(const Q8WideParams &p, int tile, int &np, int &mt)
{
    const int per_band = p.band * p.n_pairs;
    const int b = tile / per_band, r = tile - b * per_band;
    const int wide = min(p.band, p.m_tiles - b * p.band);
    np = r / wide;
    mt = b * p.band + r - np * wide;
}

__global__ void __launch_bounds__(WideShape::kThreads, 1)
q8_wide_kernel(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmX, const Q8WideParams p)
{
    using Sh = WideShape;
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
    // opfull and aempty are those of the first CTA, with arrivals from both;
    // the MMA's commits arrive at both CTAs' opempty and afull
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(drain + 1);
    volatile int *flags = reinterpret_cast<volatile int *>(tmem_slot + 1);  // [0] abort

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    // A cluster is p.split pairs, each with its part of K.  With more than one
    // there are as many clusters as tiles.
    const int rank = static_cast<int>(blockIdx.x) % kPair, pair = static_cast<int>(blockIdx.x) / kPair;
    const int part = pair % p.split, cluster = pair / p.split, first = part * kPair;
    const int clusters = static_cast<int>(gridDim.x) / (kPair * p.split);
    const uint16_t both = static_cast<uint16_t>(((1 << kPair) - 1) << first);        // the pair's ranks in the cluster
    const int my_tiles = (p.tiles - cluster + clusters - 1) / clusters;
    const int kb0 = part * p.nkb / p.split, nkb = (part + 1) * p.nkb / p.split - kb0;
    const int units = my_tiles * nkb;

    if (threadIdx.x == 0) {
        tma_prefetch_desc(&tmW);
        tma_prefetch_desc(&tmX);
        for (int i = 0; i < S; ++i) {
            mbar_init(&wfull[i], 1);
            mbar_init(&wempty[i], 4);
        }
        for (int i = 0; i < OPS; ++i) {
            mbar_init(&opfull[i], kPair * 4);
            mbar_init(&opempty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&afull[i], 1);
            mbar_init(&aempty[i], kPair * Sh::kEpiWarps);
        }
        mbar_init(drain, 1);
        flags[0] = 0;
        fence_mbar_init();
    }
    __syncthreads();
    if (warp == Sh::kMmaWarp) {
        tmem_alloc_pair(tmem_slot, Sh::kTmemCols);
        tmem_relinquish_pair();
    }
    tc_fence_before();
    cluster_sync();                      // the peer's barriers exist before anything is sent there
    tc_fence_after();
    // all 512 columns are this CTA's, so they begin at 0: as a constant it keeps
    // the MMA's addresses in uniform registers
    constexpr uint32_t tmem_base = 0;

    if (warp == Sh::kTmaWarp) {
        // -------------------------------------------------------- TMA producer
        const bool leader = elect_one();
        const uint64_t pol = policy_evict_normal();
        int np, mt;
        auto load_w = [&](int j, int kb) {
            if (leader) {
                mbar_arrive_expect_tx(&wfull[j % S], kQ8WBytes + Sh::kRawX);
                tma_load_2d(sW + j % S * kQ8WBytes, &tmW, &wfull[j % S], (kb0 + kb) * kQ8BlockK, (np * kPair + rank) * kTileN, pol);
            }
            __syncwarp();
        };
        auto load_x = [&](int j, int kb) {       // this CTA's half of the tokens
            if (leader)
                tma_load_2d(sXraw + j % S * Sh::kRawX, &tmX, &wfull[j % S], (kb0 + kb) * kQ8BlockK, mt * MT + rank * kHalfTokens, pol);
            __syncwarp();
        };
        tile_at(p, cluster, np, mt);
        const int ahead = p.static_w ? min(S, nkb) : 0;
        for (int j = 0; j < ahead; ++j)  // weights may be requested before the wait for the previous kernel
            load_w(j, j);
        pdl_wait();
        pdl_launch_dependents();         // not sooner: see skg_q8_stream.cu
        bool ok = true;
        int j = 0, issued = ahead;
        for (int tile = cluster; tile < p.tiles && ok; tile += clusters) {
            tile_at(p, tile, np, mt);
            for (int kb = 0; kb < nkb; ++kb, ++j) {
                if (j >= ahead) {
                    ok = __all_sync(0xFFFFFFFFu, mbar_wait(&wempty[j % S], ((j / S) & 1) ^ 1, p.timeout_ns, &flags[0]));
                    if (!ok)
                        break;
                    load_w(j, kb);
                    issued = j + 1;
                }
                load_x(j, kb);
            }
        }
        if (!ok)
            q8_fail(p.err, &flags[0], kErrTimeoutProducer);
        if (flags[0]) {                  // abort: let every copy land before exit
            volatile int never = 0;
            for (int k = 0; k < S && k < issued; ++k)
                mbar_wait(&wfull[k], ((issued - 1 - k) / S) & 1, kDefaultTimeoutNs, &never);
        }
    } else if (warp == Sh::kMmaWarp) {
        // ---------------------------------------------------------- MMA issuer
        if (rank == 0) {
            const bool leader = elect_one();
            const uint64_t x0 = smem_desc_kmajor_sw128(smem_u32(sX16));
            int kb = 0, in_chunk = 0, chunk = 0;
            bool ok = __all_sync(0xFFFFFFFFu, mbar_wait(&opfull[0], 0, p.timeout_ns, &flags[0]));
            // Two rounds of the operand buffers at a time, unrolled: their
            // addresses, descriptors and phases are then constants (worked out in
            // a loop over single units they took longer than the MMAs).
            for (int j0 = 0; ok && j0 < units; j0 += 2 * OPS) {
#pragma unroll
                for (int u = 0; u < 2 * OPS; ++u) {
                    if (!ok || j0 + u >= units)
                        break;
                    constexpr int kHalf = Sh::kX16 / 2 / 16;             // the second 64 k, in descriptor units
                    const uint64_t bx = x0 + static_cast<uint64_t>((u % OPS) * (Sh::kX16 / 16));
                    const uint32_t a = tmem_base + 2 * MT + (u % OPS) * 64;
                    const int t = chunk & 1;
                    const uint32_t d = tmem_base + static_cast<uint32_t>(t * MT);
                    if (in_chunk == 0)
                        ok = __all_sync(0xFFFFFFFFu, mbar_wait(&aempty[t], ((chunk >> 1) & 1) ^ 1, p.timeout_ns, &flags[0]));
                    if (!ok)
                        break;
                    tc_fence_after();
                    if (leader) {
#pragma unroll
                        for (int kk = 0; kk < 4; ++kk)
                            tc_mma_f16_ts_pair(d, a + 8 * kk, bx + 2 * kk, Sh::kIdesc, (kk > 0 || in_chunk > 0) ? 1u : 0u);
                    }
                    const bool last = j0 + u + 1 == units;
                    uint64_t *next = &opfull[(u + 1) % OPS];
                    const uint32_t next_phase = ((u + 1) / OPS) & 1;
                    const bool ready = __all_sync(0xFFFFFFFFu, last || mbar_try_wait(next, next_phase));
                    const bool end = ++kb == nkb || in_chunk == kExactBlocks - 1;
                    if (leader) {
#pragma unroll
                        for (int kk = 0; kk < 4; ++kk)
                            tc_mma_f16_ts_pair(d, a + 32 + 8 * kk, bx + kHalf + 2 * kk, Sh::kIdesc, 1u);
                        // nobody waits for the last units, and the peer may be gone by then
                        if (j0 + u + OPS < units)
                            tc_commit_pair_multicast(&opempty[u % OPS], both);
                        if (end)
                            tc_commit_pair_multicast(&afull[t], both);
                    }
                    in_chunk = end ? 0 : in_chunk + 1;
                    chunk += end;
                    kb = kb == nkb ? 0 : kb;
                    if (!ready)
                        ok = __all_sync(0xFFFFFFFFu, mbar_wait(next, next_phase, p.timeout_ns, &flags[0]));
                }
            }
            if (!ok)
                q8_fail(p.err, &flags[0], kErrTimeoutMma);
            if (!ok) {                   // abort: wait for the MMAs already issued before TMEM is freed
                if (leader)
                    tc_commit_pair(drain);
                volatile int never = 0;
                mbar_wait(drain, 0, kDefaultTimeoutNs, &never);
            }
        }
    } else if (warp < Sh::kFirstEpi) {
        // --------------------------------------------------------------- widen
        const int quarter = warp & 3, row = quarter * 32 + lane;
        const uint32_t lane_base = tmem_base + (static_cast<uint32_t>(quarter * 32) << 16) + 2 * MT;
        const XPiece piece(quarter * 4, lane, kHalfTokens);
        for (int j = (warp - Sh::kFirstWiden) >> 2; j < units; j += kWidenSets) {
            const int sl = j % S, b = j % OPS;
            // The operand buffer first: see skg_q8_split.cu
            const bool ok = mbar_wait(&opempty[b], ((j / OPS) & 1) ^ 1, p.timeout_ns, &flags[0]) &&
                            mbar_wait(&wfull[sl], (j / S) & 1, p.timeout_ns, &flags[0]);
            if (!__all_sync(0xFFFFFFFFu, ok)) {      // the whole warp goes on, or none of it
                q8_fail(p.err, &flags[0], kErrTimeoutWiden);
                break;
            }
            tc_fence_after();
            widen_row(sW + sl * kQ8WBytes, row, lane_base + b * 64);
            piece.widen<kHalfTokens / 16>(sXraw + sl * Sh::kRawX, sX16 + b * Sh::kX16, 16);
            fence_proxy_async_smem();
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(&wempty[sl]);
                mbar_arrive_cluster(map_shared_rank(smem_u32(&opfull[b]), first));
            }
        }
    } else {
        // ------------------------------------------------------------ epilogue
        constexpr int NC = Sh::kCols;
        pdl_wait();                      // scales, residual and y only from here on
        const int row = (warp & 3) * 32 + lane;
        const int col0 = ((warp - Sh::kFirstEpi) >> 2) * NC;
        const uint32_t lane_base = tmem_base + (static_cast<uint32_t>((warp & 3) * 32) << 16) + static_cast<uint32_t>(col0);
        int chunk = 0;
        bool ok = true;
        for (int tile = cluster; tile < p.tiles && ok; tile += clusters) {
            int np, mt;
            tile_at(p, tile, np, mt);
            const int n = (np * kPair + rank) * kTileN + row;
            const Scales sc = load_scales(p.g, mt * MT + col0, n);
            int acc[NC];
            for (int kb = 0; kb < nkb; kb += kExactBlocks, ++chunk) {
                const int t = chunk & 1;
                ok = __all_sync(0xFFFFFFFFu, mbar_wait(&afull[t], (chunk >> 1) & 1, p.timeout_ns, &flags[0]));
                if (!ok) {
                    q8_fail(p.err, &flags[0], kErrTimeoutEpilogue);
                    break;
                }
                tc_fence_after();
#pragma unroll
                for (int c0 = 0; c0 < NC; c0 += 8) {
                    int v[8];
                    load_sums(lane_base + static_cast<uint32_t>(t * MT + c0), v);
#pragma unroll
                    for (int c = 0; c < 8; ++c)
                        acc[c0 + c] = kb == 0 ? v[c] : acc[c0 + c] + v[c];
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0)
                    mbar_arrive_cluster(map_shared_rank(smem_u32(&aempty[t]), first));
            }
            if (ok && p.split == 1) {
                store_columns(p.g, mt * MT + col0, n, sc, acc);
            } else if (ok) {
                // in the ring's place: the last MMA has read its operands
#pragma unroll
                for (int c = 0; c < NC; ++c)
                    reinterpret_cast<int *>(smem)[(col0 + c) * kTileN + row] = acc[c];
            }
        }
    }

    __syncwarp();
    tc_fence_before();
    if (p.split == 1) {
        cluster_sync();                  // no CTA leaves while its peer may still send to it
    } else {
        int np, mt;
        tile_at(p, cluster, np, mt);
        join_and_store<kQ8WideMaxSplit, Sh::kThreads>(p.g, smem_u32(smem), mt * MT, (np * kPair + rank) * kTileN,
                                                      min(MT, p.g.M - mt * MT), p.split, part, kPair, rank, p.vec4 != 0);
    }
    if (warp == Sh::kMmaWarp) {
        tc_fence_after();
        tmem_dealloc_pair(tmem_base, Sh::kTmemCols);
    }
}

} // namespace

Q8TcShape q8_wide_shape()
{
    return {MT, 1, WideShape::kSmem, WideShape::kThreads, WideShape::kStages};
}

cudaError_t launch_q8_wide(const CUtensorMap &tmW, const CUtensorMap &tmX, const Q8WideParams &p, int grid,
                           cudaStream_t s)
{
    static int attr_set[kMaxDevices] = {};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess)
        return e;
    if (dev >= kMaxDevices)
        return cudaErrorInvalidDevice;
    if (__atomic_load_n(&attr_set[dev], __ATOMIC_ACQUIRE) == 0) {
        e = cudaFuncSetAttribute(q8_wide_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, WideShape::kSmem);
        if (e != cudaSuccess)
            return e;
        __atomic_store_n(&attr_set[dev], 1, __ATOMIC_RELEASE);
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(grid));
    cfg.blockDim = dim3(WideShape::kThreads);
    cfg.dynamicSmemBytes = WideShape::kSmem;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = static_cast<unsigned>(kPair * p.split);
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, q8_wide_kernel, tmW, tmX, p);
}

} // namespace skg

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
//   1          TMEM; in the first CTA of the pair MMA issue for both, in the second
//              a relay
//   1 + 1      TMA of W, TMA of x
//   8 warps    widen, two sets of 4 on alternate units: W into TMEM, x into
//              shared memory
//   16         epilogue: accumulators into int32 registers; at a tile's end
//              scales, residual, rounding and the store, while the next tile's
//              MMAs go on in the other accumulator
//   1          in the second CTA, the other relay
// The MMA issuer is what the rest is arranged around.  About three MMAs queue up
// behind the one that runs, and one wait on a barrier, even one already past,
// takes as long as one or two of them; so it waits once a unit, for a barrier at
// which everything the unit needs arrives, looks for the next one while half of
// this one is still to issue, and commits once a unit.
//
// What the second CTA's warps announce to the issuer in the first.  W is in TMEM:
// tcgen05.fence orders it, and the arrival is relaxed.  x is written with plain
// stores, which only a release at cluster scope orders before what a thread of
// another CTA does, and that release takes 0.7 to 1.2 us.  In the widening warps
// it took 1024 x 7168 x 7168 from 72 to 118 us.  So x is widened kAhead units
// before W, the widening warps arrive at a barrier of their own CTA, and two other
// warps in turn pass that on, with the release, for two units at a time: 76 us,
// as long as without the release.  (One relay 88 us; x two units ahead 87.)
//
// Where the tiles leave SMs idle, K is split over the up to 4 pairs of a cluster,
// which leave their sums in shared memory and add them up as the split kernel's
// CTAs do.
//
// Measured, weights from HBM: 4096 x 12288 x 7168 483-513 us (1.41-1.49 PFLOP/s of
// the 1.96 that cuBLAS reaches; it draws 1.34 kW and the clock falls to 1.8 GHz
// if it runs for seconds), 1024 x 7168 x 7168 76 us (1.38; 82 right after the
// former), 333 x 5001 x 4112 22.4 us, 256 x 4096 x 4096 16.7 us (19.3 unsplit), 128 x
// 7168 x 7168 22.0 us (29.4 unsplit).  A unit takes 0.41 us,
// where its MMAs take 0.27.  What bounds it is the widening, and how soon the ring
// is filled again: an iteration of a set of widening warps works for 1030 cycles and
// waits for 500, a load takes 2200 until it has arrived, and with the producers'
// work in one warp 1024 tokens take 83 us.  (x read by the widening warps from
// global memory instead, with 6 stages of W: 88 us; the ring's bytes taken into
// registers before the wait for the operand buffer: 86.)  Three sets of widening
// warps or 8 epilogue warps instead of 16 are no better; with all 8 widening warps
// on every unit 4096 tokens take 550 us.
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
    static constexpr int kThreads = 32 * (4 + kWidenWarps + kEpiWarps);
    static constexpr int kMmaWarp = 0, kTmaWarp = 1, kFirstWiden = 2, kFirstEpi = kFirstWiden + kWidenWarps,
                         kTmaXWarp = kFirstEpi + kEpiWarps, kRelayWarp = kTmaXWarp + 1;
    static constexpr int kStages = 4;                        // ring of int8: W of a unit, x of one kAhead later
    static constexpr int kOps = (512 - 2 * MT) / 64;         // widened W, in TMEM: 4
    static constexpr int kAhead = 4;                         // units by which x is widened before W
    static constexpr int kXOps = kOps + kAhead;              // widened x: 8
    static_assert(kStages % kWidenSets == 0 && kOps % kWidenSets == 0 && kAhead == 2 * kWidenSets && kXOps % kOps == 0 &&
                      kAhead <= kStages,
                  "a buffer is always the same set's; the prologue's and the issuer's order");
    static constexpr uint32_t kRawX = kHalfTokens * kQ8BlockK;
    static constexpr uint32_t kX16 = 2 * kRawX;              // two 64-wide halves
    static constexpr uint32_t kTmemCols = 512;
    static constexpr uint32_t kIdesc = idesc_f16_f32(2 * kTileN, MT);
    static_assert(kStages * kQ8WBytes >= MT * kTileN * 4, "the sums take the ring's place");
    static constexpr int kBars = kStages + kOps + 2 * kXOps + 7;
    static constexpr int kSmem = 1024 + kStages * (kQ8WBytes + kRawX) + kXOps * kX16 + kBars * 8 + 16;
    static_assert(kSmem <= 227 * 1024, "shared memory of a CTA");
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
    constexpr uint32_t S = Sh::kStages, OPS = Sh::kOps, XOPS = Sh::kXOps, AHEAD = Sh::kAhead;

    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    uint8_t *sW = smem;
    uint8_t *sXraw = sW + S * kQ8WBytes;
    uint8_t *sX16 = sXraw + S * Sh::kRawX;
    // int8 x of the first kAhead units: those of a set in the buffer where the set
    // widens x of its unit after them.  A warp reads and writes the same tokens,
    // which lie in the same rows.
    uint8_t *sX0 = sX16 + AHEAD * Sh::kX16;
    uint64_t *full = reinterpret_cast<uint64_t *>(sX16 + XOPS * Sh::kX16);
    uint64_t *widened = full + S;        // [XOPS] this CTA's W of a unit, and x of the one AHEAD of it
    uint64_t *opfull = widened + XOPS;   // [XOPS] operands of a unit, both CTAs'
    uint64_t *done = opfull + XOPS;      // [OPS] MMAs of a unit
    uint64_t *afull = done + OPS;        // [2] accumulators
    uint64_t *aempty = afull + 2;        // [2]
    uint64_t *x0full = aempty + 2;       // [1] int8 x of the first AHEAD units
    uint64_t *x0done = x0full + 1;       // [1] widened
    uint64_t *drain = x0done + 1;        // [1]
    // opfull and aempty are those of the first CTA, with arrivals from both;
    // the MMA's commits arrive at both CTAs' done and afull
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(drain + 1);
    volatile int *flags = reinterpret_cast<volatile int *>(tmem_slot + 1);  // [0] abort, [1] the previous kernel has ended

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
        for (int i = 0; i < S; ++i)
            mbar_init(&full[i], 2);      // W's producer and x's
        for (int i = 0; i < XOPS; ++i) {
            mbar_init(&widened[i], 4);
            // W of both CTAs, which in the first stands for its x too; the first unit of two: the second CTA's x of both
            mbar_init(&opfull[i], kPair * 4 + (i % kWidenSets == 0 ? 1 : 0));
        }
        for (int i = 0; i < OPS; ++i)
            mbar_init(&done[i], 1);
        mbar_init(x0full, 1);
        mbar_init(x0done, kWidenWarps);
        for (int i = 0; i < 2; ++i) {
            mbar_init(&afull[i], 1);
            mbar_init(&aempty[i], kPair * Sh::kEpiWarps);
        }
        mbar_init(drain, 1);
        flags[0] = flags[1] = 0;
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

    // A warp's first wait, for what comes of x: its limit does not count the previous
    // kernel's time.  (pdl_wait in these warps does the same, and a block of 64 tokens
    // took 77 us instead of 72, one of 1024 283 instead of 278.)
    auto first_wait = [&](uint64_t *bar) {
        uint64_t t0 = globaltimer_ns();
        while (!mbar_try_wait_cluster(bar, 0)) {
            if (flags[1] == 0)
                t0 = globaltimer_ns();
            if (flags[0] || globaltimer_ns() - t0 > p.timeout_ns)
                return false;
        }
        return true;
    };
    // Unit u - S has left the ring: its W has been widened, and the x that came with it.
    auto wait_widened = [&](uint32_t u) {
        return u < S || __all_sync(0xFFFFFFFFu, mbar_wait(&widened[(u - S) % XOPS], (u - S) / XOPS & 1, p.timeout_ns, &flags[0]));
    };
    // x of the second CTA's pairs of units r, r + 2, ... has been widened: passed on to the issuer.
    auto relay = [&](int r) {
        bool ok = true;
        for (uint32_t u = r * kWidenSets; ok && u < static_cast<uint32_t>(units); u += 2 * kWidenSets) {
            if (u < AHEAD)
                ok = first_wait(x0done);
            for (uint32_t v = u; ok && u >= AHEAD && v < u + kWidenSets && v < static_cast<uint32_t>(units); ++v)
                ok = mbar_wait(&widened[(v - AHEAD) % XOPS], (v - AHEAD) / XOPS & 1, p.timeout_ns, &flags[0]);
            ok = __all_sync(0xFFFFFFFFu, ok);
            if (ok && lane == 0)
                mbar_arrive_cluster_release(map_shared_rank(smem_u32(&opfull[u % XOPS]), first));
            __syncwarp();
        }
        if (!ok)
            q8_fail(p.err, &flags[0], kErrTimeoutWiden);
    };
    if (warp == Sh::kTmaWarp) {
        // ------------------------------------------------------ TMA producer of W
        const bool leader = elect_one();
        const uint64_t pol = policy_evict_normal();
        int np, mt;
        auto load = [&](uint32_t u, int kb) {
            if (leader) {
                mbar_arrive_expect_tx(&full[u % S], kQ8WBytes);
                tma_load_2d(sW + u % S * kQ8WBytes, &tmW, &full[u % S], (kb0 + kb) * kQ8BlockK, (np * kPair + rank) * kTileN, pol);
            }
            __syncwarp();
        };
        tile_at(p, cluster, np, mt);
        const uint32_t ahead = p.static_w ? min(S, nkb) : 0;
        for (uint32_t u = 0; u < ahead; ++u)     // weights may be requested before the wait for the previous kernel
            load(u, u);
        pdl_wait();
        flags[1] = 1;
        pdl_launch_dependents();         // not sooner: see skg_q8_stream.cu
        bool ok = true;
        uint32_t u = 0;
        for (int tile = cluster; tile < p.tiles && ok; tile += clusters) {
            tile_at(p, tile, np, mt);
            for (int kb = 0; kb < nkb; ++kb, ++u) {
                if (u < ahead)
                    continue;
                ok = wait_widened(u);
                if (!ok)
                    break;
                load(u, kb);
            }
        }
        if (!ok)
            q8_fail(p.err, &flags[0], kErrTimeoutProducer);
    } else if (warp == Sh::kTmaXWarp) {
        // ------------------------------------------------------ TMA producer of x
        const bool leader = elect_one();
        const uint64_t pol = policy_evict_normal();
        pdl_wait();
        if (leader)
            mbar_arrive_expect_tx(x0full, min(units, AHEAD) * Sh::kRawX);
        __syncwarp();
        bool ok = true;
        uint32_t v = 0;
        for (int tile = cluster; tile < p.tiles && ok; tile += clusters) {
            int np, mt;
            tile_at(p, tile, np, mt);
            for (int kb = 0; kb < nkb; ++kb, ++v) {
                const uint32_t u = v - AHEAD;            // with W of this unit
                uint8_t *to = sX0 + v % kWidenSets * Sh::kX16 + v / kWidenSets * Sh::kRawX;
                uint64_t *bar = x0full;
                if (v >= AHEAD) {
                    ok = wait_widened(u);
                    if (!ok)
                        break;
                    to = sXraw + u % S * Sh::kRawX;
                    bar = &full[u % S];
                }
                if (leader) {
                    if (v >= AHEAD)
                        mbar_arrive_expect_tx(bar, Sh::kRawX);
                    tma_load_2d(to, &tmX, bar, (kb0 + kb) * kQ8BlockK, mt * MT + rank * kHalfTokens, pol);
                }
                __syncwarp();
            }
        }
        const uint32_t issued = v > AHEAD ? v - AHEAD : 0;
        for (uint32_t u = issued; ok && u < static_cast<uint32_t>(units); ++u) {
            ok = wait_widened(u);        // no x comes with the last units' W
            if (ok && leader)
                mbar_arrive(&full[u % S]);
            __syncwarp();
        }
        if (!ok)
            q8_fail(p.err, &flags[0], kErrTimeoutProducer);
    } else if (warp == Sh::kMmaWarp) {
        // ---------------------------------------------------------- MMA issuer
        if (rank == 0) {
            const bool leader = elect_one();
            const uint64_t x0 = smem_desc_kmajor_sw128(smem_u32(sX16));
            int kb = 0, in_chunk = 0, chunk = 0;
            bool ok = __all_sync(0xFFFFFFFFu, first_wait(&opfull[0]));
            // A round of the operand buffers at a time, unrolled: their addresses and
            // descriptors are then constants (worked out in a loop over single units
            // they took longer than the MMAs).
            uint32_t round = 0;
            for (int j0 = 0; ok && j0 < units; j0 += XOPS, round ^= 1) {
#pragma unroll
                for (int u = 0; u < XOPS; ++u) {
                    if (!ok || j0 + u >= units)
                        break;
                    constexpr int kHalf = Sh::kX16 / 2 / 16;             // the second 64 k, in descriptor units
                    const uint64_t bx = x0 + static_cast<uint64_t>(u * (Sh::kX16 / 16));
                    const uint32_t a = tmem_base + 2 * MT + (u % OPS) * 64;
                    const int t = chunk & 1;
                    const uint32_t d = tmem_base + static_cast<uint32_t>(t * MT);
                    if (in_chunk == 0)
                        ok = __all_sync(0xFFFFFFFFu, mbar_wait_cluster(&aempty[t], ((chunk >> 1) & 1) ^ 1, p.timeout_ns, &flags[0]));
                    if (!ok)
                        break;
                    tc_fence_after();
                    if (leader) {
#pragma unroll
                        for (int kk = 0; kk < 4; ++kk)
                            tc_mma_f16_ts_pair(d, a + 8 * kk, bx + 2 * kk, Sh::kIdesc, (kk > 0 || in_chunk > 0) ? 1u : 0u);
                    }
                    const bool last = j0 + u + 1 == units;
                    uint64_t *next = &opfull[(u + 1) % XOPS];
                    const uint32_t next_phase = u + 1 < XOPS ? round : round ^ 1;
                    const bool ready = __all_sync(0xFFFFFFFFu, last || mbar_try_wait_cluster(next, next_phase));
                    const bool end = ++kb == nkb || in_chunk == kExactBlocks - 1;
                    if (leader) {
#pragma unroll
                        for (int kk = 0; kk < 4; ++kk)
                            tc_mma_f16_ts_pair(d, a + 32 + 8 * kk, bx + kHalf + 2 * kk, Sh::kIdesc, 1u);
                        // nobody waits for the last units, and the peer may be gone by then
                        if (j0 + u + OPS < units)
                            tc_commit_pair_multicast(&done[u % OPS], both);
                        if (end)
                            tc_commit_pair_multicast(&afull[t], both);
                    }
                    in_chunk = end ? 0 : in_chunk + 1;
                    chunk += end;
                    kb = kb == nkb ? 0 : kb;
                    if (!ready)
                        ok = __all_sync(0xFFFFFFFFu, mbar_wait_cluster(next, next_phase, p.timeout_ns, &flags[0]));
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
        } else {
            relay(0);
        }
    } else if (warp == Sh::kRelayWarp) {
        if (rank != 0)
            relay(1);
    } else if (warp < Sh::kFirstEpi) {
        // --------------------------------------------------------------- widen
        const int quarter = warp & 3, row = quarter * 32 + lane;
        const uint32_t lane_base = tmem_base + (static_cast<uint32_t>(quarter * 32) << 16) + 2 * MT;
        const XPiece piece(quarter * 4, lane, kHalfTokens);
        const uint32_t set = (warp - Sh::kFirstWiden) >> 2;
        const uint32_t opfull_there = map_shared_rank(smem_u32(opfull), first);
        bool ok = __all_sync(0xFFFFFFFFu, first_wait(x0full));
        for (uint32_t u = set; ok && u < AHEAD; u += kWidenSets) {
            piece.widen<kHalfTokens / 16>(sX0 + set * Sh::kX16 + u / kWidenSets * Sh::kRawX, sX16 + u * Sh::kX16, 16);
            fence_proxy_async_smem();
            __syncwarp();
        }
        if (ok && lane == 0)
            mbar_arrive(x0done);
        for (uint32_t u = set; ok && u < static_cast<uint32_t>(units); u += kWidenSets) {
            // Unit u - OPS is done, so W has its place in TMEM, and x of unit u + AHEAD =
            // u - OPS + XOPS its buffer.
            const uint32_t sl = u % S;
            ok = mbar_wait_cluster(&done[u % OPS], ((u / OPS) & 1) ^ 1, p.timeout_ns, &flags[0]) &&
                 mbar_wait(&full[sl], (u / S) & 1, p.timeout_ns, &flags[0]);
            ok = __all_sync(0xFFFFFFFFu, ok);            // the whole warp goes on, or none of it
            if (!ok)
                break;
            tc_fence_after();
            widen_row(sW + sl * kQ8WBytes, row, lane_base + u % OPS * 64);
            // (beyond the last unit: what is left in the ring, into a buffer that is not read)
            piece.widen<kHalfTokens / 16>(sXraw + sl * Sh::kRawX, sX16 + (u + AHEAD) % XOPS * Sh::kX16, 16);
            fence_proxy_async_smem();
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(&widened[u % XOPS]);
                if (rank == 0)
                    mbar_arrive(&opfull[u % XOPS]);      // W of this unit, and its x, widened before
                else
                    mbar_arrive_cluster(opfull_there + u % XOPS * 8);
            }
        }
        if (!ok)
            q8_fail(p.err, &flags[0], kErrTimeoutWiden);
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
                ok = __all_sync(0xFFFFFFFFu, mbar_wait_cluster(&afull[t], (chunk >> 1) & 1, p.timeout_ns, &flags[0]));
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
    __syncthreads();                     // from here on no role raises the abort flag any more
    // Abort: every copy lands before sums are read in the ring's place and before exit.
    if (warp == Sh::kTmaWarp && flags[0])
        wait_landed();
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

// skg_f8_wide.cu -- the projection of e4m3 rows by e4m3 weights for many tokens,
// or many of each expert: tcgen05 by pairs of CTAs.
//
//   y[m, n] = sum_b xs[m, b] ws[n / 128, b] sum_(k in block b) x[m, k] W[n, k]
//
// The arithmetic is that of skg_f8_split.cu.  Tokens are the MMA's M: a token a lane
// makes a unit's scale one number a thread, xs of its token times ws of the 128
// channels that its warp has.  Two forms:
//   PAIR = 1  a CTA computes 128 tokens x 128 channels, with four accumulators
//   PAIR = 2  two CTAs work as one (cta_group::2): 256 x 256, each with its 128 rows
//             of x (A), half of the rows of W (B) and its tokens' sums, 128 lanes x 256
//             columns; two accumulators take all of the SM's tensor memory
// Persistent over tiles, or, where those are fewer than the SMs, with K split over
// the CTAs or pairs of a cluster, joined as in skg_f8_split.cu.
//
// Roles of a CTA (one per SM):
//   1 + 1     TMA; TMEM and, in the first CTA of a pair, MMA issue for both
//   8 warps   accumulators into registers; at a tile's end the next tile's first
//             scales are requested, then residual, rounding and store, while that
//             tile's first units are computed
// An epilogue thread of a pair holds 128 sums and 64 more on their way from tensor
// memory, so the first warpgroup gives up registers (56 a thread, 224 for the others).
//
// What bounds it.  A unit of 128 k is 512 cycles of an SM's MMAs; without the epilogue's
// additions it takes 650 (operands are written to and read from shared memory at
// 100 bytes a cycle), with them 780: all 128 x 256 sums go through the registers
// once a unit, and the accumulator is free again only when they have.  Measured:
// 4096 x 12288 x 7168 269-301 us (2.4 to 2.7 PFLOP/s; cuBLAS reaches 1.96 in bf16), of which
// 8% is the last of 10.1 waves; 1024 x 7168 x 7168 52 us; 16384 rows of 32 experts,
// 4096 x 4096, 268-313 us; by tiles of 128: 128 x 7168 x 7168 17.0 us (K split in 2; 22 unsplit),
// 256 x 4096 x 4096 12.8, 333 x 5001 x 4112 20.1 (rows that begin 16 bytes off a line:
// 16 with K = 4096), 2048 rows of 32 experts, 4096 x 4096, 108 (5.0 TB/s of weights).
// Steps at 4096 x 4864 x 7168, now 105 us (with, and without it at that step):
//   sums added two at a time by fma.rn.f32x2            116, 111
//   scales requested 2, 4, 8 units ahead                150, 124, 116 (6: 113 where 8 spill)
//   scales brought to shared memory by two warps        111, 111
//   outputs stored by each lane, 8 bytes at a time      134, 116
//   the next tile's scales requested after the store    113, 105
//   16 epilogue warps of 64 columns, scales 2 ahead     154, 134
//   MMAs of half a unit, each with its own barriers     126, 128 (x is read twice)
//   waits that poll without a pause                     136, 126
// Outputs copied by the copy engine out of 68 KB of shared memory (4 stages instead of 5)
// took the same time, and tiles of 128 longer.
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

template <int PAIR>
struct WideShape {
    static constexpr int MT = 128 * PAIR, NT = 128 * PAIR;   // tokens and channels of a tile
    static constexpr int kEpiWarps = 8;
    static constexpr int kCols = NT * 4 / kEpiWarps;         // accumulator columns of an epilogue thread
    static_assert(kF8Block % kCols == 0, "one scale of W a thread");
    static constexpr int kMmaWarp = 0, kTmaWarp = 1, kFirstEpi = 4;          // two warps of the first warpgroup are idle
    static constexpr int kThreads = 32 * (kFirstEpi + kEpiWarps);
    // Registers: the launch has 3 warpgroups of 168 a thread.
    static constexpr int kRegsFew = 56, kRegsMany = 224;
    static_assert(kRegsFew + 2 * kRegsMany <= 3 * 168 && kThreads == 3 * 128, "no more than the launch has");
    static constexpr int kStages = 5;
    static constexpr int kAcc = 512 / NT;                    // accumulators in flight
    static constexpr uint32_t kTmemCols = 512;
    static constexpr uint32_t kStage = 2 * kF8TileBytes;     // a CTA's x and W of a unit
    static constexpr uint32_t kIdesc = idesc_e4m3_f32(MT, NT);
    static constexpr int kBars = 2 * kStages + 2 * kAcc + 1;
    static constexpr int kOut = 32 * 128;                    // a warp's part of the output on its way: 32 rows of 128 bytes
    static constexpr int kSmem = 1024 + kStages * kStage + kEpiWarps * kOut + kBars * 8 + 16;
    static_assert(kStages * kStage >= 128 * NT * 4, "the sums take the ring's place");
    static_assert(kSmem + f8_table_bytes(kF8MaxExperts) <= 227 * 1024, "shared memory of a CTA");
};

// A warp's 32 rows (tokens from m0 on, a lane each; the outputs are those of lanes lo
// to hi) of NC channels from n0 (the outputs are those from na on), by way of shared
// memory, so that a store's lanes cover rows: of 128 bytes at a time, bf16 or,
// where more is to be added, fp32.  (Each lane storing its own row in pieces of 8
// bytes took 8 us a tile.)  16-byte pieces are swizzled by row.
template <int EPI, int NC>
__device__ __forceinline__ void store_tile(const F8LinearParams &p, int m0, int lo, int hi, int n0, int na, const float (&acc)[NC],
                                           uint8_t *out)
{
    constexpr int W = EPI == SKG_EPI_BF16 ? 64 : 32;             // channels at a time
    const int lane = static_cast<int>(threadIdx.x) & 31;
    if (hi <= 0 || lo >= 32)
        return;
    auto piece = [&](int row, int c) { return out + row * 128 + ((c ^ (row & 7)) << 4); };
#pragma unroll
    for (int c0 = 0; c0 < NC; c0 += W) {
        const int n = n0 + c0, least = na - n, valid = p.N - n;  // channels n + least to n + valid
        if (valid <= 0 || least >= W)
            continue;
        __syncwarp();
#pragma unroll
        for (int c = 0; c < 8; ++c) {
            uint32_t w[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if constexpr (EPI == SKG_EPI_BF16) {
                    w[i] = two_bf16(acc[c0 + 8 * c + 2 * i], acc[c0 + 8 * c + 2 * i + 1]);
                } else {
                    w[i] = __float_as_uint(acc[c0 + 4 * c + i]);
                }
            }
            *reinterpret_cast<uint4 *>(piece(lane, c)) = make_uint4(w[0], w[1], w[2], w[3]);
        }
        __syncwarp();
        if (p.vec) {                     // pieces of the output are aligned, and N ends between two
            const int c = lane & 7;
            const bool in = c * (W / 8) >= least && c * (W / 8) < valid;
#pragma unroll
            for (int r0 = 0; r0 < 32; r0 += 4) {
                const int r = r0 + (lane >> 3);
                const uint4 v = *reinterpret_cast<const uint4 *>(piece(r, c));
                if (!in || r < lo || r >= hi)
                    continue;
                const size_t o = static_cast<size_t>(m0 + r) * p.N + n + c * (W / 8);
                if constexpr (EPI == SKG_EPI_BF16_RESIDUAL) {
                    const uint2 b = __ldcg(reinterpret_cast<const uint2 *>(p.res + o));
                    const float s0 = __uint_as_float(v.x) + bf16lo(b.x), s1 = __uint_as_float(v.y) + bf16hi(b.x);
                    const float s2 = __uint_as_float(v.z) + bf16lo(b.y), s3 = __uint_as_float(v.w) + bf16hi(b.y);
                    *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(p.y) + o) =
                        make_uint2(two_bf16(s0, s1), two_bf16(s2, s3));
                } else if constexpr (EPI == SKG_EPI_FP32) {
                    *reinterpret_cast<uint4 *>(static_cast<float *>(p.y) + o) = v;
                } else {
                    *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(p.y) + o) = v;
                }
            }
        } else {
#pragma unroll 4
            for (int r = max(lo, 0); r < min(hi, 32); ++r) {
#pragma unroll
                for (int c = lane; c < W; c += 32) {
                    if (c < least || c >= valid)
                        continue;
                    const size_t o = static_cast<size_t>(m0 + r) * p.N + n + c;
                    if constexpr (EPI == SKG_EPI_BF16) {
                        static_cast<uint16_t *>(p.y)[o] = *reinterpret_cast<const uint16_t *>(piece(r, c >> 3) + 2 * (c & 7));
                    } else {
                        float v = *reinterpret_cast<const float *>(piece(r, c >> 2) + 4 * (c & 3));
                        if (EPI == SKG_EPI_BF16_RESIDUAL)
                            static_cast<uint16_t *>(p.y)[o] = f32_to_bf16(v + bf16_to_f32(__ldcg(p.res + o)));
                        else
                            static_cast<float *>(p.y)[o] = v;
                    }
                }
            }
        }
    }
}

template <int PAIR>
__global__ void __launch_bounds__(WideShape<PAIR>::kThreads, 1)
f8_wide_kernel(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmX, const F8LinearParams p)
{
    using Sh = WideShape<PAIR>;
    constexpr int MT = Sh::MT, NT = Sh::NT, S = Sh::kStages, NA = Sh::kAcc, NC = Sh::kCols;

    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    uint8_t *sX = smem, *sW = smem + S * kF8TileBytes;
    uint64_t *full = reinterpret_cast<uint64_t *>(smem + S * Sh::kStage + Sh::kEpiWarps * Sh::kOut);
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
    // A cluster is p.split CTAs or pairs, each with its part of K.  With more than
    // one there is a cluster for each tile.
    const int rank = static_cast<int>(blockIdx.x) % PAIR, part = static_cast<int>(blockIdx.x) / PAIR % p.split;
    const int first = static_cast<int>(blockIdx.x) / (PAIR * p.split), step = static_cast<int>(gridDim.x) / (PAIR * p.split);
    const int lead = part * PAIR;        // the pair's first CTA, in the cluster
    const int kb0 = part * p.nkb / p.split, units = (part + 1) * p.nkb / p.split - kb0;

    if (threadIdx.x == 0) {
        tma_prefetch_desc(&tmW);
        tma_prefetch_desc(&tmX);
        for (int i = 0; i < S; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], 1);
        }
        for (int i = 0; i < NA; ++i) {
            mbar_init(&afull[i], 1);
            mbar_init(&aempty[i], PAIR * Sh::kEpiWarps);
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
    if (warp == Sh::kMmaWarp) {
        if constexpr (PAIR == 2) {
            tmem_alloc_pair(tmem_slot, Sh::kTmemCols);
            tmem_relinquish_pair();
        } else {
            tmem_alloc(tmem_slot, Sh::kTmemCols);
            tmem_relinquish();
        }
    }
    tc_fence_before();
    cluster_sync();                      // the peer's barriers exist before anything is sent there
    tc_fence_after();
    constexpr uint32_t tmem_base = 0;    // all 512 columns are this CTA's
    // Of a pair, both CTAs' copies, MMAs and epilogues arrive at these barriers (at full and
    // aempty in the first CTA, at empty and afull by the MMA's commits to both), so a
    // wait acquires at cluster scope: at the CTA's it would order nothing of the peer's
    // before what follows it, such as the MMA that overwrites an accumulator that
    // the peer has read.
    auto wait = [&](uint64_t *bar, uint32_t parity) {
        if constexpr (PAIR == 2)
            return mbar_wait_cluster(bar, parity, p.timeout_ns, &flags[0]);
        else
            return mbar_wait(bar, parity, p.timeout_ns, &flags[0]);
    };
    if (warp != Sh::kTmaWarp)            // the bounded waits do not count the previous kernel's time
        pdl_wait();

    if (warp < Sh::kFirstEpi) {
        regs_dec<Sh::kRegsFew>();
        if (warp == Sh::kTmaWarp) {
            // -------------------------------------------------------- TMA producer
            const bool leader = elect_one();
            const uint64_t pol = policy_evict_normal();
            const uint32_t full0 = map_shared_rank(smem_u32(full), lead);
            auto load = [&](uint8_t *ring, int u, const CUtensorMap *m, int kb, int row) {
                if constexpr (PAIR == 2)
                    tma_load_2d_pair(ring + u % S * kF8TileBytes, m, full0 + u % S * 8, (kb0 + kb) * kF8Block, row, pol);
                else
                    tma_load_2d(ring + u % S * kF8TileBytes, m, &full[u % S], (kb0 + kb) * kF8Block, row, pol);
            };
            auto load_w = [&](int u, const F8Tile &t, int kb) {
                if (rank == 0)           // for both CTAs' copies, which may be counted before
                    mbar_arrive_expect_tx(&full[u % S], PAIR * (p.w_box + p.x_box) * kF8Block);
                load(sW, u, &tmW, kb, f8_w_window(p, t.e, t.nt * NT + rank * 128));
            };
            auto load_x = [&](int u, const F8Tile &t, int kb) { load(sX, u, &tmX, kb, f8_x_window(p, t.m0 + rank * 128)); };
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
                    ok = __all_sync(0xFFFFFFFFu, wait(&empty[j % S], ((j / S) & 1) ^ 1));
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
        } else if (warp == Sh::kMmaWarp) {
            // ---------------------------------------------------------- MMA issuer
            if (rank == 0) {
                const bool leader = elect_one();
                const uint64_t w0 = smem_desc_kmajor_sw128(smem_u32(sW)), x0 = smem_desc_kmajor_sw128(smem_u32(sX));
                const int total = ((tiles - first + step - 1) / step) * units;
                auto commit = [&](uint64_t *bar) {
                    if constexpr (PAIR == 2)
                        tc_commit_pair_multicast(bar, static_cast<uint16_t>(3 << lead));
                    else
                        tc_commit(bar);
                };
                bool ok = true;
                int sl = 0, phase = 0;
                for (int j = 0; j < total; ++j) {
                    const int t = j % NA;
                    ok = wait(&aempty[t], ((j / NA) & 1) ^ 1) && wait(&full[sl], phase);
                    ok = __all_sync(0xFFFFFFFFu, ok);
                    if (!ok)
                        break;
                    tc_fence_after();
                    if (leader) {
                        const uint64_t a = x0 + static_cast<uint64_t>(sl * (kF8TileBytes / 16));
                        const uint64_t b = w0 + static_cast<uint64_t>(sl * (kF8TileBytes / 16));
#pragma unroll
                        for (int kk = 0; kk < 4; ++kk) {
                            if constexpr (PAIR == 2)
                                tc_mma_f8_pair(tmem_base + t * NT, a + 2 * kk, b + 2 * kk, Sh::kIdesc, kk > 0);
                            else
                                tc_mma_f8(tmem_base + t * NT, a + 2 * kk, b + 2 * kk, Sh::kIdesc, kk > 0);
                        }
                        // nobody waits for the last units' slots, and the peer's producer may be gone by then
                        if (j + S < total)
                            commit(&empty[sl]);
                        commit(&afull[t]);
                    }
                    __syncwarp();
                    if (++sl == S) {
                        sl = 0;
                        phase ^= 1;
                    }
                }
                if (!ok) {                   // abort: wait for the MMAs already issued before TMEM is freed
                    f8_fail(p.err, &flags[0], kErrTimeoutMma);
                    if (leader) {
                        if constexpr (PAIR == 2)
                            tc_commit_pair(drain);
                        else
                            tc_commit(drain);
                    }
                    volatile int never = 0;
                    mbar_wait(drain, 0, kDefaultTimeoutNs, &never);
                }
            }
        }
    } else {
        regs_inc<Sh::kRegsMany>();
        // ------------------------------------------------------------ epilogue
        pdl_launch_dependents();         // not sooner: see skg_q8_stream.cu
        const int ew = warp - Sh::kFirstEpi;
        const int col0 = (ew >> 2) * NC, row0 = (warp & 3) * 32;
        uint8_t *out = smem + S * Sh::kStage + ew * Sh::kOut;
        const uint32_t lane_base = tmem_base + (static_cast<uint32_t>((warp & 3) * 32) << 16) + static_cast<uint32_t>(col0);
        const uint32_t aempty0 = map_shared_rank(smem_u32(aempty), lead);
        constexpr int AHEAD = 6;
        bool ok = true;
        int j = 0;
        float w[AHEAD], x[AHEAD];
        const float *ws, *xs;
        bool live;
        F8Tile t;
        // A tile's scales, from its first units' on: of the next tile they are on their
        // way while the outputs of this one are stored.
        auto begin = [&](int tile) {
            t = f8_tile(p, MT, table, tile);
            // this CTA's tokens are ma to mb, the window's from m0 on
            const int ma = t.m0 + rank * 128, mb = min(t.m1, ma + 128);
            const int m = f8_x_window(p, ma) + row0 + lane, nb = t.nt * (NT / kF8Block) + col0 / kF8Block;
            live = m >= ma && m < mb && nb < p.nb;
            ws = p.w_scale + (static_cast<size_t>(t.e) * p.nb + nb) * p.nkb + kb0;
            xs = p.x_scale + static_cast<size_t>(m) * p.nkb + kb0;
#pragma unroll
            for (int i = 0; i < AHEAD; ++i) {
                w[i] = live && i < units ? __ldcg(ws + i) : 0.0f;
                x[i] = live && i < units ? __ldca(xs + i) : 0.0f;
            }
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
                    const float s = x[i] * w[i];
                    const bool more = live && kb + i + AHEAD < units;
                    w[i] = more ? __ldcg(ws + kb + i + AHEAD) : 0.0f;
                    x[i] = more ? __ldca(xs + kb + i + AHEAD) : 0.0f;
                    const int a = j % NA;
                    ok = __all_sync(0xFFFFFFFFu, wait(&afull[a], (j / NA) & 1));
                    if (!ok)
                        break;
                    tc_fence_after();
                    f8_add_unit(acc, lane_base + static_cast<uint32_t>(a * NT), s, [&] {
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0)
                            mbar_arrive_cluster(aempty0 + a * 8);
                    });
                    ++j;
                }
            }
            if (!ok)
                break;
            const int na = t.nt * NT + col0 / kF8Block * kF8Block, n0 = f8_w_window(p, t.e, na) - t.e * p.N + col0 % kF8Block;
            const int ma = t.m0 + rank * 128, m0 = f8_x_window(p, ma), lo = ma - m0 - row0, hi = min(t.m1, ma + 128) - m0 - row0;
            if (tile + step < tiles)
                begin(tile + step);
            if (p.split > 1) {
                // in the ring's place: the last MMA has read its operands
#pragma unroll
                for (int c = 0; c < NC; c += 4)
                    *reinterpret_cast<float4 *>(smem + f8_sum_at(NT, row0 + lane, col0 + c)) =
                        make_float4(acc[c], acc[c + 1], acc[c + 2], acc[c + 3]);
            } else if (p.epilogue == SKG_EPI_FP32)
                store_tile<SKG_EPI_FP32, NC>(p, m0 + row0, lo, hi, n0, na, acc, out);
            else if (p.epilogue == SKG_EPI_BF16_RESIDUAL)
                store_tile<SKG_EPI_BF16_RESIDUAL, NC>(p, m0 + row0, lo, hi, n0, na, acc, out);
            else
                store_tile<SKG_EPI_BF16, NC>(p, m0 + row0, lo, hi, n0, na, acc, out);
        }
        if (!ok)
            f8_fail(p.err, &flags[0], kErrTimeoutEpilogue);
    }

    __syncwarp();
    tc_fence_before();
    __syncthreads();                     // from here on no role raises the abort flag any more
    // Abort: every copy lands before sums are read in the ring's place and before exit.  (By
    // time: the second CTA's copies are counted in the first, whose abort that one
    // learns of as its accumulators stay away.)
    if (warp == Sh::kTmaWarp && flags[0])
        wait_landed();
    if (p.split > 1) {
        const F8Tile t = f8_tile(p, MT, table, first);
        const int ma = t.m0 + rank * 128;
        int n0[PAIR], na[PAIR];
#pragma unroll
        for (int b = 0; b < PAIR; ++b) {
            na[b] = t.nt * NT + b * kF8Block;
            n0[b] = f8_w_window(p, t.e, na[b]) - t.e * p.N;
        }
        f8_join<kF8WideMaxSplit, Sh::kThreads, PAIR>(p, smem_u32(smem), f8_x_window(p, ma), ma, min(t.m1, ma + 128), n0, na, part, rank, PAIR);
    } else if (PAIR == 2) {
        cluster_sync();                  // no CTA leaves while its peer may still send to it
    }
    if (warp == Sh::kMmaWarp) {
        tc_fence_after();
        if constexpr (PAIR == 2)
            tmem_dealloc_pair(tmem_base, Sh::kTmemCols);
        else
            tmem_dealloc(tmem_base, Sh::kTmemCols);
    }
}

template <int PAIR>
cudaError_t launch_shape(const CUtensorMap &tmW, const CUtensorMap &tmX, const F8LinearParams &p, int grid, cudaStream_t s)
{
    using Sh = WideShape<PAIR>;
    static int attr_set[kMaxDevices] = {};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess)
        return e;
    if (dev >= kMaxDevices)
        return cudaErrorInvalidDevice;
    if (__atomic_load_n(&attr_set[dev], __ATOMIC_ACQUIRE) == 0) {
        e = cudaFuncSetAttribute(f8_wide_kernel<PAIR>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 Sh::kSmem + f8_table_bytes(kF8MaxExperts));
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
    attr[1].val.clusterDim.x = static_cast<unsigned>(PAIR * p.split);
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, f8_wide_kernel<PAIR>, tmW, tmX, p);
}

template <int PAIR>
F8TcShape shape_of(int experts)
{
    using Sh = WideShape<PAIR>;
    return {Sh::MT, 1, Sh::kSmem + f8_table_bytes(experts), Sh::kThreads, Sh::kStages};
}

} // namespace

F8TcShape f8_wide_shape(int m_tile, int experts) { return m_tile == 256 ? shape_of<2>(experts) : shape_of<1>(experts); }

cudaError_t launch_f8_wide(const CUtensorMap &tmW, const CUtensorMap &tmX, const F8LinearParams &p, int m_tile, int grid,
                           cudaStream_t s)
{
    return m_tile == 256 ? launch_shape<2>(tmW, tmX, p, grid, s) : launch_shape<1>(tmW, tmX, p, grid, s);
}

} // namespace skg

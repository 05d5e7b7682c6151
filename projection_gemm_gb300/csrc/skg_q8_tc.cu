// skg_q8_tc.cu -- the 8-bit projection on the tensor cores.
//
// sm_103a has no integer kind of tcgen05.mma, and 8-bit integers are exact in
// fp16, as are their products (at most 2^14) and, in fp32, sums of up to 1024
// such products (at most 2^24).  So the integers are widened to fp16 on chip,
// multiplied with kind::f16 from a fresh accumulator every 1024 k, and the
// accumulators are added as int32: the exact integer sum, in any order and for
// any split of K.
//
// Tiles (swap-AB): 128 rows of W are the MMA's M, MT tokens its N.  Work is cut
// into units (tile, 128 k): whole waves of tiles first, one tile per CTA, then
// the units of the tiles that are left, cut evenly over the CTAs whatever tile
// they fall in.  A tile that several CTAs share is summed by integer atomics in
// the plan's workspace; the last CTA to arrive stores it and leaves the
// workspace at zero again.
//
// Roles of a CTA:
//   warps 0..3      widen: a thread reads its W row's 128 bytes of a k-block
//                   from the TMA ring, writes it as fp16 to its TMEM lane (the
//                   MMA's A operand); for M <= 64 (not WIDE) the same warps
//                   widen the x tile into shared memory (the B operand)
//   warps 4..       epilogue: TMEM accumulators to int32 registers, then
//                   scaling, residual, rounding and the store
//   then            one warp for TMA, one that issues the MMAs
// WIDE (M > 64): x was widened to fp16 in the plan's workspace before this
// kernel, since every CTA would repeat it, and arrives by TMA as the B operand.
//
// Every wait is bounded; on expiry a thread records the timeout in the plan's
// error word, raises the CTA's abort flag, waits for its own copies and MMAs,
// and the CTA frees its TMEM and returns.
#include <algorithm>

#include "skg_internal.h"
#include "skg_ptx.cuh"
#include "skg_q8_common.cuh"
#include "skg_q8_internal.h"

namespace skg {
namespace {

constexpr int kQ8BlockK = 128;                       // k of one unit: 128 bytes of a W row
constexpr int kExactBlocks = 1024 / kQ8BlockK;       // units summed by the MMA from a fresh accumulator
constexpr int kWidenSets = 2;                        // sets of 4 warps, on alternate units
constexpr int kWidenWarps = 4 * kWidenSets;
constexpr uint32_t kQ8WBytes = kTileN * kQ8BlockK;   // 16 KB

template <int MT, bool WIDE>
struct Q8Shape {
    static constexpr int kEpiWarps = WIDE ? MT / 16 : (MT == 32 ? 4 : 8);
    static constexpr int kCols = MT * 4 / kEpiWarps;         // accumulator columns of an epilogue thread
    static constexpr int kThreads = 32 * (kWidenWarps + kEpiWarps + 2);
    static constexpr int kTmaWarp = kWidenWarps + kEpiWarps;
    static constexpr int kMmaWarp = kTmaWarp + 1;
    static constexpr int kCtas = WIDE ? 1 : 2;               // per SM
    static constexpr int kStages = WIDE ? 4 : (MT == 32 ? 4 : 3);   // W (and int8 x) ring
    static constexpr int kXStages = WIDE ? (MT > 128 ? 3 : 4) : 0;                   // fp16 x ring (WIDE)
    static constexpr int kOps = WIDE && MT <= 128 ? 4 : (MT == 32 ? 3 : 2);          // widened operand buffers
    static_assert(kStages >= kOps && kOps >= kWidenSets, "the widen warps' waits need this");
    static constexpr uint32_t kRawX = WIDE ? 0 : MT * kQ8BlockK;
    static constexpr uint32_t kX16 = MT * kQ8BlockK * 2;     // fp16 x of one k-block: two 64-wide halves
    static constexpr uint32_t kTmemCols = 2 * MT + kOps * 64 <= 256 ? 256 : 512;
    static constexpr uint32_t kIdesc = idesc_f16_f32(kTileN, MT);
    static constexpr int kBars = 2 * kStages + 2 * kXStages + 2 * kOps + 5;
    static constexpr int kSmem = 1024 + kStages * (kQ8WBytes + kRawX) + (WIDE ? kXStages : kOps) * kX16 + kBars * 8 + 48;
};

// The segments of one CTA in order: whole tiles, then its share of the rest.
struct Q8Segment {
    int tile, kb0, kb1;
};

struct Q8Walk {
    int i, u, end;
    __device__ __forceinline__ Q8Walk(const Q8TcParams &p, int cta) : i(0), u(0), end(0)
    {
        if (cta < p.rem_ctas) {
            u = static_cast<int>(static_cast<long long>(cta) * p.rem_units / p.rem_ctas);
            end = static_cast<int>(static_cast<long long>(cta + 1) * p.rem_units / p.rem_ctas);
        }
    }
    __device__ __forceinline__ bool next(const Q8TcParams &p, int cta, Q8Segment &s)
    {
        if (i < p.full) {
            s = {i * static_cast<int>(gridDim.x) + cta, 0, p.nkb};
            ++i;
            return true;
        }
        if (u >= end)
            return false;
        const int t = u / p.nkb;
        s.tile = p.full * static_cast<int>(gridDim.x) + t;
        s.kb0 = u - t * p.nkb;
        s.kb1 = min(p.nkb, s.kb0 + end - u);
        u += s.kb1 - s.kb0;
        return true;
    }
};

// Tiles in bands of p.band token tiles: within a band, token tiles fastest, so
// that the CTAs of a wave share a compact block of x and W in L2.
__device__ __forceinline__ void tile_at(const Q8TcParams &p, int tile, int &nt, int &mt)
{
    const int per_band = p.band * p.n_tiles;
    const int b = tile / per_band, r = tile - b * per_band;
    const int wide = min(p.band, p.m_tiles - b * p.band);
    nt = r / wide;
    mt = b * p.band + r - nt * wide;
}

__device__ __forceinline__ void q8_fail(const Q8TcParams &p, volatile int *abort, unsigned bit)
{
    *abort = 1;
    if (p.err)
        atomicOr(p.err, bit);
}

__device__ __forceinline__ void widen16(const uint4 &v, uint32_t *r)
{
    widen4(v.x, r[0], r[1]);
    widen4(v.y, r[2], r[3]);
    widen4(v.z, r[4], r[5]);
    widen4(v.w, r[6], r[7]);
}

template <int THREADS>
__device__ __forceinline__ void q8_epi_sync()
{
    asm volatile("bar.sync 1, %0;" :: "n"(THREADS) : "memory");
}

template <int THREADS>
__device__ __forceinline__ bool q8_epi_and(bool v)
{
    uint32_t out;
    asm volatile("{\n\t.reg .pred pi, po;\n\t"
                 "setp.ne.u32 pi, %1, 0;\n\t"
                 "bar.red.and.pred po, 1, %2, pi;\n\t"
                 "selp.u32 %0, 1, 0, po;\n\t}"
                 : "=r"(out) : "r"(v ? 1u : 0u), "n"(THREADS) : "memory");
    return out != 0;
}

// NC outputs (tokens m0...) of one channel n from their sums, 4 at a time so
// that their loads are in flight together and few registers hold them.
template <int EPI, int NC>
__device__ __forceinline__ void store_columns_as(const Q8LinearParams &g, int m0, int n, const int (&acc)[NC])
{
    const int valid = g.M - m0;
    const float ws = __ldcg(g.w_scale + n);
    const float *xsp = g.x_scale + m0;
    size_t at = static_cast<size_t>(m0) * g.N + n;
#pragma unroll
    for (int c0 = 0; c0 < NC; c0 += 4) {
        float v[4];
#pragma unroll
        for (int c = 0; c < 4; ++c)
            v[c] = c0 + c < valid ? q8_scaled(acc[c0 + c], __ldcg(xsp + c0 + c), ws) : 0.0f;
        if (EPI == SKG_EPI_BF16_RESIDUAL) {
            const uint16_t *r = g.res + at;
            uint16_t b[4];
#pragma unroll
            for (int c = 0; c < 4; ++c, r += g.N)
                b[c] = c0 + c < valid ? __ldcg(r) : 0;
#pragma unroll
            for (int c = 0; c < 4; ++c)
                v[c] = __fadd_rn(v[c], bf16_to_f32(b[c]));
        }
#pragma unroll
        for (int c = 0; c < 4; ++c, at += g.N) {
            if (c0 + c < valid) {
                if (EPI == SKG_EPI_FP32)
                    static_cast<float *>(g.y)[at] = v[c];
                else
                    static_cast<uint16_t *>(g.y)[at] = f32_to_bf16(v[c]);
            }
        }
    }
}

template <int NC>
__device__ __forceinline__ void store_columns(const Q8LinearParams &g, int m0, int n, const int (&acc)[NC])
{
    if (n >= g.N || m0 >= g.M)
        return;
    if (g.epilogue == SKG_EPI_FP32)
        store_columns_as<SKG_EPI_FP32>(g, m0, n, acc);
    else if (g.epilogue == SKG_EPI_BF16_RESIDUAL)
        store_columns_as<SKG_EPI_BF16_RESIDUAL>(g, m0, n, acc);
    else
        store_columns_as<SKG_EPI_BF16>(g, m0, n, acc);
}

// 16 accumulator columns of this thread's TMEM lane as integers (they are
// integers below 2^24 in fp32: the conversion is exact).
__device__ __forceinline__ void load_sums(uint32_t taddr, int (&v)[16])
{
    uint32_t r[2][8];
    tmem_ld_x8(taddr, r[0]);
    tmem_ld_x8(taddr + 8, r[1]);
    tmem_wait_ld();
#pragma unroll
    for (int c = 0; c < 16; ++c) {
        asm volatile("" : "+r"(r[c >> 3][c & 7]));
        v[c] = __float2int_rn(__uint_as_float(r[c >> 3][c & 7]));
    }
}

// A thread's 16 columns of a slot ([m_tile][128] int32; a warp covers 32
// consecutive channels of a column).
__device__ __forceinline__ void put_sums(int *slot, int valid, const int (&v)[16])
{
#pragma unroll
    for (int c = 0; c < 16; ++c)
        if (c < valid)
            __stcg(slot + c * kTileN, v[c]);
}

// Four neighbouring channels of one token.
__device__ __forceinline__ void store_four(const Q8LinearParams &g, int m, int n, const int4 &v)
{
    const float xs = __ldcg(g.x_scale + m);
    const int s[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i)
        if (n + i < g.N)
            q8_store(g, m, n + i, s[i], xs, __ldcg(g.w_scale + n + i));
}

// The sum of a shared tile's slots, by all threads of the CTA that arrived
// last: CTA `first` holds the tile's first units in its slot 1, the others
// theirs in slot 0.  Eight 16-byte loads of a thread are in flight together.
template <int MT, int THREADS>
__device__ __forceinline__ void finish_tile(const Q8TcParams &p, int m0, int n0, int first, int last)
{
    const int items = min(MT, p.g.M - m0) * (kTileN / 4);
    const int4 *base = reinterpret_cast<const int4 *>(p.ws);
    const int4 zero = make_int4(0, 0, 0, 0);
    for (int i0 = threadIdx.x; i0 < items; i0 += 2 * THREADS) {
        int4 sum[2] = {zero, zero};
        for (int c0 = first; c0 <= last; c0 += 4) {
            int4 v[4][2];
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                const int4 *slot = base + static_cast<size_t>(2 * (c0 + c) + (c0 + c == first)) * (MT * kTileN / 4);
#pragma unroll
                for (int h = 0; h < 2; ++h)
                    v[c][h] = c0 + c <= last && i0 + h * THREADS < items ? __ldcg(slot + i0 + h * THREADS) : zero;
            }
#pragma unroll
            for (int c = 0; c < 4; ++c)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    sum[h].x += v[c][h].x;
                    sum[h].y += v[c][h].y;
                    sum[h].z += v[c][h].z;
                    sum[h].w += v[c][h].w;
                }
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int i = i0 + h * THREADS;
            if (i < items)
                store_four(p.g, m0 + i / (kTileN / 4), n0 + i % (kTileN / 4) * 4, sum[h]);
        }
    }
}

template <int MT, bool WIDE>
__global__ void __launch_bounds__(Q8Shape<MT, WIDE>::kThreads, Q8Shape<MT, WIDE>::kCtas)
q8_tc_kernel(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmX, const Q8TcParams p)
{
    using Sh = Q8Shape<MT, WIDE>;
    constexpr int S = Sh::kStages, SX = Sh::kXStages, OPS = Sh::kOps;

    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    uint8_t *sW = smem;
    uint8_t *sXraw = sW + S * kQ8WBytes;
    uint8_t *sX16 = sXraw + S * Sh::kRawX;
    uint64_t *wfull = reinterpret_cast<uint64_t *>(sX16 + (WIDE ? SX : OPS) * Sh::kX16);
    uint64_t *wempty = wfull + S;
    uint64_t *opfull = wempty + S;
    uint64_t *opempty = opfull + OPS;
    uint64_t *afull = opempty + OPS;     // [2] accumulators
    uint64_t *aempty = afull + 2;        // [2]
    uint64_t *drain = aempty + 2;        // [1]
    uint64_t *xfull = drain + 1;         // [SX]
    uint64_t *xempty = xfull + SX;       // [SX]
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(xempty + SX);
    volatile int *flags = reinterpret_cast<volatile int *>(tmem_slot + 1);  // [0] abort, [1] tiles to finish
    volatile int *finish = flags + 2;    // [2] x (tile, first CTA, last CTA)

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int cta = static_cast<int>(blockIdx.x);
    if (threadIdx.x == 0) {
        tma_prefetch_desc(&tmW);
        tma_prefetch_desc(&tmX);
        for (int i = 0; i < S; ++i) {
            mbar_init(&wfull[i], 1);
            mbar_init(&wempty[i], 4);
        }
        for (int i = 0; i < OPS; ++i) {
            mbar_init(&opfull[i], 4);
            mbar_init(&opempty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&afull[i], 1);
            mbar_init(&aempty[i], Sh::kEpiWarps);
        }
        for (int i = 0; i < SX; ++i) {
            mbar_init(&xfull[i], 1);
            mbar_init(&xempty[i], 1);
        }
        mbar_init(drain, 1);
        flags[0] = 0;
        flags[1] = 0;
        fence_mbar_init();
    }
    __syncthreads();
    pdl_launch_dependents();
    uint32_t tmem_base = 0;
    if (warp != Sh::kTmaWarp) {          // the TMA warp needs no TMEM: its first copies leave at once
        if (warp == Sh::kMmaWarp) {
            tmem_alloc(tmem_slot, Sh::kTmemCols);
            tmem_relinquish();
        }
        tc_fence_before();
        asm volatile("bar.sync 2, %0;" :: "n"(Sh::kThreads - 32) : "memory");
        tc_fence_after();
        tmem_base = *tmem_slot;
    }
    Q8Walk walk(p, cta);
    const int blocks = p.full * p.nkb + (walk.end - walk.u);     // k-blocks of this CTA

    if (warp == Sh::kTmaWarp) {
        // -------------------------------------------------------- TMA producer
        if (lane == 0 && blocks > 0) {
            // W passes once where one token tile holds all of M
            const uint64_t pol_w = p.m_tiles == 1 ? policy_evict_first() : policy_evict_normal();
            const uint64_t pol_x = p.m_tiles == 1 ? policy_evict_last() : policy_evict_normal();
            Q8Segment s;
            int j = 0, ahead = 0, issued_w = 0, issued_x = 0;
            bool ok = true;
            if (p.static_w) {            // weights may be requested before the wait for the previous kernel
                Q8Walk first(p, cta);
                while (ahead < S && first.next(p, cta, s)) {
                    int nt, mt;
                    tile_at(p, s.tile, nt, mt);
                    for (int kb = s.kb0; kb < s.kb1 && ahead < S; ++kb, ++ahead) {
                        mbar_arrive_expect_tx(&wfull[ahead], kQ8WBytes + Sh::kRawX);
                        tma_load_2d(sW + ahead * kQ8WBytes, &tmW, &wfull[ahead], kb * kQ8BlockK, nt * kTileN, pol_w);
                    }
                }
                issued_w = ahead;
                // ... and the rest of this CTA's weights from HBM into L2, up to p.ahead units
                int asked = 0;
                if (ahead == S) {
                    Q8Walk rest(p, cta);
                    int skip = ahead;
                    while (asked < p.ahead && rest.next(p, cta, s)) {
                        int nt, mt;
                        tile_at(p, s.tile, nt, mt);
                        int kb = s.kb0 + min(skip, s.kb1 - s.kb0);
                        skip -= kb - s.kb0;
                        for (; kb < s.kb1 && asked < p.ahead; ++kb, ++asked)
                            tma_prefetch_l2_2d(&tmW, kb * kQ8BlockK, nt * kTileN);
                    }
                }
            }
            pdl_wait();
            while (ok && walk.next(p, cta, s)) {
                int nt, mt;
                tile_at(p, s.tile, nt, mt);
                for (int kb = s.kb0; kb < s.kb1; ++kb, ++j) {
                    const int sl = j % S;
                    if (j >= ahead) {
                        if (!mbar_wait(&wempty[sl], ((j / S) & 1) ^ 1, p.timeout_ns, &flags[0])) {
                            q8_fail(p, &flags[0], kErrTimeoutProducer);
                            ok = false;
                            break;
                        }
                        mbar_arrive_expect_tx(&wfull[sl], kQ8WBytes + Sh::kRawX);
                        tma_load_2d(sW + sl * kQ8WBytes, &tmW, &wfull[sl], kb * kQ8BlockK, nt * kTileN, pol_w);
                        issued_w = j + 1;
                    }
                    if constexpr (!WIDE) {
                        tma_load_2d(sXraw + sl * Sh::kRawX, &tmX, &wfull[sl], kb * kQ8BlockK, mt * MT, pol_x);
                    } else {
                        const int sx = j % SX;
                        if (!mbar_wait(&xempty[sx], ((j / SX) & 1) ^ 1, p.timeout_ns, &flags[0])) {
                            q8_fail(p, &flags[0], kErrTimeoutProducer);
                            ok = false;
                            break;
                        }
                        mbar_arrive_expect_tx(&xfull[sx], Sh::kX16);
                        tma_load_2d(sX16 + sx * Sh::kX16, &tmX, &xfull[sx], kb * kQ8BlockK, mt * MT, pol_x);
                        tma_load_2d(sX16 + sx * Sh::kX16 + MT * 128, &tmX, &xfull[sx], kb * kQ8BlockK + 64, mt * MT,
                                    pol_x);
                        issued_x = j + 1;
                    }
                }
            }
            if (flags[0]) {
                // Abort: request the x tiles that begun stages still expect, and let every copy land before exit.
                if constexpr (!WIDE) {
                    for (int k = j; k < issued_w; ++k)
                        tma_load_2d(sXraw + (k % S) * Sh::kRawX, &tmX, &wfull[k % S], 0, 0, pol_x);
                }
                volatile int never = 0;
                for (int k = 0; k < S && k < issued_w; ++k)
                    mbar_wait(&wfull[k], ((issued_w - 1 - k) / S) & 1, kDefaultTimeoutNs, &never);
                if constexpr (WIDE) {
                    for (int k = 0; k < SX && k < issued_x; ++k)
                        mbar_wait(&xfull[k], ((issued_x - 1 - k) / SX) & 1, kDefaultTimeoutNs, &never);
                }
            }
        }
    } else if (warp == Sh::kMmaWarp) {
        // ---------------------------------------------------------- MMA issuer
        if (lane == 0 && blocks > 0) {
            Q8Segment s;
            bool ok = true;
            int j = 0, chunk = 0;
            while (ok && walk.next(p, cta, s)) {
                for (int kb = s.kb0; kb < s.kb1 && ok; ++kb, ++j) {
                    const int in_chunk = (kb - s.kb0) % kExactBlocks;
                    const int t = chunk & 1;
                    if (in_chunk == 0)
                        ok = mbar_wait(&aempty[t], ((chunk >> 1) & 1) ^ 1, p.timeout_ns, &flags[0]);
                    const int b = j % OPS;
                    ok = ok && mbar_wait(&opfull[b], (j / OPS) & 1, p.timeout_ns, &flags[0]);
                    uint32_t bx = smem_u32(sX16 + b * Sh::kX16);
                    if constexpr (WIDE) {
                        ok = ok && mbar_wait(&xfull[j % SX], (j / SX) & 1, p.timeout_ns, &flags[0]);
                        bx = smem_u32(sX16 + (j % SX) * Sh::kX16);
                    }
                    if (!ok) {
                        q8_fail(p, &flags[0], kErrTimeoutMma);
                        break;
                    }
                    tc_fence_after();
                    const uint32_t d = tmem_base + static_cast<uint32_t>(t * MT);
                    const uint32_t a = tmem_base + static_cast<uint32_t>(2 * MT + b * 64);
                    const uint64_t b0 = smem_desc_kmajor_sw128(bx), b1 = smem_desc_kmajor_sw128(bx + MT * 128);
#pragma unroll
                    for (int kk = 0; kk < kQ8BlockK / 16; ++kk)
                        tc_mma_f16_ts(d, a + 8 * kk, (kk < 4 ? b0 : b1) + 2 * (kk & 3), Sh::kIdesc,
                                      (in_chunk > 0 || kk > 0) ? 1u : 0u);
                    tc_commit(&opempty[b]);
                    if constexpr (WIDE)
                        tc_commit(&xempty[j % SX]);
                    if (in_chunk == kExactBlocks - 1 || kb + 1 == s.kb1) {
                        tc_commit(&afull[t]);
                        ++chunk;
                    }
                }
            }
            if (!ok) {
                // Abort: wait for the MMAs already issued before TMEM is freed.
                tc_commit(drain);
                volatile int never = 0;
                mbar_wait(drain, 0, kDefaultTimeoutNs, &never);
            }
        }
    } else if (warp < kWidenWarps) {
        // --------------------------------------------------------------- widen
        const int quarter = warp & 3, row = quarter * 32 + lane;
        const uint32_t lane_base = tmem_base + (static_cast<uint32_t>(quarter * 32) << 16) + 2 * MT;
        for (int j = warp >> 2; j < blocks; j += kWidenSets) {
            const int sl = j % S, b = j % OPS;
            // The operand buffer first: once the MMA of unit j - OPS is done, unit
            // j - S <= j - OPS has been widened, so the ring slot's barrier is at
            // most one phase behind and its parity says which.  (The sets run
            // apart: by the parity alone, a slot still waiting for unit j - S
            // looks like one that holds unit j.)
            const bool ok = mbar_wait(&opempty[b], ((j / OPS) & 1) ^ 1, p.timeout_ns, &flags[0]) &&
                            mbar_wait(&wfull[sl], (j / S) & 1, p.timeout_ns, &flags[0]);
            if (!__all_sync(0xFFFFFFFFu, ok)) {      // the whole warp goes on, or none of it
                q8_fail(p, &flags[0], kErrTimeoutWiden);
                break;
            }
            tc_fence_after();
            const uint8_t *src = sW + sl * kQ8WBytes + row * kQ8BlockK;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                uint32_t r[16];
#pragma unroll
                for (int h = 0; h < 2; ++h)
                    widen16(*reinterpret_cast<const uint4 *>(src + (((2 * i + h) ^ (row & 7)) << 4)), r + 8 * h);
                tmem_st_x16(lane_base + b * 64 + 16 * i, r);
            }
            if constexpr (!WIDE) {
                const uint8_t *xs = sXraw + sl * Sh::kRawX;
                uint8_t *xd = sX16 + b * Sh::kX16;
#pragma unroll 2
                for (int i = 0; i < MT / 16; ++i) {
                    const int c = lane & 7, m = i * 16 + quarter * 4 + (lane >> 3);
                    uint32_t r[8];
                    widen16(*reinterpret_cast<const uint4 *>(xs + m * 128 + ((c ^ (m & 7)) << 4)), r);
                    uint8_t *dst = xd + (c >> 2) * (MT * 128) + m * 128;
                    const int cc = (c & 3) * 2;
                    *reinterpret_cast<uint4 *>(dst + ((cc ^ (m & 7)) << 4)) = make_uint4(r[0], r[1], r[2], r[3]);
                    *reinterpret_cast<uint4 *>(dst + (((cc + 1) ^ (m & 7)) << 4)) = make_uint4(r[4], r[5], r[6], r[7]);
                }
                fence_proxy_async_smem();
            }
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(&opfull[b]);
                mbar_arrive(&wempty[sl]);
            }
        }
    } else {
        // ------------------------------------------------------------ epilogue
        constexpr int NC = Sh::kCols, ET = Sh::kEpiWarps * 32;
        pdl_wait();                      // scales, residual, workspace and y only from here on
        const int ew = warp - kWidenWarps;
        const int row = (warp & 3) * 32 + lane;
        const int col0 = (ew >> 2) * NC;
        const uint32_t lane_base = tmem_base + (static_cast<uint32_t>((warp & 3) * 32) << 16) + static_cast<uint32_t>(col0);
        Q8Segment s;
        int chunk = 0;
        while (walk.next(p, cta, s)) {
            int nt, mt;
            tile_at(p, s.tile, nt, mt);
            const int n = nt * kTileN + row, m0 = mt * MT + col0;
            const int valid = p.g.M - m0;
            const bool whole = s.kb0 == 0 && s.kb1 == p.nkb;
            // This CTA's two slots: 1 for a shared tile whose first units it
            // has, 0 for any other (and to carry the sums of a whole tile).
            int *slot = p.ws + static_cast<size_t>(2 * cta + (s.kb0 == 0 && !whole)) * (MT * kTileN) + col0 * kTileN + row;
            bool ok = true;
            if constexpr (WIDE) {
                // The accumulations of a segment are added in registers.
                int acc[NC];
                for (int kb = s.kb0; kb < s.kb1; kb += kExactBlocks, ++chunk) {
                    const int t = chunk & 1;
                    ok = __all_sync(0xFFFFFFFFu, mbar_wait(&afull[t], (chunk >> 1) & 1, p.timeout_ns, &flags[0]));
                    if (!ok)
                        break;
                    tc_fence_after();
#pragma unroll
                    for (int c0 = 0; c0 < NC; c0 += 16) {
                        int v[16];
                        load_sums(lane_base + static_cast<uint32_t>(t * MT + c0), v);
#pragma unroll
                        for (int c = 0; c < 16; ++c)
                            acc[c0 + c] = kb == s.kb0 ? v[c] : acc[c0 + c] + v[c];
                    }
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0)
                        mbar_arrive(&aempty[t]);
                }
                if (ok && whole) {
                    store_columns<NC>(p.g, m0, n, acc);
                } else if (ok) {
#pragma unroll
                    for (int c0 = 0; c0 < NC; c0 += 16)
                        put_sums(slot + c0 * kTileN, valid - c0, *reinterpret_cast<const int(*)[16]>(&acc[c0]));
                }
            } else {
                // Two CTAs share the SM's registers: accumulations go out in
                // pairs (both TMEM buffers at once), and where a segment has
                // more than one pair, by way of the slot.
                for (int kb = s.kb0; kb < s.kb1; kb += 2 * kExactBlocks) {
                    const bool pair = kb + kExactBlocks < s.kb1, end = kb + 2 * kExactBlocks >= s.kb1;
                    const int t = chunk & 1;
                    ok = mbar_wait(&afull[t], (chunk >> 1) & 1, p.timeout_ns, &flags[0]) &&
                         (!pair || mbar_wait(&afull[t ^ 1], ((chunk + 1) >> 1) & 1, p.timeout_ns, &flags[0]));
                    ok = __all_sync(0xFFFFFFFFu, ok);
                    if (!ok)
                        break;
                    tc_fence_after();
#pragma unroll 1
                    for (int c0 = 0; c0 < NC; c0 += 16) {
                        int v[16], u[16];
                        load_sums(lane_base + static_cast<uint32_t>(t * MT + c0), v);
                        if (pair) {
                            load_sums(lane_base + static_cast<uint32_t>((t ^ 1) * MT + c0), u);
#pragma unroll
                            for (int c = 0; c < 16; ++c)
                                v[c] += u[c];
                        }
                        if (kb > s.kb0) {
#pragma unroll
                            for (int c = 0; c < 16; ++c)
                                u[c] = c0 + c < valid ? __ldcg(slot + (c0 + c) * kTileN) : 0;
#pragma unroll
                            for (int c = 0; c < 16; ++c)
                                v[c] += u[c];
                        }
                        if (end && whole)
                            store_columns<16>(p.g, m0 + c0, n, v);
                        else
                            put_sums(slot + c0 * kTileN, valid - c0, v);
                    }
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) {
                        mbar_arrive(&aempty[t]);
                        if (pair)
                            mbar_arrive(&aempty[t ^ 1]);
                    }
                    chunk += pair ? 2 : 1;
                }
            }
            if (!ok)
                q8_fail(p, &flags[0], kErrTimeoutEpilogue);
            if (!q8_epi_and<ET>(ok && !flags[0]))
                break;
            if (!whole && ew == 0 && lane == 0) {
                // CTA c begins at unit floor(c units / ctas), so the CTA that
                // holds unit u is floor(((u + 1) ctas - 1) / units).  The
                // barrier above orders every thread's sums before this acq_rel
                // arrival; the last arrival's acquire, passed on by the CTA's
                // last barrier, orders its reads after everyone's sums.
                const long long u0 = static_cast<long long>(s.tile - p.full * static_cast<int>(gridDim.x)) * p.nkb;
                const int first = static_cast<int>(((u0 + 1) * p.rem_ctas - 1) / p.rem_units);
                const int last = static_cast<int>(((u0 + p.nkb) * p.rem_ctas - 1) / p.rem_units);
                unsigned old;
                asm volatile("atom.acq_rel.gpu.global.add.u32 %0, [%1], 1;"
                             : "=r"(old) : "l"(p.counters + first) : "memory");
                if (old == static_cast<unsigned>(last - first)) {
                    p.counters[first] = 0;
                    const int k = flags[1];
                    finish[3 * k] = s.tile;
                    finish[3 * k + 1] = first;
                    finish[3 * k + 2] = last;
                    flags[1] = k + 1;
                }
            }
        }
    }

    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if (warp == Sh::kMmaWarp) {
        tc_fence_after();
        tmem_dealloc(tmem_base, Sh::kTmemCols);
    }
    // Shared tiles that this CTA was the last to add to (at most two): every
    // warp is free by now.
    for (int k = 0; k < flags[1] && !flags[0]; ++k) {
        int nt, mt;
        tile_at(p, finish[3 * k], nt, mt);
        finish_tile<MT, Sh::kThreads>(p, mt * MT, nt * kTileN, finish[3 * k + 1], finish[3 * k + 2]);
    }
}

// x as fp16, for the tensor-core kernel's B operand.
__global__ void __launch_bounds__(256) q8_widen_kernel(const uint4 *x, uint4 *out, size_t vectors)
{
    pdl_launch_dependents();
    pdl_wait();
    for (size_t i = static_cast<size_t>(blockIdx.x) * 256 + threadIdx.x; i < vectors;
         i += static_cast<size_t>(gridDim.x) * 256) {
        uint32_t r[8];
        widen16(__ldg(x + i), r);
        out[2 * i] = make_uint4(r[0], r[1], r[2], r[3]);
        out[2 * i + 1] = make_uint4(r[4], r[5], r[6], r[7]);
    }
}

cudaError_t launch_pdl(const void *f, unsigned grid, unsigned threads, size_t smem, void **args, cudaStream_t s)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelExC(&cfg, f, args);
}

template <int MT, bool WIDE>
cudaError_t launch_shape(const CUtensorMap &tmW, const CUtensorMap &tmX, const Q8TcParams &p, int grid, cudaStream_t s)
{
    using Sh = Q8Shape<MT, WIDE>;
    static int attr_set[kMaxDevices] = {};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess)
        return e;
    if (dev >= kMaxDevices)
        return cudaErrorInvalidDevice;
    const void *f = reinterpret_cast<const void *>(&q8_tc_kernel<MT, WIDE>);
    if (__atomic_load_n(&attr_set[dev], __ATOMIC_ACQUIRE) == 0) {
        e = cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, Sh::kSmem);
        if (e == cudaSuccess)
            e = cudaFuncSetAttribute(f, cudaFuncAttributePreferredSharedMemoryCarveout, cudaSharedmemCarveoutMaxShared);
        if (e != cudaSuccess)
            return e;
        __atomic_store_n(&attr_set[dev], 1, __ATOMIC_RELEASE);
    }
    void *args[] = {const_cast<CUtensorMap *>(&tmW), const_cast<CUtensorMap *>(&tmX), const_cast<Q8TcParams *>(&p)};
    return launch_pdl(f, static_cast<unsigned>(grid), Sh::kThreads, Sh::kSmem, args, s);
}

} // namespace

Q8TcShape q8_tc_shape(int m_tile)
{
    switch (m_tile) {
    case 32: return {2, Q8Shape<32, false>::kSmem, Q8Shape<32, false>::kThreads, Q8Shape<32, false>::kStages};
    case 64: return {2, Q8Shape<64, false>::kSmem, Q8Shape<64, false>::kThreads, Q8Shape<64, false>::kStages};
    case 128: return {1, Q8Shape<128, true>::kSmem, Q8Shape<128, true>::kThreads, Q8Shape<128, true>::kStages};
    default: return {1, Q8Shape<192, true>::kSmem, Q8Shape<192, true>::kThreads, Q8Shape<192, true>::kStages};
    }
}

cudaError_t launch_q8_tc(const CUtensorMap &tmW, const CUtensorMap &tmX, const Q8TcParams &p, int m_tile, int grid,
                         cudaStream_t s)
{
    switch (m_tile) {
    case 32: return launch_shape<32, false>(tmW, tmX, p, grid, s);
    case 64: return launch_shape<64, false>(tmW, tmX, p, grid, s);
    case 128: return launch_shape<128, true>(tmW, tmX, p, grid, s);
    case 192: return launch_shape<192, true>(tmW, tmX, p, grid, s);
    default: return cudaErrorInvalidValue;
    }
}

cudaError_t launch_q8_widen(const int8_t *x, void *out, size_t elements, int num_sms, cudaStream_t s)
{
    const uint4 *src = reinterpret_cast<const uint4 *>(x);
    uint4 *dst = static_cast<uint4 *>(out);
    size_t vectors = elements / 16;
    const size_t blocks = (vectors + 255) / 256;
    const unsigned grid = static_cast<unsigned>(std::min<size_t>(blocks, static_cast<size_t>(num_sms) * 8));
    void *args[] = {&src, &dst, &vectors};
    return launch_pdl(reinterpret_cast<const void *>(&q8_widen_kernel), grid, 256, 0, args, s);
}

} // namespace skg

// skg_f8_tc_common.cuh -- device code shared by the tcgen05 kernels of the 8-bit
// floating point path: which tile is next, of one weight or of many, and the
// reading of accumulators.  Included inside namespace skg's anonymous namespace.
#pragma once

constexpr uint32_t kF8TileBytes = kTileN * kF8Block;     // 128 rows of one unit (128 k): 16 KB

__device__ __forceinline__ void f8_fail(unsigned *err, volatile int *abort, unsigned bit)
{
    *abort = 1;
    if (err)
        atomicOr(err, bit);
}

// What an expert's rows are, in shared memory: row0[e] their first, tile0[e] the
// token tiles of the experts before.  Both have experts + 1 entries.
struct F8Table {
    int *row0, *tile0;
};

__host__ __device__ constexpr int f8_table_bytes(int experts) { return experts ? 2 * (experts + 1) * 4 : 0; }

// By one warp, from offsets.  Offsets are data on the device, which nobody has
// checked: they are held to [0, M] and to ascend, so that no access of a tile is
// out of range whatever they are.
__device__ __forceinline__ void f8_build_table(const F8LinearParams &p, int m_tile, const F8Table &t)
{
    const int lane = threadIdx.x & 31;
    auto read = [&](int e) { return e <= p.experts ? min(max(__ldcg(p.offsets + e), 0), p.M) : 0; };
    int row = read(0), tiles = 0;
    if (lane == 0) {
        t.row0[0] = row;
        t.tile0[0] = 0;
    }
    for (int e0 = 1; e0 <= p.experts; e0 += 32) {
        int v = read(e0 + lane);
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int u = __shfl_up_sync(0xFFFFFFFFu, v, o);
            v = lane >= o ? max(v, u) : v;
        }
        v = max(v, row);
        int before = __shfl_up_sync(0xFFFFFFFFu, v, 1);
        before = lane ? before : row;
        int n = (v - before + m_tile - 1) / m_tile;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int u = __shfl_up_sync(0xFFFFFFFFu, n, o);
            n += lane >= o ? u : 0;
        }
        n += tiles;
        if (e0 + lane <= p.experts) {
            t.row0[e0 + lane] = v;
            t.tile0[e0 + lane] = n;
        }
        row = __shfl_sync(0xFFFFFFFFu, v, 31);
        tiles = __shfl_sync(0xFFFFFFFFu, n, 31);
    }
}

__device__ __forceinline__ int f8_tiles(const F8LinearParams &p, const F8Table &t)
{
    return (p.experts ? t.tile0[p.experts] : p.m_tiles) * p.n_tiles;
}

struct F8Tile {
    int e, nt;               // expert, tile of channels
    int m0, m1;              // first row, and the end of the expert's rows
};

// Tiles of an expert in bands of kF8Band token tiles: within a band, token tiles
// fastest, so that the CTAs of a wave share a compact block of x and W in L2.
constexpr int kF8Band = 16;

__device__ __forceinline__ F8Tile f8_tile(const F8LinearParams &p, int m_tile, const F8Table &t, int tile)
{
    F8Tile r = {0, 0, 0, p.M};
    int m_tiles = p.m_tiles;
    if (p.experts) {
        int lo = 0, hi = p.experts;              // the last expert whose tiles begin at `tile` or before
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (t.tile0[mid] * p.n_tiles <= tile)
                lo = mid;
            else
                hi = mid;
        }
        r.e = lo;
        r.m0 = t.row0[lo];
        r.m1 = t.row0[lo + 1];
        m_tiles = t.tile0[lo + 1] - t.tile0[lo];
        tile -= t.tile0[lo] * p.n_tiles;
    }
    const int per_band = kF8Band * p.n_tiles;
    const int b = tile / per_band, i = tile - b * per_band;
    const int wide = min(kF8Band, m_tiles - b * kF8Band);
    r.nt = i / wide;
    r.m0 += (b * kF8Band + i - r.nt * wide) * m_tile;
    return r;
}

// 16 accumulator columns of this thread's TMEM lane, on their way until
// tmem_wait_ld; f8_taken keeps their use behind it.
__device__ __forceinline__ void f8_taken(uint32_t (&r)[16])
{
#pragma unroll
    for (int i = 0; i < 16; ++i)
        asm volatile("" : "+r"(r[i]));
}

// A unit's sums into acc: N columns from taddr on, every one times `scale`.  The 32
// columns of a step are fetched while those before are added; `taken` is called
// when the last are in registers.  (fma.rn.f32x2 does two at a time, but not twice
// as fast: the wide kernel takes 830 cycles a unit with it, 780 with fmaf.)
template <int N, class Taken>
__device__ __forceinline__ void f8_add_unit(float (&acc)[N], uint32_t taddr, float scale, Taken &&taken)
{
    uint32_t r[2][2][16];
    auto fetch = [&](int i) {
        tmem_ld_x16(taddr + static_cast<uint32_t>(32 * i), r[i & 1][0]);
        tmem_ld_x16(taddr + static_cast<uint32_t>(32 * i + 16), r[i & 1][1]);
    };
    fetch(0);
#pragma unroll
    for (int i = 0; i < N / 32; ++i) {
        tmem_wait_ld();
        f8_taken(r[i & 1][0]);
        f8_taken(r[i & 1][1]);
        if (i + 1 < N / 32)
            fetch(i + 1);
        else
            taken();
#pragma unroll
        for (int c = 0; c < 32; ++c)
            acc[32 * i + c] = fmaf(__uint_as_float(r[i & 1][c >> 4][c & 15]), scale, acc[32 * i + c]);
    }
}

// Two outputs as bf16, the first in the low half.
__device__ __forceinline__ uint32_t two_bf16(float a, float b)
{
    uint32_t w;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w) : "f"(b), "f"(a));
    return w;
}

// One output; the residual is added in fp32, and the sum rounded once.
__device__ __forceinline__ void f8_store(const F8LinearParams &p, int m, int n, float v)
{
    const size_t o = static_cast<size_t>(m) * p.N + n;
    if (p.epilogue == SKG_EPI_FP32) {
        static_cast<float *>(p.y)[o] = v;
        return;
    }
    if (p.epilogue == SKG_EPI_BF16_RESIDUAL)
        v += bf16_to_f32(__ldcg(p.res + o));
    static_cast<uint16_t *>(p.y)[o] = f32_to_bf16(v);
}

// Where the sum of a token and channel is left for the join of a split K: rows of
// `channels` fp32, 16-byte pieces swizzled by the token, so that lanes that hold
// neighbouring tokens or neighbouring channels store without bank conflicts.
__device__ __forceinline__ uint32_t f8_sum_at(int channels, int token, int c)
{
    return static_cast<uint32_t>(token * channels * 4 + (((c >> 2) ^ (token & 7)) << 4) + (c & 3) * 4);
}

__device__ __forceinline__ float4 ld_cluster_f32x4(uint32_t addr)
{
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0,%1,%2,%3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(addr) : "memory");
    return v;
}

// The end of a tile whose K is split over p.split CTAs of the cluster, the ranks
// first, first + rank_step, ...: each has left its sums at `smem`; this CTA, the part-th of
// them, adds up and stores its share of the tokens, a warp a token and 128
// channels, always in the order of the parts.  Called by whole CTAs, all of the
// cluster's.
template <int MAX_SPLIT, int THREADS>
__device__ __forceinline__ void f8_join(const F8LinearParams &p, uint32_t smem, int channels, int m0, int n0, int tokens, int part,
                                        int first, int rank_step)
{
    const int lane = static_cast<int>(threadIdx.x) & 31;
    cluster_sync();
    const int t1 = (part + 1) * tokens / p.split, blocks = channels / kF8Block;
    const int t0 = part * tokens / p.split;
    for (int i = static_cast<int>(threadIdx.x >> 5); i < (t1 - t0) * blocks; i += THREADS / 32) {
        const int m = t0 + i / blocks, c0 = i % blocks * kF8Block;
        if (p.vec4) {
            const int c = c0 + 4 * lane, n = n0 + c;
            float4 v[MAX_SPLIT];
#pragma unroll
            for (int r = 0; r < MAX_SPLIT; ++r)
                v[r] = r < p.split ? ld_cluster_f32x4(map_shared_rank(smem + f8_sum_at(channels, m, c), first + r * rank_step))
                                   : make_float4(0, 0, 0, 0);
            float4 s = v[0];
#pragma unroll
            for (int r = 1; r < MAX_SPLIT; ++r)
                s.x += v[r].x, s.y += v[r].y, s.z += v[r].z, s.w += v[r].w;
            if (n < p.N) {
                const size_t o = static_cast<size_t>(m0 + m) * p.N + n;
                if (p.epilogue == SKG_EPI_FP32) {
                    *reinterpret_cast<float4 *>(static_cast<float *>(p.y) + o) = s;
                } else {
                    if (p.epilogue == SKG_EPI_BF16_RESIDUAL) {
                        const uint2 b = __ldcg(reinterpret_cast<const uint2 *>(p.res + o));
                        s.x += bf16lo(b.x), s.y += bf16hi(b.x), s.z += bf16lo(b.y), s.w += bf16hi(b.y);
                    }
                    *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(p.y) + o) = make_uint2(two_bf16(s.x, s.y), two_bf16(s.z, s.w));
                }
            }
        } else {
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int c = c0 + lane + 32 * k;
                float s = 0.0f;
                for (int r = 0; r < p.split; ++r)
                    s += ld_shared_cluster_f32(map_shared_rank(smem + f8_sum_at(channels, m, c), first + r * rank_step));
                if (n0 + c < p.N)
                    f8_store(p, m0 + m, n0 + c, s);
            }
        }
    }
    cluster_sync();                      // no CTA leaves while a peer reads its sums
}

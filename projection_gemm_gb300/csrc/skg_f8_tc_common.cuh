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

// 16 accumulator columns of this thread's TMEM lane; wait with tmem_wait_ld and
// take them with f8_taken before use.
__device__ __forceinline__ void f8_taken(uint32_t (&r)[16])
{
#pragma unroll
    for (int i = 0; i < 16; ++i)
        asm volatile("" : "+r"(r[i]));
}

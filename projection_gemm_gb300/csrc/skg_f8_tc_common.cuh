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
    constexpr int PER = 4;               // experts a lane: the loads of 128 are on their way together
    const int lane = threadIdx.x & 31;
    auto read = [&](int e) { return e <= p.experts ? min(max(__ldcg(p.offsets + e), 0), p.M) : 0; };
    int row = read(0), tiles = 0;
    if (lane == 0) {
        t.row0[0] = row;
        t.tile0[0] = 0;
    }
    for (int e0 = 1; e0 <= p.experts; e0 += 32 * PER) {
        const int e = e0 + lane * PER;
        int end[PER], n[PER];
#pragma unroll
        for (int i = 0; i < PER; ++i)
            end[i] = read(e + i);
#pragma unroll
        for (int i = 1; i < PER; ++i)
            end[i] = max(end[i], end[i - 1]);
        int top = end[PER - 1];          // of the lanes up to this one
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int u = __shfl_up_sync(0xFFFFFFFFu, top, o);
            top = lane >= o ? max(top, u) : top;
        }
        int before = __shfl_up_sync(0xFFFFFFFFu, top, 1);
        before = lane ? max(before, row) : row;
        int sum = 0;
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            end[i] = max(end[i], before);
            sum += (end[i] - before + m_tile - 1) / m_tile;
            n[i] = sum;
            before = end[i];
        }
        int up = sum;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int u = __shfl_up_sync(0xFFFFFFFFu, up, o);
            up += lane >= o ? u : 0;
        }
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            if (e + i <= p.experts) {
                t.row0[e + i] = end[i];
                t.tile0[e + i] = tiles + up - sum + n[i];
            }
        }
        row = max(row, __shfl_sync(0xFFFFFFFFu, top, 31));
        tiles += __shfl_sync(0xFFFFFFFFu, up, 31);
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

// Where a copy of `box` rows begins that is to have the rows from `row` on (of
// `rows` in all): there, or sooner, so that it ends with the last row.  A copy most of
// whose rows lie beyond the tensor's end takes far longer than one that has them
// all: 32 units of 128 rows of which 26, or 40, were there 65 us, or 21.  The rows
// before `row` that come with it are computed and left out.
__device__ __forceinline__ int f8_window(int row, int rows, int box) { return min(row, rows - box); }

__device__ __forceinline__ int f8_x_window(const F8LinearParams &p, int m0) { return f8_window(m0, p.M, p.x_box); }

// Of the channels from n0 on of expert e: in rows of all experts' weights.
__device__ __forceinline__ int f8_w_window(const F8LinearParams &p, int e, int n0)
{
    return f8_window(e * p.N + n0, max(1, p.experts) * p.N, p.w_box);
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
// first, first + rank_step, ...: each has left its sums at `smem`, tokens from m0 on
// and blocks of 128 channels from n[0], n[1] on (windows); the outputs are those of
// tokens ma to mb and channels na[b] to p.N.  This CTA, the part-th of them, adds up and
// stores its share of the tokens, a warp a token and block, always in the order of
// the parts.  Called by whole CTAs, all of the cluster's.
template <int MAX_SPLIT, int THREADS, int BLOCKS>
__device__ __forceinline__ void f8_join(const F8LinearParams &p, uint32_t smem, int m0, int ma, int mb, const int (&n0)[BLOCKS],
                                        const int (&na)[BLOCKS], int part, int first, int rank_step)
{
    constexpr int channels = BLOCKS * kF8Block;
    const int lane = static_cast<int>(threadIdx.x) & 31;
    cluster_sync();
    const int tokens = max(0, mb - ma), t0 = part * tokens / p.split, t1 = (part + 1) * tokens / p.split;
    for (int i = static_cast<int>(threadIdx.x >> 5); i < (t1 - t0) * BLOCKS; i += THREADS / 32) {
        const int m = ma + t0 + i / BLOCKS, b = i % BLOCKS;
        const int first_n = BLOCKS == 1 || b == 0 ? n0[0] : n0[BLOCKS - 1], least = BLOCKS == 1 || b == 0 ? na[0] : na[BLOCKS - 1];
        if (p.vec4) {
            const int c = b * kF8Block + 4 * lane, n = first_n + 4 * lane;
            float4 v[MAX_SPLIT];
#pragma unroll
            for (int r = 0; r < MAX_SPLIT; ++r)
                v[r] = r < p.split ? ld_cluster_f32x4(map_shared_rank(smem + f8_sum_at(channels, m - m0, c), first + r * rank_step))
                                   : make_float4(0, 0, 0, 0);
            float4 s = v[0];
#pragma unroll
            for (int r = 1; r < MAX_SPLIT; ++r)
                s.x += v[r].x, s.y += v[r].y, s.z += v[r].z, s.w += v[r].w;
            if (n >= least && n < p.N) {
                const size_t o = static_cast<size_t>(m) * p.N + n;
                if (p.epilogue == SKG_EPI_FP32) {
                    *reinterpret_cast<float4 *>(static_cast<float *>(p.y) + o) = s;
                } else {
                    if (p.epilogue == SKG_EPI_BF16_RESIDUAL) {
                        const uint2 r = __ldcg(reinterpret_cast<const uint2 *>(p.res + o));
                        s.x += bf16lo(r.x), s.y += bf16hi(r.x), s.z += bf16lo(r.y), s.w += bf16hi(r.y);
                    }
                    *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(p.y) + o) = make_uint2(two_bf16(s.x, s.y), two_bf16(s.z, s.w));
                }
            }
        } else {
            float s[4] = {};
#pragma unroll
            for (int r = 0; r < MAX_SPLIT; ++r) {
                if (r < p.split) {
                    float v[4];
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        v[k] = ld_shared_cluster_f32(map_shared_rank(smem + f8_sum_at(channels, m - m0, b * kF8Block + lane + 32 * k),
                                                                     first + r * rank_step));
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        s[k] += v[k];
                }
            }
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int n = first_n + lane + 32 * k;
                if (n >= least && n < p.N)
                    f8_store(p, m, n, s[k]);
            }
        }
    }
    cluster_sync();                      // no CTA leaves while a peer reads its sums
}

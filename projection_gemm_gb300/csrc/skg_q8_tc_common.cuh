// skg_q8_tc_common.cuh -- device code shared by the 8-bit path's tcgen05 kernels:
// widening, the epilogue's reading of accumulators, its stores, and the join of a
// split K.  Included inside namespace skg's anonymous namespace.
#pragma once

constexpr int kQ8BlockK = 128;                       // k of one unit: 128 bytes of a W row
constexpr int kExactBlocks = 1024 / kQ8BlockK;       // units summed by the MMA from a fresh accumulator
constexpr int kWidenSets = 2;                        // sets of 4 warps (a set covers the 128 TMEM lanes)
constexpr int kWidenWarps = 4 * kWidenSets;
constexpr uint32_t kQ8WBytes = kTileN * kQ8BlockK;   // 16 KB

__device__ __forceinline__ void q8_fail(unsigned *err, volatile int *abort, unsigned bit)
{
    *abort = 1;
    if (err)
        atomicOr(err, bit);
}

__device__ __forceinline__ void widen16(const uint4 &v, uint32_t *r)
{
    widen4(v.x, r[0], r[1]);
    widen4(v.y, r[2], r[3]);
    widen4(v.z, r[4], r[5]);
    widen4(v.w, r[6], r[7]);
}

// A W row's 128 bytes of a unit (a tile of 128-byte rows, 128-byte swizzle) as
// fp16 into this thread's TMEM lane: 64 columns.
__device__ __forceinline__ void widen_row(const uint8_t *tile, int row, uint32_t taddr)
{
    const uint8_t *src = tile + row * kQ8BlockK;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        uint32_t r[16];
#pragma unroll
        for (int h = 0; h < 2; ++h)
            widen16(*reinterpret_cast<const uint4 *>(src + (((2 * i + h) ^ (row & 7)) << 4)), r + 8 * h);
        tmem_st_x16(taddr + 16 * i, r);
    }
}

// A thread's 16-byte pieces of an x tile (128 bytes a token, 128-byte swizzle):
// piece c of token m and of every `step`-th token after it; a warp has the 32
// pieces of 4 tokens.  In fp16 a token is 128 bytes of each of two 64-wide
// halves, swizzled too.  8 lanes take half of an even token and the other half
// of the odd one after it: then neither their loads nor their stores share a
// bank.  (8 lanes to a token stored 2-way: 93,600 wavefronts an SM in the wide
// kernel at 1024 x 7168 x 7168 instead of 69,800, and 73.1 us instead of 71.4.)
struct XPiece {
    int from, to0, to1;

    __device__ __forceinline__ XPiece(int m0, int lane, int tokens)
    {
        const int odd = (lane >> 2) & 1;
        const int m = m0 + (lane >> 4) * 2 + odd, c = (lane & 3) + 4 * (odd ^ ((lane >> 3) & 1));
        const int cc = (c & 3) * 2;
        from = m * 128 + ((c ^ (m & 7)) << 4);
        to0 = (c >> 2) * (tokens * 128) + m * 128 + ((cc ^ (m & 7)) << 4);
        to1 = to0 ^ 16;
    }

    template <int N>
    __device__ __forceinline__ void widen(const uint8_t *raw, uint8_t *x16, int step) const      // step: of whole swizzle periods
    {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            uint32_t r[8];
            widen16(*reinterpret_cast<const uint4 *>(raw + from + i * step * 128), r);
            uint8_t *dst = x16 + i * step * 128;
            *reinterpret_cast<uint4 *>(dst + to0) = make_uint4(r[0], r[1], r[2], r[3]);
            *reinterpret_cast<uint4 *>(dst + to1) = make_uint4(r[4], r[5], r[6], r[7]);
        }
    }
};

// What a warp's 32 channels x 32 tokens need besides their sums, fetched before
// those are complete: a thread holds the scale of its channel n and of token
// m0 + lane.
struct Scales {
    float w, x;
};

__device__ __forceinline__ Scales load_scales(const Q8LinearParams &g, int m0, int n)
{
    const int m = m0 + (threadIdx.x & 31);
    return {n < g.N ? __ldcg(g.w_scale + n) : 0.0f, m < g.M ? __ldcg(g.x_scale + m) : 0.0f};
}

// 32 outputs (tokens m0...) of one channel n from their sums; the residual's
// loads 8 at a time.  Called by whole warps.
template <int EPI>
__device__ __forceinline__ void store_columns_as(const Q8LinearParams &g, int m0, int n, const Scales &sc, const int (&acc)[32])
{
    const int valid = n < g.N ? g.M - m0 : 0;
    size_t at = static_cast<size_t>(m0) * g.N + n;
#pragma unroll
    for (int c0 = 0; c0 < 32; c0 += 8) {
        uint16_t b[8];
        if (EPI == SKG_EPI_BF16_RESIDUAL) {
            const uint16_t *r = g.res + at;
#pragma unroll
            for (int c = 0; c < 8; ++c, r += g.N)
                b[c] = c0 + c < valid ? __ldcg(r) : 0;
        }
#pragma unroll
        for (int c = 0; c < 8; ++c, at += g.N) {
            float v = q8_scaled(acc[c0 + c], __shfl_sync(0xFFFFFFFFu, sc.x, c0 + c), sc.w);
            if (EPI == SKG_EPI_BF16_RESIDUAL)
                v = __fadd_rn(v, bf16_to_f32(b[c]));
            if (c0 + c < valid) {
                if (EPI == SKG_EPI_FP32)
                    static_cast<float *>(g.y)[at] = v;
                else
                    static_cast<uint16_t *>(g.y)[at] = f32_to_bf16(v);
            }
        }
    }
}

__device__ __forceinline__ void store_columns(const Q8LinearParams &g, int m0, int n, const Scales &sc, const int (&acc)[32])
{
    if (g.epilogue == SKG_EPI_FP32)
        store_columns_as<SKG_EPI_FP32>(g, m0, n, sc, acc);
    else if (g.epilogue == SKG_EPI_BF16_RESIDUAL)
        store_columns_as<SKG_EPI_BF16_RESIDUAL>(g, m0, n, sc, acc);
    else
        store_columns_as<SKG_EPI_BF16>(g, m0, n, sc, acc);
}

// NC accumulator columns of this thread's TMEM lane as integers (they are
// integers of at most 2^24 in fp32: the conversion is exact).
template <int NC>
__device__ __forceinline__ void load_sums(uint32_t taddr, int (&v)[NC])
{
    uint32_t r[NC / 8][8];
#pragma unroll
    for (int i = 0; i < NC / 8; ++i)
        tmem_ld_x8(taddr + 8 * i, r[i]);
    tmem_wait_ld();
#pragma unroll
    for (int c = 0; c < NC; ++c) {
        asm volatile("" : "+r"(r[c >> 3][c & 7]));
        v[c] = __float2int_rn(__uint_as_float(r[c >> 3][c & 7]));
    }
}

__device__ __forceinline__ int4 ld_cluster_v4(uint32_t addr)
{
    int4 v;
    asm volatile("ld.shared::cluster.v4.s32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr) : "memory");
    return v;
}

// Four 32-bit words of a CTA of the cluster: 16 neighbouring bytes, or words 128
// bytes apart.
__device__ __forceinline__ int4 ld_cluster_four(uint32_t addr, bool vec4)
{
    if (vec4)
        return ld_cluster_v4(addr);
    int v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v[i]) : "r"(addr + 128 * i) : "memory");
    return make_int4(v[0], v[1], v[2], v[3]);
}

// What four outputs of a token (channels n, n + 1, ... with vec4, else n, n + 32,
// ..., so that a warp's loads and stores cover neighbouring channels) need
// besides their sums.
struct Four {
    float xs, ws[4];
    uint16_t res[4];
};

__device__ __forceinline__ Four load_four(const Q8LinearParams &g, int m, int n, bool vec4)
{
    Four f;
    f.xs = __ldcg(g.x_scale + m);
    const size_t o = static_cast<size_t>(m) * g.N + n;
    const bool res = g.epilogue == SKG_EPI_BF16_RESIDUAL;
    if (vec4) {                          // n is a multiple of 4 and N too
        const float4 w = n < g.N ? __ldcg(reinterpret_cast<const float4 *>(g.w_scale + n)) : make_float4(0, 0, 0, 0);
        f.ws[0] = w.x, f.ws[1] = w.y, f.ws[2] = w.z, f.ws[3] = w.w;
        const uint2 r = res && n < g.N ? __ldcg(reinterpret_cast<const uint2 *>(g.res + o)) : make_uint2(0, 0);
        f.res[0] = r.x & 0xFFFF, f.res[1] = r.x >> 16, f.res[2] = r.y & 0xFFFF, f.res[3] = r.y >> 16;
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f.ws[i] = n + 32 * i < g.N ? __ldcg(g.w_scale + n + 32 * i) : 0.0f;
            f.res[i] = res && n + 32 * i < g.N ? __ldcg(g.res + o + 32 * i) : 0;
        }
    }
    return f;
}

__device__ __forceinline__ void store_four(const Q8LinearParams &g, int m, int n, bool vec4, const Four &f, const int4 &sum)
{
    const int s[4] = {sum.x, sum.y, sum.z, sum.w};
    float v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[i] = q8_scaled(s[i], f.xs, f.ws[i]);
        if (g.epilogue == SKG_EPI_BF16_RESIDUAL)
            v[i] = __fadd_rn(v[i], bf16_to_f32(f.res[i]));
    }
    const size_t o = static_cast<size_t>(m) * g.N + n;
    if (g.epilogue == SKG_EPI_FP32) {
        float *y = static_cast<float *>(g.y) + o;
        if (vec4 && n < g.N) {
            *reinterpret_cast<float4 *>(y) = make_float4(v[0], v[1], v[2], v[3]);
            return;
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (n + 32 * i < g.N)
                y[32 * i] = v[i];
        return;
    }
    uint16_t *y = static_cast<uint16_t *>(g.y) + o;
    if (vec4 && n < g.N) {
        *reinterpret_cast<uint2 *>(y) = make_uint2(f32_to_bf16(v[0]) | static_cast<uint32_t>(f32_to_bf16(v[1])) << 16,
                                                   f32_to_bf16(v[2]) | static_cast<uint32_t>(f32_to_bf16(v[3])) << 16);
        return;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
        if (n + 32 * i < g.N)
            y[32 * i] = f32_to_bf16(v[i]);
}

// The end of a tile whose K is split over `split` CTAs of the cluster, the
// ranks first, first + step, ...: each has left its sums [token][128 channels]
// as int32 at `smem`; this CTA, the part-th of them, adds up and stores its
// share of the tokens, four channels a thread.  Called by whole CTAs, all of
// the cluster's.
template <int MAX_SPLIT, int THREADS>
__device__ __forceinline__ void join_and_store(const Q8LinearParams &g, uint32_t smem, int m0, int n0, int tokens, int split,
                                               int part, int step, int first, bool vec4)
{
    const int lane = static_cast<int>(threadIdx.x) & 31;
    const int t1 = (part + 1) * tokens / split, n = n0 + (vec4 ? 4 * lane : lane);
    int m = part * tokens / split + static_cast<int>(threadIdx.x >> 5);
    Four f = {};
    pdl_wait();
    if (m < t1)
        f = load_four(g, m0 + m, n, vec4);           // on its way while the cluster meets
    cluster_sync();
    const uint32_t base = smem + (vec4 ? 16 * lane : 4 * lane);
    while (m < t1) {
        int4 sum = make_int4(0, 0, 0, 0);
        int4 v[MAX_SPLIT];
#pragma unroll
        for (int r = 0; r < MAX_SPLIT; ++r)
            v[r] = r < split ? ld_cluster_four(map_shared_rank(base + m * (kTileN * 4), first + r * step), vec4) : make_int4(0, 0, 0, 0);
#pragma unroll
        for (int r = 0; r < MAX_SPLIT; ++r) {
            sum.x += v[r].x;
            sum.y += v[r].y;
            sum.z += v[r].z;
            sum.w += v[r].w;
        }
        store_four(g, m0 + m, n, vec4, f, sum);
        m += THREADS / 32;
        if (m < t1)
            f = load_four(g, m0 + m, n, vec4);
    }
    cluster_sync();                      // no CTA leaves while a peer reads its sums
}

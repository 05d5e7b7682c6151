// skg_f8_api.cu -- host side of the 8-bit floating point path of include/skg.h:
// argument checks, plans and launches.
#include <algorithm>
#include <cmath>
#include <cstdint>
#include <new>

#include <cuda.h>
#include <cuda_runtime.h>

#include "skg.h"
#include "skg_f8_internal.h"
#include "skg_internal.h"

using namespace skg;

struct skg_f8_plan_s {
    skg_f8_plan_desc d;
    int device = 0, num_sms = 0;
    unsigned int *err_host = nullptr; // mapped pinned word
    unsigned int *err_dev = nullptr;
    cudaStream_t last_stream = nullptr;
};

namespace {

constexpr int kF8MaxK = 131072;
constexpr int kF8MaxM = 1 << 20;
constexpr int kF8MaxRow = 1 << 30;    // quantisers: element indexes of a row, and those just behind it, fit 32 bits

bool aligned(const void *p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }      // null is aligned

skg_status launched(cudaError_t e, const char *who)
{
    return e == cudaSuccess ? SKG_OK
                            : set_error(SKG_ERR_CUDA, "%s: %s (%s)", who, cudaGetErrorName(e), cudaGetErrorString(e));
}

int ceil_div(int a, int b) { return a / b + (a % b != 0); }

// Clusters of the split kernel resident at once on 152 SMs, by the CTAs of a
// cluster, two to an SM (cudaOccupancyMaxActiveClusters; a cluster stays within
// one GPC).  (With another number of SMs the counts are scaled; a launch that does
// not fit takes longer and gives the same result.)
constexpr int kSplitResident[] = {0, 304, 152, 97, 74, 58, 46, 38, 36};
static_assert(sizeof(kSplitResident) / sizeof(int) == kF8SplitMax + 1, "a count for each split");

long long resident(int on_152, int num_sms) { return std::max(1ll, static_cast<long long>(on_152) * num_sms / 152); }

// Experts with a row, about: the rows' choices taken as even.
double taken(const skg_f8_plan_desc &d)
{
    return d.experts ? d.experts * (1.0 - std::pow(1.0 - 1.0 / d.experts, d.M)) : 1.0;
}

// Token tiles: of one weight exactly; of experts as many as they take about, for
// the choice of a launch (`most` false), or at the most.
double token_tiles(const skg_f8_plan_desc &d, int m_tile, bool most)
{
    if (!d.experts)
        return ceil_div(d.M, m_tile);
    if (most)
        return std::min(d.experts, d.M) + d.M / m_tile;
    return taken(d) * std::max(1.0, d.M / taken(d) / m_tile + 0.5);
}

// The same of the wide kernel, a CTA an SM: single CTAs (128 tokens) and pairs (256).
constexpr int kWideResident1[] = {0, 152, 76, 48, 36};
constexpr int kWideResident2[] = {0, 76, 36, 23, 15};

struct Choice {
    int kind, m_tile, split;
    double us;
};

int n_tile_of(int kind, int m_tile) { return kind == SKG_F8_KERNEL_WIDE ? m_tile : kTileN; }

int max_split(int kind) { return kind == SKG_F8_KERNEL_WIDE ? kF8WideMaxSplit : kF8SplitMax; }

long long slots_of(int kind, int m_tile, int split, int num_sms)
{
    const int *r = kind == SKG_F8_KERNEL_SPLIT ? kSplitResident : m_tile == 128 ? kWideResident1 : kWideResident2;
    return resident(r[split], num_sms);
}

// The kernels' times (us) as measured: what a unit of 128 k takes a CTA's MMAs and
// its epilogue, a tile's end, and a launch's ends.
//
//                     unit: one CTA an SM, two   tile   ends   with K split
//   SPLIT 16 tokens         0.27  0.36           0.6    2.8    4.9
//         32                0.30  0.38           1.2    2.8    4.9
//         64                0.31  0.60           1.2    2.8    4.9
//   WIDE 128                0.33  -              1.0    2.5    6.3
//        256 (pairs)        0.39  -              2.0    4.0    7.8
//
// A unit takes a quarter more where rows of x and W begin between lines of 128 bytes,
// a tile of the wide kernel 2 more where rows of the output are not aligned.  The
// weights come from HBM at 6.3 TB/s at the most, by the wide kernel at 5.6.  Where that
// is about what bounds the split kernel, its ends with K split are 8.3 less 0.0225 a
// CTA: few CTAs take longer until enough of the weights is on its way.  Clusters of 3,
// 5, 6 or 7 take 0.4 longer, and with experts all start 1.3 later.  (Of 123 shapes of
// 1 to 5952 rows, with and without experts, the launch chosen is within 8% of the
// fastest for 114 and within 16% for all.)
double launch_us(const skg_f8_plan_desc &d, int kind, int m_tile, int split, int num_sms)
{
    const double sms = num_sms, tiles = token_tiles(d, m_tile, false) * ceil_div(d.N, n_tile_of(kind, m_tile));
    const int units = ceil_div(ceil_div(d.K, kF8Block), split);
    const double slots = static_cast<double>(slots_of(kind, m_tile, split, num_sms));
    const double at_once = std::min(tiles, slots) * split;            // CTAs, or pairs of them
    double waves = std::ceil(tiles / slots);
    if (split == 1 && (d.experts ? tiles > 0.8 * slots : waves > 2.0))
        waves = tiles / slots + 0.5;     // persistent, not all end together; or not known exactly
    const double hbm = taken(d) * d.N * d.K / (kind == SKG_F8_KERNEL_WIDE ? 5.6e6 : 6.3e6);
    double unit, tile, ends;
    if (kind == SKG_F8_KERNEL_WIDE) {
        unit = m_tile == 128 ? 0.33 : 0.39;
        tile = (m_tile == 128 ? 1.0 : 2.0) + (d.N % 8 != 0 ? 2.0 : 0.0);
        ends = (m_tile == 128 ? 2.5 : 4.0) + (split > 1 ? 3.8 : 0.0);
    } else {
        const bool two = at_once > sms;
        unit = m_tile == 16 ? (two ? 0.36 : 0.27) : m_tile == 32 ? (two ? 0.38 : 0.30) : (two ? 0.60 : 0.31);
        tile = m_tile == 16 ? 0.6 : 1.2;
        ends = split == 1 ? 2.8 : 4.9;
    }
    const double own = waves * (unit * (d.K % kF8Block ? 1.25 : 1.0) * units + tile);
    if (kind == SKG_F8_KERNEL_SPLIT && split > 1 && own < 1.3 * hbm && hbm > 4.0)
        ends = std::max(2.0, 8.3 - 0.0225 * at_once * 152.0 / sms);
    ends += ((split & (split - 1)) != 0 ? 0.4 : 0.0) + (d.experts && split > 1 ? 1.3 : 0.0);
    return std::pow(std::pow(hbm, 4) + std::pow(own, 4), 0.25) + ends;       // the larger, or a little more where they are close
}

// The launch that takes the least time, given a kernel, a tile and the CTAs that
// share a tile's K, or none of them (0).  K is split only into clusters that are
// resident at once.
Choice choose(const skg_f8_plan_desc &d, int kind, int m_tile, int split, int num_sms)
{
    const int nkb = ceil_div(d.K, kF8Block);
    Choice best = {0, 0, 0, 0.0};
    for (int mt = 16; mt <= 256; mt *= 2) {
        const int k = mt <= 64 ? SKG_F8_KERNEL_SPLIT : SKG_F8_KERNEL_WIDE;
        if ((kind && k != kind) || (m_tile && mt != m_tile))
            continue;
        for (int s = 1; s <= std::min(max_split(k), nkb); ++s) {
            const double tiles = token_tiles(d, mt, false) * ceil_div(d.N, n_tile_of(k, mt));
            if (split ? s != std::min(split, nkb) : s > 1 && tiles > slots_of(k, mt, s, num_sms))
                continue;
            const double us = launch_us(d, k, mt, s, num_sms);
            if (!best.kind || us < best.us)
                best = {k, mt, s, us};
        }
    }
    return best;
}

skg_status fill_launch(skg_f8_plan_desc *d, int kind, int m_tile, int split, int num_sms, const char *who)
{
    const Choice c = choose(*d, kind, m_tile, split, num_sms);
    const bool wide = c.kind == SKG_F8_KERNEL_WIDE;
    const F8TcShape sh = wide ? f8_wide_shape(c.m_tile, d->experts) : f8_split_shape(c.m_tile, d->experts);
    d->kernel_kind = c.kind;
    d->m_tile = sh.m_tile;
    d->n_tile = n_tile_of(c.kind, c.m_tile);
    d->split_k = c.split;
    d->threads = sh.threads;
    d->smem_bytes = sh.smem_bytes;
    d->stages = sh.stages;
    d->ctas_per_sm = sh.ctas_per_sm;
    const double tiles = token_tiles(*d, d->m_tile, true) * ceil_div(d->N, d->n_tile);
    if (tiles > (1 << 27))
        return set_error(SKG_ERR_UNSUPPORTED, "%s: more than 2^27 tiles", who);
    d->tiles = static_cast<int>(tiles);
    const int ctas = (c.m_tile == 256 ? 2 : 1) * c.split, slots = std::max(1, num_sms * sh.ctas_per_sm / ctas);
    d->grid = ctas * (c.split > 1 ? d->tiles : std::min(d->tiles, slots));
    return SKG_OK;
}

} // namespace

extern "C" {

skg_status skg_quantize_f8(int M, int K, const void *x, size_t ldx, const void *gate, size_t ldg, const int *rows, int x_rows,
                           void *q, float *scale, void *stream)
{
    static const char who[] = "skg_quantize_f8";
    if (M < 0 || K < 1 || (rows && x_rows < 0))
        return set_error(SKG_ERR_INVALID_ARG, "%s: M and x_rows must be >= 0 and K >= 1 (got M=%d, x_rows=%d, K=%d)", who, M,
                         x_rows, K);
    if (M > 0 && ((!x && !(rows && x_rows == 0)) || !q || !scale))
        return set_error(SKG_ERR_INVALID_ARG, "%s: x, q and scale must be non-NULL", who);
    if (K > kF8MaxRow)
        return set_error(SKG_ERR_UNSUPPORTED, "%s: K must be at most 2^30 (got %d)", who, K);
    if (ldx < static_cast<size_t>(K) || (gate && ldg < static_cast<size_t>(K)))
        return set_error(SKG_ERR_INVALID_ARG, "%s: a row stride of x / gate is below K = %d", who, K);
    if (!aligned(x, 2) || !aligned(gate, 2) || !aligned(rows, 4) || !aligned(scale, 4))
        return set_error(SKG_ERR_ALIGNMENT, "%s: x, gate, rows or scale misses its element alignment", who);
    if (M == 0)
        return SKG_OK;
    F8RowParams p = {};
    p.x = static_cast<const uint16_t *>(x);
    p.gate = static_cast<const uint16_t *>(gate);
    p.rows = rows;
    p.q = static_cast<uint8_t *>(q);
    p.scale = scale;
    p.ldx = ldx;
    p.ldg = ldg;
    p.M = M;
    p.K = K;
    p.kb = ceil_div(K, kF8Block);
    p.x_rows = x_rows;
    return launched(launch_f8_quantize(p, static_cast<cudaStream_t>(stream)), who);
}

skg_status skg_quantize_f8_weights(int experts, int N, int K, const void *W, void *q, float *scale, void *stream)
{
    static const char who[] = "skg_quantize_f8_weights";
    if (experts < 1 || N < 1 || K < 1)
        return set_error(SKG_ERR_INVALID_ARG, "%s: experts, N and K must be positive (got %d, %d, %d)", who, experts, N, K);
    if (!W || !q || !scale)
        return set_error(SKG_ERR_INVALID_ARG, "%s: W, q and scale must be non-NULL", who);
    if (!aligned(W, 2) || !aligned(scale, 4))
        return set_error(SKG_ERR_ALIGNMENT, "%s: W or scale misses its element alignment", who);
    if (K > kF8MaxRow)
        return set_error(SKG_ERR_UNSUPPORTED, "%s: K must be at most 2^30 (got %d)", who, K);
    F8WeightParams p = {static_cast<const uint16_t *>(W), static_cast<uint8_t *>(q), scale, experts, N, K,
                        ceil_div(N, kF8Block), ceil_div(K, kF8Block)};
    if (static_cast<double>(experts) * p.nb * p.kb > 2147483647.0)
        return set_error(SKG_ERR_UNSUPPORTED, "%s: more than 2^31 - 1 blocks", who);
    return launched(launch_f8_quantize_weights(p, static_cast<cudaStream_t>(stream)), who);
}

skg_status skg_f8_plan_query(int M, int N, int K, int epilogue, int experts, int num_sms, skg_f8_plan_desc *out)
{
    static const char who[] = "skg_f8_plan_query";
    if (!out)
        return set_error(SKG_ERR_INVALID_ARG, "%s: out is NULL", who);
    if (M < 1 || N < 1 || num_sms < 1 || experts < 0)
        return set_error(SKG_ERR_INVALID_ARG, "%s: M, N and num_sms must be positive, experts >= 0 (got %d, %d, %d, %d)", who,
                         M, N, num_sms, experts);
    if (epilogue < SKG_EPI_BF16 || epilogue > SKG_EPI_FP32)
        return set_error(SKG_ERR_INVALID_ARG, "%s: unknown epilogue %d", who, epilogue);
    if (K < 16 || K % 16 != 0 || K > kF8MaxK)
        return set_error(SKG_ERR_UNSUPPORTED, "%s: K must be a multiple of 16 in [16, %d] (got %d)", who, kF8MaxK, K);
    if (M > kF8MaxM || experts > kF8MaxExperts)
        return set_error(SKG_ERR_UNSUPPORTED, "%s: M must be at most %d and experts %d (got %d, %d)", who, kF8MaxM,
                         kF8MaxExperts, M, experts);
    if (static_cast<long long>(std::max(1, experts)) * N > 0x7FFFFF00ll)
        return set_error(SKG_ERR_UNSUPPORTED, "%s: more than 2^31 - 256 channels in all (%d experts, N=%d)", who, experts, N);
    skg_f8_plan_desc d = {};
    d.M = M;
    d.N = N;
    d.K = K;
    d.epilogue = epilogue;
    d.experts = experts;
    const skg_status st = fill_launch(&d, 0, 0, 0, num_sms, who);
    if (st == SKG_OK)
        *out = d;
    return st;
}

skg_status skg_f8_plan(int M, int N, int K, int epilogue, int experts, int static_weights, skg_f8_plan_t *out)
{
    static const char who[] = "skg_f8_plan";
    if (!out)
        return set_error(SKG_ERR_INVALID_ARG, "%s: out is NULL", who);
    *out = nullptr;
    skg_f8_plan_desc d;
    skg_status st = skg_f8_plan_query(M, N, K, epilogue, experts, 1, &d);     // the arguments alone
    if (st != SKG_OK)
        return st;
    int dev = 0, sms = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess)
        e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess)
        return launched(e, who);
    skg_f8_plan_s *p = new (std::nothrow) skg_f8_plan_s();
    if (!p)
        return set_error(SKG_ERR_CUDA, "%s: out of host memory", who);
    p->d = d;
    p->d.static_weights = static_weights != 0;
    p->device = dev;
    p->num_sms = sms;
    st = fill_launch(&p->d, 0, 0, 0, sms, who);
    if (st == SKG_OK)
        st = launched(cudaHostAlloc(reinterpret_cast<void **>(&p->err_host), sizeof(unsigned int), cudaHostAllocMapped), who);
    if (st == SKG_OK) {
        *p->err_host = 0;
        st = launched(cudaHostGetDevicePointer(reinterpret_cast<void **>(&p->err_dev), p->err_host, 0), who);
    }
    if (st != SKG_OK) {
        skg_f8_plan_destroy(p);
        return st;
    }
    *out = p;
    return SKG_OK;
}

skg_status skg_f8_plan_force(skg_f8_plan_t p, int kind, int m_tile, int split_k)
{
    static const char who[] = "skg_f8_plan_force";
    if (!p)
        return set_error(SKG_ERR_INVALID_ARG, "%s: plan is NULL", who);
    if (kind < 0 || kind > SKG_F8_KERNEL_WIDE)
        return set_error(SKG_ERR_INVALID_ARG, "%s: unknown kernel kind %d", who, kind);
    const int k = kind ? kind : p->d.kernel_kind;
    const bool wide = k == SKG_F8_KERNEL_WIDE;
    if (m_tile != 0 && !(wide ? m_tile == 128 || m_tile == 256 : m_tile == 16 || m_tile == 32 || m_tile == 64))
        return set_error(SKG_ERR_INVALID_ARG, "%s: m_tile %d is none of this kernel's", who, m_tile);
    if (split_k < 0 || split_k > max_split(k))
        return set_error(SKG_ERR_INVALID_ARG, "%s: this kernel takes a split_k of at most %d (got %d)", who, max_split(k), split_k);
    skg_f8_plan_desc d = p->d;
    const skg_status st = fill_launch(&d, k, m_tile, split_k, p->num_sms, who);
    if (st == SKG_OK)
        p->d = d;
    return st;
}

skg_status skg_f8_plan_info(skg_f8_plan_t p, skg_f8_plan_desc *out)
{
    if (!p || !out)
        return set_error(SKG_ERR_INVALID_ARG, "skg_f8_plan_info: plan and out must be non-NULL");
    *out = p->d;
    return SKG_OK;
}

skg_status skg_f8_run(skg_f8_plan_t p, const void *x, const float *x_scale, const void *W, const float *w_scale,
                      const void *residual, const int *offsets, void *y, void *stream)
{
    static const char who[] = "skg_f8_run";
    if (!p)
        return set_error(SKG_ERR_INVALID_ARG, "%s: plan is NULL", who);
    if (!x || !x_scale || !W || !w_scale || !y)
        return set_error(SKG_ERR_INVALID_ARG, "%s: x, x_scale, W, w_scale and y must be non-NULL", who);
    const skg_f8_plan_desc &d = p->d;
    const bool want = d.epilogue == SKG_EPI_BF16_RESIDUAL;
    if (want != (residual != nullptr))
        return set_error(SKG_ERR_INVALID_ARG, want ? "%s: this plan's epilogue needs a residual"
                                                   : "%s: this plan's epilogue takes no residual", who);
    if ((d.experts != 0) != (offsets != nullptr))
        return set_error(SKG_ERR_INVALID_ARG, d.experts ? "%s: this plan's experts need offsets"
                                                        : "%s: this plan has no experts and takes no offsets", who);
    if (!aligned(x, 16) || !aligned(W, 16))
        return set_error(SKG_ERR_ALIGNMENT, "%s: x and W must be 16-byte aligned", who);
    if (!aligned(x_scale, 4) || !aligned(w_scale, 4) || !aligned(y, d.epilogue == SKG_EPI_FP32 ? 4 : 2) ||
        !aligned(residual, 2) || !aligned(offsets, 4))
        return set_error(SKG_ERR_ALIGNMENT, "%s: a scale, y, residual or offsets misses its element alignment", who);
    int dev = 0;
    const cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess)
        return launched(e, who);
    if (dev != p->device)
        return set_error(SKG_ERR_INVALID_ARG, "%s: the plan is of device %d, the current one is %d", who, p->device, dev);
    if (__atomic_exchange_n(p->err_host, 0u, __ATOMIC_ACQ_REL) != 0)
        return set_error(SKG_ERR_DEVICE_TIMEOUT, "%s: an earlier launch of this plan ran out of a bounded wait", who);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    p->last_stream = s;
    F8LinearParams g = {};
    g.x_scale = x_scale;
    g.w_scale = w_scale;
    g.res = static_cast<const uint16_t *>(residual);
    g.y = y;
    g.offsets = offsets;
    g.err = p->err_dev;
    g.M = d.M;
    g.N = d.N;
    g.K = d.K;
    g.epilogue = d.epilogue;
    g.experts = d.experts;
    g.nkb = ceil_div(d.K, kF8Block);
    g.nb = ceil_div(d.N, kF8Block);
    g.m_tiles = ceil_div(d.M, d.m_tile);
    g.n_tiles = ceil_div(d.N, d.n_tile);
    g.split = d.split_k;
    g.static_w = d.static_weights;
    g.vec4 = d.N % 4 == 0 && aligned(residual, 8) && aligned(y, d.epilogue == SKG_EPI_FP32 ? 16 : 8);
    g.vec = d.epilogue == SKG_EPI_BF16 ? d.N % 8 == 0 && aligned(y, 16) : g.vec4;
    g.timeout_ns = kDefaultTimeoutNs;
    const bool wide = d.kernel_kind == SKG_F8_KERNEL_WIDE;
    const int w_rows = d.N * std::max(1, d.experts);
    g.w_box = std::min(kTileN, w_rows);
    g.x_box = std::min(wide ? 128 : d.m_tile, d.M);
    CUtensorMap tmW, tmX;
    // Rows that begin between two lines of 128 bytes: with the L2 fetching 256 at a
    // time the wide kernel takes longer, 4096 x 4864 x 7184 144 us instead of 132.
    const CUtensorMapL2promotion promotion = wide && d.K % 128 != 0 ? CU_TENSOR_MAP_L2_PROMOTION_L2_128B : CU_TENSOR_MAP_L2_PROMOTION_L2_256B;
    skg_status st = encode_tiled_2d(&tmW, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, W, w_rows, d.K, g.w_box, promotion);
    if (st == SKG_OK)
        st = encode_tiled_2d(&tmX, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, x, d.M, d.K, g.x_box, promotion);
    if (st != SKG_OK)
        return st;
    return launched(wide ? launch_f8_wide(tmW, tmX, g, d.m_tile, d.grid, s) : launch_f8_split(tmW, tmX, g, d.m_tile, d.grid, s), who);
}

skg_status skg_f8_plan_check(skg_f8_plan_t p)
{
    static const char who[] = "skg_f8_plan_check";
    if (!p)
        return set_error(SKG_ERR_INVALID_ARG, "%s: plan is NULL", who);
    cudaError_t e = p->last_stream ? cudaStreamSynchronize(p->last_stream) : cudaDeviceSynchronize();
    if (e == cudaSuccess)
        e = cudaGetLastError();
    if (e != cudaSuccess)
        return launched(e, who);
    const unsigned w = __atomic_exchange_n(p->err_host, 0u, __ATOMIC_ACQ_REL);
    if (w != 0)
        return set_error(SKG_ERR_DEVICE_TIMEOUT, "a kernel of this plan ran out of a bounded wait (bits 0x%x)", w);
    return SKG_OK;
}

skg_status skg_f8_debug_wait_timeout(skg_f8_plan_t p, unsigned long long timeout_ns, void *stream)
{
    static const char who[] = "skg_f8_debug_wait_timeout";
    if (!p)
        return set_error(SKG_ERR_INVALID_ARG, "%s: plan is NULL", who);
    if (timeout_ns == 0 || timeout_ns > 10000000000ull)
        return set_error(SKG_ERR_INVALID_ARG, "%s: timeout_ns must be in (0, 10 s]", who);
    p->last_stream = static_cast<cudaStream_t>(stream);
    return launched(launch_debug_wait(p->err_dev, timeout_ns, p->last_stream), who);
}

skg_status skg_f8_plan_destroy(skg_f8_plan_t p)
{
    if (!p)
        return SKG_OK;
    if (p->err_host)
        cudaFreeHost(p->err_host);
    delete p;
    return SKG_OK;
}

} // extern "C"

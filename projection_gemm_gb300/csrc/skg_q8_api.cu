// skg_q8_api.cu -- host side of the 8-bit path of include/skg.h: argument
// checks, plans and launches.
#include <algorithm>
#include <cstdint>
#include <new>
#include <vector>

#include <cuda.h>
#include <cuda_runtime.h>

#include "skg.h"
#include "skg_internal.h"
#include "skg_q8_internal.h"

using namespace skg;

struct skg_q8_plan_s {
    skg_q8_plan_desc d;
    int num_sms = 0;
    void *ws = nullptr;               // sums put away by the split kernel
    size_t ws_cap = 0;
    std::vector<void *> retired;      // outgrown workspaces: a captured graph may still use them
    unsigned int *err_host = nullptr; // mapped pinned word
    unsigned int *err_dev = nullptr;
    cudaStream_t last_stream = nullptr;
};

namespace {

constexpr int kQ8MaxK = 131056;       // (-128)^2 K < 2^31, K a multiple of 16
constexpr int kQ8MaxM = 1 << 18;

bool aligned(const void *p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

skg_status check_rows(const char *who, int M, int K, const void *x, size_t ldx, const void *q, const float *scale)
{
    if (M < 0 || K < 1)
        return set_error(SKG_ERR_INVALID_ARG, "%s: M must be >= 0 and K >= 1 (got M=%d, K=%d)", who, M, K);
    if (M > 0 && (!x || !q || !scale))
        return set_error(SKG_ERR_INVALID_ARG, "%s: x, q and scale must be non-NULL", who);
    if (ldx < static_cast<size_t>(K))
        return set_error(SKG_ERR_INVALID_ARG, "%s: row stride %zu of x is below K = %d", who, ldx, K);
    if (!aligned(x, 2) || !aligned(scale, 4))
        return set_error(SKG_ERR_ALIGNMENT, "%s: x / scale miss their element alignment", who);
    return SKG_OK;
}

skg_status launched(cudaError_t e, const char *who)
{
    return e == cudaSuccess ? SKG_OK
                            : set_error(SKG_ERR_CUDA, "%s: %s (%s)", who, cudaGetErrorName(e), cudaGetErrorString(e));
}

constexpr int kQ8Band = 8;            // token tiles per band of the tile order
constexpr int kQ8BlockK = 128;        // k per unit of the tcgen05 kernels
constexpr int kStreamMaxM = 16;

int ceil_div(int a, int b) { return a / b + (a % b != 0); }

// Clusters resident at once on 152 SMs, by what a cluster's tile has its K
// split into (cudaOccupancyMaxActiveClusters; a cluster stays within one GPC):
// CTAs of the split kernel, two to an SM; pairs of the wide kernel, one CTA to
// an SM.  43 tiles split in 7 are 301 CTAs, but 38 clusters at a time.  (With
// another number of SMs the counts are scaled, which clusters need not follow; a
// launch that does not fit takes longer and gives the same result.)
constexpr int kSplitResident[] = {0, 304, 152, 97, 74, 58, 46, 38, 36};
constexpr int kWideResident[] = {0, 76, 36, 23, 15};
static_assert(sizeof(kWideResident) / sizeof(int) == kQ8WideMaxSplit + 1, "a count for each split");

long long resident(int on_152, int num_sms) { return std::max(1ll, static_cast<long long>(on_152) * num_sms / 152); }

// The tcgen05 kernels' times (us) as measured.  A CTA of the split kernel takes
// 0.93 a unit of 128 k, 0.52 if it has the SM to itself (0.69 and 0.40 with
// tiles of 32 tokens), and 2.8 for its ends, 2.2 more to join a split K.
double split_us(long long tiles, int nkb, int m_tile, int split, int num_sms)
{
    const long long slots = resident(kSplitResident[split], num_sms), waves = (tiles + slots - 1) / slots;
    const bool alone = tiles * split <= num_sms;
    const double unit = m_tile == 32 ? (alone ? 0.40 : 0.69) : (alone ? 0.52 : 0.93);
    return static_cast<double>(waves) * ((split > 1 ? 5.0 : 2.8) + unit * ceil_div(nkb, split));
}

// A pair of the wide kernel takes 0.42 a unit and 0.9 a tile, but no less than
// its epilogue's 2.6, and 5.4 for its ends, 3.5 more to join a split K.
double wide_us(long long tiles, int nkb, int split, int num_sms)
{
    const long long slots = resident(kWideResident[split], num_sms), waves = (tiles + slots - 1) / slots;
    return (split > 1 ? 8.9 : 5.4) + static_cast<double>(waves) * std::max(2.6, 0.9 + 0.42 * ceil_div(nkb, split));
}

struct TcChoice {
    int m_tile, split;
    double us;
};

long long tiles_of(const skg_q8_plan_desc &d, int n_tile, int m_tile)
{
    return static_cast<long long>(ceil_div(d.N, n_tile)) * ceil_div(d.M, m_tile);
}

// The split kernel's tile and the CTAs that share its K, given either or none
// (0): the fastest of those whose clusters are resident at once.  Measured, with
// 1 ... CTAs of 64-token tiles, then of 32: 428 x 1560 x 976 6.7, 8.2, 9.1 and
// 7.4, 13.6; 204 x 120 x 10800 44, 26, 19, 14.8, (8) 9.4 and 34, 19.9, (4) 10.9,
// (8) 7.2; 64 x 7168 x 7168 31, 20.1, 20.6, (5) 15.3.
TcChoice choose_split(const skg_q8_plan_desc &d, int m_tile, int split, int num_sms)
{
    const int nkb = ceil_div(d.K, kQ8BlockK);
    TcChoice best = {0, 0, 0.0};
    for (int mt = 64; mt >= 32; mt -= 32) {
        if (m_tile ? mt != m_tile : mt == 64 && d.M <= 32)
            continue;
        const long long tiles = tiles_of(d, kTileN, mt);
        for (int s = 1; s <= std::min(8, nkb); ++s) {
            if (split ? s != std::min(split, nkb) : s > 1 && tiles > resident(kSplitResident[s], num_sms))
                continue;
            const double us = split_us(tiles, nkb, mt, s, num_sms);
            if (!best.split || us < best.us)
                best = {mt, s, us};
        }
    }
    return best;
}

// Pairs that share a tile's K in the wide kernel, in the same way.  Measured
// with 1, 2, 3 and 4: 128 x 7168 x 7168 29.4, 22.0, 34.7, 32.9; 65 x 7168 x 16384
// 58, 36.1, 53, 46; 128 x 2048 x 4096 19.0, 14.6, 12.7, 12.8; 100 x 8192 x 2048
// 13.7, 13.0, 22.8, 32.7.
TcChoice choose_wide(const skg_q8_plan_desc &d, int split, int num_sms)
{
    const int nkb = ceil_div(d.K, kQ8BlockK), mt = q8_wide_shape().m_tile;
    const long long tiles = tiles_of(d, 2 * kTileN, mt);
    TcChoice best = {0, 0, 0.0};
    for (int s = 1; s <= std::min(kQ8WideMaxSplit, nkb); ++s) {
        if (split ? s != std::min(split, nkb) : s > 1 && tiles > resident(kWideResident[s], num_sms))
            continue;
        const double us = wide_us(tiles, nkb, s, num_sms);
        if (!best.split || us < best.us)
            best = {mt, s, us};
    }
    return best;
}

// The streaming kernel up to 8 tokens, and up to 16 while its CTAs fit in one
// wave (three to an SM) or W is so small that the split kernel's ends weigh more.  Measured, stream then split: 8 x 12288 x 7168 16.9 and
// 19.0, 8 x 28672 x 8192 39.6 and 45; 16 x 2432 x 7168 6.1 and 7.9, 16 x 7296 x
// 7168 11.9 and 12.5, 9 x 5000 x 4112 7.9 and 8.4; beyond, 16 x 9216 x 4096 14.0
// and 9.9, 9 x 16384 x 7168 29 and 24, 16 x 16384 x 2048 11.5 and 9.3, but 16 x
// 12288 x 1024 6.1 and 6.8.  It is furthest off at 16 x 4096 x 16384, 16.9 and 15.0.
bool prefer_stream(const skg_q8_plan_desc &d, int num_sms)
{
    return d.M <= 8 || (d.M <= kStreamMaxM && (ceil_div(d.N, 16) <= 3 * num_sms || static_cast<long long>(d.N) * d.K <= (16 << 20)));
}

// The split or the wide kernel.  Measured, split then wide: 24 x 28672 x 8192
// 47 and 63, 128 x 1024 x 7168 10.0 and 13.9, 128 x 7168 x 7168 26.5 and 21.9,
// 256 x 4096 x 4096 18.5 and 16.7, 1849 x 680 x 320 5.5 and 8.7, 1000 x 4096 x
// 4096 52 and 33.6.  It is furthest off at 64 x 28672 x 8192, 55.6 and 63.5, where
// the wide kernel is taken.
bool prefer_split(const skg_q8_plan_desc &d, int num_sms)
{
    return choose_split(d, 0, 0, num_sms).us <= choose_wide(d, 0, num_sms).us;
}

// Accumulations of 1024 k that a CTA of the split kernel puts away: all but two.
int carried(const skg_q8_plan_desc &d)
{
    const int units = ceil_div(ceil_div(d.K, kQ8BlockK), d.split_k);
    return std::max(0, ceil_div(units * kQ8BlockK, 1024) - 2);
}

skg_status fill_launch(skg_q8_plan_desc *d, int kind, int m_tile, int split, int num_sms, const char *who)
{
    if (!kind)
        kind = prefer_stream(*d, num_sms)  ? SKG_Q8_KERNEL_STREAM
               : prefer_split(*d, num_sms) ? SKG_Q8_KERNEL_SPLIT
                                           : SKG_Q8_KERNEL_WIDE;
    d->kernel_kind = kind;
    d->split_k = 1;
    d->smem_bytes = d->stages = 0;
    d->workspace_bytes = 0;
    if (kind == SKG_Q8_KERNEL_STREAM) {
        if (d->M > kStreamMaxM)
            return set_error(SKG_ERR_UNSUPPORTED, "%s: the streaming kernel takes at most %d tokens (M=%d)", who,
                             kStreamMaxM, d->M);
        const Q8StreamShape sh = q8_stream_shape(d->M, d->N, num_sms);
        d->m_tile = d->M <= 8 ? 8 : 16;
        d->n_tile = 16 * sh.groups;
        d->tiles = d->grid = ceil_div(d->N, d->n_tile);
        d->threads = 32 * sh.warps;
        d->ctas_per_sm = sh.ctas_per_sm;
        return SKG_OK;
    }
    const bool wide = kind == SKG_Q8_KERNEL_WIDE;
    const TcChoice c = wide ? choose_wide(*d, split, num_sms) : choose_split(*d, m_tile, split, num_sms);
    d->m_tile = c.m_tile;
    d->split_k = c.split;
    d->n_tile = wide ? 2 * kTileN : kTileN;
    const long long tiles = tiles_of(*d, d->n_tile, d->m_tile);
    if (tiles > (1ll << 27))
        return set_error(SKG_ERR_UNSUPPORTED, "%s: more than 2^27 tiles", who);
    d->tiles = static_cast<int>(tiles);
    const Q8TcShape sh = wide ? q8_wide_shape() : q8_split_shape(d->m_tile);
    d->threads = sh.threads;
    d->smem_bytes = sh.smem_bytes;
    d->stages = sh.stages;
    d->ctas_per_sm = sh.ctas_per_sm;
    if (wide) {
        d->grid = 2 * d->split_k * (d->split_k > 1 ? d->tiles : std::min(d->tiles, std::max(1, num_sms / 2)));
        return SKG_OK;
    }
    d->grid = d->tiles * d->split_k;
    d->workspace_bytes = static_cast<size_t>(d->grid) * carried(*d) * d->m_tile * kTileN * 4;
    return SKG_OK;
}

skg_status ensure_workspace(skg_q8_plan_s *p, const char *who)
{
    const size_t need = p->d.workspace_bytes;
    if (need <= p->ws_cap)
        return SKG_OK;
    try {                             // the only allocation that could throw, out of a C entry
        p->retired.reserve(p->retired.size() + 1);
    } catch (const std::bad_alloc &) {
        return set_error(SKG_ERR_CUDA, "%s: out of host memory", who);
    }
    void *ws = nullptr;
    const cudaError_t e = cudaMalloc(&ws, need);
    if (e != cudaSuccess)
        return launched(e, who);
    if (p->ws)
        p->retired.push_back(p->ws);  // has its place
    p->ws = ws;
    p->ws_cap = need;
    return SKG_OK;
}

} // namespace

extern "C" {

skg_status skg_rmsnorm_q8(int M, int K, float eps, const void *x, size_t ldx, const void *residual, size_t ldr,
                          const void *gamma, void *h, size_t ldh, void *y, void *q, float *scale, void *stream)
{
    static const char who[] = "skg_rmsnorm_q8";
    const skg_status st = check_rows(who, M, K, x, ldx, q, scale);
    if (st != SKG_OK)
        return st;
    if (!(eps >= 0.0f) || eps > 3.402823466e38f)
        return set_error(SKG_ERR_INVALID_ARG, "%s: eps must be a finite number >= 0", who);
    if (h && !residual)
        return set_error(SKG_ERR_INVALID_ARG, "%s: h is written only where a residual is added", who);
    if ((residual && ldr < static_cast<size_t>(K)) || (h && ldh < static_cast<size_t>(K)))
        return set_error(SKG_ERR_INVALID_ARG, "%s: a row stride of residual / h is below K = %d", who, K);
    if (!aligned(residual, 2) || !aligned(gamma, 2) || !aligned(h, 2) || !aligned(y, 2))
        return set_error(SKG_ERR_ALIGNMENT, "%s: a bf16 tensor misses its element alignment", who);
    if (M == 0)
        return SKG_OK;
    Q8RowParams p = {};
    p.x = static_cast<const uint16_t *>(x);
    p.second = static_cast<const uint16_t *>(residual);
    p.gamma = static_cast<const uint16_t *>(gamma);
    p.h = static_cast<uint16_t *>(h);
    p.y = static_cast<uint16_t *>(y);
    p.q = static_cast<int8_t *>(q);
    p.scale = scale;
    p.ldx = ldx;
    p.ld2 = ldr;
    p.ldh = ldh;
    p.M = M;
    p.K = K;
    p.eps = eps;
    return launched(launch_q8_norm(p, static_cast<cudaStream_t>(stream)), who);
}

skg_status skg_quantize_q8(int M, int K, const void *x, size_t ldx, const void *gate, size_t ldg, void *q,
                           float *scale, void *stream)
{
    static const char who[] = "skg_quantize_q8";
    const skg_status st = check_rows(who, M, K, x, ldx, q, scale);
    if (st != SKG_OK)
        return st;
    if (gate && ldg < static_cast<size_t>(K))
        return set_error(SKG_ERR_INVALID_ARG, "%s: row stride %zu of gate is below K = %d", who, ldg, K);
    if (!aligned(gate, 2))
        return set_error(SKG_ERR_ALIGNMENT, "%s: gate misses its element alignment", who);
    if (M == 0)
        return SKG_OK;
    Q8RowParams p = {};
    p.x = static_cast<const uint16_t *>(x);
    p.second = static_cast<const uint16_t *>(gate);
    p.q = static_cast<int8_t *>(q);
    p.scale = scale;
    p.ldx = ldx;
    p.ld2 = ldg;
    p.M = M;
    p.K = K;
    return launched(launch_q8_quantize(p, static_cast<cudaStream_t>(stream)), who);
}

skg_status skg_q8_plan_query(int M, int N, int K, int epilogue, int num_sms, skg_q8_plan_desc *out)
{
    static const char who[] = "skg_q8_plan_query";
    if (!out)
        return set_error(SKG_ERR_INVALID_ARG, "%s: out is NULL", who);
    if (M < 1 || N < 1 || num_sms < 1)
        return set_error(SKG_ERR_INVALID_ARG, "%s: M, N and num_sms must be positive (got %d, %d, %d)", who, M, N,
                         num_sms);
    if (epilogue < SKG_EPI_BF16 || epilogue > SKG_EPI_FP32)
        return set_error(SKG_ERR_INVALID_ARG, "%s: unknown epilogue %d", who, epilogue);
    if (K < 16 || K % 16 != 0 || K > kQ8MaxK)
        return set_error(SKG_ERR_UNSUPPORTED, "%s: K must be a multiple of 16 in [16, %d] (got %d)", who, kQ8MaxK, K);
    if (M > kQ8MaxM)
        return set_error(SKG_ERR_UNSUPPORTED, "%s: M must be at most %d (got %d)", who, kQ8MaxM, M);
    skg_q8_plan_desc d = {};
    d.M = M;
    d.N = N;
    d.K = K;
    d.epilogue = epilogue;
    const skg_status st = fill_launch(&d, 0, 0, 0, num_sms, who);
    if (st == SKG_OK)
        *out = d;
    return st;
}

skg_status skg_q8_plan(int M, int N, int K, int epilogue, int static_weights, skg_q8_plan_t *out)
{
    static const char who[] = "skg_q8_plan";
    if (!out)
        return set_error(SKG_ERR_INVALID_ARG, "%s: out is NULL", who);
    *out = nullptr;
    skg_q8_plan_desc d;
    skg_status st = skg_q8_plan_query(M, N, K, epilogue, 1, &d);     // the arguments alone
    if (st != SKG_OK)
        return st;
    int dev = 0, sms = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess)
        e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess)
        return launched(e, who);
    skg_q8_plan_s *p = new (std::nothrow) skg_q8_plan_s();
    if (!p)
        return set_error(SKG_ERR_CUDA, "%s: out of host memory", who);
    p->d = d;
    p->d.static_weights = static_weights != 0;
    p->num_sms = sms;
    st = fill_launch(&p->d, 0, 0, 0, sms, who);
    if (st == SKG_OK)
        st = launched(cudaHostAlloc(reinterpret_cast<void **>(&p->err_host), sizeof(unsigned int), cudaHostAllocMapped), who);
    if (st == SKG_OK) {
        *p->err_host = 0;
        st = launched(cudaHostGetDevicePointer(reinterpret_cast<void **>(&p->err_dev), p->err_host, 0), who);
    }
    if (st == SKG_OK)
        st = ensure_workspace(p, who);
    if (st != SKG_OK) {
        skg_q8_plan_destroy(p);
        return st;
    }
    *out = p;
    return SKG_OK;
}

skg_status skg_q8_plan_force(skg_q8_plan_t p, int kind, int m_tile, int split_k)
{
    static const char who[] = "skg_q8_plan_force";
    if (!p)
        return set_error(SKG_ERR_INVALID_ARG, "%s: plan is NULL", who);
    if (kind < 0 || kind > SKG_Q8_KERNEL_WIDE)
        return set_error(SKG_ERR_INVALID_ARG, "%s: unknown kernel kind %d", who, kind);
    skg_q8_plan_desc d = p->d;
    const int k = kind ? kind : d.kernel_kind;
    const bool tile_ok = m_tile == 0 || (k == SKG_Q8_KERNEL_SPLIT && (m_tile == 32 || m_tile == 64)) ||
                         (k == SKG_Q8_KERNEL_WIDE && m_tile == q8_wide_shape().m_tile);
    if (!tile_ok)
        return set_error(SKG_ERR_INVALID_ARG, "%s: m_tile %d is none of this kernel's", who, m_tile);
    const int most = k == SKG_Q8_KERNEL_SPLIT ? 8 : k == SKG_Q8_KERNEL_WIDE ? kQ8WideMaxSplit : 0;
    if (split_k < 0 || split_k > most)
        return set_error(SKG_ERR_INVALID_ARG, "%s: this kernel takes a split_k of at most %d (got %d)", who, most, split_k);
    skg_status st = fill_launch(&d, k, m_tile, split_k, p->num_sms, who);
    if (st != SKG_OK)
        return st;
    const skg_q8_plan_desc old = p->d;
    p->d = d;
    st = ensure_workspace(p, who);
    if (st != SKG_OK)
        p->d = old;
    return st;
}

skg_status skg_q8_plan_info(skg_q8_plan_t p, skg_q8_plan_desc *out)
{
    if (!p || !out)
        return set_error(SKG_ERR_INVALID_ARG, "skg_q8_plan_info: plan and out must be non-NULL");
    *out = p->d;
    return SKG_OK;
}

skg_status skg_q8_run(skg_q8_plan_t p, const void *x, const float *x_scale, const void *W, const float *w_scale,
                      const void *residual, void *y, void *stream)
{
    static const char who[] = "skg_q8_run";
    if (!p)
        return set_error(SKG_ERR_INVALID_ARG, "%s: plan is NULL", who);
    if (!x || !x_scale || !W || !w_scale || !y)
        return set_error(SKG_ERR_INVALID_ARG, "%s: x, x_scale, W, w_scale and y must be non-NULL", who);
    const skg_q8_plan_desc &d = p->d;
    const bool want = d.epilogue == SKG_EPI_BF16_RESIDUAL;
    if (want != (residual != nullptr))
        return set_error(SKG_ERR_INVALID_ARG, want ? "%s: this plan's epilogue needs a residual"
                                                   : "%s: this plan's epilogue takes no residual", who);
    if (!aligned(x, 16) || !aligned(W, 16))
        return set_error(SKG_ERR_ALIGNMENT, "%s: x and W must be 16-byte aligned", who);
    if (!aligned(x_scale, 4) || !aligned(w_scale, 4) || !aligned(y, d.epilogue == SKG_EPI_FP32 ? 4 : 2) ||
        !aligned(residual, 2))
        return set_error(SKG_ERR_ALIGNMENT, "%s: a scale, y or residual misses its element alignment", who);
    if (__atomic_exchange_n(p->err_host, 0u, __ATOMIC_ACQ_REL) != 0)
        return set_error(SKG_ERR_DEVICE_TIMEOUT, "%s: an earlier launch of this plan ran out of a bounded wait", who);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    p->last_stream = s;
    Q8LinearParams g = {};
    g.x = static_cast<const int8_t *>(x);
    g.x_scale = x_scale;
    g.W = static_cast<const int8_t *>(W);
    g.w_scale = w_scale;
    g.res = static_cast<const uint16_t *>(residual);
    g.y = y;
    g.M = d.M;
    g.N = d.N;
    g.K = d.K;
    g.epilogue = d.epilogue;
    if (d.kernel_kind == SKG_Q8_KERNEL_STREAM)
        return launched(launch_q8_stream(g, {d.n_tile / 16, d.threads / 32, d.ctas_per_sm}, d.static_weights != 0, s), who);

    const int nkb = ceil_div(d.K, kQ8BlockK), m_tiles = ceil_div(d.M, d.m_tile);
    const int vec4 = d.N % 4 == 0 && aligned(w_scale, 16) && aligned(residual, 8) &&
                     aligned(y, d.epilogue == SKG_EPI_FP32 ? 16 : 8);
    CUtensorMap tmW, tmX;
    skg_status st = encode_tiled_2d(&tmW, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, W, d.N, d.K, kTileN);
    if (st != SKG_OK)
        return st;
    if (d.kernel_kind == SKG_Q8_KERNEL_SPLIT) {
        st = encode_tiled_2d(&tmX, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, x, d.M, d.K, d.m_tile);
        if (st != SKG_OK)
            return st;
        Q8SplitParams t = {};
        t.g = g;
        t.carry = static_cast<int *>(p->ws);
        t.carried = carried(d);
        t.err = p->err_dev;
        t.nkb = nkb;
        t.m_tiles = m_tiles;
        t.split = d.split_k;
        t.static_w = d.static_weights;
        t.vec4 = vec4;
        t.timeout_ns = kDefaultTimeoutNs;
        return launched(launch_q8_split(tmW, tmX, t, d.m_tile, d.grid, s), who);
    }
    st = encode_tiled_2d(&tmX, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, x, d.M, d.K, d.m_tile / 2);
    if (st != SKG_OK)
        return st;
    Q8WideParams t = {};
    t.g = g;
    t.err = p->err_dev;
    t.nkb = nkb;
    t.n_pairs = ceil_div(d.N, 2 * kTileN);
    t.m_tiles = m_tiles;
    t.tiles = d.tiles;
    t.band = kQ8Band;
    t.split = d.split_k;
    t.vec4 = vec4;
    t.static_w = d.static_weights;
    t.timeout_ns = kDefaultTimeoutNs;
    return launched(launch_q8_wide(tmW, tmX, t, d.grid, s), who);
}

skg_status skg_q8_plan_check(skg_q8_plan_t p)
{
    static const char who[] = "skg_q8_plan_check";
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

skg_status skg_q8_debug_wait_timeout(skg_q8_plan_t p, unsigned long long timeout_ns, void *stream)
{
    static const char who[] = "skg_q8_debug_wait_timeout";
    if (!p)
        return set_error(SKG_ERR_INVALID_ARG, "%s: plan is NULL", who);
    if (timeout_ns == 0 || timeout_ns > 10000000000ull)
        return set_error(SKG_ERR_INVALID_ARG, "%s: timeout_ns must be in (0, 10 s]", who);
    p->last_stream = static_cast<cudaStream_t>(stream);
    return launched(launch_debug_wait(p->err_dev, timeout_ns, p->last_stream), who);
}

skg_status skg_q8_plan_destroy(skg_q8_plan_t p)
{
    if (!p)
        return SKG_OK;
    if (p->ws)
        cudaFree(p->ws);
    for (void *w : p->retired)
        cudaFree(w);
    if (p->err_host)
        cudaFreeHost(p->err_host);
    delete p;
    return SKG_OK;
}

} // extern "C"

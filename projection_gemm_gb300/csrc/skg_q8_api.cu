// skg_q8_api.cu -- host side of the 8-bit path of include/skg.h: argument
// checks, plans and launches.
#include <cstdint>
#include <new>

#include <cuda.h>
#include <cuda_runtime.h>

#include "skg.h"
#include "skg_internal.h"
#include "skg_q8_internal.h"

using namespace skg;

struct skg_q8_plan_s {
    skg_q8_plan_desc d;
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
    *out = d;
    return SKG_OK;
}

skg_status skg_q8_plan(int M, int N, int K, int epilogue, int static_weights, skg_q8_plan_t *out)
{
    static const char who[] = "skg_q8_plan";
    if (!out)
        return set_error(SKG_ERR_INVALID_ARG, "%s: out is NULL", who);
    *out = nullptr;
    skg_q8_plan_desc d;
    const skg_status st = skg_q8_plan_query(M, N, K, epilogue, 1, &d);
    if (st != SKG_OK)
        return st;
    d.static_weights = static_weights != 0;
    skg_q8_plan_s *p = new (std::nothrow) skg_q8_plan_s();
    if (!p)
        return set_error(SKG_ERR_CUDA, "%s: out of host memory", who);
    p->d = d;
    *out = p;
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
    return launched(launch_q8_gemv(g, static_cast<cudaStream_t>(stream)), who);
}

skg_status skg_q8_plan_destroy(skg_q8_plan_t p)
{
    delete p;
    return SKG_OK;
}

} // extern "C"

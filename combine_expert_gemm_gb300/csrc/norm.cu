// Residual add + layer norm of token rows, and its backward with the
// reduction of the weight gradients (include/moe_block.h).
//
//   s = x + add (rounded to x's type);  mean = sum s / d
//   rstd = (sum (s - mean)^2 / d + eps)^-1/2;  y = (s - mean) rstd gamma + beta
//   dx = dres + rstd (w - sum w / d - xh sum(w xh) / d),  w = dy gamma,
//   xh = (s - mean) rstd;  dgamma = sum_t dy xh;  dbeta = sum_t dy
//
// All of it is bound by HBM: a few operations per element moved.
#include <math.h>

#include "../../include/moe_block.h"
#include "moe_common.cuh"

namespace moe {
namespace {

constexpr int kNormMaxD = 16384;
constexpr int kNormThreads = 256;

// Eight consecutive elements of a row as fp32.
template <typename T>
__device__ __forceinline__ void load8(const T *p, float (&f)[8]);
template <>
__device__ __forceinline__ void load8<uint16_t>(const uint16_t *p, float (&f)[8]) {
    const uint4 v = *reinterpret_cast<const uint4 *>(p);
    f[0] = bf16_lo(v.x); f[1] = bf16_hi(v.x);
    f[2] = bf16_lo(v.y); f[3] = bf16_hi(v.y);
    f[4] = bf16_lo(v.z); f[5] = bf16_hi(v.z);
    f[6] = bf16_lo(v.w); f[7] = bf16_hi(v.w);
}
template <>
__device__ __forceinline__ void load8<float>(const float *p, float (&f)[8]) {
    const float4 a = reinterpret_cast<const float4 *>(p)[0];
    const float4 b = reinterpret_cast<const float4 *>(p)[1];
    f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
    f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
}
__device__ __forceinline__ void store8(uint16_t *p, const float (&f)[8]) {
    *reinterpret_cast<uint4 *>(p) =
        make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                   pack_bf16x2(f[6], f[7]));
}
__device__ __forceinline__ void store8(float *p, const float (&f)[8]) {
    reinterpret_cast<float4 *>(p)[0] = make_float4(f[0], f[1], f[2], f[3]);
    reinterpret_cast<float4 *>(p)[1] = make_float4(f[4], f[5], f[6], f[7]);
}

__device__ __forceinline__ float block_sum(float v, float *red) {
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, off);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
    __syncthreads();
    v = 0.f;
    for (int w = 0; w < kNormThreads / 32; ++w) v += red[w];
    return v;
}

// One CTA per row; three passes over the row, the last two from L1.
template <typename XT>
__global__ void __launch_bounds__(kNormThreads)
norm_fwd_rows(int d, const XT *x, const uint16_t *add, const float *__restrict__ gamma,
              const float *__restrict__ beta, float eps, XT *x_sum, uint16_t *__restrict__ y,
              float *__restrict__ mean, float *__restrict__ rstd) {
    pdl_enter();
    __shared__ float red[kNormThreads / 32];
    const int64_t base = (int64_t)blockIdx.x * d;
    const XT *s = add ? x_sum + base : x + base;
    float sum = 0.f;
    for (int c = threadIdx.x * 8; c < d; c += kNormThreads * 8) {
        float f[8];
        load8(x + base + c, f);
        if (add) {
            float a[8];
            load8(add + base + c, a);
#pragma unroll
            for (int i = 0; i < 8; ++i) f[i] += a[i];
            store8(x_sum + base + c, f);
            load8(x_sum + base + c, f);  // the rounded sum, this thread's own store
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) sum += f[i];
    }
    const float mu = block_sum(sum, red) / (float)d;
    float sq = 0.f;
    for (int c = threadIdx.x * 8; c < d; c += kNormThreads * 8) {
        float f[8];
        load8(s + c, f);
#pragma unroll
        for (int i = 0; i < 8; ++i) sq = fmaf(f[i] - mu, f[i] - mu, sq);
    }
    const float rs = 1.f / sqrtf(block_sum(sq, red) / (float)d + eps);
    if (mean && threadIdx.x == 0) {
        mean[blockIdx.x] = mu;
        rstd[blockIdx.x] = rs;
    }
    for (int c = threadIdx.x * 8; c < d; c += kNormThreads * 8) {
        float f[8];
        load8(s + c, f);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            f[i] = (f[i] - mu) * rs;
            if (gamma) f[i] *= gamma[c + i];
            if (beta) f[i] += beta[c + i];
        }
        store8(y + base + c, f);
    }
}

template <typename XT, typename YT, typename GT>
__global__ void __launch_bounds__(kNormThreads)
norm_bwd_rows(int d, const XT *__restrict__ x, const YT *__restrict__ dy,
              const float *__restrict__ gamma, const float *__restrict__ mean,
              const float *__restrict__ rstd, const GT *dres, GT *dx) {
    pdl_enter();
    __shared__ float red[kNormThreads / 32];
    const int64_t base = (int64_t)blockIdx.x * d;
    const float mu = mean[blockIdx.x], rs = rstd[blockIdx.x];
    float sa = 0.f, sb = 0.f;
    for (int c = threadIdx.x * 8; c < d; c += kNormThreads * 8) {
        float f[8], w[8];
        load8(x + base + c, f);
        load8(dy + base + c, w);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            if (gamma) w[i] *= gamma[c + i];
            sa += w[i];
            sb = fmaf(w[i], (f[i] - mu) * rs, sb);
        }
    }
    const float a = block_sum(sa, red) / (float)d, b = block_sum(sb, red) / (float)d;
    for (int c = threadIdx.x * 8; c < d; c += kNormThreads * 8) {
        float f[8], w[8], r[8] = {0, 0, 0, 0, 0, 0, 0, 0};
        load8(x + base + c, f);
        load8(dy + base + c, w);
        if (dres) load8(dres + base + c, r);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            if (gamma) w[i] *= gamma[c + i];
            r[i] += rs * (w[i] - a - (f[i] - mu) * rs * b);
        }
        store8(dx + base + c, r);
    }
}

constexpr int kWgSplits = 64;  // row splits of the weight gradients' partial sums

// Partial dgamma / dbeta of one row split: part[split][2][d].
template <typename XT, typename YT>
__global__ void __launch_bounds__(kNormThreads)
norm_bwd_weight(int rows, int d, const XT *__restrict__ x, const YT *__restrict__ dy,
                const float *__restrict__ mean, const float *__restrict__ rstd,
                float *__restrict__ part) {
    pdl_enter();
    const int c = (blockIdx.x * kNormThreads + threadIdx.x) * 8;
    if (c >= d) return;
    const int64_t per = ((int64_t)rows + kWgSplits - 1) / kWgSplits;
    const int64_t t0 = blockIdx.y * per, t1 = min((int64_t)rows, t0 + per);
    float g[8] = {0, 0, 0, 0, 0, 0, 0, 0}, b[8] = {0, 0, 0, 0, 0, 0, 0, 0};
    for (int64_t t = t0; t < t1; ++t) {
        float f[8], w[8];
        load8(x + t * d + c, f);
        load8(dy + t * d + c, w);
        const float mu = mean[t], rs = rstd[t];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            g[i] = fmaf(w[i], (f[i] - mu) * rs, g[i]);
            b[i] += w[i];
        }
    }
    store8(part + ((int64_t)blockIdx.y * 2) * d + c, g);
    store8(part + ((int64_t)blockIdx.y * 2 + 1) * d + c, b);
}

__global__ void __launch_bounds__(kNormThreads)
norm_bwd_weight_sum(int d, const float *__restrict__ part, float *__restrict__ dgamma,
                    float *__restrict__ dbeta) {
    pdl_enter();
    const int c = blockIdx.x * kNormThreads + threadIdx.x;
    if (c >= d) return;
    float g = 0.f, b = 0.f;
    for (int s = 0; s < kWgSplits; ++s) {
        g += part[(int64_t)(2 * s) * d + c];
        b += part[(int64_t)(2 * s + 1) * d + c];
    }
    if (dgamma) dgamma[c] = g;
    if (dbeta) dbeta[c] = b;
}

inline moe_status check_norm(int32_t rows, int32_t d) {
    if (rows < 0 || d <= 0) return MOE_ERR_INVALID_ARG;
    if (d % 8 != 0) return MOE_ERR_ALIGNMENT;
    if (d > kNormMaxD) return MOE_ERR_UNSUPPORTED;
    return MOE_OK;
}

inline bool dtype_ok(int32_t t) { return t == MOE_BF16 || t == MOE_FP32; }

template <typename XT, typename YT, typename GT>
moe_status launch_norm_bwd(int32_t rows, int32_t d, const void *x, const void *dy,
                           const float *gamma, const float *mean, const float *rstd,
                           const void *dres, void *dx, float *dgamma, float *dbeta, void *ws,
                           cudaStream_t stream) {
    if (rows > 0)
        launch_pdl(norm_bwd_rows<XT, YT, GT>, rows, kNormThreads, 0, stream, d,
                   static_cast<const XT *>(x), static_cast<const YT *>(dy), gamma, mean, rstd,
                   static_cast<const GT *>(dres), static_cast<GT *>(dx));
    if (dgamma || dbeta) {
        float *part = reinterpret_cast<float *>(static_cast<uint8_t *>(ws) + 256);
        const unsigned cols = (unsigned)((d / 8 + kNormThreads - 1) / kNormThreads);
        launch_pdl(norm_bwd_weight<XT, YT>, dim3(cols, kWgSplits), kNormThreads, 0, stream, rows, d,
                   static_cast<const XT *>(x), static_cast<const YT *>(dy), mean, rstd, part);
        launch_pdl(norm_bwd_weight_sum, (d + kNormThreads - 1) / kNormThreads, kNormThreads, 0,
                   stream, d, static_cast<const float *>(part), dgamma, dbeta);
    }
    return launch_status();
}

}  // namespace
}  // namespace moe

using namespace moe;

MOE_API moe_status moe_layer_norm(int32_t rows, int32_t d, int32_t x_dtype, const void *x,
                                  const moe_bf16 *add, const float *gamma, const float *beta,
                                  float eps, void *x_sum, moe_bf16 *y, float *mean, float *rstd,
                                  cudaStream_t stream) {
    moe_status r = check_norm(rows, d);
    if (r != MOE_OK) return r;
    if (!dtype_ok(x_dtype) || !(eps > 0.f) || isinf(eps)) return MOE_ERR_INVALID_ARG;
    if (rows == 0) return MOE_OK;
    if (!x || !y || (add != nullptr) != (x_sum != nullptr) || (mean != nullptr) != (rstd != nullptr))
        return MOE_ERR_INVALID_ARG;
    const void *ptrs[] = {x, add, gamma, beta, x_sum, y, mean, rstd};
    for (const void *p : ptrs)
        if (!aligned16(p)) return MOE_ERR_ALIGNMENT;
    if (x_dtype == MOE_BF16)
        launch_pdl(norm_fwd_rows<uint16_t>, rows, kNormThreads, 0, stream, d,
                   static_cast<const uint16_t *>(x), add, gamma, beta, eps,
                   static_cast<uint16_t *>(x_sum), y, mean, rstd);
    else
        launch_pdl(norm_fwd_rows<float>, rows, kNormThreads, 0, stream, d,
                   static_cast<const float *>(x), add, gamma, beta, eps,
                   static_cast<float *>(x_sum), y, mean, rstd);
    return launch_status();
}

MOE_API size_t moe_layer_norm_backward_workspace_bytes(int32_t rows, int32_t d) {
    if (check_norm(rows, d) != MOE_OK) return 0;
    return 256 + (size_t)kWgSplits * 2 * d * sizeof(float);
}

MOE_API moe_status moe_layer_norm_backward(int32_t rows, int32_t d, int32_t x_dtype, const void *x,
                                           int32_t dy_dtype, const void *dy, const float *gamma,
                                           const float *mean, const float *rstd, int32_t dx_dtype,
                                           const void *dres, void *dx, float *dgamma, float *dbeta,
                                           void *ws, size_t ws_bytes, cudaStream_t stream) {
    moe_status r = check_norm(rows, d);
    if (r != MOE_OK) return r;
    if (!dtype_ok(x_dtype) || !dtype_ok(dy_dtype) || !dtype_ok(dx_dtype)) return MOE_ERR_INVALID_ARG;
    if (rows > 0 && (!x || !dy || !mean || !rstd || !dx)) return MOE_ERR_INVALID_ARG;
    const void *ptrs[] = {x, dy, gamma, mean, rstd, dres, dx, dgamma, dbeta};
    for (const void *p : ptrs)
        if (!aligned16(p)) return MOE_ERR_ALIGNMENT;
    if (!ws || (reinterpret_cast<uintptr_t>(ws) & 255u) ||
        ws_bytes < moe_layer_norm_backward_workspace_bytes(rows, d))
        return MOE_ERR_WORKSPACE;
    auto go = [&](auto xt, auto yt, auto gt) {
        return launch_norm_bwd<decltype(xt), decltype(yt), decltype(gt)>(
            rows, d, x, dy, gamma, mean, rstd, dres, dx, dgamma, dbeta, ws, stream);
    };
    auto go_g = [&](auto xt, auto yt) {
        return dx_dtype == MOE_BF16 ? go(xt, yt, uint16_t()) : go(xt, yt, float());
    };
    auto go_y = [&](auto xt) {
        return dy_dtype == MOE_BF16 ? go_g(xt, uint16_t()) : go_g(xt, float());
    };
    return x_dtype == MOE_BF16 ? go_y(uint16_t()) : go_y(float());
}

// The router's products for a gradient of every logit (include/moe_block.h):
//   dx = dx_in + dl W;  dW = dl^T x;  dbias = column sums of dl
// with dl [T, N] fp32, W [N, d] fp32, x [T, d] bf16.
#include "../../include/moe_block.h"
#include "moe_common.cuh"

namespace moe {
namespace {

constexpr int kRdCols = 256;    // threads per CTA, one output column each
constexpr int kRdTok = 32;      // tokens per CTA of the dx kernel
constexpr int kRdExp = 16;      // experts per CTA of the dW kernel
constexpr int kRdChunk = 64;    // experts or tokens staged at a time
constexpr int kRdSplits = 32;   // token splits of dW

__global__ void __launch_bounds__(kRdCols)
router_dense_dx(int T, int N, int d, const float *__restrict__ dl, const float *__restrict__ w,
                const float *dx_in, float *dx) {
    pdl_enter();
    __shared__ float sm[kRdTok][kRdChunk];
    const int col = blockIdx.y * kRdCols + threadIdx.x;
    const int64_t t0 = (int64_t)blockIdx.x * kRdTok;
    float acc[kRdTok];
#pragma unroll
    for (int i = 0; i < kRdTok; ++i) acc[i] = 0.f;
    for (int e0 = 0; e0 < N; e0 += kRdChunk) {
        __syncthreads();
        for (int i = threadIdx.x; i < kRdTok * kRdChunk; i += kRdCols) {
            const int64_t t = t0 + i / kRdChunk;
            const int e = e0 + i % kRdChunk;
            sm[i / kRdChunk][i % kRdChunk] = t < T && e < N ? dl[t * N + e] : 0.f;
        }
        __syncthreads();
        if (col >= d) continue;
        for (int j = 0; j < kRdChunk && e0 + j < N; ++j) {
            const float v = w[(int64_t)(e0 + j) * d + col];
#pragma unroll
            for (int i = 0; i < kRdTok; ++i) acc[i] = fmaf(sm[i][j], v, acc[i]);
        }
    }
    if (col >= d) return;
#pragma unroll
    for (int i = 0; i < kRdTok; ++i) {
        const int64_t t = t0 + i;
        if (t < T) dx[t * d + col] = (dx_in ? dx_in[t * d + col] : 0.f) + acc[i];
    }
}

// part[split][N][d + 1]: column d holds the sums of dl (dbias).
__global__ void __launch_bounds__(kRdCols)
router_dense_dw(int T, int N, int d, const float *__restrict__ dl, const uint16_t *__restrict__ x,
                float *__restrict__ part) {
    pdl_enter();
    __shared__ float sm[kRdChunk][kRdExp];
    // without x only the extra column, dbias, is summed
    const int col = x ? blockIdx.x * kRdCols + threadIdx.x : d + threadIdx.x;
    const int e0 = blockIdx.y * kRdExp;
    const int64_t per = ((int64_t)T + kRdSplits - 1) / kRdSplits;
    const int64_t t0 = blockIdx.z * per, t1 = min((int64_t)T, t0 + per);
    float acc[kRdExp];
#pragma unroll
    for (int i = 0; i < kRdExp; ++i) acc[i] = 0.f;
    for (int64_t tc = t0; tc < t1; tc += kRdChunk) {
        __syncthreads();
        for (int i = threadIdx.x; i < kRdChunk * kRdExp; i += kRdCols) {
            const int64_t t = tc + i / kRdExp;
            const int e = e0 + i % kRdExp;
            sm[i / kRdExp][i % kRdExp] = t < t1 && e < N ? dl[t * N + e] : 0.f;
        }
        __syncthreads();
        if (col > d) continue;
        for (int j = 0; j < kRdChunk && tc + j < t1; ++j) {
            const float v = col < d ? bf16_lo(x[(tc + j) * d + col]) : 1.f;
#pragma unroll
            for (int i = 0; i < kRdExp; ++i) acc[i] = fmaf(sm[j][i], v, acc[i]);
        }
    }
    if (col > d) return;
#pragma unroll
    for (int i = 0; i < kRdExp; ++i)
        if (e0 + i < N) part[((int64_t)blockIdx.z * N + e0 + i) * (d + 1) + col] = acc[i];
}

__global__ void __launch_bounds__(kRdCols)
router_dense_sum(int N, int d, const float *__restrict__ part, float *__restrict__ dw,
                 float *__restrict__ dbias) {
    pdl_enter();
    const int64_t n = (int64_t)N * (d + 1);
    const int64_t i = (int64_t)blockIdx.x * kRdCols + threadIdx.x;
    if (i >= n) return;
    float v = 0.f;
    for (int s = 0; s < kRdSplits; ++s) v += part[s * n + i];
    const int64_t e = i / (d + 1);
    const int c = (int)(i % (d + 1));
    if (c < d) {
        if (dw) dw[e * d + c] = v;
    } else if (dbias) {
        dbias[e] = v;
    }
}

}  // namespace
}  // namespace moe

using namespace moe;

MOE_API size_t moe_router_dense_backward_workspace_bytes(const moe_shape *s) {
    if (check_shape(s) != MOE_OK) return 0;
    return 256 + (size_t)kRdSplits * s->N * (s->d + 1) * sizeof(float);
}

MOE_API moe_status moe_router_dense_backward(const moe_shape *s, const moe_bf16 *x,
                                             const float *w_router, const float *dlogits,
                                             const float *dx_in, float *dx, float *dw_router,
                                             float *dbias, void *ws, size_t ws_bytes,
                                             cudaStream_t stream) {
    moe_status r = check_shape(s);
    if (r != MOE_OK) return r;
    if (s->T > 0 && (!dlogits || (dx && !w_router) || (dw_router && !x) || (dx_in && !dx)))
        return MOE_ERR_INVALID_ARG;
    const void *ptrs[] = {x, w_router, dlogits, dx_in, dx, dw_router, dbias};
    for (const void *p : ptrs)
        if (!aligned16(p)) return MOE_ERR_ALIGNMENT;
    if (!ws || (reinterpret_cast<uintptr_t>(ws) & 255u) ||
        ws_bytes < moe_router_dense_backward_workspace_bytes(s))
        return MOE_ERR_WORKSPACE;
    const int T = s->T, N = s->N, d = s->d;
    if (!dx && !dw_router && !dbias) return MOE_OK;
    if (dx && T > 0)
        launch_pdl(router_dense_dx, dim3((T + kRdTok - 1) / kRdTok, (d + kRdCols - 1) / kRdCols),
                   kRdCols, 0, stream, T, N, d, dlogits, w_router, dx_in, dx);
    if (dw_router || dbias) {
        float *part = reinterpret_cast<float *>(static_cast<uint8_t *>(ws) + 256);
        launch_pdl(router_dense_dw,
                   dim3(dw_router ? d / kRdCols + 1 : 1, (N + kRdExp - 1) / kRdExp, kRdSplits),
                   kRdCols, 0, stream, T, N, d, dlogits,
                   dw_router ? x : static_cast<const moe_bf16 *>(nullptr), part);
        const int64_t n = (int64_t)N * (d + 1);
        launch_pdl(router_dense_sum, (unsigned)((n + kRdCols - 1) / kRdCols), kRdCols, 0, stream, N,
                   d, static_cast<const float *>(part), dw_router, dbias);
    }
    return launch_status();
}

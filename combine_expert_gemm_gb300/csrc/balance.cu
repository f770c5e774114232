// The router's balance loss and z loss, and their gradient with respect to
// every logit (include/moe_block.h).
//
//   p = softmax(logits[t]);  balance = N sum_e c_e / (Tc K) sum_t p_te / Tc
//   z = sum_t lse_t^2 / Tc
//   dlogits = p (gb N / Tc (f - sum_e p_e f_e) + gz 2 lse / Tc) + scattered dlogit
//
// One warp per token.  Both kernels move the [T, N] logits once and are bound
// by HBM at length and by their launches when short.
#include "../../include/moe_block.h"
#include "moe_common.cuh"

namespace moe {
namespace {

constexpr int kBalWarps = 8;
constexpr int kBalThreads = kBalWarps * 32;
constexpr int kBalMaxCtas = 304;

// Partial sums of one CTA in the workspace, N + 2 words of each kind:
// int32 counts [N], token count, padding; then fp32 probability sums [N],
// sum of lse^2, padding.
inline __host__ __device__ int64_t bal_stride(int N) { return (N + 2 + 3) / 4 * 4; }

__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) v = fmaxf(v, __shfl_xor_sync(0xFFFFFFFFu, v, off));
    return v;
}
__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, off);
    return v;
}

__global__ void __launch_bounds__(kBalThreads)
balance_partial(int T, int N, int K, const float *__restrict__ logits,
                const int32_t *__restrict__ topk_idx, const uint8_t *__restrict__ mask,
                float *__restrict__ lse, int32_t *__restrict__ part_i, float *__restrict__ part_f) {
    pdl_enter();
    extern __shared__ float sm[];
    float *acc = sm;                                              // [warps][N]
    int *cnt = reinterpret_cast<int *>(sm + kBalWarps * N);       // [N]
    float *zs = reinterpret_cast<float *>(cnt + N);               // [warps]
    int *ts = reinterpret_cast<int *>(zs + kBalWarps);            // [warps]
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    for (int i = threadIdx.x; i < (kBalWarps + 1) * N; i += kBalThreads) sm[i] = 0.f;
    __syncthreads();
    float z = 0.f;
    int tok = 0;
    float *my = acc + warp * N;
    for (int64_t t = (int64_t)blockIdx.x * kBalWarps + warp; t < T; t += gridDim.x * kBalWarps) {
        if (mask && mask[t] == 0) {
            if (lane == 0) lse[t] = 0.f;
            continue;
        }
        const float *l = logits + t * N;
        float m = -INFINITY;
        for (int e = lane; e < N; e += 32) m = fmaxf(m, l[e]);
        m = warp_max(m);
        if (m == -INFINITY) m = 0.f;  // all -inf: probabilities 0; all NaN: NaN below
        float sum = 0.f;
        for (int e = lane; e < N; e += 32) sum += expf(l[e] - m);
        sum = warp_sum(sum);
        const float inv = sum == 0.f ? 0.f : 1.f / sum;
        for (int e = lane; e < N; e += 32) my[e] += expf(l[e] - m) * inv;
        const float v = m + logf(sum);
        if (sum != 0.f) z = fmaf(v, v, z);
        ++tok;
        if (lane == 0) lse[t] = v;
        if (lane < K) {
            const int e = topk_idx[t * K + lane];
            if (e >= 0 && e < N) atomicAdd(cnt + e, 1);
        }
    }
    if (lane == 0) {
        zs[warp] = z;
        ts[warp] = tok;
    }
    __syncthreads();
    part_i += blockIdx.x * bal_stride(N);
    part_f += blockIdx.x * bal_stride(N);
    for (int e = threadIdx.x; e < N; e += kBalThreads) {
        float p = 0.f;
        for (int w = 0; w < kBalWarps; ++w) p += acc[w * N + e];
        part_i[e] = cnt[e];
        part_f[e] = p;
    }
    if (threadIdx.x == 0) {
        float p = 0.f;
        int n = 0;
        for (int w = 0; w < kBalWarps; ++w) {
            p += zs[w];
            n += ts[w];
        }
        part_i[N] = n;
        part_f[N] = p;
    }
}

// One CTA: the partial sums over CTAs in order, and the two losses.
__global__ void __launch_bounds__(1024)
balance_finish(int N, int K, int ctas, const int32_t *__restrict__ part_i,
               const float *__restrict__ part_f, int32_t *__restrict__ count,
               int32_t *__restrict__ token_count, float *__restrict__ prob,
               float *__restrict__ losses) {
    pdl_enter();
    __shared__ float sum_f[1025];
    __shared__ int sum_i[1025];
    __shared__ float red[32];
    const int64_t st = bal_stride(N);
    for (int e = threadIdx.x; e <= N; e += blockDim.x) {
        float p = 0.f;
        int c = 0;
        for (int g = 0; g < ctas; ++g) {
            p += part_f[g * st + e];
            c += part_i[g * st + e];
        }
        sum_f[e] = p;
        sum_i[e] = c;
    }
    __syncthreads();
    const int tc = sum_i[N];
    const float inv = tc > 0 ? 1.f / (float)tc : 0.f;
    float dot = 0.f;
    const int e = threadIdx.x;
    if (e < N) {
        const float p = sum_f[e] * inv;
        count[e] = sum_i[e];
        prob[e] = p;
        dot = (float)sum_i[e] * inv / (float)K * p;
    }
    dot = warp_sum(dot);
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = dot;
    __syncthreads();
    if (threadIdx.x == 0) {
        float b = 0.f;
        for (int w = 0; w < (int)blockDim.x / 32; ++w) b += red[w];
        token_count[0] = tc;
        losses[0] = (float)N * b;
        losses[1] = sum_f[N] * inv;
    }
}

__global__ void __launch_bounds__(kBalThreads)
balance_bwd_rows(int T, int N, int K, const float *__restrict__ logits,
                 const int32_t *__restrict__ topk_idx, const uint8_t *__restrict__ mask,
                 const int32_t *__restrict__ count, const int32_t *__restrict__ token_count,
                 const float *__restrict__ lse, const float *__restrict__ dlosses,
                 const float *__restrict__ dlogit, float *__restrict__ dlogits) {
    pdl_enter();
    extern __shared__ float sm[];
    float *f = sm;  // [N]
    const int tc = token_count[0];
    const float inv = tc > 0 ? 1.f / (float)tc : 0.f;
    for (int e = threadIdx.x; e < N; e += kBalThreads) f[e] = (float)count[e] * inv / (float)K;
    __syncthreads();
    const float cb = dlosses[0] * (float)N * inv, cz = 2.f * dlosses[1] * inv;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    for (int64_t t = (int64_t)blockIdx.x * kBalWarps + warp; t < T; t += gridDim.x * kBalWarps) {
        const float *l = logits + t * N;
        float *o = dlogits + t * N;
        const bool live = !(mask && mask[t] == 0);
        float v = 0.f, dot = 0.f;
        bool none = true;  // no probability: masked, or every logit -inf
        if (live) {
            v = lse[t];
            none = v == -INFINITY;
            if (!none)
                for (int e = lane; e < N; e += 32) dot = fmaf(expf(l[e] - v), f[e], dot);
            dot = warp_sum(dot);
        }
        int my_e = -1;
        float my_d = 0.f;
        if (dlogit && lane < K) {
            my_e = topk_idx[t * K + lane];
            my_d = dlogit[t * K + lane];
        }
        for (int e0 = 0; e0 < N; e0 += 32) {
            const int e = e0 + lane;
            float r = 0.f;
            if (!none && e < N) r = expf(l[e] - v) * (cb * (f[e] - dot) + cz * v);
            if (dlogit)
                for (int k = 0; k < K; ++k) {
                    const int ek = __shfl_sync(0xFFFFFFFFu, my_e, k);
                    const float dk = __shfl_sync(0xFFFFFFFFu, my_d, k);
                    if (ek == e) r += dk;
                }
            if (e < N) o[e] = r;
        }
    }
}

inline int bal_ctas(int T) {
    const int want = (T + kBalWarps - 1) / kBalWarps;
    return want < kBalMaxCtas ? (want < 1 ? 1 : want) : kBalMaxCtas;
}

inline bool ws_ok(const void *ws, size_t have, size_t need) {
    return ws && (reinterpret_cast<uintptr_t>(ws) & 255u) == 0 && have >= need;
}

}  // namespace
}  // namespace moe

using namespace moe;

MOE_API size_t moe_balance_loss_workspace_bytes(const moe_shape *s) {
    if (check_shape(s) != MOE_OK) return 0;
    return 256 + (size_t)kBalMaxCtas * bal_stride(s->N) * 8;
}

MOE_API moe_status moe_balance_loss(const moe_shape *s, const float *logits,
                                    const int32_t *topk_idx, const uint8_t *token_mask,
                                    int32_t *expert_count, int32_t *token_count,
                                    float *expert_prob, float *lse, float *losses, void *ws,
                                    size_t ws_bytes, cudaStream_t stream) {
    moe_status r = check_shape(s);
    if (r != MOE_OK) return r;
    if (!expert_count || !token_count || !expert_prob || !losses ||
        (s->T > 0 && (!logits || !topk_idx || !lse)))
        return MOE_ERR_INVALID_ARG;
    const void *ptrs[] = {logits, topk_idx, token_mask, expert_count, token_count, expert_prob,
                          lse, losses};
    for (const void *p : ptrs)
        if (!aligned16(p)) return MOE_ERR_ALIGNMENT;
    if (!ws_ok(ws, ws_bytes, moe_balance_loss_workspace_bytes(s))) return MOE_ERR_WORKSPACE;
    const int ctas = bal_ctas(s->T);
    int32_t *part_i = reinterpret_cast<int32_t *>(static_cast<uint8_t *>(ws) + 256);
    float *part_f = reinterpret_cast<float *>(part_i + kBalMaxCtas * bal_stride(s->N));
    const size_t smem = sizeof(float) * ((kBalWarps + 1) * s->N + 2 * kBalWarps);
    launch_pdl(balance_partial, ctas, kBalThreads, smem, stream, s->T, s->N, s->K, logits, topk_idx,
               token_mask, lse, part_i, part_f);
    launch_pdl(balance_finish, 1, 1024, 0, stream, s->N, s->K, ctas,
               static_cast<const int32_t *>(part_i), static_cast<const float *>(part_f),
               expert_count, token_count, expert_prob, losses);
    return launch_status();
}

MOE_API moe_status moe_balance_loss_backward(const moe_shape *s, const float *logits,
                                             const int32_t *topk_idx, const uint8_t *token_mask,
                                             const int32_t *expert_count,
                                             const int32_t *token_count, const float *lse,
                                             const float *dlosses, const float *dlogit,
                                             float *dlogits, cudaStream_t stream) {
    moe_status r = check_shape(s);
    if (r != MOE_OK) return r;
    if (s->T == 0) return MOE_OK;
    if (!logits || !expert_count || !token_count || !lse || !dlosses || !dlogits ||
        (dlogit && !topk_idx))
        return MOE_ERR_INVALID_ARG;
    const void *ptrs[] = {logits, topk_idx, token_mask, expert_count, token_count, lse, dlosses,
                          dlogit, dlogits};
    for (const void *p : ptrs)
        if (!aligned16(p)) return MOE_ERR_ALIGNMENT;
    const int want = (s->T + kBalWarps - 1) / kBalWarps, most = num_sms() * 8;
    launch_pdl(balance_bwd_rows, want < most ? want : most, kBalThreads, sizeof(float) * s->N, stream,
               s->T, s->N, s->K, logits, topk_idx, token_mask, expert_count, token_count, lse,
               dlosses, dlogit, dlogits);
    return launch_status();
}

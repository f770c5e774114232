// The router's balance loss and z loss, and their gradient with respect to
// every logit (include/moe_block.h).
//
//   p = softmax(logits[t]);  balance = N sum_e c_e / (Tc K) sum_t p_te / Tc
//   z = sum_t lse_t^2 / Tc
//   dlogits = p (gb N / Tc (f - sum_e p_e f_e) + gz 2 lse / Tc) + scattered dlogit
//
// A token's row of logits is held in the registers of a group of LANES lanes,
// VPT logits each (8 x 4 for N <= 32 up to 32 x 32), so both kernels read the
// logits once and need one exponential per logit.  Rows of a multiple of four
// logits are read and written in 16-byte vectors (8 bytes for an even number).
//
// The bytes would be the bound (131072 x 250 masked logits: 20 us forward, 36
// backward), but issue slots come close: about 200 instructions a row forward
// with a whole warp per row.  So each probability is a packed subtraction and
// product and the hardware's 2^x, and the forward takes as few lanes a row as
// its registers allow (27 us).  The product with log2 e is rounded at the size
// of the argument, which costs d u of a probability e^-d of the row's largest
// (u = 2^-24); what is done once a row, the logarithm and the division, is
// rounded to fp32's last bit.  expf with scalar arithmetic took 40 us forward
// instead of 32.  The 2-norm error of dlogits is 1.0e-7 at 131072 x 60 and 1.2e-7
// at 131072 x 250, that of a plain fp32 form with expf 0.8e-7 and 1.0e-7;
// probabilities, log sums and losses are as good as that form's.
#include <algorithm>

#include "../../include/moe_block.h"
#include "moe_common.cuh"

namespace moe {
namespace {

constexpr int kBalCtas = 152;  // partial sums of the forward: one CTA per SM
constexpr int kAlone = 4;      // rows a group when one CTA takes all tokens
constexpr int kBalSlots = 8;   // warps that add up side by side in shared memory

// Partial sums of one CTA in the workspace, rounded up to 16 bytes: int32
// counts [N] and the tokens, then fp32 probability sums [N] and the sum of lse^2.
inline __host__ __device__ int64_t bal_stride(int N) { return (N + 1 + 3) / 4 * 4; }

constexpr float kLog2e = 1.44269504f;

__device__ __forceinline__ float ex2(float v) {
    float r;
    asm("ex2.approx.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}

template <int LANES>
__device__ __forceinline__ float group_max(float v) {
#pragma unroll
    for (int off = LANES / 2; off > 0; off >>= 1) v = fmaxf(v, __shfl_xor_sync(0xFFFFFFFFu, v, off));
    return v;
}
template <int LANES>
__device__ __forceinline__ float group_sum(float v) {
#pragma unroll
    for (int off = LANES / 2; off > 0; off >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, off);
    return v;
}

// The experts of lane `sub` of a group: register i holds expert
// first(sub) + step(i), in vectors of VEC logits.  HALF: the row fills every
// vector that starts in the first half of the registers (of 12 registers in
// vectors of 4, the first 8), and these need no bounds check.
template <int LANES, int VPT, int VEC, bool HALF>
struct Row {
    static __device__ __forceinline__ int first(int sub) { return VEC * sub; }
    static __device__ __forceinline__ constexpr int step(int i) {
        return i / VEC * VEC * LANES + i % VEC;
    }
    static __device__ __forceinline__ bool in_row(int e0, int i, int N) {
        return (HALF && i < VPT / 2 && VEC <= VPT / 2) || e0 + step(i) < N;
    }
    // a row's logits; experts past N (or all of them) read as -inf
    static __device__ __forceinline__ void load(const float *row, int sub, int N, bool on, float (&v)[VPT]) {
        const int e0 = first(sub);
#pragma unroll
        for (int i = 0; i < VPT; i += VEC) {
#pragma unroll
            for (int j = 0; j < VEC; ++j) v[i + j] = -INFINITY;
            if (!on || !in_row(e0, i, N)) continue;
            const float *p = row + e0 + step(i);
            if (VEC == 4) {
                const float4 q = __ldcs(reinterpret_cast<const float4 *>(p));
                v[i] = q.x; v[i + 1] = q.y; v[i + 2] = q.z; v[i + 3] = q.w;
            } else if (VEC == 2) {
                const float2 q = __ldcs(reinterpret_cast<const float2 *>(p));
                v[i] = q.x; v[i + 1] = q.y;
            } else {
                v[i] = __ldcs(p);
            }
        }
    }
    // adds a row in shared memory, aligned as the vectors want it
    static __device__ __forceinline__ void add(const float *row, int sub, int N, float (&v)[VPT]) {
        const int e0 = first(sub);
#pragma unroll
        for (int i = 0; i < VPT; i += VEC) {
            if (!in_row(e0, i, N)) continue;
            const float *p = row + e0 + step(i);
            if (VEC == 4) {
                const float4 q = *reinterpret_cast<const float4 *>(p);
                v[i] += q.x; v[i + 1] += q.y; v[i + 2] += q.z; v[i + 3] += q.w;
            } else if (VEC == 2) {
                const float2 q = *reinterpret_cast<const float2 *>(p);
                v[i] += q.x; v[i + 1] += q.y;
            } else {
                v[i] += *p;
            }
        }
    }
    static __device__ __forceinline__ void store(float *row, int sub, int N, const float (&v)[VPT]) {
        const int e0 = first(sub);
#pragma unroll
        for (int i = 0; i < VPT; i += VEC) {
            if (!in_row(e0, i, N)) continue;
            float *p = row + e0 + step(i);
            if (VEC == 4) *reinterpret_cast<float4 *>(p) = make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
            else if (VEC == 2) *reinterpret_cast<float2 *>(p) = make_float2(v[i], v[i + 1]);
            else *p = v[i];
        }
    }
};

// The outputs that follow from the sums over all tokens.
struct LossOut {
    int32_t *count, *token_count;
    float *prob, *losses;

    static __device__ __forceinline__ float inv(int tc) { return tc > 0 ? 1.f / (float)tc : 0.f; }
    // expert e's count and mean probability; its term of the balance loss over N
    __device__ __forceinline__ float expert(int e, int c, float sum, int tc, int K) const {
        const float p = sum * inv(tc);
        count[e] = c;
        prob[e] = p;
        return (float)c * inv(tc) / (float)K * p;
    }
    __device__ __forceinline__ void losses_of(float dot, float z, int tc, int N) const {
        token_count[0] = tc;
        losses[0] = (float)N * dot;
        losses[1] = z * inv(tc);
    }
};

__host__ __device__ constexpr int bal_threads(int vpt) { return vpt >= 16 ? 512 : 1024; }

template <int LANES, int VPT, int VEC, bool HALF>
__global__ void __launch_bounds__(bal_threads(VPT), 1)
balance_partial(int T, int N, int K, const float *__restrict__ logits,
                const int32_t *__restrict__ topk_idx, const uint8_t *__restrict__ mask,
                float *__restrict__ lse, int32_t *__restrict__ part_i, float *__restrict__ part_f,
                const LossOut out) {
    pdl_enter();
    using R = Row<LANES, VPT, VEC, HALF>;
    constexpr int kThreads = bal_threads(VPT), kWarps = kThreads / 32;
    constexpr int kGroups = kThreads / LANES;
    extern __shared__ float sm[];
    float *acc_s = sm;                                          // [kBalSlots][N]
    int *cnt = reinterpret_cast<int *>(sm + kBalSlots * N);     // [N]
    __shared__ float zs[kWarps];
    __shared__ int ts[kWarps];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, sub = threadIdx.x % LANES;
    for (int i = threadIdx.x; i < (kBalSlots + 1) * N; i += kThreads) sm[i] = 0.f;
    __syncthreads();
    alignas(float2) float acc[VPT];  // read in pairs, should it ever leave the registers
    float2 *acc2 = reinterpret_cast<float2 *>(acc);
#pragma unroll
    for (int i = 0; i < VPT; ++i) acc[i] = 0.f;
    float z = 0.f;
    int tok = 0;
    // Whole warps step together: a group past T, or at a masked token, idles.
    // A row's logits and chosen experts are loaded one step ahead and its mask
    // two, so that no load of a step waits for another one.
    constexpr int kIdx = (kMaxK + LANES - 1) / LANES;
    const int64_t step = (int64_t)gridDim.x * kGroups;
    auto counted = [&](int64_t t) { return t < T && !(mask && mask[t] == 0); };
    int64_t w0 = (int64_t)blockIdx.x * kGroups + warp * (32 / LANES);
    float ahead[VPT];
    int idx[kIdx];
    bool ahead_on = false, later_on = false;
    auto load_idx = [&](int64_t t, bool on) {
#pragma unroll
        for (int j = 0; j < kIdx; ++j) {
            const int k = sub + j * LANES;
            idx[j] = on && k < K ? topk_idx[t * K + k] : -1;
        }
    };
    {
        const int64_t t = w0 + lane / LANES;
        ahead_on = counted(t);
        later_on = counted(t + step);
        R::load(logits + t * N, sub, N, ahead_on, ahead);
        load_idx(t, ahead_on);
    }
    for (; w0 < T; w0 += step) {
        const int64_t t = w0 + lane / LANES;
        const bool in = t < T;
        const bool on = ahead_on;
        alignas(float2) float v[VPT];
        int mine[kIdx];
#pragma unroll
        for (int i = 0; i < VPT; ++i) v[i] = ahead[i];
#pragma unroll
        for (int j = 0; j < kIdx; ++j) mine[j] = idx[j];
        ahead_on = later_on;
        later_on = counted(t + 2 * step);
        R::load(logits + (t + step) * N, sub, N, ahead_on, ahead);
        load_idx(t + step, ahead_on);
        float m = v[0];
#pragma unroll
        for (int i = 1; i < VPT; ++i) m = fmaxf(m, v[i]);
        m = group_max<LANES>(m);
        if (m == -INFINITY) m = 0.f;  // all -inf: probabilities 0; all NaN: NaN below
        // exp(v - m) = 2^((v - m) log2 e); the difference comes first, because
        // v log2 e overflows for the lowest values that masks are made of
        const float2 mul = make_float2(kLog2e, kLog2e), off = make_float2(-m, -m);
        float2 sum2 = make_float2(0.f, 0.f);
        float2 *v2 = reinterpret_cast<float2 *>(v);
#pragma unroll
        for (int i = 0; i < VPT / 2; ++i) {
            const float2 a = __fmul2_rn(__fadd2_rn(v2[i], off), mul);
            v2[i] = make_float2(ex2(a.x), ex2(a.y));
            sum2 = __fadd2_rn(sum2, v2[i]);
        }
        const float sum = group_sum<LANES>(sum2.x + sum2.y);
        const float inv = sum == 0.f ? 0.f : __frcp_rn(sum);
        const float2 inv2 = make_float2(inv, inv);
#pragma unroll
        for (int i = 0; i < VPT / 2; ++i) acc2[i] = __ffma2_rn(v2[i], inv2, acc2[i]);
#pragma unroll
        for (int j = 0; j < kIdx; ++j)
            if (mine[j] >= 0 && mine[j] < N) atomicAdd(cnt + mine[j], 1);
        if (in && sub == 0) {
            const float l = m + logf(sum);
            lse[t] = on ? l : 0.f;
            if (on) {
                ++tok;
                if (sum != 0.f) z = fmaf(l, l, z);
            }
        }
    }
    // the warp's groups, then the warps, in a fixed order
#pragma unroll
    for (int i = 0; i < VPT; ++i)
#pragma unroll
        for (int off = LANES; off < 32; off <<= 1) acc[i] += __shfl_xor_sync(0xFFFFFFFFu, acc[i], off);
    z = group_sum<32>(z);
    tok = __reduce_add_sync(0xFFFFFFFFu, tok);
    if (lane == 0) {
        zs[warp] = z;
        ts[warp] = tok;
    }
    for (int w = 0; w < kWarps; w += kBalSlots) {
        if (warp >= w && warp < w + kBalSlots && lane < LANES) {
            float *my = acc_s + (warp - w) * N + R::first(sub);
#pragma unroll
            for (int i = 0; i < VPT; ++i)
                if (R::first(sub) + R::step(i) < N) my[R::step(i)] += acc[i];
        }
        __syncthreads();
    }
    // the warps' sums as a tree: one after the other, 32 of them could each lose
    // half an ulp of the whole
    z = group_sum<32>(lane < kWarps ? zs[lane] : 0.f);
    tok = __reduce_add_sync(0xFFFFFFFFu, lane < kWarps ? ts[lane] : 0);
    float dot = 0.f;
    part_i += blockIdx.x * bal_stride(N);
    part_f += blockIdx.x * bal_stride(N);
    for (int e = threadIdx.x; e < N; e += kThreads) {
        float p = 0.f;
#pragma unroll
        for (int w = 0; w < kBalSlots; ++w) p += acc_s[w * N + e];
        if (gridDim.x == 1) {
            dot += out.expert(e, cnt[e], p, tok, K);
        } else {
            part_i[e] = cnt[e];
            part_f[e] = p;
        }
    }
    if (gridDim.x > 1) {
        if (threadIdx.x == 0) {
            part_i[N] = tok;
            part_f[N] = z;
        }
        return;
    }
    // few tokens: this CTA has all of them, and no second launch is needed
    __syncthreads();  // zs is read above
    dot = group_sum<32>(dot);
    if (lane == 0) zs[warp] = dot;
    __syncthreads();
    if (warp > 0) return;
    dot = group_sum<32>(lane < kWarps ? zs[lane] : 0.f);
    if (lane == 0) out.losses_of(dot, z, tok, N);
}

constexpr int kFinishCtas = 8;

// The CTAs' partial sums and the two losses.  Each thread takes four experts (a
// 16-byte vector) of every slices-th CTA; the slices are then added pairwise.
// The loads of a thread are independent, so this is one or two rounds of L2
// latency: an expert per thread took 9 to 12 us here.
// One cluster of CTAs: what one SM can read in time bounds many experts' sums
// (588 KB for 152 CTAs of 481 experts), so each CTA adds its share of the rows
// and the first one adds the others' sums from their shared memory.
__device__ __forceinline__ float4 peer_f4(const float4 *p, uint32_t rank) {
    float4 v;
    asm volatile("{\n .reg .b32 a;\n mapa.shared::cluster.u32 a, %4, %5;\n"
                 " ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [a];\n}"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "r"(smem_u32(p)), "r"(rank)
                 : "memory");
    return v;
}

__global__ void __launch_bounds__(1024)
balance_finish(int N, int K, int ctas, int slices, const int32_t *__restrict__ part_i,
               const float *__restrict__ part_f, const LossOut out) {
    pdl_enter();
    __shared__ float4 sf4[1024];
    __shared__ int4 si4[1024];
    __shared__ float red[32];
    float *sf = reinterpret_cast<float *>(sf4);
    int *si = reinterpret_cast<int *>(si4);
    const int st = (int)bal_stride(N), vec = st / 4;
    // the last vector's padding holds nothing that is read back
    const int rank = (int)cluster_rank(), peers = (int)gridDim.x;
    if ((int)threadIdx.x < slices * vec) {
        const int e = threadIdx.x % vec, q = threadIdx.x / vec;
        float4 p = make_float4(0.f, 0.f, 0.f, 0.f);
        int4 c = make_int4(0, 0, 0, 0);
#pragma unroll 8
        for (int g = rank * slices + q; g < ctas; g += peers * slices) {
            const float4 a = reinterpret_cast<const float4 *>(part_f)[g * vec + e];
            const int4 b = reinterpret_cast<const int4 *>(part_i)[g * vec + e];
            p.x += a.x; p.y += a.y; p.z += a.z; p.w += a.w;
            c.x += b.x; c.y += b.y; c.z += b.z; c.w += b.w;
        }
        sf4[threadIdx.x] = p;
        si4[threadIdx.x] = c;
    }
    for (int h = slices; h > 1;) {
        const int half = (h + 1) / 2;
        __syncthreads();
        for (int j = threadIdx.x; j < (h - half) * st; j += blockDim.x) {
            sf[j] += sf[j + half * st];
            si[j] += si[j + half * st];
        }
        h = half;
    }
    if (peers > 1) {
        cluster_sync_all();
        if (rank == 0 && (int)threadIdx.x < vec) {
            float4 p = sf4[threadIdx.x];
            int4 c = si4[threadIdx.x];
#pragma unroll
            for (int r = 1; r < kFinishCtas; ++r) {
                const float4 a = peer_f4(&sf4[threadIdx.x], r);
                const float4 b = peer_f4(reinterpret_cast<float4 *>(&si4[threadIdx.x]), r);
                p.x += a.x; p.y += a.y; p.z += a.z; p.w += a.w;
                c.x += __float_as_int(b.x); c.y += __float_as_int(b.y);
                c.z += __float_as_int(b.z); c.w += __float_as_int(b.w);
            }
            sf4[threadIdx.x] = p;
            si4[threadIdx.x] = c;
        }
        cluster_sync_all();  // the others' shared memory stays until it is read
        if (rank != 0) return;
    }
    __syncthreads();
    const int tc = si[N];
    float dot = (int)threadIdx.x < N ? out.expert(threadIdx.x, si[threadIdx.x], sf[threadIdx.x], tc, K) : 0.f;
    dot = group_sum<32>(dot);
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = dot;
    __syncthreads();
    if (threadIdx.x >= 32) return;
    dot = group_sum<32>(red[threadIdx.x]);  // 1024 threads
    if (threadIdx.x == 0) out.losses_of(dot, sf[N], tc, N);
}

constexpr int kBwdThreads = 256;

inline __host__ __device__ int bal_gate_stride(int N) { return (N + 3) / 4 * 4; }

template <int LANES, int VPT, int VEC, bool HALF>
__global__ void __launch_bounds__(kBwdThreads)
balance_bwd_rows(int T, int N, int K, const float *__restrict__ logits,
                 const int32_t *__restrict__ topk_idx, const uint8_t *__restrict__ mask,
                 const int32_t *__restrict__ count, const int32_t *__restrict__ token_count,
                 const float *__restrict__ lse, const float *__restrict__ dlosses,
                 const float *__restrict__ dlogit, float *__restrict__ dlogits) {
    pdl_enter();
    using R = Row<LANES, VPT, VEC, HALF>;
    constexpr int kGroups = kBwdThreads / LANES;
    constexpr int kIdx = (kMaxK + LANES - 1) / LANES;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, sub = threadIdx.x % LANES;
    // this token's gates by expert, zero between rows
    extern __shared__ float gate_s[];
    const int stride = bal_gate_stride(N);
    float *gates = gate_s + threadIdx.x / LANES * stride;
    if (dlogit) {
        for (int e = sub; e < stride; e += LANES) gates[e] = 0.f;
        __syncwarp();
    }
    const int tc = token_count[0];
    const float inv = tc > 0 ? 1.f / (float)tc : 0.f;
    const float cb = dlosses[0] * (float)N * inv, cz = 2.f * dlosses[1] * inv;
    // one division: sixteen a thread were two thirds of the instructions of a
    // launch with one row a warp
    const float share = inv / (float)K;
    alignas(float2) float f[VPT];
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        const int e = R::first(sub) + R::step(i);
        f[i] = e < N ? (float)count[e] * share : 0.f;
    }
    for (int64_t w0 = (int64_t)blockIdx.x * kGroups + warp * (32 / LANES); w0 < T;
         w0 += (int64_t)gridDim.x * kGroups) {
        const int64_t t = w0 + lane / LANES;
        const bool in = t < T;
        bool on = in && !(mask && mask[t] == 0);
        alignas(float2) float v[VPT];
        R::load(logits + t * N, sub, N, on, v);
        // lane `sub` holds the token's routes sub, sub + LANES, ...
        int idx[kIdx];
        float gate[kIdx];
#pragma unroll
        for (int j = 0; j < kIdx; ++j) {
            const int k = sub + j * LANES;
            const bool is = dlogit && in && k < K;
            idx[j] = is ? topk_idx[t * K + k] : -1;
            gate[j] = is ? dlogit[t * K + k] : 0.f;
        }
        const float l = on ? lse[t] : 0.f;
        on = on && l != -INFINITY;  // every logit -inf: no probability, no gradient
        // e_j = exp(v_j - lse) holds the error of a log sum rounded at the row's
        // size (at 1e9 it equals every logit, and each e_j is 1), so it is only a
        // shifted exponential: p_j = e_j / sum e.  lse is at most half an ulp off, 4
        // where an ulp is 8, and equals the largest logit where it is more: the
        // largest e_j is between e^-4 / N and e^4.
        const float2 mul = make_float2(kLog2e, kLog2e), off = make_float2(-l, -l);
        float2 dot2 = make_float2(0.f, 0.f), sum2 = make_float2(0.f, 0.f);
        float2 *v2 = reinterpret_cast<float2 *>(v), *f2 = reinterpret_cast<float2 *>(f);
#pragma unroll
        for (int i = 0; i < VPT / 2; ++i) {
            const float2 a = __fmul2_rn(__fadd2_rn(v2[i], off), mul);
            v2[i] = make_float2(ex2(a.x), ex2(a.y));
            sum2 = __fadd2_rn(sum2, v2[i]);
            dot2 = __ffma2_rn(v2[i], f2[i], dot2);
        }
        float sum = sum2.x + sum2.y, dot = dot2.x + dot2.y;
#pragma unroll
        for (int o = LANES / 2; o > 0; o >>= 1) {
            sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
            dot += __shfl_xor_sync(0xFFFFFFFFu, dot, o);
        }
        // p_j (cb (f_j - sum_e p_e f_e) + cz lse), the two divisions in the factors
        const float scale = __frcp_rn(sum);
        const float cs = cb * scale, c = fmaf(-cb, dot * scale, cz * l) * scale;
        const float2 c2 = make_float2(c, c), cs2 = make_float2(cs, cs);
#pragma unroll
        for (int i = 0; i < VPT / 2; ++i) {
            const float2 g = __fmul2_rn(v2[i], __ffma2_rn(cs2, f2[i], c2));
            v2[i] = on ? g : make_float2(0.f, 0.f);
        }
        if (dlogit) {
            // The lane of each route puts its gate where the lane that holds the
            // expert finds it.  Comparing every expert with every route took 36
            // us instead of 31 (both calls) at T = 65536, N = 128, K = 16, and a
            // second write of the routes' elements 82 instead of 75 at T =
            // 131072, N = 250, K = 10; with K = 1 or 2 comparing would gain 3%.
            int *tag = reinterpret_cast<int *>(gates);
            bool is[kIdx], dup = false;
#pragma unroll
            for (int j = 0; j < kIdx; ++j) {
                is[j] = idx[j] >= 0 && idx[j] < N;
                if (is[j]) tag[idx[j]] = sub + j * LANES;
            }
            __syncwarp();
#pragma unroll
            for (int j = 0; j < kIdx; ++j) dup |= is[j] && tag[idx[j]] != sub + j * LANES;
            const bool any = __any_sync(0xFFFFFFFFu, dup);
#pragma unroll
            for (int j = 0; j < kIdx; ++j)
                if (is[j]) gates[idx[j]] = any ? 0.f : gate[j];
            __syncwarp();
            // one expert in several routes (moe_route never does this): their
            // gates are added one after the other
            for (int k = 0; any && k < K; ++k) {
#pragma unroll
                for (int j = 0; j < kIdx; ++j)
                    if (is[j] && sub + j * LANES == k) gates[idx[j]] += gate[j];
                __syncwarp();
            }
            R::add(gates, sub, N, v);
            __syncwarp();
#pragma unroll
            for (int j = 0; j < kIdx; ++j)
                if (is[j]) gates[idx[j]] = 0.f;
            __syncwarp();
        }
        if (in) R::store(dlogits + t * N, sub, N, v);
    }
}

// How a row of N logits is held: calls fn with LANES, VPT, the vector length
// that keeps rows aligned, and whether N fills half of it (each type's N begins
// where the type before it ends).  Few lanes, because
// what a kernel does once a row (statistics, counts, sums over the lanes) then
// serves several rows an instruction, as long as the registers leave enough
// warps.  Both calls, us, with these lanes (forward, backward) and with others:
//   T = 131072, N = 33,  K = 4    (8, 8)   28   (8, 16)  30
//   T = 131072, N = 64,  K = 8    (8, 8)   34   (8, 16)  37
//   T = 131072, N = 96,  K = 8    (8, 8)   40   (8, 16)  43
//   T = 131072, N = 128, K = 8    (8, 8)   48   (8, 16)  50   (16, 8)  48
//   T = 65536,  N = 160, K = 6    (8, 16)  36   (8, 8)   40   (8, 32)  41
//   T = 131072, N = 250, K = 10   (8, 16)  75   (8, 8)   83   (8, 32)  82   (16, 16) 80
//   T = 61814,  N = 259, K = 14   (32, 32) 52   (32, 16) 54   (16, 32) 52
//   T = 7886,   N = 481, K = 1    (32, 32) 18   (32, 16) 21   (16, 32) 19
//   T = 30000,  N = 512, K = 8    (32, 32) 46   (32, 16) 53   (16, 32) 44
// From N = 96 on these were measured before the backward took its row's sum; with
// the lanes of the first column they are now 39, 46, 35, 77, 53, 20 and 44.  For
// 385 to 512 experts (16, 32) then takes 3 to 6% less at 60000 tokens (N = 400: 62
// against 65, N = 512: 71 against 76), as much at 30000 and 4 to 5% more at 15000
// and 8000 (30 against 29, 20.6 against 19.5): a whole warp a row stays.
// Room for 96, 192 and 384 experts beside the powers of two: N = 96 in a row of
// 128 takes 44 us, N = 160 in one of 256 39, N = 259 in one of 512 59.
template <int L, int V, int W, bool H>
struct RowOf {
    static constexpr int lanes = L, vpt = V, vec = W;
    static constexpr bool half = H;
};
template <int V>
struct Int {
    static constexpr int value = V;
};
template <bool FWD, typename Fn>
inline void with_row(int N, Fn &&fn) {
    auto go = [&](auto w) {
        constexpr int kVec = decltype(w)::value;
        if (N <= 32) fn(RowOf<8, 4, kVec, false>());
        else if (N <= 64) fn(RowOf<8, 8, kVec, true>());
        else if (N <= 96) fn(RowOf<8, 12, kVec, true>());
        else if (N <= 128) fn(RowOf<8, 16, kVec, true>());
        else if (N <= 192) fn(RowOf<FWD ? 8 : 16, FWD ? 24 : 12, kVec, true>());
        else if (N <= 256) fn(RowOf<FWD ? 8 : 16, FWD ? 32 : 16, kVec, true>());
        else if (N <= 384) fn(RowOf<32, 12, kVec, true>());
        else if (N <= 512) fn(RowOf<32, 16, kVec, true>());
        else fn(RowOf<32, 32, kVec, true>());
    };
    if (N % 4 == 0) go(Int<4>());
    else if (N % 2 == 0) go(Int<2>());
    else go(Int<1>());
}

inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

inline bool ws_ok(const void *ws, size_t have, size_t need) {
    return ws && (reinterpret_cast<uintptr_t>(ws) & 255u) == 0 && have >= need;
}

}  // namespace
}  // namespace moe

using namespace moe;

MOE_API size_t moe_balance_loss_workspace_bytes(const moe_shape *s) {
    if (check_shape(s) != MOE_OK) return 0;
    return 256 + (size_t)kBalCtas * bal_stride(s->N) * 8;
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
    const int N = s->N;
    int32_t *part_i = reinterpret_cast<int32_t *>(static_cast<uint8_t *>(ws) + 256);
    float *part_f = reinterpret_cast<float *>(part_i + kBalCtas * bal_stride(N));
    const LossOut out = {expert_count, token_count, expert_prob, losses};
    int ctas = 1;
    with_row<true>(N, [&](auto q) {
        using Q = decltype(q);
        constexpr int kThreads = bal_threads(Q::vpt), kGroups = kThreads / Q::lanes;
        // up to kAlone rows a group one CTA takes less than a second launch
        ctas = s->T <= kAlone * kGroups ? 1 : (int)std::min<int64_t>(kBalCtas, ceil_div(s->T, kGroups));
        launch_pdl(balance_partial<Q::lanes, Q::vpt, Q::vec, Q::half>, ctas, kThreads,
                   sizeof(float) * (kBalSlots + 1) * N, stream, s->T, N, s->K, logits, topk_idx,
                   token_mask, lse, part_i, part_f, out);
    });
    if (ctas > 1) {
        // one CTA up to 128 KB of sums: 152 x 71 experts took 31.5 us with eight and
        // 30.7 with one, 152 x 128 the same, 152 x 250 85.7 and 88.3, 152 x 1000 85
        // and 99 (both calls)
        const unsigned peers = ctas * bal_stride(N) > 16384 ? kFinishCtas : 1;
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(peers);
        cfg.blockDim = dim3(1024);
        cfg.stream = stream;
        cudaLaunchAttribute attr[2];
        set_pdl_attr(attr[0]);
        attr[1].id = cudaLaunchAttributeClusterDimension;
        attr[1].val.clusterDim.x = peers;
        attr[1].val.clusterDim.y = 1;
        attr[1].val.clusterDim.z = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 2;
        if (cudaLaunchKernelEx(&cfg, balance_finish, N, s->K, ctas,
                               std::min(ctas, 1024 / (int)(bal_stride(N) / 4)),
                               static_cast<const int32_t *>(part_i), static_cast<const float *>(part_f),
                               out) != cudaSuccess)
            return MOE_ERR_CUDA;
    }
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
    with_row<false>(s->N, [&](auto q) {
        using Q = decltype(q);
        const int64_t want = ceil_div(s->T, kBwdThreads / Q::lanes);
        launch_pdl(balance_bwd_rows<Q::lanes, Q::vpt, Q::vec, Q::half>,
                   (unsigned)std::min<int64_t>(want, (int64_t)num_sms() * 8), kBwdThreads,
                   dlogit ? sizeof(float) * (kBwdThreads / Q::lanes) * bal_gate_stride(s->N) : 0, stream,
                   s->T, s->N, s->K, logits, topk_idx, token_mask, expert_count, token_count, lse,
                   dlosses, dlogit, dlogits);
    });
    return launch_status();
}

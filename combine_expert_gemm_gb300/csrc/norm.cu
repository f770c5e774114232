// Residual add + layer norm of token rows, and its backward with the
// reduction of the weight gradients (include/moe_block.h).
//
//   s = x + add (rounded to x's type);  mean = sum s / d
//   rstd = (sum (s - mean)^2 / d + eps)^-1/2;  y = (s - mean) rstd gamma + beta
//   dx = dres + rstd (w - sum w / d - xh sum(w xh) / d),  w = dy gamma,
//   xh = (s - mean) rstd;  dgamma = sum_t dy xh;  dbeta = sum_t dy
//
// Bound by HBM: a few operations per element moved, so both kernels read every
// row once.  Persistent CTAs of up to 512 threads, one per SM, are cut into
// groups of whole warps; a group takes one row at a time and each of its
// threads keeps the same columns (8 to 32 of them) from row to row.  The
// forward's gamma and beta and the backward's share of dgamma and dbeta
// therefore stay in registers, and the weight gradients cost no second pass
// over x and dy (the two-pass version took 74 of 172 us at 8192 x 2048).
//
// The forward's bf16 rows arrive through a ring of cp.async copies, kStages - 1
// rows ahead (fp32 rows in registers).  A thread copies exactly the bytes that it will read itself, so the
// ring needs no barrier and no wait but the thread's own cp.async.wait_group.
// The backward moves three tensors in, and there the copies' and the ring's own
// instructions were what it waited for (353 a warp-row, 0.34 issued a cycle): it
// loads the next row's x and dy straight into registers as soon as the current
// row's are unpacked, and gamma, in shared memory, makes room for them.
// 32768 x 4096: 246 -> 210 us, of which the reads take 174 at the rate a plain
// read reaches.
//
// A row's sums cross the group's warps through shared memory with one barrier
// per row (two alternating buffers); every warp then adds the warps' pairs
// with lane shuffles.  The forward exchanges each warp's sum and its squares
// centred at the warp's own mean, which combine exactly into the variance
// around the row's mean:
//   M2 = sum_w M2_w + n_w (mean_w - mean)^2.
// Issue slots are the second limit: 8 columns a thread and every thread adding
// all the warps' pairs in a loop took 370 us for the forward of 32768 x 4096,
// whose bytes take 158.
#include <math.h>

#include <algorithm>

#include "../../include/moe_block.h"
#include "moe_common.cuh"

namespace moe {
namespace {

constexpr int kNormMaxD = 16384;
constexpr int kNormMaxThreads = 512;
constexpr int kNormCtas = 152;        // one per SM; the order of the weight sums follows it
constexpr size_t kNormRing = 196608;  // most shared memory a kernel takes

// Two fp32 values side by side: the packed instructions halve the issue slots
// of the element-wise work.
typedef float2 f2;

__device__ __forceinline__ f2 make2(float lo, float hi) { return make_float2(lo, hi); }
__device__ __forceinline__ f2 both(float v) { return make_float2(v, v); }
__device__ __forceinline__ f2 fma2(f2 a, f2 b, f2 c) { return __ffma2_rn(a, b, c); }
__device__ __forceinline__ f2 add2(f2 a, f2 b) { return __fadd2_rn(a, b); }
__device__ __forceinline__ f2 mul2(f2 a, f2 b) { return __fmul2_rn(a, b); }
__device__ __forceinline__ float sum_of(f2 v) { return v.x + v.y; }

// Eight elements (a chunk) as four pairs.
__device__ __forceinline__ void unpack(const uint4 &v, f2 (&f)[4]) {
    f[0] = make2(bf16_lo(v.x), bf16_hi(v.x));
    f[1] = make2(bf16_lo(v.y), bf16_hi(v.y));
    f[2] = make2(bf16_lo(v.z), bf16_hi(v.z));
    f[3] = make2(bf16_lo(v.w), bf16_hi(v.w));
}
__device__ __forceinline__ uint32_t pack2(f2 v) { return pack_bf16x2(v.x, v.y); }
__device__ __forceinline__ uint4 pack(const f2 (&f)[4]) {
    return make_uint4(pack2(f[0]), pack2(f[1]), pack2(f[2]), pack2(f[3]));
}
__device__ __forceinline__ void store8(uint16_t *p, const f2 (&f)[4]) {
    *reinterpret_cast<uint4 *>(p) = pack(f);
}
__device__ __forceinline__ void store8(float *p, const f2 (&f)[4]) {
    reinterpret_cast<float4 *>(p)[0] = make_float4(f[0].x, f[0].y, f[1].x, f[1].y);
    reinterpret_cast<float4 *>(p)[1] = make_float4(f[2].x, f[2].y, f[3].x, f[3].y);
}
// Stores a chunk (if on) and replaces it by what the store holds.
__device__ __forceinline__ void store_round8(uint16_t *p, f2 (&f)[4], bool on) {
    const uint4 v = pack(f);
    if (on) *reinterpret_cast<uint4 *>(p) = v;
    unpack(v, f);
}
__device__ __forceinline__ void store_round8(float *p, f2 (&f)[4], bool on) {
    if (on) store8(p, f);
}

// A thread's slot of one ring stage: 16-byte words kNormMaxThreads words apart
// (a constant, so that words are addressed by offsets in the instruction), a
// warp's accesses consecutive.  T's 8 elements take 1 or 2 words.
template <typename T>
constexpr __host__ __device__ int words() { return (int)sizeof(T) / 2; }

// Copies 8 elements (bytes = 16), or zeros without reading src (bytes = 0): a
// thread past the row's end, or a tensor that is not there, then needs no
// branch where the slot is read.
template <typename T>
__device__ __forceinline__ void ring_copy(uint4 *slot, const T *src, int bytes) {
    const uint4 *g = reinterpret_cast<const uint4 *>(src);
#pragma unroll
    for (int i = 0; i < words<T>(); ++i)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(
                         smem_u32(slot + i * kNormMaxThreads)),
                     "l"(g + i), "r"(bytes)
                     : "memory");
}
template <typename T>
__device__ __forceinline__ void ring_read(const uint4 *slot, f2 (&f)[4]);
template <>
__device__ __forceinline__ void ring_read<uint16_t>(const uint4 *slot, f2 (&f)[4]) {
    unpack(*slot, f);
}
template <>
__device__ __forceinline__ void ring_read<float>(const uint4 *slot, f2 (&f)[4]) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const uint4 v = slot[i * kNormMaxThreads];
        f[2 * i] = make2(__uint_as_float(v.x), __uint_as_float(v.y));
        f[2 * i + 1] = make2(__uint_as_float(v.z), __uint_as_float(v.w));
    }
}
// Eight consecutive fp32 parameters, or `none` where there are none.
__device__ __forceinline__ void load_param(const float *p, int col, int d, float none, f2 (&f)[4]) {
    float4 a = make_float4(none, none, none, none), b = a;
    if (p && col < d) {
        a = __ldg(reinterpret_cast<const float4 *>(p + col));
        b = __ldg(reinterpret_cast<const float4 *>(p + col) + 1);
    }
    f[0] = make2(a.x, a.y); f[1] = make2(a.z, a.w);
    f[2] = make2(b.x, b.y); f[3] = make2(b.z, b.w);
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, off);
    return v;
}

// Barrier among the warps of one group (ids 1..15; a group of one warp needs
// no barrier between warps).
__device__ __forceinline__ void group_sync(int id, int warps) {
    if (warps == 1) __syncwarp();
    else asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(warps * 32) : "memory");
}

// Sum over 16 lanes (the group's warps, at most 16, one per lane of each half
// warp), in every lane.
__device__ __forceinline__ float half_sum(float v) {
#pragma unroll
    for (int off = 8; off > 0; off >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, off);
    return v;
}

// How a row of d columns is laid over threads.
struct NormPlan {
    int cpt;      // chunks of 8 columns per thread: 1, 2 or 4
    int warps;    // warps per group
    int groups;   // groups per CTA
    int ctas;
};

// 16 columns a thread halve a row's exchange between warps against 8; more
// than 16 only where 512 threads do not reach, the registers being short.
inline int norm_cpt(int d) { return d <= 256 ? 1 : d <= 16 * kNormMaxThreads ? 2 : 4; }

// The backward holds two rows of x and dy: with both in fp32 the registers want
// 8 columns a thread where 512 threads reach (23872 x 2040: 118 us against 144).
inline int bwd_cpt(int d, size_t bytes) {
    return bytes == 8 && d <= 8 * kNormMaxThreads ? 1 : norm_cpt(d);
}

inline NormPlan norm_plan(int rows, int d, int cpt) {
    NormPlan p;
    const int chunks = d / 8;
    p.cpt = cpt;
    p.warps = (chunks + 32 * p.cpt - 1) / (32 * p.cpt);
    p.groups = std::min(p.warps == 1 ? 16 : 15, kNormMaxThreads / 32 / p.warps);
    // few rows: one group per CTA before a second one on any SM
    p.groups = std::max(1, std::min(p.groups, rows / kNormCtas));
    p.ctas = std::max(1, std::min(kNormCtas, (rows + p.groups - 1) / p.groups));
    return p;
}

// Eight elements as loaded: 16 bytes of bf16 or 32 of fp32.
template <typename T>
struct Raw {
    uint4 w[words<T>()];
    __device__ __forceinline__ void load(const T *p, bool on) {
        const uint4 *g = reinterpret_cast<const uint4 *>(p);
#pragma unroll
        for (int i = 0; i < words<T>(); ++i) w[i] = on ? __ldcs(g + i) : make_uint4(0u, 0u, 0u, 0u);
    }
    __device__ __forceinline__ void get(f2 (&f)[4]) const {
        if (words<T>() == 1) {
            unpack(w[0], f);
        } else {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const uint4 v = w[i % words<T>()];
                f[2 * i] = make2(__uint_as_float(v.x), __uint_as_float(v.y));
                f[2 * i + 1] = make2(__uint_as_float(v.z), __uint_as_float(v.w));
            }
        }
    }
};

template <typename XT, int CPT, int STAGES>
__global__ void __launch_bounds__(kNormMaxThreads, 1)
norm_fwd(int rows, int d, int warps, const XT *x, const uint16_t *add, const float *__restrict__ gamma,
         const float *__restrict__ beta, float eps, XT *x_sum, uint16_t *__restrict__ y,
         float *__restrict__ mean, float *__restrict__ rstd) {
    pdl_enter();
    extern __shared__ uint4 ring[];
    __shared__ float2 red[2][32];
    constexpr int kChunkWords = words<XT>() + 1, kStage = CPT * kChunkWords * kNormMaxThreads;
    const int gthreads = warps * 32, group = threadIdx.x / gthreads, tid = threadIdx.x % gthreads;
    const int groups = blockDim.x / gthreads, lane = threadIdx.x & 31, gw = tid >> 5;
    const int chunks = d / 8;
    bool on[CPT];
    f2 ga[CPT][4], be[CPT][4];
#pragma unroll
    for (int c = 0; c < CPT; ++c) {
        on[c] = tid + c * gthreads < chunks;  // a thread past the row works on zeros
        load_param(gamma, (tid + c * gthreads) * 8, d, 1.f, ga[c]);
        load_param(beta, (tid + c * gthreads) * 8, d, 0.f, be[c]);
    }
    const int64_t step = (int64_t)gridDim.x * groups;
    const int64_t first = (int64_t)blockIdx.x * groups + group;
    uint4 *mine = ring + threadIdx.x;
    // kRing: a cp.async ring, STAGES - 1 rows ahead; otherwise the next row waits
    // in registers
    constexpr bool kRing = STAGES > 0;
    Raw<XT> nx[kRing ? 1 : CPT];
    Raw<uint16_t> na[kRing ? 1 : CPT];
    auto fetch = [&](int64_t t, int stage) {
        if (t < rows) {
            const int64_t at = t * d + tid * 8;
#pragma unroll
            for (int c = 0; c < CPT; ++c) {
                const XT *px = x + at + c * gthreads * 8;
                const uint16_t *pa = add + at + c * gthreads * 8;
                if (kRing) {
                    uint4 *s = mine + stage * kStage + c * kChunkWords * kNormMaxThreads;
                    ring_copy(s, px, on[c] ? 16 : 0);
                    if (add) ring_copy(s + words<XT>() * kNormMaxThreads, pa, on[c] ? 16 : 0);
                } else {
                    nx[c % (kRing ? 1 : CPT)].load(px, on[c]);
                    if (add) na[c % (kRing ? 1 : CPT)].load(pa, on[c]);
                }
            }
        }
        if (kRing) cp_async_commit();
    };
    if (kRing) {
#pragma unroll
        for (int s = 0; s < STAGES - 1; ++s) fetch(first + s * step, s);
    } else {
        fetch(first, 0);
    }
    // columns of warp w: chunks [32 w, 32 w + 32) of each of the CPT parts
    auto columns = [&](int w) {
        int n = 0;
#pragma unroll
        for (int c = 0; c < CPT; ++c) n += 8 * max(0, min(32, chunks - c * gthreads - w * 32));
        return (float)n;
    };
    const float inv_nw = 1.f / columns(gw), inv_d = 1.f / (float)d;
    // lane w stands for warp w of the group when the warps' pairs are added
    const int other = lane & 15;
    const float lane_n = other < warps ? columns(other) : 0.f;
    const float lane_inv_n = other < warps ? 1.f / lane_n : 0.f;
    int stage = 0, buf = 0;
    for (int64_t t = first; t < rows; t += step) {
        if (kRing) {
            fetch(t + (STAGES - 1) * step, stage == 0 ? STAGES - 1 : stage - 1);
            cp_async_wait<kRing ? STAGES - 1 : 0>();
        }
        const int64_t at = t * d + tid * 8;
        const uint4 *s = mine + stage * kStage;
        if (++stage == STAGES) stage = 0;
        f2 f[CPT][4];
        f2 sum2 = both(0.f);
#pragma unroll
        for (int c = 0; c < CPT; ++c) {
            if (kRing) ring_read<XT>(s + c * kChunkWords * kNormMaxThreads, f[c]);
            else nx[c % (kRing ? 1 : CPT)].get(f[c]);
            if (add) {
                f2 a[4];
                if (kRing) ring_read<uint16_t>(s + (c * kChunkWords + words<XT>()) * kNormMaxThreads, a);
                else na[c % (kRing ? 1 : CPT)].get(a);
#pragma unroll
                for (int i = 0; i < 4; ++i) f[c][i] = add2(f[c][i], a[i]);
                store_round8(x_sum + at + c * gthreads * 8, f[c], on[c]);
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) sum2 = add2(sum2, f[c][i]);
        }
        if (!kRing) fetch(t + step, 0);
        const float sum = warp_sum(sum_of(sum2));
        const float mw = sum * inv_nw;
        f2 sq2 = both(0.f);
#pragma unroll
        for (int c = 0; c < CPT; ++c) {
            const f2 neg_mw = both(on[c] ? -mw : 0.f);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const f2 v = add2(f[c][i], neg_mw);
                sq2 = fma2(v, v, sq2);
            }
        }
        float mu = mw, var = warp_sum(sum_of(sq2));
        if (warps > 1) {
            float2 *r = red[buf] + group * warps;
            if (lane == 0) r[gw] = make_float2(sum, var);
            group_sync(1 + group, warps);
            buf ^= 1;
            const float2 pair = other < warps ? r[other] : make_float2(0.f, 0.f);
            mu = half_sum(pair.x) * inv_d;
            const float dm = fmaf(pair.x, lane_inv_n, -mu);
            var = half_sum(other < warps ? fmaf(lane_n * dm, dm, pair.y) : 0.f);
        }
        const float rs = rsqrtf(fmaf(var, inv_d, eps));  // within 2 ulp
        if (mean && tid == 0) {
            mean[t] = mu;
            rstd[t] = rs;
        }
        const f2 neg_mu = both(-mu), rs2 = both(rs);
#pragma unroll
        for (int c = 0; c < CPT; ++c) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                f[c][i] = fma2(mul2(add2(f[c][i], neg_mu), rs2), ga[c][i], be[c][i]);
            if (on[c]) store8(y + at + c * gthreads * 8, f[c]);
        }
    }
    if (kRing) cp_async_wait<0>();
}

// part[cta][2][d]: this CTA's sums of dgamma and dbeta (part may be NULL).
template <typename XT, typename YT, typename GT, int CPT>
__global__ void __launch_bounds__(kNormMaxThreads, 1)
norm_bwd(int rows, int d, int warps, const XT *__restrict__ x, const YT *__restrict__ dy,
         const float *__restrict__ gamma, const float *__restrict__ mean,
         const float *__restrict__ rstd, const GT *dres, GT *dx, float *__restrict__ part) {
    pdl_enter();
    extern __shared__ uint4 ring[];
    __shared__ float2 red[2][32];
    const int gthreads = warps * 32, group = threadIdx.x / gthreads, tid = threadIdx.x % gthreads;
    const int groups = blockDim.x / gthreads, lane = threadIdx.x & 31, gw = tid >> 5;
    const int chunks = d / 8;
    // past 16 columns a thread the registers hold only the weight gradients:
    // gamma, x and dy are read again for the row's second half
    constexpr bool kKeep = CPT <= 2;
    constexpr int kHeld = kKeep ? CPT : 1;
    bool on[CPT];
    f2 dg[CPT][4], db[CPT][4];
    // gamma of this thread's columns waits in its own words of shared memory
    uint4 *gamma_s = ring + threadIdx.x;
#pragma unroll
    for (int c = 0; c < CPT; ++c) {
        on[c] = tid + c * gthreads < chunks;
        f2 g[4];
        load_param(gamma, (tid + c * gthreads) * 8, d, 1.f, g);
#pragma unroll
        for (int i = 0; i < 2; ++i)
            gamma_s[(2 * c + i) * kNormMaxThreads] =
                make_uint4(__float_as_uint(g[2 * i].x), __float_as_uint(g[2 * i].y),
                           __float_as_uint(g[2 * i + 1].x), __float_as_uint(g[2 * i + 1].y));
#pragma unroll
        for (int i = 0; i < 4; ++i) dg[c][i] = db[c][i] = both(0.f);
    }
    const int64_t step = (int64_t)gridDim.x * groups;
    const int64_t first = (int64_t)blockIdx.x * groups + group;
    const float inv_d = 1.f / (float)d;
    int buf = 0;
    Raw<XT> nx[kHeld];
    Raw<YT> ny[kHeld];
    float mu_n = 0.f, rs_n = 0.f;
    auto fetch = [&](int64_t t) {
        const int64_t at = t * d + tid * 8;
        mu_n = mean[t];
        rs_n = rstd[t];
#pragma unroll
        for (int c = 0; c < (kKeep ? CPT : 0); ++c) {
            nx[c % kHeld].load(x + at + c * gthreads * 8, on[c]);
            ny[c % kHeld].load(dy + at + c * gthreads * 8, on[c]);
        }
    };
    if (first < rows) fetch(first);
    for (int64_t t = first; t < rows; t += step) {
        const float mu = mu_n, rs = rs_n;
        const int64_t at = t * d + tid * 8;
        const f2 neg_mu = both(-mu), rs2 = both(rs);
        f2 xh[kHeld][4], w[kHeld][4];
        // xh and w = dy gamma of one chunk; take: dgamma and dbeta get their share
        auto chunk = [&](int c, bool take, const Raw<XT> &rx, const Raw<YT> &ry, f2 (&xh)[4], f2 (&w)[4]) {
            rx.get(xh);
            ry.get(w);
            f2 ga[4];
            ring_read<float>(gamma_s + 2 * c * kNormMaxThreads, ga);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                xh[i] = mul2(add2(xh[i], neg_mu), rs2);
                if (take) {
                    dg[c][i] = fma2(w[i], xh[i], dg[c][i]);
                    db[c][i] = add2(db[c][i], w[i]);
                }
                w[i] = mul2(w[i], ga[i]);
            }
        };
        f2 sa2 = both(0.f), sb2 = both(0.f);
#pragma unroll
        for (int c = 0; c < CPT; ++c) {
            if (!kKeep) {
                nx[0].load(x + at + c * gthreads * 8, on[c]);
                ny[0].load(dy + at + c * gthreads * 8, on[c]);
            }
            chunk(c, true, nx[c % kHeld], ny[c % kHeld], xh[c % kHeld], w[c % kHeld]);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                sa2 = add2(sa2, w[c % kHeld][i]);
                sb2 = fma2(w[c % kHeld][i], xh[c % kHeld][i], sb2);
            }
        }
        if (t + step < rows) fetch(t + step);
        Raw<GT> res[kHeld];
        if (kKeep) {
#pragma unroll
            for (int c = 0; c < kHeld; ++c)
                res[c].load((dres ? dres : dx) + at + c * gthreads * 8, on[c] && dres);
        }
        float sa = warp_sum(sum_of(sa2)), sb = warp_sum(sum_of(sb2));
        if (warps > 1) {
            float2 *r = red[buf] + group * warps;
            if (lane == 0) r[gw] = make_float2(sa, sb);
            group_sync(1 + group, warps);
            buf ^= 1;
            const float2 pair = (lane & 15) < warps ? r[lane & 15] : make_float2(0.f, 0.f);
            sa = half_sum(pair.x);
            sb = half_sum(pair.y);
        }
        // dx = dres + rs w - rs sa / d - rs sb / d xh
        const f2 a2 = both(-sa * inv_d * rs), b2 = both(-sb * inv_d * rs);
#pragma unroll
        for (int c = 0; c < CPT; ++c) {
            if (!kKeep) {
                Raw<XT> rx;
                Raw<YT> ry;
                rx.load(x + at + c * gthreads * 8, on[c]);
                ry.load(dy + at + c * gthreads * 8, on[c]);
                res[0].load((dres ? dres : dx) + at + c * gthreads * 8, on[c] && dres);
                chunk(c, false, rx, ry, xh[0], w[0]);
            }
            f2 r[4];
            res[c % kHeld].get(r);
#pragma unroll
            for (int i = 0; i < 4; ++i)
                r[i] = add2(r[i], fma2(rs2, w[c % kHeld][i], fma2(b2, xh[c % kHeld][i], a2)));
            if (on[c]) store8(dx + at + c * gthreads * 8, r);
        }
    }
    if (!part) return;
    // the CTA's groups, in order, through the shared memory that held gamma
    float *acc = reinterpret_cast<float *>(ring);  // [groups][2][d]
    __syncthreads();
#pragma unroll
    for (int c = 0; c < CPT; ++c) {
        const int at = tid + c * gthreads;
        if (at >= chunks) continue;
        store8(acc + ((size_t)group * 2) * d + at * 8, dg[c]);
        store8(acc + ((size_t)group * 2 + 1) * d + at * 8, db[c]);
    }
    __syncthreads();
    for (int i = threadIdx.x; i < 2 * d / 4; i += blockDim.x) {
        float4 v = reinterpret_cast<const float4 *>(acc)[i];
        for (int g = 1; g < groups; ++g) {
            const float4 q = reinterpret_cast<const float4 *>(acc + (size_t)g * 2 * d)[i];
            v.x += q.x;
            v.y += q.y;
            v.z += q.z;
            v.w += q.w;
        }
        reinterpret_cast<float4 *>(part + (int64_t)blockIdx.x * 2 * d)[i] = v;
    }
}

// dgamma and dbeta from the CTAs' sums: 64 of the 2 d columns per CTA, 16
// slices of the CTAs' rows side by side, added in order.
constexpr int kSumThreads = 256;

__global__ void __launch_bounds__(kSumThreads)
norm_bwd_sum(int d, int ctas, const float *__restrict__ part, float *__restrict__ dgamma,
             float *__restrict__ dbeta) {
    pdl_enter();
    __shared__ float4 sm[16][16];
    const int q = threadIdx.x & 15, s = threadIdx.x >> 4;
    const int i = blockIdx.x * 16 + q;  // float4 index within [2][d]
    const int n = 2 * d / 4;
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
    if (i < n) {
#pragma unroll 5
        for (int g = s; g < ctas; g += 16) {
            const float4 p = reinterpret_cast<const float4 *>(part)[(int64_t)g * n + i];
            v.x += p.x;
            v.y += p.y;
            v.z += p.z;
            v.w += p.w;
        }
    }
    sm[s][q] = v;
    __syncthreads();
    if (s != 0 || i >= n) return;
    for (int k = 1; k < 16; ++k) {
        const float4 p = sm[k][q];
        v.x += p.x;
        v.y += p.y;
        v.z += p.z;
        v.w += p.w;
    }
    // d is a multiple of 8, so a vector lies in one of the two rows
    if (i < d / 4) {
        if (dgamma) reinterpret_cast<float4 *>(dgamma)[i] = v;
    } else if (dbeta) {
        reinterpret_cast<float4 *>(dbeta)[i - d / 4] = v;
    }
}

inline moe_status check_norm(int32_t rows, int32_t d) {
    if (rows < 0 || d <= 0) return MOE_ERR_INVALID_ARG;
    if (d % 8 != 0) return MOE_ERR_ALIGNMENT;
    if (d > kNormMaxD) return MOE_ERR_UNSUPPORTED;
    return MOE_OK;
}

inline bool dtype_ok(int32_t t) { return t == MOE_BF16 || t == MOE_FP32; }

// As many ring stages as fit, 4 at most.
constexpr int ring_stages(int words_per_thread) {
    const int n = (int)(kNormRing / ((size_t)words_per_thread * 16 * kNormMaxThreads));
    return n > 4 ? 4 : n;
}

template <int V>
struct Cpt {
    static constexpr int value = V;
};
template <typename Fn>
inline moe_status with_cpt(int c, Fn &&fn) {
    return c == 1 ? fn(Cpt<1>()) : c == 2 ? fn(Cpt<2>()) : fn(Cpt<4>());
}

template <typename XT, int CPT>
moe_status launch_norm_fwd(int32_t rows, int32_t d, const void *x, const moe_bf16 *add,
                           const float *gamma, const float *beta, float eps, void *x_sum,
                           moe_bf16 *y, float *mean, float *rstd, cudaStream_t stream) {
    // fp32 rows through the ring took 71 us at 23872 x 2040 and 110 with add,
    // through registers 51 and 92; bf16 rows 36 and 68 against 42 and 63 to 67,
    // and more where a row is longer (8000 x 5120: 52 against 65)
    constexpr int kWords = CPT * (words<XT>() + 1);
    constexpr int kStages = sizeof(XT) == 4 && CPT <= 2 ? 0 : ring_stages(kWords);
    const NormPlan p = norm_plan(rows, d, CPT);
    const int threads = p.groups * p.warps * 32;
    auto *kern = norm_fwd<XT, CPT, kStages>;
    static PerDeviceOnce attr;
    if (!device_once(attr, [&] { return set_smem_limit(kern, kNormRing); })) return MOE_ERR_CUDA;
    launch_pdl(kern, p.ctas, threads, (size_t)kStages * kWords * 16 * kNormMaxThreads, stream, rows, d, p.warps,
               static_cast<const XT *>(x), add, gamma, beta, eps, static_cast<XT *>(x_sum), y, mean,
               rstd);
    return launch_status();
}

template <typename XT, typename YT, typename GT, int CPT>
moe_status launch_norm_bwd(int32_t rows, int32_t d, const void *x, const void *dy,
                           const float *gamma, const float *mean, const float *rstd,
                           const void *dres, void *dx, float *dgamma, float *dbeta, void *ws,
                           cudaStream_t stream) {
    const NormPlan p = norm_plan(rows, d, CPT);
    const int threads = p.groups * p.warps * 32;
    float *part = dgamma || dbeta ? reinterpret_cast<float *>(static_cast<uint8_t *>(ws) + 256) : nullptr;
    if (rows > 0) {
        auto *kern = norm_bwd<XT, YT, GT, CPT>;
        static PerDeviceOnce attr;
        if (!device_once(attr, [&] { return set_smem_limit(kern, kNormRing); })) return MOE_ERR_CUDA;
        // gamma, and the groups' weight sums at the end
        const size_t smem = std::max((size_t)p.groups * 2 * d * sizeof(float),
                                     (size_t)CPT * 2 * 16 * kNormMaxThreads);
        launch_pdl(kern, p.ctas, threads, smem, stream, rows, d, p.warps, static_cast<const XT *>(x),
                   static_cast<const YT *>(dy), gamma, mean, rstd, static_cast<const GT *>(dres),
                   static_cast<GT *>(dx), part);
    }
    if (part)
        launch_pdl(norm_bwd_sum, (2 * d / 4 + 15) / 16, kSumThreads, 0, stream, d,
                   rows > 0 ? p.ctas : 0, static_cast<const float *>(part), dgamma, dbeta);
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
    auto go = [&](auto xt) {
        return with_cpt(norm_cpt(d), [&](auto c) {
            return launch_norm_fwd<decltype(xt), decltype(c)::value>(rows, d, x, add, gamma, beta, eps,
                                                                     x_sum, y, mean, rstd, stream);
        });
    };
    return x_dtype == MOE_BF16 ? go(uint16_t()) : go(float());
}

MOE_API size_t moe_layer_norm_backward_workspace_bytes(int32_t rows, int32_t d) {
    if (check_norm(rows, d) != MOE_OK) return 0;
    return 256 + (size_t)kNormCtas * 2 * d * sizeof(float);
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
        return with_cpt(bwd_cpt(d, sizeof(xt) + sizeof(yt)), [&](auto c) {
            return launch_norm_bwd<decltype(xt), decltype(yt), decltype(gt), decltype(c)::value>(
                rows, d, x, dy, gamma, mean, rstd, dres, dx, dgamma, dbeta, ws, stream);
        });
    };
    auto go_g = [&](auto xt, auto yt) {
        return dx_dtype == MOE_BF16 ? go(xt, yt, uint16_t()) : go(xt, yt, float());
    };
    auto go_y = [&](auto xt) {
        return dy_dtype == MOE_BF16 ? go_g(xt, uint16_t()) : go_g(xt, float());
    };
    return x_dtype == MOE_BF16 ? go_y(uint16_t()) : go_y(float());
}

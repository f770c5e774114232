// Activation checkpoints in MXINT8 and the backward steps that read them
// (include/moe_block.h).
//
// Block of 32 elements along a row: E = floor(log2 max|v|) >= -127, codes
// c = rne(v 2^(6-E)) held to +-127, value c 2^(E-6).  v 2^(6-E) is exact in
// fp32 (a power-of-two multiple of a bf16), so the rounding decision, and
// with it every code, is a function of the input alone; the value has at most
// 7 significant bits and is exact in bf16.
//
// A lane takes 8 elements (16 bytes of bf16), a block is four lanes.  All
// kernels are bound by HBM.
#include <algorithm>

#include "../../include/moe_block.h"
#include "moe_common.cuh"

namespace moe {
namespace {

constexpr int kCkThreads = 256;
constexpr int kCkBlock = 32;

// |v| of both bf16 halves of a word, as two 16-bit integers; the larger of
// each pair orders like the magnitudes (NaN above infinity above the rest).
__device__ __forceinline__ uint32_t abs_max2(uint32_t a, uint32_t b) {
    return __vmaxu2(a & 0x7FFF7FFFu, b & 0x7FFF7FFFu);
}

// Scale byte of the block held by this lane and its three neighbours.
__device__ __forceinline__ uint32_t block_byte(const uint4 &v) {
    uint32_t m = abs_max2(v.x, v.y);
    m = __vmaxu2(m, abs_max2(v.z, v.w));
    m = __vmaxu2(m, __shfl_xor_sync(0xFFFFFFFFu, m, 1));
    m = __vmaxu2(m, __shfl_xor_sync(0xFFFFFFFFu, m, 2));
    return max(m & 0xFFFFu, m >> 16) >> 7;  // the exponent field, E + 127
}

// 2^(127 - byte), that is 2^-E, for byte <= 254.
__device__ __forceinline__ float inv_scale(uint32_t byte) {
    return byte == 254u ? __uint_as_float(0x00400000u) : __uint_as_float((254u - byte) << 23);
}

// Adding 1.5 * 2^23 leaves the nearest integer, ties to even, in a float's low
// bits, and a byte of them is the code.  With conversions and shifts the save was
// bound by its instructions (118 per 8 elements a lane, 78% of the issue slots):
// 136 us on the OLMoE-like layer's buffers against 128.
constexpr float kRound = 12582912.f;

// The codes of two values, as the low bytes of a pair of words.
__device__ __forceinline__ float2 code_pair(uint32_t w, float2 inv) {
    float2 v = __fmul2_rn(make_float2(bf16_lo(w), bf16_hi(w)), inv);
    v = make_float2(fminf(fmaxf(v.x, -1.984375f), 1.984375f), fminf(fmaxf(v.y, -1.984375f), 1.984375f));
    return __ffma2_rn(v, make_float2(64.f, 64.f), make_float2(kRound, kRound));
}

__device__ __forceinline__ uint32_t codes4(uint32_t w0, uint32_t w1, float2 inv) {
    const float2 a = code_pair(w0, inv), b = code_pair(w1, inv);
    const uint32_t lo = __byte_perm(__float_as_uint(a.x), __float_as_uint(a.y), 0x0040);
    const uint32_t hi = __byte_perm(__float_as_uint(b.x), __float_as_uint(b.y), 0x0040);
    return __byte_perm(lo, hi, 0x5410);
}

__device__ __forceinline__ uint2 codes8(const uint4 &v, uint32_t byte) {
    if (byte == 255u) return make_uint2(0u, 0u);
    const float s = inv_scale(byte);
    const float2 inv = make_float2(s, s);
    return make_uint2(codes4(v.x, v.y, inv), codes4(v.z, v.w, inv));
}

// 2^(byte - 133), the value of one code step; NaN for byte 255.
__device__ __forceinline__ float code_step(uint32_t byte) {
    if (byte == 255u) return __uint_as_float(0x7FC00000u);
    return e8m0_value(byte) * 0.015625f;
}

__device__ __forceinline__ void values8(const uint2 &q, float step, float (&f)[8]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[i] = (float)(int8_t)(q.x >> (8 * i)) * step;
        f[4 + i] = (float)(int8_t)(q.y >> (8 * i)) * step;
    }
}

// silu(z) = z / (1 + exp(-z)) from exp(-|z|) <= 1, which never overflows: with
// exp(-z) a z below -88 would give 0 where z exp(z) is still a normal number.
__device__ __forceinline__ float silu(float z) {
    const float t = __expf(-fabsf(z));
    const float r = __fdividef(1.f, 1.f + t);
    return z * (z < 0.f ? t * r : r);
}

__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
    return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                      pack_bf16x2(f[6], f[7]));
}

struct SaveBuf {
    const uint4 *src;
    uint2 *q;
    uint8_t *scale;
    int chunks;  // 8-element chunks per row, a multiple of 4; 0: left out
};
struct SaveBufs {
    SaveBuf b[3];
};

// The valid rows of a packed buffer are one contiguous run of chunks; a warp
// takes kUnroll x 32 of them at a time, all loads before the first use, so
// that an SM keeps 80 KB of loads in flight (5 CTAs of 48 registers a thread;
// one chunk a lane at a time moved 5.2 TB/s on the OLMoE-like layer's buffers).
constexpr int kUnroll = 4;

__global__ void __launch_bounds__(kCkThreads)
checkpoint_save_rows(const int32_t *__restrict__ offset, int N, int64_t R, const SaveBufs bufs) {
    pdl_enter();
    const int64_t A = min((int64_t)max(offset[N], 0), R);
    const int lane = threadIdx.x & 31;
    const int64_t warp0 = ((int64_t)blockIdx.x * kCkThreads + threadIdx.x) >> 5;
    const int64_t warps = (int64_t)gridDim.x * (kCkThreads / 32);
#pragma unroll
    for (int i = 0; i < 3; ++i) {
        const SaveBuf b = bufs.b[i];
        const int64_t n = A * b.chunks;
        // whole warps step together: the shuffles need every lane
        for (int64_t c0 = warp0 * (32 * kUnroll); c0 < n; c0 += warps * (32 * kUnroll)) {
            uint4 v[kUnroll];
#pragma unroll
            for (int u = 0; u < kUnroll; ++u) {
                const int64_t c = c0 + u * 32 + lane;
                v[u] = c < n ? __ldcs(b.src + c) : make_uint4(0u, 0u, 0u, 0u);
            }
#pragma unroll
            for (int u = 0; u < kUnroll; ++u) {
                const int64_t c = c0 + u * 32 + lane;
                const uint32_t byte = block_byte(v[u]);
                if (c >= n) continue;
                b.q[c] = codes8(v[u], byte);
                if ((c & 3) == 0) b.scale[c >> 2] = (uint8_t)byte;
            }
        }
    }
}

constexpr int kRestoreUnroll = 2;

__global__ void __launch_bounds__(kCkThreads)
checkpoint_restore_rows(const int32_t *__restrict__ offset, int N, int64_t R, int chunks,
                        const uint2 *__restrict__ g_q, const uint8_t *__restrict__ g_scale,
                        const uint2 *__restrict__ u_q, const uint8_t *__restrict__ u_scale,
                        uint4 *__restrict__ g_save, uint4 *__restrict__ u_save,
                        uint4 *__restrict__ h_act) {
    pdl_enter();
    const int64_t n = min((int64_t)max(offset[N], 0), R) * chunks;
    const int lane = threadIdx.x & 31;
    const int64_t warp0 = ((int64_t)blockIdx.x * kCkThreads + threadIdx.x) >> 5;
    const int64_t warps = (int64_t)gridDim.x * (kCkThreads / 32);
    for (int64_t c0 = warp0 * (32 * kRestoreUnroll) + lane; c0 < n; c0 += warps * (32 * kRestoreUnroll)) {
        uint2 gq[kRestoreUnroll], uq[kRestoreUnroll];
        uint32_t gs[kRestoreUnroll], us[kRestoreUnroll];
#pragma unroll
        for (int v = 0; v < kRestoreUnroll; ++v) {
            const int64_t c = c0 + v * 32;
            if (c >= n) continue;
            gq[v] = __ldcs(g_q + c);
            uq[v] = __ldcs(u_q + c);
            gs[v] = g_scale[c >> 2];
            us[v] = u_scale[c >> 2];
        }
#pragma unroll
        for (int v = 0; v < kRestoreUnroll; ++v) {
            const int64_t c = c0 + v * 32;
            if (c >= n) continue;
            float g[8], u[8], h[8];
            values8(gq[v], code_step(gs[v]), g);
            values8(uq[v], code_step(us[v]), u);
#pragma unroll
            for (int i = 0; i < 8; ++i) h[i] = silu(g[i]) * u[i];
            g_save[c] = pack8(g);
            u_save[c] = pack8(u);
            h_act[c] = pack8(h);
        }
    }
}

// One warp per token, as moe_combine_backward's kernel: for each chunk of the
// token's dy the K route rows' codes are read at once, and the K partial dot
// products stay in registers.  Two warps a CTA: a token's work goes by its
// accepted routes, and with 8 warps a CTA waited for its longest (84 and 98 us
// on the OLMoE-like and a drop-heavy layer, 76 and 86 with 2).
constexpr int kTokWarps = 2;
constexpr int kTokUnroll = 2;

template <int MAXK>
__global__ void __launch_bounds__(kTokWarps * 32)
combine_bwd_checkpoint_rows(int T, int nchunk, int K, const uint4 *__restrict__ dy,
                            const uint2 *__restrict__ y_q, const uint8_t *__restrict__ y_scale,
                            const int32_t *__restrict__ route_row, const float *__restrict__ gate,
                            uint4 *__restrict__ dy_disp, float *__restrict__ dgate,
                            float *__restrict__ dlogit) {
    pdl_enter();
    const int lane = threadIdx.x & 31;
    const int64_t t = (int64_t)blockIdx.x * kTokWarps + (threadIdx.x >> 5);
    if (t >= T) return;
    const int32_t my_row = lane < K ? route_row[t * K + lane] : -1;
    const float my_g = lane < K ? gate[t * K + lane] : 0.0f;
    int32_t rows[MAXK];
    float gs[MAXK], part[MAXK];
#pragma unroll
    for (int k = 0; k < MAXK; ++k) {
        rows[k] = __shfl_sync(0xFFFFFFFFu, my_row, k);
        gs[k] = __shfl_sync(0xFFFFFFFFu, my_g, k);
        part[k] = 0.0f;
    }
    for (int c0 = lane; c0 < nchunk; c0 += 32 * kTokUnroll) {
        uint4 w[kTokUnroll];
        uint2 q[kTokUnroll][MAXK];
        uint32_t sc[kTokUnroll][MAXK];
#pragma unroll
        for (int u = 0; u < kTokUnroll; ++u) {
            const int c = c0 + 32 * u;
            if (c >= nchunk) continue;
            w[u] = dy[t * nchunk + c];
#pragma unroll
            for (int k = 0; k < MAXK; ++k)
                if (k < K && rows[k] >= 0) {
                    const int64_t at = (int64_t)rows[k] * nchunk + c;
                    q[u][k] = __ldcs(y_q + at);
                    sc[u][k] = y_scale[at >> 2];
                }
        }
#pragma unroll
        for (int u = 0; u < kTokUnroll; ++u) {
            const int c = c0 + 32 * u;
            if (c >= nchunk) continue;
            const float f[8] = {bf16_lo(w[u].x), bf16_hi(w[u].x), bf16_lo(w[u].y), bf16_hi(w[u].y),
                                bf16_lo(w[u].z), bf16_hi(w[u].z), bf16_lo(w[u].w), bf16_hi(w[u].w)};
#pragma unroll
            for (int k = 0; k < MAXK; ++k) {
                if (k >= K || rows[k] < 0) continue;
                float o[8], pr[8];
                values8(q[u][k], code_step(sc[u][k]), o);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    pr[i] = __fmul_rn(gs[k], f[i]);
                    part[k] = __fmaf_rn(f[i], o[i], part[k]);
                }
                dy_disp[(int64_t)rows[k] * nchunk + c] = pack8(pr);
            }
        }
    }
    // lane k < K ends up with route k's dgate; dot is the chain over k ascending
    // that the dispatch's router backward takes
    float mine = 0.f, dot = 0.f;
#pragma unroll
    for (int k = 0; k < MAXK; ++k) {
        if (k >= K) break;
        float v = part[k];
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, off);
        if (rows[k] < 0) v = 0.f;
        if (lane == k) mine = v;
        dot = fmaf(gs[k], v, dot);
    }
    if (lane < K) {
        dgate[t * K + lane] = mine;
        if (dlogit) dlogit[t * K + lane] = my_g * (mine - dot);
    }
}

// CTAs for `chunks`, `waves` per SM at most: several times what is resident (5
// of 48 registers a thread), so that SMs which finish early take more, but few
// enough that the rows past expert_offset[N], which the host does not know, cost
// nothing.  8 per SM, 1.6 waves, took 140 us to save and 94 to restore the
// OLMoE-like layer's buffers, 40 and 80 take 135 and 86; one CTA per 1024 chunks
// of the whole buffer took 134 instead of 112 us to save a drop-heavy layer's.
constexpr int kSaveWaves = 40, kRestoreWaves = 80;

inline int ck_grid(int64_t chunks, int unroll, int waves) {
    const int64_t per = (int64_t)kCkThreads * unroll, want = (chunks + per - 1) / per;
    return (int)std::min<int64_t>(want, (int64_t)num_sms() * waves);
}

}  // namespace
}  // namespace moe

using namespace moe;

MOE_API moe_status moe_checkpoint_save(const moe_shape *s, const int32_t *expert_offset,
                                       const moe_bf16 *g_save, const moe_bf16 *u_save,
                                       const moe_bf16 *y_disp, int8_t *g_q, uint8_t *g_scale,
                                       int8_t *u_q, uint8_t *u_scale, int8_t *y_q, uint8_t *y_scale,
                                       cudaStream_t stream) {
    moe_status r = check_shape(s);
    if (r != MOE_OK) return r;
    if (s->d % kCkBlock != 0 || s->h % kCkBlock != 0) return MOE_ERR_UNSUPPORTED;
    const int64_t R = buffer_rows(s);
    if (R == 0) return MOE_OK;
    if (!expert_offset || (g_save && (!g_q || !g_scale)) || (u_save && (!u_q || !u_scale)) ||
        (y_disp && (!y_q || !y_scale)))
        return MOE_ERR_INVALID_ARG;
    const void *ptrs[] = {expert_offset, g_save, u_save, y_disp, g_q, g_scale, u_q, u_scale, y_q,
                          y_scale};
    for (const void *p : ptrs)
        if (!aligned16(p)) return MOE_ERR_ALIGNMENT;
    const moe_bf16 *src[3] = {g_save, u_save, y_disp};
    int8_t *q[3] = {g_q, u_q, y_q};
    uint8_t *sc[3] = {g_scale, u_scale, y_scale};
    SaveBufs bufs;
    int64_t most = 0;
    for (int i = 0; i < 3; ++i) {
        const int chunks = src[i] ? (i < 2 ? s->h : s->d) / 8 : 0;
        bufs.b[i] = SaveBuf{reinterpret_cast<const uint4 *>(src[i]), reinterpret_cast<uint2 *>(q[i]),
                            sc[i], chunks};
        if (R * chunks > most) most = R * chunks;
    }
    if (most == 0) return MOE_OK;
    launch_pdl(checkpoint_save_rows, ck_grid(most, kUnroll, kSaveWaves), kCkThreads, 0, stream, expert_offset, s->N, R, bufs);
    return launch_status();
}

MOE_API moe_status moe_checkpoint_restore(const moe_shape *s, const int32_t *expert_offset,
                                          const int8_t *g_q, const uint8_t *g_scale,
                                          const int8_t *u_q, const uint8_t *u_scale,
                                          moe_bf16 *g_save, moe_bf16 *u_save, moe_bf16 *h_act,
                                          cudaStream_t stream) {
    moe_status r = check_shape(s);
    if (r != MOE_OK) return r;
    if (s->d % kCkBlock != 0 || s->h % kCkBlock != 0) return MOE_ERR_UNSUPPORTED;
    const int64_t R = buffer_rows(s);
    if (R == 0) return MOE_OK;
    const void *ptrs[] = {expert_offset, g_q, g_scale, u_q, u_scale, g_save, u_save, h_act};
    for (const void *p : ptrs)
        if (!p) return MOE_ERR_INVALID_ARG;
    for (const void *p : ptrs)
        if (!aligned16(p)) return MOE_ERR_ALIGNMENT;
    const int chunks = s->h / 8;
    launch_pdl(checkpoint_restore_rows, ck_grid(R * chunks, kRestoreUnroll, kRestoreWaves), kCkThreads, 0, stream, expert_offset,
               s->N, R, chunks, reinterpret_cast<const uint2 *>(g_q), g_scale,
               reinterpret_cast<const uint2 *>(u_q), u_scale, reinterpret_cast<uint4 *>(g_save),
               reinterpret_cast<uint4 *>(u_save), reinterpret_cast<uint4 *>(h_act));
    return launch_status();
}

MOE_API moe_status moe_combine_backward_checkpoint(const moe_shape *s, const moe_bf16 *dy,
                                                   const int8_t *y_q, const uint8_t *y_scale,
                                                   const int32_t *route_row,
                                                   const float *topk_gate, moe_bf16 *dy_disp,
                                                   float *dgate, float *dlogit,
                                                   cudaStream_t stream) {
    moe_status r = check_shape(s);
    if (r != MOE_OK) return r;
    if (s->d % kCkBlock != 0 || s->h % kCkBlock != 0) return MOE_ERR_UNSUPPORTED;
    if (s->T == 0) return MOE_OK;
    if (!dy || !route_row || !topk_gate || !dgate ||
        (s->cap > 0 && (!y_q || !y_scale || !dy_disp)))
        return MOE_ERR_INVALID_ARG;
    const void *ptrs[] = {dy, y_q, y_scale, route_row, topk_gate, dy_disp, dgate, dlogit};
    for (const void *p : ptrs)
        if (!aligned16(p)) return MOE_ERR_ALIGNMENT;
    auto *kern = s->K <= 8 ? combine_bwd_checkpoint_rows<8> : combine_bwd_checkpoint_rows<16>;
    const int grid = (int)(((int64_t)s->T + kTokWarps - 1) / kTokWarps);
    launch_pdl(kern, grid, kTokWarps * 32, 0, stream, s->T, s->d / 8, s->K,
               reinterpret_cast<const uint4 *>(dy), reinterpret_cast<const uint2 *>(y_q), y_scale,
               route_row, topk_gate, reinterpret_cast<uint4 *>(dy_disp), dgate, dlogit);
    return launch_status();
}

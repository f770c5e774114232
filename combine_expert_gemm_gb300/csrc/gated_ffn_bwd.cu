// Backward of the dense gated feed-forward block (include/moe_dense.h), from the
// factors P = act(G), Q = U act'(G) and H that its forward saved:
//
//   R = dy Wd;  dU = s R P,  dG = s R Q,  Hs = s H,  ds = row sums of R H
//   dx = dx_in + dG Wg + dU Wu;  dWg = dG^T x, dWu = dU^T x, dWd = dy^T Hs
//
// Three products of CTA pairs (pair_gemm.cuh): R with the factors in its
// epilogue; dx over the 2 h columns of dG and dU; and the three weight gradients
// in one launch.  Operands that are transposed against their storage (weights in
// the first two, activations in the third) are read MN-major, so nothing is
// transposed in memory.  dG and dU are rounded to bf16 between the products, as
// the tensor core's operands have to be; all sums are fp32.
#include "ffn_common.cuh"

namespace moe {
namespace {

using namespace pair;

// Row sums of R H: one fp32 a row and 128-column half tile.
struct FactorArgs {
    CUtensorMap dy, wd, odg, odu, ohs;
    int T, d, h, mt, nt;
    const uint16_t *p, *q, *hact;
    const float *scale;
    float *part;  // [2 nt][T], or NULL
    int *status;
};

template <bool SCALE>
struct Factor {
    using Args = FactorArgs;
    struct Regs {
        float s;
        uint4 p[4], q[4], h[4];  // the factors of the 32 columns to come
    };
    static constexpr int kStages = 6;
    static constexpr int kStageBytes = 2 * OPERAND;
    static constexpr int kGroup = 0;
    static __device__ __forceinline__ int tiles(const Args &p) { return p.mt * p.nt; }
    static __device__ __forceinline__ Tile tile(const Args &p, int g) {
        int m, n;
        band_tile(g, p.mt, p.nt, m, n);
        return Tile{0, m * PM, n * BN};
    }
    static __device__ __forceinline__ int k_blocks(const Args &p, const Tile &) { return (p.d + BK - 1) / BK; }
    static __device__ __forceinline__ void load(const Args &p, const Tile &t, int kb, uint32_t s, uint32_t bar,
                                                int rank) {
        load_k(s, &p.dy, bar, kb * BK, t.m + rank * BM, 0);
        load_mn(s + OPERAND, &p.wd, bar, t.n + rank * BM, kb * BK, 0);
    }
    static __device__ __forceinline__ void mma(const Args &, const Tile &, uint32_t d, uint32_t s, bool first) {
        mma_block<1, false, true>(d, s, s + OPERAND, first);
    }
    static __device__ __forceinline__ void before(const Args &p, const Tile &t, Epi &e, int wrow, Regs &r) {
        const int row = t.m + wrow + e.lane;
        if (SCALE) r.s = row < p.T ? p.scale[row] : 0.0f;
        factors(p, row, t.n + e.col, r);
    }
    static __device__ __forceinline__ void fetch(const uint16_t *src, bool row_ok, int col, int h, uint4 (&v)[4]) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            v[i] = row_ok && col + 8 * i < h ? __ldcs(reinterpret_cast<const uint4 *>(src) + i) : make_uint4(0, 0, 0, 0);
    }
    static __device__ __forceinline__ void factors(const Args &p, int row, int col, Regs &r) {
        const int64_t at = (int64_t)row * p.h + col;
        fetch(p.p + at, row < p.T, col, p.h, r.p);
        fetch(p.q + at, row < p.T, col, p.h, r.q);
        if (SCALE) fetch(p.hact + at, row < p.T, col, p.h, r.h);
    }
    static __device__ __forceinline__ void epilogue(const Args &p, const Tile &t, Epi &e, int wrow, Regs &r) {
        const int row0 = t.m + wrow, row = row0 + e.lane;
        if (row0 >= p.T) return;
        float ds = 0.0f;
        const int colh = t.n + e.col;
#pragma unroll 1
        for (int c = 0; c < BN / 2; c += 32) {
            const int col = colh + c;
            if (col >= p.h) break;
            float v[32];
            read32(e.taddr + c, v);
            const uint32_t *pw = reinterpret_cast<const uint32_t *>(r.p);
            const uint32_t *qw = reinterpret_cast<const uint32_t *>(r.q);
            const uint32_t *hw = reinterpret_cast<const uint32_t *>(r.h);
            uint32_t du[16], dg[16], hs[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                float a = v[2 * i], b = v[2 * i + 1];
                if (SCALE) {
                    const float h0 = bf16_lo(hw[i]), h1 = bf16_hi(hw[i]);
                    // columns past h: the accumulator is 0 there
                    ds = fmaf(a, h0, ds);
                    ds = fmaf(b, h1, ds);
                    hs[i] = pack_bf16x2(r.s * h0, r.s * h1);
                    a *= r.s;
                    b *= r.s;
                }
                du[i] = pack_bf16x2(a * bf16_lo(pw[i]), b * bf16_hi(pw[i]));
                dg[i] = pack_bf16x2(a * bf16_lo(qw[i]), b * bf16_hi(qw[i]));
            }
            if (c + 32 < BN / 2) factors(p, row, col + 32, r);
            store_block16(e, du, &p.odu, col, row0, 0);
            store_block16(e, dg, &p.odg, col, row0, 0);
            if (SCALE) store_block16(e, hs, &p.ohs, col, row0, 0);
        }
        if (SCALE && p.part && row < p.T) p.part[(int64_t)(colh / (BN / 2)) * p.T + row] = ds;
    }
};

struct DxArgs {
    CUtensorMap dg, du, wg, wu, o;
    int T, d, h, mt, nt, hb;
    const void *dx_in;
    float *dx32;
    int *status;
};

template <bool F32>
struct Dx {
    using Args = DxArgs;
    struct Regs {};
    static constexpr int kStages = 6;
    static constexpr int kStageBytes = 2 * OPERAND;
    static constexpr int kGroup = 0;
    static __device__ __forceinline__ int tiles(const Args &p) { return p.mt * p.nt; }
    static __device__ __forceinline__ Tile tile(const Args &p, int g) {
        int m, n;
        band_tile(g, p.mt, p.nt, m, n);
        return Tile{0, m * PM, n * BN};
    }
    static __device__ __forceinline__ int k_blocks(const Args &p, const Tile &) { return 2 * p.hb; }
    static __device__ __forceinline__ void load(const Args &p, const Tile &t, int kb, uint32_t s, uint32_t bar,
                                                int rank) {
        const bool up = kb >= p.hb;
        const int k = (up ? kb - p.hb : kb) * BK;
        load_k(s, up ? &p.du : &p.dg, bar, k, t.m + rank * BM, 0);
        load_mn(s + OPERAND, up ? &p.wu : &p.wg, bar, t.n + rank * BM, k, 0);
    }
    static __device__ __forceinline__ void mma(const Args &, const Tile &, uint32_t d, uint32_t s, bool first) {
        mma_block<1, false, true>(d, s, s + OPERAND, first);
    }
    static __device__ __forceinline__ void before(const Args &, const Tile &, const Epi &, int, Regs &) {}
    static __device__ __forceinline__ void epilogue(const Args &p, const Tile &t, Epi &e, int wrow, Regs &) {
        const int row0 = t.m + wrow, row = row0 + e.lane;
        if (row0 >= p.T) return;
#pragma unroll 1
        for (int c = 0; c < BN / 2; c += 32) {
            const int col = t.n + e.col + c;
            if (col >= p.d) break;
            const int64_t at = (int64_t)row * p.d + col;
            float v[32];
            if (F32) {
                const float4 *src = reinterpret_cast<const float4 *>(static_cast<const float *>(p.dx_in) + at);
                float4 in[8];
                if (p.dx_in) {
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        in[i] = row < p.T && col + 4 * i < p.d ? __ldcs(src + i) : make_float4(0, 0, 0, 0);
                }
                read32(e.taddr + c, v);
                float4 *dst = reinterpret_cast<float4 *>(p.dx32 + at);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    float4 o = make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
                    if (p.dx_in) o = make_float4(o.x + in[i].x, o.y + in[i].y, o.z + in[i].z, o.w + in[i].w);
                    if (row < p.T && col + 4 * i < p.d) __stcs(dst + i, o);
                }
            } else {
                const uint4 *src = reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(p.dx_in) + at);
                uint4 in[4];
                if (p.dx_in) {
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        in[i] = row < p.T && col + 8 * i < p.d ? __ldcs(src + i) : make_uint4(0, 0, 0, 0);
                }
                read32(e.taddr + c, v);
                const uint32_t *iw = reinterpret_cast<const uint32_t *>(in);
                uint32_t w[16];
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    w[i] = p.dx_in ? pack_bf16x2(v[2 * i] + bf16_lo(iw[i]), v[2 * i + 1] + bf16_hi(iw[i]))
                                   : pack_bf16x2(v[2 * i], v[2 * i + 1]);
                store_block16(e, w, &p.o, col, row0, 0);
            }
        }
    }
};

// The three weight gradients: their tiles one after the other, dWd first.  The
// reduction runs over the tokens.
struct WeightArgs {
    CUtensorMap a[3];  // dy, dG, dU: rows of the gradient
    CUtensorMap b[2];  // Hs, x: its columns
    CUtensorMap o[3];
    int T, d, h;
    int md, nd;        // 256-tiles of d and h
    int *status;
};

template <bool F32>
struct Weight {
    using Args = WeightArgs;
    struct Regs {};
    static constexpr int kStages = 6;
    static constexpr int kStageBytes = 2 * OPERAND;
    static constexpr int kGroup = 0;
    static __device__ __forceinline__ int tiles(const Args &p) { return 3 * p.md * p.nd; }
    // z: which weight.  dWd [d, h], dWg and dWu [h, d]
    static __device__ __forceinline__ Tile tile(const Args &p, int g) {
        const int per = p.md * p.nd, z = g / per;
        int m, n;
        band_tile(g - z * per, z ? p.nd : p.md, z ? p.md : p.nd, m, n);
        return Tile{z, m * PM, n * BN};
    }
    static __device__ __forceinline__ int k_blocks(const Args &p, const Tile &) { return (p.T + BK - 1) / BK; }
    static __device__ __forceinline__ void load(const Args &p, const Tile &t, int kb, uint32_t s, uint32_t bar,
                                                int rank) {
        load_mn(s, &p.a[t.z], bar, t.m + rank * BM, kb * BK, 0);
        load_mn(s + OPERAND, &p.b[t.z ? 1 : 0], bar, t.n + rank * BM, kb * BK, 0);
    }
    static __device__ __forceinline__ void mma(const Args &, const Tile &, uint32_t d, uint32_t s, bool first) {
        mma_block<1, true, true>(d, s, s + OPERAND, first);
    }
    static __device__ __forceinline__ void before(const Args &, const Tile &, const Epi &, int, Regs &) {}
    static __device__ __forceinline__ void epilogue(const Args &p, const Tile &t, Epi &e, int wrow, Regs &) {
        const int row0 = t.m + wrow, rows = t.z ? p.h : p.d, cols = t.z ? p.d : p.h;
        if (row0 >= rows) return;
        const CUtensorMap *map = &p.o[t.z];
#pragma unroll 1
        for (int c = 0; c < BN / 2; c += 32) {
            const int col = t.n + e.col + c;
            if (col >= cols) break;
            float v[32];
            read32(e.taddr + c, v);
            if (F32) {
                if (e.lane == 0) bulk_wait_read<0>();
                __syncwarp();
#pragma unroll
                for (int q = 0; q < 8; ++q)
                    *reinterpret_cast<float4 *>(e.blk + e.lane * 128 + ((q ^ (e.lane & 7)) * 16)) =
                        make_float4(v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]);
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                __syncwarp();
                if (e.lane == 0) {
                    tma_store_3d(map, smem_u32(e.blk), col, row0, 0);
                    bulk_commit();
                }
            } else {
                uint32_t w[16];
#pragma unroll
                for (int i = 0; i < 16; ++i) w[i] = pack_bf16x2(v[2 * i], v[2 * i + 1]);
                store_block16(e, w, map, col, row0, 0);
            }
        }
    }
};

// out[t] = the sum of part[0..n)[t], in order.
template <bool F32>
__global__ void __launch_bounds__(256) token_scale_sum(int T, int n, const float *__restrict__ part, void *out) {
    pdl_enter();
    const int t = blockIdx.x * 256 + threadIdx.x;
    if (t >= T) return;
    float s = 0.0f;
    for (int i = 0; i < n; ++i) s += part[(int64_t)i * T + t];
    if (F32) static_cast<float *>(out)[t] = s;
    else static_cast<__nv_bfloat16 *>(out)[t] = __float2bfloat16_rn(s);
}

inline size_t align256(size_t v) { return (v + 255) & ~(size_t)255; }

// Workspace: status, dG, dU, Hs [T, h] bf16, the parts of dtoken_scale.
struct Layout {
    size_t dg, du, hs, part, bytes;
    Layout(int64_t T, int64_t h) {
        const size_t a = align256((size_t)(T * h * 2));
        dg = 256;
        du = dg + a;
        hs = du + a;
        part = hs + a;
        bytes = part + align256((size_t)(2 * ((h + BN - 1) / BN) * T * 4));
    }
};

}  // namespace
}  // namespace moe

using namespace moe;

MOE_API size_t moe_gated_ffn_backward_workspace_bytes(int32_t T, int32_t d, int32_t h) {
    if (check_ffn(T, d, h) != MOE_OK) return 0;
    return Layout(T, h).bytes;
}

MOE_API moe_status moe_gated_ffn_backward(int32_t T, int32_t d, int32_t h, const moe_bf16 *x,
                                          const moe_bf16 *w_gate, const moe_bf16 *w_up,
                                          const moe_bf16 *w_down, const float *token_scale,
                                          const moe_bf16 *h_act, const moe_bf16 *p_save,
                                          const moe_bf16 *q_save, const moe_bf16 *dy, int32_t dx_dtype,
                                          const void *dx_in, void *dx, int32_t dw_dtype, void *dw_gate,
                                          void *dw_up, void *dw_down, void *dtoken_scale, void *ws,
                                          size_t ws_bytes, cudaStream_t stream) {
    moe_status r = check_ffn(T, d, h);
    if (r != MOE_OK) return r;
    if ((dx_dtype != MOE_BF16 && dx_dtype != MOE_FP32) || (dw_dtype != MOE_BF16 && dw_dtype != MOE_FP32))
        return MOE_ERR_INVALID_ARG;
    if (dtoken_scale && !token_scale) return MOE_ERR_INVALID_ARG;
    if (!w_gate || !w_up || !w_down || !dw_gate || !dw_up || !dw_down) return MOE_ERR_INVALID_ARG;
    if (T > 0 && (!x || !h_act || !p_save || !q_save || !dy || !dx)) return MOE_ERR_INVALID_ARG;
    // the weights' gradients read x and dy after dx is written
    if (T > 0 && (dx == x || dx == dy)) return MOE_ERR_INVALID_ARG;
    const Layout at(T, h);
    if (!ws || ws_bytes < at.bytes || (reinterpret_cast<uintptr_t>(ws) & 255u)) return MOE_ERR_WORKSPACE;
    const void *ptrs[] = {x,  w_gate, w_up, w_down,  token_scale, h_act,   p_save,      q_save,
                          dy, dx_in,  dx,   dw_gate, dw_up,       dw_down, dtoken_scale};
    for (const void *q : ptrs)
        if (!aligned16(q)) return MOE_ERR_ALIGNMENT;
    const bool dw32 = dw_dtype == MOE_FP32;
    if (T == 0) {
        const size_t n = (size_t)d * h * (dw32 ? 4 : 2);
        if (cudaMemsetAsync(dw_gate, 0, n, stream) != cudaSuccess ||
            cudaMemsetAsync(dw_up, 0, n, stream) != cudaSuccess ||
            cudaMemsetAsync(dw_down, 0, n, stream) != cudaSuccess)
            return MOE_ERR_CUDA;
        return MOE_OK;
    }
    char *base = static_cast<char *>(ws);
    int *status = reinterpret_cast<int *>(base);
    const void *hs = token_scale ? base + at.hs : static_cast<const void *>(h_act);

    FactorArgs f{};
    f.T = T;
    f.d = d;
    f.h = h;
    f.mt = (T + PM - 1) / PM;
    f.nt = (h + BN - 1) / BN;
    f.p = reinterpret_cast<const uint16_t *>(p_save);
    f.q = reinterpret_cast<const uint16_t *>(q_save);
    f.hact = reinterpret_cast<const uint16_t *>(h_act);
    f.scale = token_scale;
    f.part = dtoken_scale ? reinterpret_cast<float *>(base + at.part) : nullptr;
    f.status = status;
    DxArgs g{};
    g.T = T;
    g.d = d;
    g.h = h;
    g.mt = f.mt;
    g.nt = (d + BN - 1) / BN;
    g.hb = (h + BK - 1) / BK;
    g.dx_in = dx_in;
    g.dx32 = static_cast<float *>(dx);
    g.status = status;
    WeightArgs w{};
    w.T = T;
    w.d = d;
    w.h = h;
    w.md = g.nt;
    w.nd = f.nt;
    w.status = status;
    const bool dx32 = dx_dtype == MOE_FP32;
    if (!map_k(&f.dy, dy, d, T) || !map_mn(&f.wd, w_down, h, d) || !map_store(&f.odg, base + at.dg, h, T) ||
        !map_store(&f.odu, base + at.du, h, T) || !map_store(&f.ohs, base + at.hs, h, T) ||
        !map_k(&g.dg, base + at.dg, h, T) || !map_k(&g.du, base + at.du, h, T) || !map_mn(&g.wg, w_gate, d, h) ||
        !map_mn(&g.wu, w_up, d, h) || (!dx32 && !map_store(&g.o, dx, d, T)) || !map_mn(&w.a[0], dy, d, T) ||
        !map_mn(&w.a[1], base + at.dg, h, T) || !map_mn(&w.a[2], base + at.du, h, T) ||
        !map_mn(&w.b[0], hs, h, T) || !map_mn(&w.b[1], x, d, T))
        return MOE_ERR_CUDA;
    void *dw[3] = {dw_down, dw_gate, dw_up};
    for (int i = 0; i < 3; ++i) {
        const uint64_t inner = i ? d : h, rows = i ? h : d;
        if (!(dw32 ? make_map_f32_3d(&w.o[i], dw[i], inner, rows, 1) : map_store(&w.o[i], dw[i], inner, rows)))
            return MOE_ERR_CUDA;
    }
    const int64_t ftiles = (int64_t)f.mt * f.nt, gtiles = (int64_t)g.mt * g.nt;
    r = token_scale ? launch<Factor<true>>(f, ftiles, stream) : launch<Factor<false>>(f, ftiles, stream);
    if (r != MOE_OK) return r;
    if (dtoken_scale) {
        launch_pdl(dw32 ? token_scale_sum<true> : token_scale_sum<false>, (unsigned)((T + 255) / 256), 256, 0, stream,
                   (int)T, 2 * f.nt, f.part, dtoken_scale);
        if ((r = launch_status()) != MOE_OK) return r;
    }
    r = dx32 ? launch<Dx<true>>(g, gtiles, stream) : launch<Dx<false>>(g, gtiles, stream);
    if (r != MOE_OK) return r;
    const int64_t wtiles = (int64_t)3 * w.md * w.nd;
    return dw32 ? launch<Weight<true>>(w, wtiles, stream) : launch<Weight<false>>(w, wtiles, stream);
}

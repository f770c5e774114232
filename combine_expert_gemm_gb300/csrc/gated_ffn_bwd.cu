// Backward of the dense gated feed-forward block (include/moe_dense.h), from the
// factors P = act(G), Q = U act'(G) and H that its forward saved:
//
//   R = dy Wd;  dU = s R P,  dG = s R Q,  Hs = s H,  ds = row sums of R H
//   dx = dx_in + dG Wg + dU Wu;  dWg = dG^T x, dWu = dU^T x, dWd = dy^T Hs
//
// Two launches of CTA pairs (pair_gemm.cuh): R with the factors in its epilogue,
// then dx and the three weight gradients together.  Operands that are transposed
// against their storage (weights in R and dx, activations in the weight gradients)
// are read MN-major, so nothing is transposed in memory.  dG and dU are rounded to bf16 between the products, as
// the tensor core's operands have to be; all sums are fp32.
#include "ffn_common.cuh"
#include "small_gemm.cuh"

namespace moe {
namespace {

using namespace pair;

// Row sums of R H: one fp32 a row and half tile.
struct FactorArgs {
    CUtensorMap dy, wd, odg, odu, ohs;
    int T, d, h, mt, nt;
    const uint16_t *p, *q, *hact;
    const float *scale;
    float *part;  // [2 nt][T], or NULL
    int *status;
};

template <bool SCALE, int N>
struct Factor {
    using Args = FactorArgs;
    struct Regs {
        float s;
        uint4 p[4], q[4], h[4];  // the factors of the 32 columns to come
    };
    static constexpr int kN = N, kStages = N == 256 ? 6 : 8;
    static constexpr int kStageBytes = OPERAND + b_bytes(N);
    static constexpr int kGroup = 0;
    static __device__ __forceinline__ int count(const Args &p, int unit, int units) {
        return strided_count(p.mt * p.nt, unit, units);
    }
    static __device__ __forceinline__ Tile tile(const Args &p, int unit, int units, int i) {
        int m, n;
        band_tile(unit + i * units, p.mt, p.nt, m, n);
        return Tile{0, m * PM, n * N};
    }
    static __device__ __forceinline__ int k_blocks(const Args &p, const Tile &) { return (p.d + BK - 1) / BK; }
    static __device__ __forceinline__ void load(const Args &p, const Tile &t, int kb, uint32_t s, uint32_t bar,
                                                int rank) {
        load_k(s, &p.dy, bar, kb * BK, t.m + rank * BM, 0);
        load_mn<N / 2>(s + OPERAND, &p.wd, bar, t.n + rank * (N / 2), kb * BK, 0);
    }
    static __device__ __forceinline__ void mma(const Args &, const Tile &, uint32_t d, uint32_t s, bool first) {
        mma_block<1, N, false, true>(d, s, s + OPERAND, first);
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
        for (int c = 0; c < N / 2; c += 32) {
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
            if (c + 32 < N / 2) factors(p, row, col + 32, r);
            store_block16(e, du, &p.odu, col, row0, 0);
            store_block16(e, dg, &p.odg, col, row0, 0);
            if (SCALE) store_block16(e, hs, &p.ohs, col, row0, 0);
        }
        if (SCALE && p.part && row < p.T) p.part[(int64_t)(colh / (N / 2)) * p.T + row] = ds;
    }
};

// The same for few tokens (small_gemm.cuh): the features are hidden units, Wd is
// read MN-major.
struct SmallFactorArgs {
    CUtensorMap wd, dy;
    int T, h, nk, split, tt;
    const uint16_t *p, *q, *hact;
    const float *scale;
    uint16_t *dg, *du, *hs;
    float *part;  // [ceil(h / 128) split][T], or NULL
    int *status;
};

template <bool SCALE, int N>
struct SmallFactor {
    using Args = SmallFactorArgs;
    static constexpr int kN = N;
    static constexpr bool kPairs = false, kEarly = false;
    static constexpr int kAMn = 1, kBMn = 0, kFmt = 1, kPieces = 1;
    static constexpr bool kMirror = false;
    static __device__ __forceinline__ void load_a(const Args &p, uint32_t s, uint32_t bar, int kb, int f0, int, int) {
        small::load_box(s, &p.wd, bar, f0, kb * BK);
        small::load_box(s + BLK, &p.wd, bar, f0 + 64, kb * BK);
    }
    static __device__ __forceinline__ void load_b(const Args &p, uint32_t s, uint32_t bar, int kb, int t0, int, int) {
        small::load_box(s, &p.dy, bar, kb * BK, t0);
    }
    static __device__ __forceinline__ void prefetch_maps(const Args &p) {
        tma_prefetch_desc(&p.wd);
        tma_prefetch_desc(&p.dy);
    }
    struct In {
        uint2 p, q, h;
        float s;
    };
    static __device__ __forceinline__ void fetch(const Args &p, int t, int f, int, In &in) {
        if (f >= p.h) return;
        const int64_t at = (int64_t)t * p.h + f;
        in.p = *reinterpret_cast<const uint2 *>(p.p + at);
        in.q = *reinterpret_cast<const uint2 *>(p.q + at);
        if (SCALE) {
            in.h = *reinterpret_cast<const uint2 *>(p.hact + at);
            in.s = p.scale[t];
        }
    }
    static __device__ __forceinline__ void emit(const Args &p, bool ok, int t, int f, int, const float4 &r,
                                                const float4 &, const In &in) {
        const int64_t at = (int64_t)t * p.h + f;
        float ds = 0.0f;
        if (ok && f < p.h) {
            const uint2 a = in.p, b = in.q;
            float4 v = r;
            if (SCALE) {
                const uint2 c = in.h;
                const float s = in.s;
                const float h0 = bf16_lo(c.x), h1 = bf16_hi(c.x), h2 = bf16_lo(c.y), h3 = bf16_hi(c.y);
                ds = fmaf(r.x, h0, fmaf(r.y, h1, fmaf(r.z, h2, r.w * h3)));
                *reinterpret_cast<uint2 *>(p.hs + at) = make_uint2(pack_bf16x2(s * h0, s * h1), pack_bf16x2(s * h2, s * h3));
                v = make_float4(s * r.x, s * r.y, s * r.z, s * r.w);
            }
            *reinterpret_cast<uint2 *>(p.du + at) = make_uint2(pack_bf16x2(v.x * bf16_lo(a.x), v.y * bf16_hi(a.x)),
                                                               pack_bf16x2(v.z * bf16_lo(a.y), v.w * bf16_hi(a.y)));
            *reinterpret_cast<uint2 *>(p.dg + at) = make_uint2(pack_bf16x2(v.x * bf16_lo(b.x), v.y * bf16_hi(b.x)),
                                                               pack_bf16x2(v.z * bf16_lo(b.y), v.w * bf16_hi(b.y)));
        }
        if (SCALE && p.part) {
            // the lanes of a token: this CTA's share of the tile's features (0 where
            // it lies past h)
            const int per = small::kM / 4 / p.split;
            for (int o = per / 2; o; o >>= 1) ds += __shfl_xor_sync(0xFFFFFFFFu, ds, o);
            if (ok && (threadIdx.x & (per - 1)) == 0) p.part[(int64_t)(f / (small::kM / p.split)) * p.T + t] = ds;
        }
    }
};

// dx and the three weight gradients in one launch: z = 0..2 are tiles of dWd
// [d, h], dWg and dWu [h, d], reduced over the tokens, z = 3 tiles of dx, reduced over
// the 2 h columns of dG and dU.  Alone, 96 weight tiles of an 8192-token step on 76
// pairs take two rounds and 256 tiles of dx four, 127 us where the products take 90;
// together the pairs get equal shares: first the kind with the longer tiles, in
// turn, then of the other kind as many as even the shares out (share).
//
// The weights' sums run over all tokens, dx's over 2 h.  In one accumulator the gradients
// of a million tokens came out 0.7% short, as the tensor core cuts where an fp32 addition
// rounds (pair_gemm.cuh).  Past kMostBlocks an accumulator holds that many, 8192
// tokens, and they are added in registers: a sum of terms of one sign is at most 2^-14
// short, whatever its length.  Sums that fit one accumulator stay there: tiles of 96
// tokens are all epilogue, and took 77 us for 69 through registers.
constexpr int kMostBlocks = 128;
struct GradArgs {
    CUtensorMap wa[3];     // dy, dG, dU: rows of a weight gradient
    CUtensorMap wb[2];     // Hs, x: its columns
    CUtensorMap wo[3];
    CUtensorMap xa[2];     // dG, dU
    CUtensorMap xb[2];     // Wg, Wu
    CUtensorMap xo;
    int T, d, h;
    int mt, md, mh;        // 256-row tiles of T, d and h
    int nd, nh;            // N-column tiles of d and h
    int hb, tb;            // k-blocks of h and T
    const void *dx_in;
    int long_x;            // the longer tiles are dx's
    // `r` units have q + 1 long tiles, the others q; of the short ones they get sa each, and
    // the others sb each, the first `se` of them one more
    int q, r, sa, sb, se;
    int *status;
};

template <bool DX32, bool DW32, int N, bool LONG>
struct Grad {
    using Args = GradArgs;
    struct Regs {};
    static constexpr int kN = N, kStages = N == 256 ? 6 : 8;
    static constexpr int kStageBytes = OPERAND + b_bytes(N);
    static constexpr int kGroup = LONG ? kMostBlocks : 0;
    static constexpr int COLS = N / 2;
    static __device__ __forceinline__ int longs(const Args &p, int unit) { return p.q + (unit < p.r ? 1 : 0); }
    static __device__ __forceinline__ int count(const Args &p, int unit, int) {
        const int v = unit - p.r;
        return longs(p, unit) + (v < 0 ? p.sa : p.sb + (v < p.se ? 1 : 0));
    }
    static __device__ __forceinline__ Tile tile(const Args &p, int unit, int units, int i) {
        const int nl = longs(p, unit);
        bool x = p.long_x;
        int g = unit + i * units;
        if (i >= nl) {
            x = !x;
            // the short tiles: first those of the units from r on, then of the others
            const int v = unit - p.r, rest = units - p.r;
            g = (v >= 0 ? v * p.sb + min(v, p.se) : rest * p.sb + p.se + unit * p.sa) + i - nl;
        }
        int m, n;
        if (x) {
            band_tile(g, p.mt, p.nd, m, n);
            return Tile{3, m * PM, n * N};
        }
        const int down = p.md * p.nh, per = p.mh * p.nd;  // tiles of dWd, of dWg and dWu each
        if (g < down) {
            band_tile(g, p.md, p.nh, m, n);
            return Tile{0, m * PM, n * N};
        }
        const int z = 1 + (g - down) / per;
        band_tile(g - down - (z - 1) * per, p.mh, p.nd, m, n);
        return Tile{z, m * PM, n * N};
    }
    static __device__ __forceinline__ int k_blocks(const Args &p, const Tile &t) { return t.z == 3 ? 2 * p.hb : p.tb; }
    static __device__ __forceinline__ void load(const Args &p, const Tile &t, int kb, uint32_t s, uint32_t bar,
                                                int rank) {
        if (t.z == 3) {
            const int up = kb >= p.hb, k = (kb - up * p.hb) * BK;
            load_k(s, &p.xa[up], bar, k, t.m + rank * BM, 0);
            load_mn<N / 2>(s + OPERAND, &p.xb[up], bar, t.n + rank * (N / 2), k, 0);
        } else {
            load_mn<BM>(s, &p.wa[t.z], bar, t.m + rank * BM, kb * BK, 0);
            load_mn<N / 2>(s + OPERAND, &p.wb[t.z ? 1 : 0], bar, t.n + rank * (N / 2), kb * BK, 0);
        }
    }
    static __device__ __forceinline__ void mma(const Args &, const Tile &t, uint32_t d, uint32_t s, bool first) {
        if (t.z == 3) mma_block<1, N, false, true>(d, s, s + OPERAND, first);
        else mma_block<1, N, true, true>(d, s, s + OPERAND, first);
    }
    static __device__ __forceinline__ void before(const Args &, const Tile &, const Epi &, int, Regs &) {}
    static __device__ __forceinline__ void epilogue(const Args &p, const Tile &t, Epi &e, int wrow, Regs &) {
        store(p, t, e, wrow, [&](int c, float (&v)[32]) { read32(e.taddr + 32 * c, v); });
    }
    static __device__ __forceinline__ void finish(const Args &p, const Tile &t, Epi &e, int wrow,
                                                  const float (&sum)[COLS]) {
        store(p, t, e, wrow, [&](int c, float (&v)[32]) { pick32(sum, c, v); });
    }
    // The tile's sums, 32 columns of a lane's row at a time from get.
    template <typename Get>
    static __device__ __forceinline__ void store(const Args &p, const Tile &t, Epi &e, int wrow, Get &&get) {
        const bool x = t.z == 3;
        const int row0 = t.m + wrow, row = row0 + e.lane;
        const int rows = x ? p.T : t.z ? p.h : p.d, cols = t.z ? p.d : p.h;
        if (row0 >= rows) return;
        const CUtensorMap *map = x ? &p.xo : &p.wo[t.z];
        const bool f32 = x ? DX32 : DW32;
        // a store of 2 KB only waits for the one before the last: a 4 KB one of another
        // tile has to have left both blocks
        if (DX32 != DW32 && e.lane == 0) bulk_wait_read<0>();
#pragma unroll 1
        for (int c = 0; c < COLS / 32; ++c) {
            const int col = t.n + e.col + 32 * c;
            if (col >= cols) break;
            float add[32];
            const bool more = x && p.dx_in;
            if (more) fetch_dx(p, row, col, add);
            float v[32];
            get(c, v);
            if (more) {
#pragma unroll
                for (int i = 0; i < 32; ++i) v[i] += add[i];
            }
            if (f32) {
                store_block32(e, v, map, col, row0);
            } else {
                uint32_t w[16];
#pragma unroll
                for (int i = 0; i < 16; ++i) w[i] = pack_bf16x2(v[2 * i], v[2 * i + 1]);
                store_block16(e, w, map, col, row0, 0);
            }
        }
    }
    // 32 columns of this lane's row of dx_in.
    static __device__ __forceinline__ void fetch_dx(const Args &p, int row, int col, float (&v)[32]) {
        const int64_t at = (int64_t)row * p.d + col;
        if (DX32) {
            const float4 *src = reinterpret_cast<const float4 *>(static_cast<const float *>(p.dx_in) + at);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float4 q = row < p.T && col + 4 * i < p.d ? __ldcs(src + i) : make_float4(0, 0, 0, 0);
                v[4 * i] = q.x;
                v[4 * i + 1] = q.y;
                v[4 * i + 2] = q.z;
                v[4 * i + 3] = q.w;
            }
        } else {
            const uint4 *src = reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(p.dx_in) + at);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint4 q = row < p.T && col + 8 * i < p.d ? __ldcs(src + i) : make_uint4(0, 0, 0, 0);
                const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    v[8 * i + 2 * k] = bf16_lo(w[k]);
                    v[8 * i + 2 * k + 1] = bf16_hi(w[k]);
                }
            }
        }
    }
    // A 32 x 32 block of fp32 through the warp's 4 KB.
    static __device__ __forceinline__ void store_block32(Epi &e, const float (&v)[32], const CUtensorMap *map, int x,
                                                         int y) {
        if (e.lane == 0) bulk_wait_read<0>();
        __syncwarp();
#pragma unroll
        for (int q = 0; q < 8; ++q)
            *reinterpret_cast<float4 *>(e.blk + e.lane * 128 + ((q ^ (e.lane & 7)) * 16)) =
                make_float4(v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]);
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncwarp();
        if (e.lane == 0) {
            tma_store_3d(map, smem_u32(e.blk), x, y, 0);
            bulk_commit();
        }
    }
};

// Shares of `units` pairs: nl long tiles of cost cl in turn, and ns short ones of cost cs
// so that the pairs' costs come out even.
inline void share(GradArgs &p, int units, int64_t nl, int64_t cl, int64_t ns, int64_t cs) {
    p.q = (int)(nl / units);
    p.r = (int)(nl % units);
    const int64_t even = (nl * cl + ns * cs) / units;
    const int64_t left = even - (p.q + 1) * cl;
    p.sa = p.r == 0 || left <= 0 ? 0 : (int)std::min<int64_t>(left / cs, ns / p.r);
    const int64_t rest = ns - (int64_t)p.r * p.sa;
    p.sb = (int)(rest / (units - p.r));
    p.se = (int)(rest % (units - p.r));
}

template <int N, bool LONG>
moe_status launch_grad(const GradArgs &g, bool dx32, bool dw32, int64_t tiles, cudaStream_t st) {
    if (dx32)
        return dw32 ? launch<Grad<true, true, N, LONG>>(g, tiles, st) : launch<Grad<true, false, N, LONG>>(g, tiles, st);
    return dw32 ? launch<Grad<false, true, N, LONG>>(g, tiles, st) : launch<Grad<false, false, N, LONG>>(g, tiles, st);
}

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

// Cluster size of SmallFactor, or 0 where the tiles are too many for it.
inline int small_split(int T, int d, int h) {
    const int ft = (h + small::kM - 1) / small::kM, n = small::tile_tokens(T);
    return small::fits(ft, T) ? small::split_for((int64_t)ft * ((T + n - 1) / n), (d + BK - 1) / BK,
                                                  small::tiles_per_sm(n)) : 0;
}

// Columns of Factor's tiles.
inline int factor_columns(int T, int h) {
    const int64_t mt = (T + PM - 1) / PM;
    return narrow(mt * ((h + 255) / 256), mt * ((h + 127) / 128)) ? 128 : 256;
}

// Parts of dtoken_scale: half tiles, or the shares of small tiles.
inline int scale_parts(int T, int d, int h) {
    const int split = small_split(T, d, h), n = factor_columns(T, h);
    return split ? (h + small::kM - 1) / small::kM * split : 2 * ((h + n - 1) / n);
}

// Workspace: status, dG, dU, Hs [T, h] bf16, the parts of dtoken_scale.
struct Layout {
    size_t dg, du, hs, part, bytes;
    Layout(int64_t T, int64_t d, int64_t h) {
        const size_t a = align256((size_t)(T * h * 2));
        dg = 256;
        du = dg + a;
        hs = du + a;
        part = hs + a;
        bytes = part + align256((size_t)(scale_parts((int)T, (int)d, (int)h) * T * 4));
    }
};

}  // namespace
}  // namespace moe

using namespace moe;

MOE_API size_t moe_gated_ffn_backward_workspace_bytes(int32_t T, int32_t d, int32_t h) {
    if (check_ffn(T, d, h) != MOE_OK) return 0;
    return Layout(T, d, h).bytes;
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
    const Layout at(T, d, h);
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
    const int fn = factor_columns(T, h);
    f.nt = (h + fn - 1) / fn;
    f.p = reinterpret_cast<const uint16_t *>(p_save);
    f.q = reinterpret_cast<const uint16_t *>(q_save);
    f.hact = reinterpret_cast<const uint16_t *>(h_act);
    f.scale = token_scale;
    f.part = dtoken_scale ? reinterpret_cast<float *>(base + at.part) : nullptr;
    f.status = status;
    GradArgs g{};
    g.T = T;
    g.d = d;
    g.h = h;
    g.mt = f.mt;
    g.md = (d + PM - 1) / PM;
    g.mh = (h + PM - 1) / PM;
    g.hb = (h + BK - 1) / BK;
    g.tb = (T + BK - 1) / BK;
    g.dx_in = dx_in;
    g.status = status;
    const bool dx32 = dx_dtype == MOE_FP32;
    if (!map_k(&f.dy, dy, d, T) || !map_mn(&f.wd, w_down, h, d) || !map_store(&f.odg, base + at.dg, h, T) ||
        !map_store(&f.odu, base + at.du, h, T) || !map_store(&f.ohs, base + at.hs, h, T) ||
        !map_k(&g.xa[0], base + at.dg, h, T) || !map_k(&g.xa[1], base + at.du, h, T) ||
        !map_mn(&g.xb[0], w_gate, d, h) || !map_mn(&g.xb[1], w_up, d, h) ||
        !(dx32 ? make_map_f32_3d(&g.xo, dx, d, T, 1) : map_store(&g.xo, dx, d, T)) || !map_mn(&g.wa[0], dy, d, T) ||
        !map_mn(&g.wa[1], base + at.dg, h, T) || !map_mn(&g.wa[2], base + at.du, h, T) ||
        !map_mn(&g.wb[0], hs, h, T) || !map_mn(&g.wb[1], x, d, T))
        return MOE_ERR_CUDA;
    void *dw[3] = {dw_down, dw_gate, dw_up};
    for (int i = 0; i < 3; ++i) {
        const uint64_t inner = i ? d : h, rows = i ? h : d;
        if (!(dw32 ? make_map_f32_3d(&g.wo[i], dw[i], inner, rows, 1) : map_store(&g.wo[i], dw[i], inner, rows)))
            return MOE_ERR_CUDA;
    }
    const int64_t ftiles = (int64_t)f.mt * f.nt;
    const int split = small_split(T, d, h);
    if (split) {
        SmallFactorArgs a{};
        const int n = small::tile_tokens(T);
        a.T = T;
        a.h = h;
        a.nk = (d + BK - 1) / BK;
        a.split = split;
        a.tt = (T + n - 1) / n;
        a.p = f.p;
        a.q = f.q;
        a.hact = f.hact;
        a.scale = token_scale;
        a.dg = reinterpret_cast<uint16_t *>(base + at.dg);
        a.du = reinterpret_cast<uint16_t *>(base + at.du);
        a.hs = reinterpret_cast<uint16_t *>(base + at.hs);
        a.part = f.part;
        a.status = status;
        a.wd = f.wd;
        if (!make_map_16(&a.dy, dy, d, T, 1, d, 64, n)) return MOE_ERR_CUDA;
        r = small::with_tokens(T, [&](auto k) {
            constexpr int N = decltype(k)::value;
            const int ft = (h + small::kM - 1) / small::kM;
            return token_scale ? small::launch<SmallFactor<true, N>>(a, ft, 1, stream)
                               : small::launch<SmallFactor<false, N>>(a, ft, 1, stream);
        });
    } else {
        r = fn == 256 ? (token_scale ? launch<Factor<true, 256>>(f, ftiles, stream)
                                     : launch<Factor<false, 256>>(f, ftiles, stream))
                      : (token_scale ? launch<Factor<true, 128>>(f, ftiles, stream)
                                     : launch<Factor<false, 128>>(f, ftiles, stream));
    }
    if (r != MOE_OK) return r;
    if (dtoken_scale) {
        launch_pdl(dw32 ? token_scale_sum<true> : token_scale_sum<false>, (unsigned)((T + 255) / 256), 256, 0, stream,
                   (int)T, scale_parts(T, d, h), f.part, dtoken_scale);
        if ((r = launch_status()) != MOE_OK) return r;
    }
    // tiles of 128 columns, which take 1.7 times as long for the same products, where a
    // pair's share of those is still less than the longest tile of 256
    const int64_t cx = 2 * g.hb, cw = g.tb;
    auto count = [&](int n, int64_t &wt, int64_t &xt) {
        g.nd = (d + n - 1) / n;
        g.nh = (h + n - 1) / n;
        wt = (int64_t)g.md * g.nh + (int64_t)2 * g.mh * g.nd;
        xt = (int64_t)g.mt * g.nd;
    };
    int64_t wt, xt;
    count(256, wt, xt);
    const bool wide = 17 * (wt * cw + xt * cx) > 10 * std::max(cx, cw) * pairs_for((int64_t)1 << 40);
    if (!wide) count(128, wt, xt);
    const int64_t tiles = wt + xt;
    const int units = pairs_for(tiles);
    g.long_x = cx > cw;
    if (g.long_x) share(g, units, xt, cx, wt, cw);
    else share(g, units, wt, cw, xt, cx);
    if (std::max(cx, cw) > kMostBlocks)
        return wide ? launch_grad<256, true>(g, dx32, dw32, tiles, stream)
                    : launch_grad<128, true>(g, dx32, dw32, tiles, stream);
    return wide ? launch_grad<256, false>(g, dx32, dw32, tiles, stream)
                : launch_grad<128, false>(g, dx32, dw32, tiles, stream);
}

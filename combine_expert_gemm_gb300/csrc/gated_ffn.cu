// The dense gated feed-forward block (include/moe_dense.h): a shared expert that
// every token passes.
//
//   G = x Wg^T, U = x Wu^T;  H = act(G) U;  y = add + s (H Wd^T)
//
// Two products.  The first computes G and U of the same 128 hidden units in one
// 256-column tile (the pair's leader holds the gate rows, its peer the up rows)
// and leaves H and, for the backward, P = act(G) and Q = U act'(G): with these
// dU = dH P and dG = dH Q, so the backward takes no exponential and does
// not depend on the activation, at the memory that G and U would take.  The second
// adds and scales in its epilogue.  Widths are multiples of 8 only: what a tile
// reaches past T, d or h is read as zeros and never stored.
#include "ffn_common.cuh"
#include "small_gemm.cuh"

namespace moe {
namespace {

using namespace pair;

struct HiddenArgs {
    CUtensorMap x, wg, wu, o, p, q;
    int T, d, h, mt, nt;
    int *status;
};

// act(g) and act'(g).  silu and gelu are both g sigmoid(z): z = g, or
// 2 sqrt(2 / pi) (g + 0.044715 g^3).
template <int ACT>
__device__ __forceinline__ void activate(float g, float &a, float &da) {
    if (ACT == MOE_ACT_RELU) {
        // not fmaxf, which would drop a NaN
        a = g < 0.0f ? 0.0f : g;
        da = g > 0.0f ? 1.0f : 0.0f;
        return;
    }
    float z = g, dz = 1.0f;
    if (ACT == MOE_ACT_GELU) {
        constexpr float k = 1.5957691216057308f;  // 2 sqrt(2 / pi)
        const float g2 = g * g;
        z = k * g * fmaf(0.044715f, g2, 1.0f);
        dz = k * fmaf(3.0f * 0.044715f, g2, 1.0f);
    }
    // 1 + e^-z past 2^126 gives 0, which is what s is then to fp32
    const float s = __fdividef(1.0f, 1.0f + __expf(-z));
    a = g * s;
    const float gz = ACT == MOE_ACT_GELU ? g * dz : g;
    // far from 0 the slope is s itself, also where g dz overflows
    da = s == 0.0f || s == 1.0f ? s : fmaf(gz * s, 1.0f - s, s);
}

template <int ACT, bool SAVE, int N>
struct Hidden {
    using Args = HiddenArgs;
    struct Regs {};
    static constexpr int kN = N, kStages = N == 256 ? 6 : 8;
    static constexpr int kStageBytes = OPERAND + b_bytes(N);
    static constexpr int kGroup = 0;
    static __device__ __forceinline__ int count(const Args &p, int unit, int units) {
        return strided_count(p.mt * p.nt, unit, units);
    }
    static __device__ __forceinline__ Tile tile(const Args &p, int unit, int units, int i) {
        int m, n;
        band_tile(unit + i * units, p.mt, p.nt, m, n);
        return Tile{0, m * PM, n * (N / 2)};
    }
    static __device__ __forceinline__ int k_blocks(const Args &p, const Tile &) { return (p.d + BK - 1) / BK; }
    static __device__ __forceinline__ void load(const Args &p, const Tile &t, int kb, uint32_t s, uint32_t bar,
                                                int rank) {
        load_k(s, &p.x, bar, kb * BK, t.m + rank * BM, 0);
        load_k(s + OPERAND, rank ? &p.wu : &p.wg, bar, kb * BK, t.n, 0);
    }
    static __device__ __forceinline__ void mma(const Args &, const Tile &, uint32_t d, uint32_t s, bool first) {
        mma_block<1, N, false, false>(d, s, s + OPERAND, first);
    }
    static __device__ __forceinline__ void before(const Args &, const Tile &, const Epi &, int, Regs &) {}
    static __device__ __forceinline__ void epilogue(const Args &p, const Tile &t, Epi &e, int wrow, Regs &) {
        const int row0 = t.m + wrow;
        if (row0 >= p.T) return;
        // G in the first half of the tile's columns, U in the second: this warp's N / 4 units
        const int unit = e.col / 2;
        const uint32_t gat = e.taddr - (uint32_t)(e.col - unit);
#pragma unroll 1
        for (int c = 0; c < N / 4; c += 32) {
            const int col = t.n + unit + c;
            if (col >= p.h) break;
            float g[32], u[32];
            read32(gat + c, g);
            read32(gat + N / 2 + c, u);
            uint32_t hw[16], pw[16], qw[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                float a0, a1, d0, d1;
                activate<ACT>(g[2 * i], a0, d0);
                activate<ACT>(g[2 * i + 1], a1, d1);
                hw[i] = pack_bf16x2(a0 * u[2 * i], a1 * u[2 * i + 1]);
                if (SAVE) {
                    pw[i] = pack_bf16x2(a0, a1);
                    qw[i] = pack_bf16x2(u[2 * i] * d0, u[2 * i + 1] * d1);
                }
            }
            store_block16(e, hw, &p.o, col, row0, 0);
            if (SAVE) {
                store_block16(e, pw, &p.p, col, row0, 0);
                store_block16(e, qw, &p.q, col, row0, 0);
            }
        }
    }
};

struct OutArgs {
    CUtensorMap hact, wd, o;
    int T, d, h, mt, nt;
    const uint16_t *add;
    const float *scale;
    int *status;
};

template <int N>
struct Out {
    using Args = OutArgs;
    struct Regs {
        uint4 add[N / 16];  // this lane's columns of add
        float s;
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
    static __device__ __forceinline__ int k_blocks(const Args &p, const Tile &) { return (p.h + BK - 1) / BK; }
    static __device__ __forceinline__ void load(const Args &p, const Tile &t, int kb, uint32_t s, uint32_t bar,
                                                int rank) {
        load_k(s, &p.hact, bar, kb * BK, t.m + rank * BM, 0);
        load_k(s + OPERAND, &p.wd, bar, kb * BK, t.n + rank * (N / 2), 0);
    }
    static __device__ __forceinline__ void mma(const Args &, const Tile &, uint32_t d, uint32_t s, bool first) {
        mma_block<1, N, false, false>(d, s, s + OPERAND, first);
    }
    static __device__ __forceinline__ void before(const Args &p, const Tile &t, Epi &e, int wrow, Regs &r) {
        const int row = t.m + wrow + e.lane;
        r.s = p.scale && row < p.T ? p.scale[row] : 1.0f;
        if (p.add) {
            const int col = t.n + e.col;
            const uint16_t *src = p.add + (int64_t)row * p.d + col;
#pragma unroll
            for (int i = 0; i < N / 16; ++i)
                r.add[i] = row < p.T && col + 8 * i < p.d ? __ldcs(reinterpret_cast<const uint4 *>(src) + i)
                                                          : make_uint4(0, 0, 0, 0);
        }
    }
    static __device__ __forceinline__ void epilogue(const Args &p, const Tile &t, Epi &e, int wrow, Regs &r) {
        const int row0 = t.m + wrow;
        if (row0 >= p.T) return;
#pragma unroll
        for (int c = 0; c < N / 2; c += 32) {
            const int col = t.n + e.col + c;
            if (col >= p.d) break;
            float v[32];
            read32(e.taddr + c, v);
            uint32_t w[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                float a = v[2 * i], b = v[2 * i + 1];
                if (p.add) {
                    const uint4 &q = r.add[c / 8 + i / 4];
                    const uint32_t z = i % 4 == 0 ? q.x : i % 4 == 1 ? q.y : i % 4 == 2 ? q.z : q.w;
                    a = fmaf(r.s, a, bf16_lo(z));
                    b = fmaf(r.s, b, bf16_hi(z));
                } else if (p.scale) {
                    a *= r.s;
                    b *= r.s;
                }
                w[i] = pack_bf16x2(a, b);
            }
            store_block16(e, w, &p.o, col, row0, 0);
        }
    }
};

// ------------------------------------------------------------- few tokens --

__device__ __forceinline__ uint2 pack4(float a, float b, float c, float d) {
    return make_uint2(pack_bf16x2(a, b), pack_bf16x2(c, d));
}

struct SmallHiddenArgs {
    CUtensorMap wg, wu, x;
    int T, h, nk, split, tt;
    uint16_t *o, *p, *q;
    int *status;
};

// The tile's rows 0-63 are gate rows, 64-127 the up rows of the same units.
template <int ACT, bool SAVE, int N>
struct SmallHidden {
    using Args = SmallHiddenArgs;
    static constexpr int kN = N;
    static constexpr bool kPairs = true, kEarly = false;
    static constexpr int kAMn = 0, kBMn = 0, kFmt = 1, kPieces = 1;
    static constexpr bool kMirror = false;
    static __device__ __forceinline__ void load_a(const Args &p, uint32_t s, uint32_t bar, int kb, int f0, int,
                                                  int) {
        small::load_box(s, &p.wg, bar, kb * BK, f0);
        small::load_box(s + small::kABytes / 2, &p.wu, bar, kb * BK, f0);
    }
    static __device__ __forceinline__ void load_b(const Args &p, uint32_t s, uint32_t bar, int kb, int t0, int,
                                                  int) {
        small::load_box(s, &p.x, bar, kb * BK, t0);
    }
    static __device__ __forceinline__ void prefetch_maps(const Args &p) {
        tma_prefetch_desc(&p.wg);
        tma_prefetch_desc(&p.wu);
        tma_prefetch_desc(&p.x);
    }
    struct In {};
    static __device__ __forceinline__ void fetch(const Args &, int, int, int, In &) {}
    static __device__ __forceinline__ void emit(const Args &p, bool ok, int t, int f, int, const float4 &g,
                                                const float4 &u, const In &) {
        if (!ok || f >= p.h) return;
        float a[4], d[4];
        activate<ACT>(g.x, a[0], d[0]);
        activate<ACT>(g.y, a[1], d[1]);
        activate<ACT>(g.z, a[2], d[2]);
        activate<ACT>(g.w, a[3], d[3]);
        const int64_t at = (int64_t)t * p.h + f;
        *reinterpret_cast<uint2 *>(p.o + at) = pack4(a[0] * u.x, a[1] * u.y, a[2] * u.z, a[3] * u.w);
        if (SAVE) {
            *reinterpret_cast<uint2 *>(p.p + at) = pack4(a[0], a[1], a[2], a[3]);
            *reinterpret_cast<uint2 *>(p.q + at) = pack4(u.x * d[0], u.y * d[1], u.z * d[2], u.w * d[3]);
        }
    }
};

struct SmallOutArgs {
    CUtensorMap wd, hact;
    int T, d, nk, split, tt;
    const uint16_t *add;
    const float *scale;
    uint16_t *y;
    int *status;
};

// Runs right behind the product that makes H, which reads no more than its grid ahead
// has left and writes no weights, so Wd is on its way before that has finished.
template <int N>
struct SmallOut {
    using Args = SmallOutArgs;
    static constexpr int kN = N;
    static constexpr bool kPairs = false, kEarly = true;
    static constexpr int kAMn = 0, kBMn = 0, kFmt = 1, kPieces = 1;
    static constexpr bool kMirror = false;
    static __device__ __forceinline__ void load_a(const Args &p, uint32_t s, uint32_t bar, int kb, int f0, int,
                                                  int) {
        small::load_box(s, &p.wd, bar, kb * BK, f0);
    }
    static __device__ __forceinline__ void load_b(const Args &p, uint32_t s, uint32_t bar, int kb, int t0, int,
                                                  int) {
        small::load_box(s, &p.hact, bar, kb * BK, t0);
    }
    static __device__ __forceinline__ void prefetch_maps(const Args &p) {
        tma_prefetch_desc(&p.wd);
        tma_prefetch_desc(&p.hact);
    }
    struct In {
        uint2 add;
        float s;
    };
    static __device__ __forceinline__ void fetch(const Args &p, int t, int f, int, In &in) {
        in.s = p.scale ? p.scale[t] : 1.0f;
        in.add = p.add && f < p.d ? *reinterpret_cast<const uint2 *>(p.add + (int64_t)t * p.d + f) : make_uint2(0, 0);
    }
    static __device__ __forceinline__ void emit(const Args &p, bool ok, int t, int f, int, const float4 &v,
                                                const float4 &, const In &in) {
        if (!ok || f >= p.d) return;
        float4 o = make_float4(in.s * v.x, in.s * v.y, in.s * v.z, in.s * v.w);
        if (p.add)
            o = make_float4(fmaf(in.s, v.x, bf16_lo(in.add.x)), fmaf(in.s, v.y, bf16_hi(in.add.x)),
                            fmaf(in.s, v.z, bf16_lo(in.add.y)), fmaf(in.s, v.w, bf16_hi(in.add.y)));
        *reinterpret_cast<uint2 *>(p.y + (int64_t)t * p.d + f) = pack4(o.x, o.y, o.z, o.w);
    }
};

template <int ACT>
moe_status launch_small_hidden(const SmallHiddenArgs &a, bool save, int ft, cudaStream_t st) {
    return small::with_tokens(a.T, [&](auto n) {
        constexpr int N = decltype(n)::value;
        return save ? small::launch<SmallHidden<ACT, true, N>>(a, ft, 1, st)
                    : small::launch<SmallHidden<ACT, false, N>>(a, ft, 1, st);
    });
}

template <int ACT>
moe_status launch_hidden(const HiddenArgs &a, bool wide, bool save, cudaStream_t st) {
    const int64_t tiles = (int64_t)a.mt * a.nt;
    if (wide)
        return save ? launch<Hidden<ACT, true, 256>>(a, tiles, st) : launch<Hidden<ACT, false, 256>>(a, tiles, st);
    return save ? launch<Hidden<ACT, true, 128>>(a, tiles, st) : launch<Hidden<ACT, false, 128>>(a, tiles, st);
}

}  // namespace
}  // namespace moe

using namespace moe;

MOE_API size_t moe_gated_ffn_workspace_bytes(int32_t T, int32_t d, int32_t h) {
    if (check_ffn(T, d, h) != MOE_OK) return 0;
    return 256;
}

MOE_API moe_status moe_gated_ffn(int32_t T, int32_t d, int32_t h, int32_t act, const moe_bf16 *x,
                                 const moe_bf16 *w_gate, const moe_bf16 *w_up,
                                 const moe_bf16 *w_down, const moe_bf16 *add,
                                 const float *token_scale, moe_bf16 *y, moe_bf16 *h_act,
                                 moe_bf16 *p_save, moe_bf16 *q_save, void *ws, size_t ws_bytes,
                                 cudaStream_t stream) {
    moe_status r = check_ffn(T, d, h);
    if (r != MOE_OK) return r;
    if (act < MOE_ACT_SILU || act > MOE_ACT_RELU) return MOE_ERR_INVALID_ARG;
    if (!p_save != !q_save) return MOE_ERR_INVALID_ARG;
    if (!ws || ws_bytes < moe_gated_ffn_workspace_bytes(T, d, h) || (reinterpret_cast<uintptr_t>(ws) & 255u))
        return MOE_ERR_WORKSPACE;
    if (T == 0) return MOE_OK;
    if (!x || !w_gate || !w_up || !w_down || !y || !h_act || x == y) return MOE_ERR_INVALID_ARG;
    const void *ptrs[] = {x, w_gate, w_up, w_down, add, token_scale, y, h_act, p_save, q_save};
    for (const void *q : ptrs)
        if (!aligned16(q)) return MOE_ERR_ALIGNMENT;

    const bool save = p_save != nullptr;
    int *const status = static_cast<int *>(ws);
    // each product in the form that its tiles are made for
    const int n = small::tile_tokens(T), tt = (T + n - 1) / n;
    const int ft1 = (h + small::kM / 2 - 1) / (small::kM / 2), ft2 = (d + small::kM - 1) / small::kM;
    const bool few1 = small::fits(ft1, T), few2 = small::fits(ft2, T);
    if (few1) {
        SmallHiddenArgs a{};
        a.T = T;
        a.h = h;
        a.nk = (d + BK - 1) / BK;
        a.tt = tt;
        a.split = small::split_for((int64_t)ft1 * tt, a.nk, small::tiles_per_sm(n));
        a.o = reinterpret_cast<uint16_t *>(h_act);
        a.p = reinterpret_cast<uint16_t *>(p_save);
        a.q = reinterpret_cast<uint16_t *>(q_save);
        a.status = status;
        if (!make_map_16(&a.wg, w_gate, d, h, 1, d, 64, small::kM / 2) ||
            !make_map_16(&a.wu, w_up, d, h, 1, d, 64, small::kM / 2) || !make_map_16(&a.x, x, d, T, 1, d, 64, n))
            return MOE_ERR_CUDA;
        r = act == MOE_ACT_SILU   ? launch_small_hidden<MOE_ACT_SILU>(a, save, ft1, stream)
            : act == MOE_ACT_GELU ? launch_small_hidden<MOE_ACT_GELU>(a, save, ft1, stream)
                                  : launch_small_hidden<MOE_ACT_RELU>(a, save, ft1, stream);
    } else {
        HiddenArgs a{};
        a.T = T;
        a.d = d;
        a.h = h;
        a.mt = (T + PM - 1) / PM;
        const bool wide = !narrow((int64_t)a.mt * ((h + 127) / 128), (int64_t)a.mt * ((h + 63) / 64));
        const int units = wide ? 128 : 64;  // hidden units of a tile
        a.nt = (h + units - 1) / units;
        a.status = status;
        if (!map_k(&a.x, x, d, T) || !map_k(&a.wg, w_gate, d, h, 1, 0, units) ||
            !map_k(&a.wu, w_up, d, h, 1, 0, units) ||
            !map_store(&a.o, h_act, h, T) || (save && (!map_store(&a.p, p_save, h, T) || !map_store(&a.q, q_save, h, T))))
            return MOE_ERR_CUDA;
        r = act == MOE_ACT_SILU   ? launch_hidden<MOE_ACT_SILU>(a, wide, save, stream)
            : act == MOE_ACT_GELU ? launch_hidden<MOE_ACT_GELU>(a, wide, save, stream)
                                  : launch_hidden<MOE_ACT_RELU>(a, wide, save, stream);
    }
    if (r != MOE_OK) return r;
    if (few2) {
        SmallOutArgs o{};
        o.T = T;
        o.d = d;
        o.nk = (h + BK - 1) / BK;
        o.tt = tt;
        o.split = small::split_for((int64_t)ft2 * tt, o.nk, small::tiles_per_sm(n));
        o.add = reinterpret_cast<const uint16_t *>(add);
        o.scale = token_scale;
        o.y = reinterpret_cast<uint16_t *>(y);
        o.status = status;
        if (!make_map_16(&o.wd, w_down, h, d, 1, h, 64, small::kM) || !make_map_16(&o.hact, h_act, h, T, 1, h, 64, n))
            return MOE_ERR_CUDA;
        return small::with_tokens(T, [&](auto k) {
            return small::launch<SmallOut<decltype(k)::value>>(o, ft2, 1, stream);
        });
    }
    OutArgs o{};
    o.T = T;
    o.d = d;
    o.h = h;
    o.mt = (T + PM - 1) / PM;
    const bool wide = !narrow((int64_t)o.mt * ((d + 255) / 256), (int64_t)o.mt * ((d + 127) / 128));
    o.nt = wide ? (d + 255) / 256 : (d + 127) / 128;
    o.add = reinterpret_cast<const uint16_t *>(add);
    o.scale = token_scale;
    o.status = status;
    if (!map_k(&o.hact, h_act, h, T) || !map_k(&o.wd, w_down, h, d, 1, 0, wide ? 128 : 64) ||
        !map_store(&o.o, y, d, T))
        return MOE_ERR_CUDA;
    return wide ? launch<Out<256>>(o, (int64_t)o.mt * o.nt, stream) : launch<Out<128>>(o, (int64_t)o.mt * o.nt, stream);
}

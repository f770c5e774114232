// The matrix product of few tiles (gated_ffn.cu, gated_ffn_bwd.cu, newton_schulz.cu).
// The result's contiguous dimension (features: the weights' rows or columns) is the
// 128 rows of a tile, its rows (tokens) are the up to 128 columns, so few tokens are
// multiplied as few and not as 256 padded rows; and the reduction is split
// over the S CTAs of a cluster where there are fewer tiles than SMs.
//
// What bounds it is the operands' way from memory and the latency of each step, so a
// CTA keeps its loads in flight ahead of the MMAs; the partial accumulators
// are added through distributed shared memory, each CTA a share of the features,
// in rank order; and the epilogue runs over (token, 4 features) items with
// neighbouring threads on neighbouring features, so loads and stores are whole
// rows.  An epilogue thread has several of them on their way at once, the first before
// the product is done (one at a time, a tile of 128 tokens took 15 us).  The sums
// wait where the stages were.
//
// A problem P says what is loaded and what happens to a sum:
//   kN       tokens of a tile (16, 32, 64 or 128);
//   kPairs   the features are 64 pairs (rows 0-63 and 64-127 belong together);
//   kFmt     1 for bf16 operands, 0 for fp16;
//   kPieces  1, or 2: each operand is a high and a low piece, a product the three
//            of them that count (newton_schulz.cu), and an accumulator holds one
//            k-block, which are added in fp32 registers (pair_gemm.cuh says why);
//   kAMn / kBMn  the operand's rows are its inner dimension (MN-major);
//   kMirror  the result is symmetric and the operands one: only tiles on and above the
//            diagonal are computed (kN is 128), and each is stored twice, once from
//            a transposed copy of the sums; one on the diagonal loads A alone;
//   kEarly   A may be loaded before the wait for the grid ahead: that grid is one of ours
//            that waited for all before it and does not write A;
//   load_a / load_b (of piece q), prefetch_maps; In and fetch, what an item needs from memory; emit.
#pragma once

#include "pair_gemm.cuh"

namespace moe {
namespace small {

constexpr int kM = 128;                       // features of a tile
constexpr int kBK = 64;
constexpr int kABytes = kM * kBK * 2;         // 16 KB
constexpr int kThreads = 256;                  // of the epilogue; a producer and an MMA warp follow
constexpr int kMaxSplit = 8;

template <class P>
__host__ __device__ constexpr int a_bytes() { return P::kPieces * kABytes; }
template <class P>
__host__ __device__ constexpr int stage_bytes() { return a_bytes<P>() + P::kPieces * P::kN * kBK * 2; }
// Up to 64 tokens without pieces: about 96 KB, so that two CTAs share an SM and the
// grid behind starts beside this one.  More: as many as an SM holds.
template <class P>
__host__ __device__ constexpr int stages() {
    return P::kPieces == 2 ? (P::kN >= 128 ? 3 : P::kN == 64 ? 4 : 5) : P::kN >= 128 ? 6 : P::kN == 64 ? 4 : 5;
}
// Items of an epilogue thread in flight: as many as the larger tiles have work for (with
// four for 16 tokens, the longer code came in 2 us later for one token).
template <class P>
__host__ __device__ constexpr int items_ahead() { return P::kN >= 128 ? 4 : P::kN == 64 ? 2 : 1; }
// Accumulators, used in turn, and the TMEM columns of all of them.
template <class P>
__host__ __device__ constexpr int accs() { return P::kPieces == 2 ? 4 : 1; }
constexpr int kGroup = 1;  // k-blocks of an accumulator with pieces (with two: 8e-6 for 128 x 4096)
template <class P>
__host__ __device__ constexpr int columns() { return accs<P>() * P::kN < 32 ? 32 : accs<P>() * P::kN; }

struct alignas(8) Bars {
    uint64_t full[6], empty[6], tfull[4], tempty[4], done;
    uint32_t tmem_base;
    int abort;
};

// Floats of a row of the transposed sums: 16-byte stores of 8 lanes hit 32 banks.
constexpr int kPitchT = kM + 4;

template <class P>
constexpr size_t smem_bytes() {
    static_assert(!P::kMirror || (P::kN == kM && (size_t)stages<P>() * stage_bytes<P>() >=
                                                     (size_t)kM * (kM + kPitchT) * 4), "both copies fit");
    static_assert((size_t)stages<P>() * stage_bytes<P>() >= (size_t)P::kN * kM * 4, "the sums fit the stages");
    return 1024 + (size_t)stages<P>() * stage_bytes<P>() + sizeof(Bars) + 16;
}

__device__ __forceinline__ void load_box(uint32_t dst, const CUtensorMap *map, uint32_t bar, int x, int y,
                                         int z = 0) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(bar)
        : "memory");
}

__device__ __forceinline__ float4 ld_cluster(uint32_t addr) {
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "r"(addr)
                 : "memory");
    return v;
}

template <class P>
__global__ void __launch_bounds__(kThreads + 64) small_gemm(const __grid_constant__ typename P::Args p) {
    constexpr int STAGES = stages<P>(), SB = stage_bytes<P>(), AB = a_bytes<P>(), N = P::kN;
    constexpr int kBBytes = N * kBK * 2, kItems = items_ahead<P>();
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem =
        reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
    float *part = reinterpret_cast<float *>(smem);  // [N tokens][128 features], once the stages are done
    Bars *bars = reinterpret_cast<Bars *>(smem + STAGES * SB);
    volatile int *abort = &bars->abort;
    int *status = p.status;
    const int split = p.split, rank = split > 1 ? (int)cluster_rank() : 0;
    const int z = (int)blockIdx.z / p.tt;
    int f0 = (int)blockIdx.y * (P::kPairs ? kM / 2 : kM), t0 = ((int)blockIdx.z - z * p.tt) * N;
    if (P::kMirror) {  // blockIdx.y runs over the tiles of the upper triangle, row by row
        const int mt = (p.T + kM - 1) / kM;
        int r = (int)blockIdx.y, m = 0;
        while (r >= mt - m) r -= mt - m++;
        t0 = m * kM;
        f0 = (m + r) * kM;
    }
    const bool diagonal = P::kMirror && t0 == f0;  // B is A
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int kb0 = p.nk * rank / split, kb1 = p.nk * (rank + 1) / split, nk = kb1 - kb0;
    constexpr int ACCS = accs<P>();
    const int group = P::kPieces == 2 ? kGroup : nk;  // k-blocks of an accumulator

    if (threadIdx.x == 0) {
        for (int s = 0; s < STAGES; ++s) {
            mbar_init(smem_u32(&bars->full[s]), 1);
            mbar_init(smem_u32(&bars->empty[s]), 1);
        }
        mbar_init(smem_u32(&bars->done), 1);
        for (int a = 0; a < ACCS; ++a) {
            mbar_init(smem_u32(&bars->tfull[a]), 1);
            mbar_init(smem_u32(&bars->tempty[a]), kThreads / 32);
        }
        bars->abort = 0;
        fence_mbar_init();
    }
    if (threadIdx.x == 32) P::prefetch_maps(p);
    __syncthreads();

    const int first = min(nk, STAGES);
    auto stage_at = [&](int s) { return smem_u32(smem + s * SB); };
    auto issue_a = [&](int i) {
        const uint32_t bar = smem_u32(&bars->full[i % STAGES]);
        mbar_arrive_expect_tx(bar, diagonal ? AB : SB);
#pragma unroll
        for (int q = 0; q < P::kPieces; ++q)
            P::load_a(p, stage_at(i % STAGES) + q * kABytes, bar, kb0 + i, f0, z, q);
    };
    if (P::kEarly && threadIdx.x == kThreads)
        for (int i = 0; i < first; ++i) issue_a(i);
    pdl_enter();
    // tensor memory behind the wait, as in pair_gemm.cuh: nothing that holds it waits for
    // another grid
    if (warp == kThreads / 32 + 1) tmem_alloc(smem_u32(&bars->tmem_base), columns<P>());
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = bars->tmem_base;

    // this CTA's share of the features (pairs): items of 4 features a token
    constexpr int kF = P::kPairs ? kM / 2 : kM;
    const int share = kF / split, per = share / 4, shift = 31 - __clz(per);  // a power of two
    auto item_f = [&](int i) { return rank * share + (i & (per - 1)) * 4; };
    typename P::In in[kItems];
    auto fetch = [&](int i0, int items, int row0, int col0) {
#pragma unroll
        for (int u = 0; u < kItems; ++u) {
            const int i = i0 + u * kThreads + (int)threadIdx.x;
            if (i < items) P::fetch(p, row0 + (i >> shift), col0 + item_f(i), z, in[u]);
        }
    };

    if (threadIdx.x == kThreads) {
        bool ok = true;
        int issued = 0;
        for (int i = 0; i < nk; ++i, ++issued) {
            const int s = i % STAGES;
            if (i >= STAGES &&
                !mbar_wait(smem_u32(&bars->empty[s]), (uint32_t)((i / STAGES - 1) & 1), status, abort)) {
                ok = false;
                break;
            }
            if (!P::kEarly || i >= first) issue_a(i);
            if (diagonal) continue;
#pragma unroll
            for (int q = 0; q < P::kPieces; ++q)
                P::load_b(p, stage_at(s) + AB + q * kBBytes, smem_u32(&bars->full[s]), kb0 + i, t0, z, q);
        }
        if (!ok) {  // copies in flight land before the CTA leaves
            for (int i = max(0, issued - STAGES); i < issued; ++i) {
                volatile int no_abort = 0;
                mbar_wait(smem_u32(&bars->full[i % STAGES]), (uint32_t)((i / STAGES) & 1), status, &no_abort);
            }
        }
    } else if (threadIdx.x == kThreads + 32) {
        constexpr uint32_t idesc = (1u << 4) | ((uint32_t)P::kFmt << 7) | ((uint32_t)P::kFmt << 10) |
                                   ((uint32_t)P::kAMn << 15) | ((uint32_t)P::kBMn << 16) | ((uint32_t)(N >> 3) << 17) |
                                   ((uint32_t)(kM >> 4) << 24);
        auto mma = [&](uint32_t d, uint32_t sa, uint32_t sb, bool fresh) {
#pragma unroll
            for (int kk = 0; kk < kBK / 16; ++kk)
                tc_mma_bf16(d, P::kAMn ? pair::mn_desc(sa + kk * 2048) : sw128_kmajor_desc(sa + kk * 32),
                            P::kBMn ? pair::mn_desc(sb + kk * 2048) : sw128_kmajor_desc(sb + kk * 32), idesc,
                            fresh && kk == 0 ? 0u : 1u);
        };
        int in_group = 0, g = 0, i = 0;
        for (; i < nk; ++i) {
            const int s = i % STAGES, acc = g % ACCS;
            const bool fresh = in_group == 0;
            if (fresh && g >= ACCS &&
                !mbar_wait(smem_u32(&bars->tempty[acc]), (uint32_t)((g / ACCS - 1) & 1), status, abort))
                break;
            if (!mbar_wait(smem_u32(&bars->full[s]), (uint32_t)((i / STAGES) & 1), status, abort)) break;
            tc_fence_after();
            const uint32_t sa = stage_at(s), sb = diagonal ? sa : sa + AB, d = tmem + acc * N;
            if (P::kPieces == 2) {  // the small products first
                mma(d, sa + kABytes, sb, fresh);
                mma(d, sa, sb + kBBytes, false);
                mma(d, sa, sb, false);
            } else {
                mma(d, sa, sb, fresh);
            }
            tc_commit(smem_u32(&bars->empty[s]));
            if (++in_group == group || i + 1 == nk) {
                tc_commit(smem_u32(&bars->tfull[acc]));
                in_group = 0;
                ++g;
            }
        }
        if (i < nk) {  // a wait gave up: what was issued completes before the CTA leaves
            tc_commit(smem_u32(&bars->done));
            volatile int no_abort = 0;
            mbar_wait(smem_u32(&bars->done), 0, status, &no_abort);
        }
    } else if (warp < kThreads / 32) {
        fetch(0, min(N, p.T - t0) * per, t0, f0);
        // two warps a lane quadrant, each with half of the tokens
        constexpr int kCols = N == 16 ? 16 : N / 2;
        const int quad = warp & 3, c0 = (warp >> 2) * kCols;
        const bool mine = c0 < N;  // 16 tokens: the first four warps
        const uint32_t at = tmem + ((uint32_t)(quad * 32) << 16) + (uint32_t)c0;
        float *dst = part + quad * 32 + lane;
        if constexpr (P::kPieces == 1) {
            // one accumulator, which goes straight to the place of the stages, all of them
            // read by then
            mbar_wait(smem_u32(&bars->tfull[0]), 0, status, abort);
            tc_fence_after();
#pragma unroll 1
            for (int c = 0; c < kCols && mine; c += 16) {
                uint32_t v[16];
                tmem_ld16(at + c, v);
                tmem_ld_wait();
                reg_fence(v);
#pragma unroll
                for (int i = 0; i < 16; ++i) dst[(c0 + c + i) * kM] = __uint_as_float(v[i]);
            }
            tc_fence_before();
        } else {
            // the groups' sums in registers, and then in the place of the stages
            const int groups = (nk + group - 1) / group;
            float sum[kCols];
#pragma unroll 1
            for (int g = 0; g < groups; ++g) {
                const int acc = g % ACCS;
                if (!mbar_wait(smem_u32(&bars->tfull[acc]), (uint32_t)((g / ACCS) & 1), status, abort)) break;
                tc_fence_after();
#pragma unroll
                for (int c = 0; c < kCols; c += 16) {
                    uint32_t v[16];
                    tmem_ld16(at + acc * N + c, v);
                    tmem_ld_wait();
                    reg_fence(v);
#pragma unroll
                    for (int i = 0; i < 16; ++i)
                        sum[c + i] = g == 0 ? __uint_as_float(v[i]) : sum[c + i] + __uint_as_float(v[i]);
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(&bars->tempty[acc]));
            }
#pragma unroll
            for (int i = 0; i < kCols; ++i) dst[(c0 + i) * kM] = sum[i];
            if (P::kMirror) {  // row feature, columns tokens
                float4 *dt = reinterpret_cast<float4 *>(part + kM * kM + (quad * 32 + lane) * kPitchT + c0);
#pragma unroll
                for (int i = 0; i < kCols / 4; ++i)
                    dt[i] = make_float4(sum[4 * i], sum[4 * i + 1], sum[4 * i + 2], sum[4 * i + 3]);
            }
        }
    }
    __syncwarp();
    if (split > 1) cluster_sync_all();
    else __syncthreads();

    // the sums over the cluster, in rank order; the mirrored tile in a second pass
    const int passes = warp >= kThreads / 32 ? 0 : P::kMirror && !diagonal ? 2 : 1;
#pragma unroll 1
    for (int pass = 0; pass < passes; ++pass) {
        const int row0 = pass ? f0 : t0, col0 = pass ? t0 : f0;
        const float *const own = pass ? part + kM * kM : part;
        const uint32_t base = smem_u32(own);
        const int pitch = pass ? kPitchT : kM;
        const int items = min(pass ? kM : N, p.T - row0) * per;
#pragma unroll 1
        for (int i0 = 0; i0 < items; i0 += kItems * kThreads) {
            if (i0 || pass) fetch(i0, items, row0, col0);
            float4 a[kItems], b[kItems];
            const float4 zero = make_float4(0, 0, 0, 0);
#pragma unroll
            for (int u = 0; u < kItems; ++u) a[u] = b[u] = zero;
            if (split == 1) {
#pragma unroll
                for (int u = 0; u < kItems; ++u) {
                    const int i = i0 + u * kThreads + (int)threadIdx.x;
                    if (i >= items) continue;
                    const float4 *at = reinterpret_cast<const float4 *>(own + (i >> shift) * pitch + item_f(i));
                    a[u] = at[0];
                    if (P::kPairs) b[u] = at[kM / 2 / 4];
                }
            }
#pragma unroll 4
            for (int r = 0; r < split && split > 1; ++r) {
                // all items' loads of up to four ranks at once: one by one they take the
                // distributed memory's latency each
                const uint32_t from = cluster_map(base, r);
                float4 q[kItems], w[kItems];
#pragma unroll
                for (int u = 0; u < kItems; ++u) {
                    const int i = i0 + u * kThreads + (int)threadIdx.x;
                    if (i >= items) continue;
                    const uint32_t at = from + (uint32_t)((i >> shift) * pitch + item_f(i)) * 4;
                    q[u] = ld_cluster(at);
                    if (P::kPairs) w[u] = ld_cluster(at + kM / 2 * 4);
                }
#pragma unroll
                for (int u = 0; u < kItems; ++u) {
                    a[u] = make_float4(a[u].x + q[u].x, a[u].y + q[u].y, a[u].z + q[u].z, a[u].w + q[u].w);
                    if (P::kPairs)
                        b[u] = make_float4(b[u].x + w[u].x, b[u].y + w[u].y, b[u].z + w[u].z, b[u].w + w[u].w);
                }
            }
#pragma unroll
            for (int u = 0; u < kItems; ++u) {
                const int i = i0 + u * kThreads + (int)threadIdx.x;
                if (i - lane >= items) break;  // the whole warp
                P::emit(p, i < items, row0 + (i >> shift), col0 + item_f(i), z, a[u], b[u], in[u]);
            }
        }
    }
    if (split > 1) cluster_sync_all();  // no CTA leaves while its sums are read
    else __syncthreads();
    if (warp == kThreads / 32 + 1) {
        tc_fence_after();
        tmem_dealloc(tmem, columns<P>());
    }
}

// CTAs of a cluster: as many as the SMs hold beside the other tiles, `slots` CTAs in
// all, with two k-blocks each at least.  Clusters of eight leave SMs of a GPC unused: 16
// of them fit at once with an SM a CTA.
inline int split_for(int64_t tiles, int nk, int per_sm) {
    const int slots = per_sm * (num_sms() - num_sms() % 8);
    int s = 1;
    while (s < kMaxSplit && tiles * (2 * s) <= (s == 4 ? per_sm * 128 : slots) && nk >= 4 * s) s *= 2;
    return s;
}

template <class P>
moe_status launch(const typename P::Args &args, int ftiles, int64_t planes, cudaStream_t st) {
    static PerDeviceOnce smem_attr;
    if (!device_once(smem_attr, [] { return set_smem_limit(small_gemm<P>, smem_bytes<P>()); }))
        return MOE_ERR_CUDA;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)args.split, (unsigned)ftiles, (unsigned)(args.tt * planes));
    cfg.blockDim = dim3(kThreads + 64);
    cfg.dynamicSmemBytes = smem_bytes<P>();
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    set_pdl_attr(attr[0]);
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)args.split;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    if (cudaLaunchKernelEx(&cfg, small_gemm<P>, args) != cudaSuccess) return MOE_ERR_CUDA;
    return launch_status();
}

// Tokens of a tile: the smallest that holds them all, or 128 with several tiles (a
// weight row is then read by fewer tiles: 96 tokens in tiles of 64 took 1 us more than in
// one of 128, 1537 in 300 tiles of 64 half as long again as the pairs' 42).
inline int tile_tokens(int T) { return T <= 16 ? 16 : T <= 32 ? 32 : T <= 64 ? 64 : 128; }
inline int tiles_per_sm(int n) { return n == 128 ? 1 : 2; }

// Calls f with std::integral_constant-like N of tile_tokens(T).
template <int N>
struct Tokens {
    static constexpr int value = N;
};
template <typename F>
inline moe_status with_tokens(int T, F &&f) {
    switch (tile_tokens(T)) {
        case 16: return f(Tokens<16>{});
        case 32: return f(Tokens<32>{});
        case 64: return f(Tokens<64>{});
        default: return f(Tokens<128>{});
    }
}

// Whether so many feature tiles of T tokens fit the SMs in one round.
inline bool fits(int64_t ftiles, int T) {
    const int n = tile_tokens(T);
    return ftiles * ((T + n - 1) / n) <= tiles_per_sm(n) * num_sms();
}

}  // namespace small
}  // namespace moe

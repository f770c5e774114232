// The matrix product of few tokens (gated_ffn.cu, gated_ffn_bwd.cu): the weights'
// rows or columns are the 128 rows of a tile (features), up to 128 tokens its
// columns, so a tile multiplies what there is and not 256 padded rows; and the
// reduction is split over the S CTAs of a cluster when there are fewer tiles than SMs.
//
// What bounds it is the weights' way from memory and the latency of each step, so a
// CTA keeps as many loads in flight as it has k-blocks, up to kStages; the partial
// accumulators are added through distributed shared memory, each CTA a share of
// the features, in rank order; and the epilogue runs over (token, 4 features) items
// with neighbouring threads on neighbouring features, so loads and stores are
// whole rows.
//
// A problem P says what is loaded and what happens to a sum:
//   kN       tokens of a tile (16, 32, 64 or 128), kPairs: the features are 64 pairs
//            (rows 0-63 and 64-127 of the tile belong together);
//   kAMn     the features are the inner dimension of the weight (MN-major);
//   kEarly   the weights may be loaded before the wait for the grid ahead: that grid
//            is one of ours that waited for all before it and writes no weights;
//   load_a / load_b, emit.
#pragma once

#include "pair_gemm.cuh"

namespace moe {
namespace small {

constexpr int kM = 128;                       // features of a tile
constexpr int kBK = 64;
constexpr int kABytes = kM * kBK * 2;         // 16 KB
constexpr int kThreads = 256;
constexpr int kMaxSplit = 8;

template <class P>
__host__ __device__ constexpr int stage_bytes() { return kABytes + P::kN * kBK * 2; }
template <class P>
__host__ __device__ constexpr int stages() { return P::kN >= 128 ? 4 : 5; }

struct alignas(8) Bars {
    uint64_t full[5], empty[5], done;
    uint32_t tmem_base;
    int abort;
};

template <class P>
constexpr size_t smem_bytes() {
    return 1024 + (size_t)stages<P>() * stage_bytes<P>() + (size_t)P::kN * kM * 4 + sizeof(Bars) + 16;
}

__device__ __forceinline__ void load_box(uint32_t dst, const CUtensorMap *map, uint32_t bar, int x, int y) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(0), "r"(bar)
        : "memory");
}

__device__ __forceinline__ float4 ld_cluster(uint32_t addr) {
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "r"(addr));
    return v;
}

template <class P>
__global__ void __launch_bounds__(kThreads) small_gemm(const __grid_constant__ typename P::Args p) {
    constexpr int STAGES = stages<P>(), SB = stage_bytes<P>(), N = P::kN;
    constexpr int kCols = N < 32 ? 32 : N;  // TMEM columns
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem =
        reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
    float *part = reinterpret_cast<float *>(smem + STAGES * SB);  // [N tokens][128 features]
    Bars *bars = reinterpret_cast<Bars *>(part + N * kM);
    volatile int *abort = &bars->abort;
    int *status = p.status;
    const int split = p.split, rank = split > 1 ? (int)cluster_rank() : 0;
    const int f0 = (int)blockIdx.y * (P::kPairs ? kM / 2 : kM), t0 = (int)blockIdx.z * N;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int kb0 = p.nk * rank / split, kb1 = p.nk * (rank + 1) / split, nk = kb1 - kb0;

    if (threadIdx.x == 0) {
        for (int s = 0; s < STAGES; ++s) {
            mbar_init(smem_u32(&bars->full[s]), 1);
            mbar_init(smem_u32(&bars->empty[s]), 1);
        }
        mbar_init(smem_u32(&bars->done), 1);
        bars->abort = 0;
        fence_mbar_init();
    }
    if (warp == 1) tmem_alloc(smem_u32(&bars->tmem_base), kCols);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = bars->tmem_base;

    const int first = min(nk, STAGES);
    auto stage_at = [&](int s) { return smem_u32(smem + s * SB); };
    if (P::kEarly && threadIdx.x == 0) {
        for (int i = 0; i < first; ++i) {
            const uint32_t bar = smem_u32(&bars->full[i]);
            mbar_arrive_expect_tx(bar, SB);
            P::load_a(p, stage_at(i), bar, kb0 + i, f0);
        }
    }
    pdl_enter();
    if (threadIdx.x == 0) {
        bool ok = true;
        int issued = 0;
        for (int i = 0; i < nk; ++i, ++issued) {
            const int s = i % STAGES;
            const uint32_t bar = smem_u32(&bars->full[s]);
            if (i >= STAGES &&
                !mbar_wait(smem_u32(&bars->empty[s]), (uint32_t)((i / STAGES - 1) & 1), status, abort)) {
                ok = false;
                break;
            }
            if (!P::kEarly || i >= first) {
                mbar_arrive_expect_tx(bar, SB);
                P::load_a(p, stage_at(s), bar, kb0 + i, f0);
            }
            P::load_b(p, stage_at(s) + kABytes, bar, kb0 + i, t0);
        }
        if (!ok) {  // copies in flight land before the CTA leaves
            for (int i = max(0, issued - STAGES); i < issued; ++i) {
                volatile int no_abort = 0;
                mbar_wait(smem_u32(&bars->full[i % STAGES]), (uint32_t)((i / STAGES) & 1), status, &no_abort);
            }
        }
    } else if (threadIdx.x == 32) {
        constexpr uint32_t idesc = (1u << 4) | (1u << 7) | (1u << 10) | ((uint32_t)P::kAMn << 15) |
                                   ((uint32_t)(N >> 3) << 17) | ((uint32_t)(kM >> 4) << 24);
        for (int i = 0; i < nk; ++i) {
            const int s = i % STAGES;
            if (!mbar_wait(smem_u32(&bars->full[s]), (uint32_t)((i / STAGES) & 1), status, abort)) break;
            tc_fence_after();
            const uint32_t sa = stage_at(s), sb = sa + kABytes;
#pragma unroll
            for (int kk = 0; kk < kBK / 16; ++kk)
                tc_mma_bf16(tmem, P::kAMn ? pair::mn_desc(sa + kk * 2048) : sw128_kmajor_desc(sa + kk * 32),
                            sw128_kmajor_desc(sb + kk * 32), idesc, (i | kk) != 0 ? 1u : 0u);
            tc_commit(smem_u32(&bars->empty[s]));
        }
        // also after a wait that gave up: what was issued completes here
        tc_commit(smem_u32(&bars->done));
    }
    __syncwarp();
    // the accumulator to shared memory, token by token: two warps a lane quadrant
    mbar_wait(smem_u32(&bars->done), 0, status, abort);
    tc_fence_after();
    {
        const int quad = warp & 3;
        constexpr int kHalf = N / 2;  // columns of a warp, at least 8
        const int c0 = (warp >> 2) * kHalf;
        const uint32_t at = tmem + ((uint32_t)(quad * 32) << 16);
        float *dst = part + quad * 32 + lane;
        if (N == 16) {
            if (warp < 4) {
                uint32_t v[16];
                tmem_ld16(at, v);
                tmem_ld_wait();
                reg_fence(v);
#pragma unroll
                for (int i = 0; i < 16; ++i) dst[i * kM] = __uint_as_float(v[i]);
            }
        } else {
#pragma unroll 1
            for (int c = c0; c < c0 + kHalf; c += 16) {
                uint32_t v[16];
                tmem_ld16(at + c, v);
                tmem_ld_wait();
                reg_fence(v);
#pragma unroll
                for (int i = 0; i < 16; ++i) dst[(c + i) * kM] = __uint_as_float(v[i]);
            }
        }
        tc_fence_before();
    }
    if (split > 1) cluster_sync_all();
    else __syncthreads();

    // this CTA's share of the features (pairs), summed over the cluster in rank order
    constexpr int kF = P::kPairs ? kM / 2 : kM;
    const int share = kF / split, per = share / 4;  // float4 items a token; a power of two
    const int tokens = min(N, p.T - t0);
    const uint32_t base = smem_u32(part);
    const int items = tokens * per;
#pragma unroll 1
    for (int i0 = warp * 32; i0 < items; i0 += kThreads) {
        const int i = i0 + lane;
        const bool ok = i < items;
        const int t = ok ? i / per : 0, f = rank * share + (i % per) * 4;
        float4 a = make_float4(0, 0, 0, 0), b = a;
        const uint32_t at = base + (uint32_t)(t * kM + f) * 4;
        for (int r = 0; r < split; ++r) {
            const uint32_t src = split > 1 ? cluster_map(at, r) : at;
            const float4 q = ld_cluster(src);
            a = make_float4(a.x + q.x, a.y + q.y, a.z + q.z, a.w + q.w);
            if (P::kPairs) {
                const float4 w = ld_cluster(src + kM / 2 * 4);
                b = make_float4(b.x + w.x, b.y + w.y, b.z + w.z, b.w + w.w);
            }
        }
        P::emit(p, ok, t0 + t, f0 + f, a, b, per);
    }
    if (split > 1) cluster_sync_all();  // no CTA leaves while its sums are read
    else __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, kCols);
    }
}

// CTAs of a cluster: as many as the SMs hold beside the other tiles (clusters of
// eight need eight SMs of one GPC: 16 of them fit at once), with two k-blocks each at
// least.
inline int split_for(int64_t tiles, int nk) {
    int s = 1;
    while (s < kMaxSplit && tiles * (2 * s) <= (s == 4 ? 128 : num_sms() - num_sms() % 8) && nk >= 4 * s) s *= 2;
    return s;
}

template <class P>
moe_status launch(const typename P::Args &args, int ftiles, int ttiles, cudaStream_t st) {
    static PerDeviceOnce smem_attr;
    if (!device_once(smem_attr, [] { return set_smem_limit(small_gemm<P>, smem_bytes<P>()); }))
        return MOE_ERR_CUDA;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)args.split, (unsigned)ftiles, (unsigned)ttiles);
    cfg.blockDim = dim3(kThreads);
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

// Tokens of a tile: the smallest that holds them all, or 128 with several tiles.
inline int tile_tokens(int T) { return T <= 16 ? 16 : T <= 32 ? 32 : T <= 64 ? 64 : 128; }

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

// Whether `features` of a tile each and T tokens fit the SMs in one round.
inline bool fits(int64_t ftiles, int T) {
    const int n = tile_tokens(T);
    return ftiles * ((T + n - 1) / n) <= num_sms();
}

}  // namespace small
}  // namespace moe

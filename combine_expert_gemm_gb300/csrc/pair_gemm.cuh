// The CTA-pair matrix product that the dense operators share (gated_ffn.cu,
// gated_ffn_bwd.cu, newton_schulz.cu): one persistent kernel, parametrised by a
// problem P that says which tiles there are, what a k-block loads, which MMAs
// it takes and what happens to a finished tile.
//
// Clusters of two CTAs, one CTA per SM:
//   warp 0     TMA producer (both CTAs) into a ring of P::kStages stages;
//   warp 1     in the leader one thread issues tcgen05.mma.cta_group::2 (M = 256
//              across the pair, N = P::kN, K = 16) into two fp32 accumulators of
//              kN TMEM columns, used in turn;
//   8 more     epilogue, two warps per TMEM lane quadrant, each with half of the
//              kN columns of its 32 rows.
// kN is 256, or 128 where tiles of 256 columns leave too many pairs without one.
// Both CTAs' loads complete on the leader's full barrier; the leader's commits
// release stages and announce accumulators in both CTAs; both CTAs' epilogue
// warps release an accumulator on the leader's barrier.
//
// P::kGroup = 0: an accumulator holds a whole tile, and P::epilogue reads it;
// what it needs from memory P::before fetches while the tile is multiplied.
// P::kGroup > 0: an accumulator holds kGroup k-blocks.  The tensor core cuts
// where an fp32 addition rounds, always towards zero, so a long sum in one
// accumulator drifts by up to 2^-23 of its size per MMA; the epilogue warps
// add the groups in fp32 registers instead, and P::finish gets the sums.
//
// Every store of the epilogues goes through maps or guards that end at the
// matrix's extent, every load of a tile past it reads zeros.
#pragma once

#include <algorithm>

#include "moe_common.cuh"

namespace moe {
namespace pair {

constexpr int BM = 128;              // rows of A a CTA
constexpr int PM = 2 * BM;           // rows of A a pair
constexpr int BK = 64;               // k of a k-block
constexpr int OPERAND = BM * BK * 2; // one CTA's 128 x 64 16-bit operand: 16 KB
// One CTA's half of the N columns of B in a k-block.
__host__ __device__ constexpr int b_bytes(int n) { return n / 2 * BK * 2; }
constexpr int BLK = 64 * BK * 2;     // a 64 x 64 MN-major block: 8 KB
constexpr int kTmemCols = 512;
constexpr int kEpiWarps = 8;
constexpr int kEpiBlock = 4096;      // shared memory of an epilogue warp

// With kGroup > 0 an epilogue thread keeps up to 128 sums, more than 168 registers hold
// beside what it works with (2-3 KB of spills): two idle warps fill the
// first warpgroup, which gives up its registers: 128 x 40 + 256 x 232 = 384 x 168.
template <class P>
__host__ __device__ constexpr int epi_warp0() { return P::kGroup ? 4 : 2; }
template <class P>
__host__ __device__ constexpr int threads() { return 32 * (epi_warp0<P>() + kEpiWarps); }

struct Tile {
    int z, m, n;  // matrix of the batch, first row, first column
};

template <int STAGES>
struct alignas(8) Bars {
    uint64_t full[STAGES];
    uint64_t empty[STAGES];
    uint64_t tfull[2];
    uint64_t tempty[2];
    uint32_t tmem_base;
    int abort;
};

template <class P>
constexpr size_t smem_bytes() {
    return 1024 + (size_t)P::kStages * P::kStageBytes + kEpiWarps * kEpiBlock + sizeof(Bars<P::kStages>) + 16;
}

// ------------------------------------------------------------- host: maps --

// 3-D map over [planes, rows, inner] of 16-bit elements, rows `ld` elements
// apart: loads of box_inner x box_rows with the swizzle of a box's width (64
// elements: 128 bytes; 32: 64 bytes), stores of 32 x 32 blocks.  What lies past
// `inner` or `rows` reads as zeros and is not written, whatever ld is.
inline bool make_map_16(CUtensorMap *m, const void *base, uint64_t inner, uint64_t rows, uint64_t planes,
                        uint64_t ld, uint32_t box_inner, uint32_t box_rows) {
    EncodeTiledFn fn = encode_fn();
    if (!fn) return false;
    const cuuint64_t dims[3] = {inner, rows, planes};
    const cuuint64_t strides[2] = {ld * 2, ld * 2 * rows};
    const cuuint32_t box[3] = {box_inner, box_rows, 1};
    const cuuint32_t estr[3] = {1, 1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(base), dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE,
              box_inner == 64 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// K-major operand (128 or `box` rows of 64 k), MN-major operand (64 k of 64 columns a
// box) and 32 x 32 store blocks of one [planes, rows, inner] matrix.
inline bool map_k(CUtensorMap *m, const void *p, uint64_t inner, uint64_t rows, uint64_t planes = 1,
                  uint64_t ld = 0, int box = BM) {
    return make_map_16(m, p, inner, rows, planes, ld ? ld : inner, 64, (uint32_t)box);
}
inline bool map_mn(CUtensorMap *m, const void *p, uint64_t inner, uint64_t rows, uint64_t planes = 1,
                   uint64_t ld = 0) {
    return make_map_16(m, p, inner, rows, planes, ld ? ld : inner, 64, BK);
}
inline bool map_store(CUtensorMap *m, const void *p, uint64_t inner, uint64_t rows, uint64_t planes = 1,
                      uint64_t ld = 0) {
    return make_map_16(m, p, inner, rows, planes, ld ? ld : inner, 32, 32);
}

// --------------------------------------------------------------- device --

__device__ __forceinline__ void load_box(uint32_t dst, const CUtensorMap *map, uint32_t bar, int x, int y,
                                         int z) {
    asm volatile(
        "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(bar)
        : "memory");
}

// This CTA's operand: K-major rows row.. of k.., or MN-major columns col.. of k-rows
// k.. in blocks of 64 columns.
__device__ __forceinline__ void load_k(uint32_t dst, const CUtensorMap *map, uint32_t bar, int k, int row,
                                       int z) {
    load_box(dst, map, bar, k, row, z);
}
template <int COLS>
__device__ __forceinline__ void load_mn(uint32_t dst, const CUtensorMap *map, uint32_t bar, int col, int k,
                                        int z) {
#pragma unroll
    for (int c = 0; c < COLS; c += 64) load_box(dst + c / 64 * BLK, map, bar, col + c, k, z);
}

// Descriptor of an MN-major operand: 128-byte rows of 64 elements of one k, 8-row
// groups 1 KB apart, 64-element blocks 8 KB apart.
__device__ __forceinline__ uint64_t mn_desc(uint32_t smem_addr) {
    uint64_t d = 0;
    d |= (uint64_t)((smem_addr >> 4) & 0x3FFFu);
    d |= (uint64_t)(BLK >> 4) << 16;
    d |= (uint64_t)(1024u >> 4) << 32;
    d |= (uint64_t)1u << 46;
    d |= (uint64_t)2u << 61;
    return d;
}

// Instruction descriptor: fp32 accumulator, A and B both bf16 (fmt 1) or both
// fp16 (fmt 0), each K-major (0) or MN-major (1).
__host__ __device__ constexpr uint32_t idesc16(int fmt, int n, int a_mn, int b_mn) {
    return (1u << 4) | ((uint32_t)fmt << 7) | ((uint32_t)fmt << 10) | ((uint32_t)a_mn << 15) |
           ((uint32_t)b_mn << 16) | ((uint32_t)(n >> 3) << 17) | ((uint32_t)(PM >> 4) << 24);
}

// The four K = 16 steps of one k-block.
template <int FMT, int N, bool A_MN, bool B_MN>
__device__ __forceinline__ void mma_block(uint32_t d_tmem, uint32_t sa, uint32_t sb, bool first) {
    constexpr uint32_t idesc = idesc16(FMT, N, A_MN, B_MN);
#pragma unroll
    for (int kk = 0; kk < BK / 16; ++kk)
        tc_mma_bf16_pair(d_tmem, A_MN ? mn_desc(sa + kk * 2048) : sw128_kmajor_desc(sa + kk * 32),
                         B_MN ? mn_desc(sb + kk * 2048) : sw128_kmajor_desc(sb + kk * 32), idesc,
                         first && kk == 0 ? 0u : 1u);
}

// Tile order: bands of kBand row tiles, columns slowest inside a band, so that
// the tiles in flight share few panels of A and of B.
constexpr int kBand = 8;
__device__ __forceinline__ void band_tile(int g, int mt, int nt, int &m, int &n) {
    const int band = g / (kBand * nt);
    const int r = g - band * kBand * nt;
    const int rows = min(kBand, mt - band * kBand);
    m = band * kBand + r % rows;
    n = r / rows;
}

// Tiles g = unit, unit + units, ... of `total`.
__device__ __forceinline__ int strided_count(int total, int unit, int units) {
    return unit < total ? (total - unit - 1) / units + 1 : 0;
}

// 32 columns of the accumulator at taddr.
__device__ __forceinline__ void read32(uint32_t taddr, float (&v)[32]) {
    uint32_t a[16], b[16];
    tmem_ld16(taddr, a);
    tmem_ld16(taddr + 16, b);
    tmem_ld_wait();
    reg_fence(a);
    reg_fence(b);
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        v[i] = __uint_as_float(a[i]);
        v[16 + i] = __uint_as_float(b[i]);
    }
}

// Columns 32 c .. 32 c + 31 of a row's 64 or 128 sums, by selections: registers have no
// index, and a loop over c is short where its unrolled code is not.
template <int COLS>
__device__ __forceinline__ void pick32(const float (&sum)[COLS], int c, float (&v)[32]) {
#pragma unroll
    for (int i = 0; i < 32; ++i) {
        v[i] = c & 1 ? sum[32 + i] : sum[i];
        if constexpr (COLS > 64) {
            const float b = c & 1 ? sum[96 + i] : sum[64 + i];
            v[i] = c & 2 ? b : v[i];
        }
    }
}

// What an epilogue warp knows: the accumulator at its 32 lanes (rows) and its
// first column, that column within the tile, and its shared memory (1 KB aligned),
// two 2 KB blocks used in turn.
struct Epi {
    uint32_t taddr;
    int col, lane, turn;
    uint8_t *blk;
};

// A warp's 32 x 32 block of 16-bit pairs to (x, y, z) of a map_store map.  The block
// of shared memory is the one that the store before the last one left from:
// waiting for that one alone keeps the next in flight (with one block a warp the
// update's products waited 0.6 us a store, 10 us a tile).
__device__ __forceinline__ void store_block16(Epi &e, const uint32_t (&w)[16], const CUtensorMap *map, int x,
                                              int y, int z) {
    uint8_t *blk = e.blk + (e.turn ^= 2048);
    if (e.lane == 0) bulk_wait_read<1>();
    __syncwarp();
#pragma unroll
    for (int q = 0; q < 4; ++q)
        *reinterpret_cast<uint4 *>(blk + e.lane * 64 + ((q ^ ((e.lane >> 1) & 3)) * 16)) =
            make_uint4(w[4 * q], w[4 * q + 1], w[4 * q + 2], w[4 * q + 3]);
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    __syncwarp();
    if (e.lane == 0) {
        tma_store_3d(map, smem_u32(blk), x, y, z);
        bulk_commit();
    }
}

template <class P>
__global__ void __launch_bounds__(threads<P>(), 1) pair_gemm(const __grid_constant__ typename P::Args p) {
    constexpr int STAGES = P::kStages;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem =
        reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
    uint8_t *epi_smem = smem + (size_t)STAGES * P::kStageBytes;
    Bars<STAGES> *bars = reinterpret_cast<Bars<STAGES> *>(epi_smem + kEpiWarps * kEpiBlock);
    volatile int *abort = &bars->abort;
    int *status = p.status;
    const uint32_t rank = cluster_rank();
    const bool leader = rank == 0;
    const int unit = (int)blockIdx.x / 2, units = (int)gridDim.x / 2;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        for (int s = 0; s < STAGES; ++s) {
            mbar_init(smem_u32(&bars->full[s]), 1);
            mbar_init(smem_u32(&bars->empty[s]), 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(smem_u32(&bars->tfull[b]), 1);
            mbar_init(smem_u32(&bars->tempty[b]), 2 * kEpiWarps);
        }
        bars->abort = 0;
        fence_mbar_init();
    }
    // What came so far touches only this pair's own shared memory and may run beside the
    // grid before this one.  Tensor memory is taken behind the wait: a grid
    // ahead that takes its own after letting this one start would wait for ours.
    pdl_enter();
    if (warp == 1) tmem_alloc_pair(smem_u32(&bars->tmem_base), kTmemCols);
    tc_fence_before();
    __syncthreads();
    cluster_sync_all();  // barriers of both CTAs exist before any remote arrival
    tc_fence_after();
    const uint32_t tmem_base = bars->tmem_base;
    const int count = P::count(p, unit, units);  // tiles of this pair

    if (warp < epi_warp0<P>()) {
        // with kGroup > 0 the whole first warpgroup, at this one instruction
        if constexpr (P::kGroup > 0) asm volatile("setmaxnreg.dec.sync.aligned.u32 40;");
        if (warp == 0 && lane == 0) {
            int stage = 0;
            uint32_t phase = 0;
            int issued = 0;
            bool ok = true;
            for (int i = 0; i < count && ok; ++i) {
                const Tile t = P::tile(p, unit, units, i);
                const int nk = P::k_blocks(p, t);
                for (int kb = 0; kb < nk; ++kb) {
                    if (!mbar_wait(smem_u32(&bars->empty[stage]), phase ^ 1, status, abort)) {
                        ok = false;
                        break;
                    }
                    const uint32_t own_full = smem_u32(&bars->full[stage]);
                    if (leader) mbar_arrive_expect_tx(own_full, 2 * P::kStageBytes);
                    P::load(p, t, kb, smem_u32(smem + (size_t)stage * P::kStageBytes), cluster_map(own_full, 0),
                            (int)rank);
                    ++issued;
                    if (++stage == STAGES) {
                        stage = 0;
                        phase ^= 1;
                    }
                }
            }
            if (!ok && leader) {
                // the leader's full barriers count both CTAs' copies: let the
                // ones already issued land before the pair leaves
                for (int s = 0; s < STAGES; ++s) {
                    volatile int no_abort = 0;
                    mbar_wait(smem_u32(&bars->full[s]), phase ^ (s >= stage ? 1 : 0), status, &no_abort);
                }
            }
            // the leader's MMAs read this CTA's stages: every use is released
            for (int s = 0; s < STAGES; ++s) {
                const int uses = issued / STAGES + (s < issued % STAGES ? 1 : 0);
                if (uses > 0) mbar_wait(smem_u32(&bars->empty[s]), (uint32_t)((uses - 1) & 1), status, abort);
            }
        }
        if (warp == 1 && lane == 0 && leader) {
            int stage = 0;
            uint32_t phase = 0;
            int acc = 0;
            uint32_t acc_phase = 0;
            bool ok = true;
            for (int i = 0; i < count && ok; ++i) {
                const Tile t = P::tile(p, unit, units, i);
                const int nk = P::k_blocks(p, t);
                for (int k0 = 0; k0 < nk && ok; k0 += P::kGroup ? P::kGroup : nk) {
                    const int k1 = P::kGroup ? min(nk, k0 + P::kGroup) : nk;
                    if (!mbar_wait(smem_u32(&bars->tempty[acc]), acc_phase ^ 1, status, abort)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint32_t d_tmem = tmem_base + (uint32_t)(acc * P::kN);
                    for (int kb = k0; kb < k1; ++kb) {
                        if (!mbar_wait(smem_u32(&bars->full[stage]), phase, status, abort)) {
                            ok = false;
                            break;
                        }
                        tc_fence_after();
                        P::mma(p, t, d_tmem, smem_u32(smem + (size_t)stage * P::kStageBytes), kb == k0);
                        tc_commit_pair(smem_u32(&bars->empty[stage]));
                        if (++stage == STAGES) {
                            stage = 0;
                            phase ^= 1;
                        }
                    }
                    if (!ok) break;
                    tc_commit_pair(smem_u32(&bars->tfull[acc]));
                    if (++acc == 2) {
                        acc = 0;
                        acc_phase ^= 1;
                    }
                }
            }
        }
    } else {
        if constexpr (P::kGroup > 0) asm volatile("setmaxnreg.inc.sync.aligned.u32 232;");
        const int quad = warp & 3, ew = warp - epi_warp0<P>();
        constexpr int COLS = P::kN / 2;
        Epi e;
        e.col = (ew >> 2) * COLS;
        e.lane = lane;
        e.turn = 0;
        e.blk = epi_smem + ew * kEpiBlock;
        const int wrow = (int)rank * BM + quad * 32;
        const uint32_t tlane = tmem_base + ((uint32_t)(quad * 32) << 16) + (uint32_t)e.col;
        int acc = 0;
        uint32_t acc_phase = 0;
        bool ok = true;
        auto release = [&] {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_cluster_relaxed(cluster_map(smem_u32(&bars->tempty[acc]), 0));
            if (++acc == 2) {
                acc = 0;
                acc_phase ^= 1;
            }
        };
        for (int i = 0; i < count && ok; ++i) {
            const Tile t = P::tile(p, unit, units, i);
            if constexpr (P::kGroup == 0) {
                typename P::Regs regs;
                P::before(p, t, e, wrow, regs);
                if (!mbar_wait(smem_u32(&bars->tfull[acc]), acc_phase, status, abort)) break;
                tc_fence_after();
                e.taddr = tlane + (uint32_t)(acc * P::kN);
                P::epilogue(p, t, e, wrow, regs);
                release();
            } else {
                float sum[COLS];
                const int nk = P::k_blocks(p, t);
                for (int k0 = 0; k0 < nk; k0 += P::kGroup) {
                    if (!mbar_wait(smem_u32(&bars->tfull[acc]), acc_phase, status, abort)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint32_t at = tlane + (uint32_t)(acc * P::kN);
#pragma unroll
                    for (int c = 0; c < COLS; c += 16) {
                        uint32_t v[16];
                        tmem_ld16(at + c, v);
                        tmem_ld_wait();
                        reg_fence(v);
#pragma unroll
                        for (int i = 0; i < 16; ++i)
                            sum[c + i] = k0 == 0 ? __uint_as_float(v[i]) : sum[c + i] + __uint_as_float(v[i]);
                    }
                    release();
                }
                if (ok) P::finish(p, t, e, wrow, sum);
            }
        }
        if (lane == 0) bulk_wait<0>();  // stores complete before the CTA ends
    }

    tc_fence_before();
    __syncthreads();
    cluster_sync_all();  // both CTAs are done with every barrier and every MMA
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc_pair(tmem_base, kTmemCols);
    }
}

// CTA pairs of a launch over so many tiles.
inline int pairs_for(int64_t tiles) {
    return (int)std::min<int64_t>(std::max(num_sms() / 2, 1), std::max<int64_t>(tiles, 1));
}

// Whether tiles of 128 columns serve better than half as many of 256.  They read as much
// of A for half the products and take 0.6 to 0.86 of a wide tile's time (the Gram
// product of one 2048 x 4096 matrix, 72 narrow tiles or 36 wide ones on 76 pairs: 50
// against 63 us; the hidden units of 8192 tokens, 512 or 256 tiles: 72 against 48), so only
// where they need no more rounds.
inline bool narrow(int64_t wide_tiles, int64_t narrow_tiles) {
    const int64_t pairs = std::max(num_sms() / 2, 1);
    return (narrow_tiles + pairs - 1) / pairs <= (wide_tiles + pairs - 1) / pairs;
}

template <class P>
moe_status launch(const typename P::Args &args, int64_t tiles, cudaStream_t st) {
    static PerDeviceOnce smem_attr;
    if (!device_once(smem_attr, [] {
            if (P::kGroup > 0) {
                // the epilogue's share has to fit what the block is launched with: a
                // setmaxnreg past it would wait for ever
                cudaFuncAttributes at;
                if (cudaFuncGetAttributes(&at, pair_gemm<P>) != cudaSuccess ||
                    at.numRegs * threads<P>() < 128 * 40 + 256 * 232)
                    return false;
            }
            return set_smem_limit(pair_gemm<P>, smem_bytes<P>());
        }))
        return MOE_ERR_CUDA;
    const int pairs = pairs_for(tiles);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(2 * pairs));
    cfg.blockDim = dim3(threads<P>());
    cfg.dynamicSmemBytes = smem_bytes<P>();
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    set_pdl_attr(attr[1]);
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    if (cudaLaunchKernelEx(&cfg, pair_gemm<P>, args) != cudaSuccess) return MOE_ERR_CUDA;
    return launch_status();
}

}  // namespace pair
}  // namespace moe

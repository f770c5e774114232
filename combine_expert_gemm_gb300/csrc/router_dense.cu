// The router's products for a gradient of every logit (include/moe_block.h):
//   dx = dx_in + dl W;  dW = dl^T x;  dbias = column sums of dl
// with dl [T, N] fp32, W [N, d] fp32, x [T, d] bf16.
//
// Both products are skinny (N experts deep or wide against d columns), so what
// they cannot do without is the traffic of dx_in, dx and x: 10 bytes per token
// and column against 4 N fp32 operations.  On the fp32 pipes the operations
// would take longer than the bytes (the simple kernel of 32 fused multiply-adds
// per load took 1747 us where the bytes take 199: T = 32768, d = 4096, N = 32),
// so the products run on the tensor cores, with fp32 accuracy from bf16 pieces:
//   v = v0 + v1 + v2,  v0 = bf16(v), v1 = bf16(v - v0), v2 = bf16(v - v0 - v1)
// holds all 24 bits of an fp32 value, the residuals are exact, and a product
// of two bf16 values is exact in the fp32 accumulator.  dl W sums the six piece
// products whose size is at least 2^-16 of the leading one (what is left out is
// below 2^-24 of it); dl^T x needs three, x being bf16 already.
//
// Launches: router_dense_prep writes the pieces (dl's transposed, so that both
// products read them in a layout of the tensor cores) and partial sums of
// dbias; router_dense_dw and router_dense_dx are the products.  The partial sums
// of dw and dbias are added, in a fixed order, by router_dense_dx's epilogue
// warps while its first tile is loaded and multiplied (a launch of its own took
// 5 us), or by router_dense_sum when dx is not wanted.
#include <algorithm>

#include "../../include/moe_block.h"
#include "moe_common.cuh"

namespace moe {
namespace {

constexpr int kSms = 152;  // the machine the work is split for (results do not depend on it)

// ------------------------------------------------------------------ pieces --

struct Pieces {
    uint16_t p[3];
};

// The three bf16 pieces of v.  Past the largest bf16 the first piece is cut
// instead of rounded, so that it stays finite; a non-finite v is its own first
// piece and the others are 0.
__device__ __forceinline__ Pieces split3(float v) {
    Pieces r;
    if ((__float_as_uint(v) & 0x7F800000u) == 0x7F800000u) {
        const __nv_bfloat16 b = __float2bfloat16_rn(v);
        r.p[0] = *reinterpret_cast<const uint16_t *>(&b);
        r.p[1] = r.p[2] = 0;
        return r;
    }
#pragma unroll
    for (int i = 0; i < 3; ++i) {
        const __nv_bfloat16 b = __float2bfloat16_rn(v);
        uint32_t w = *reinterpret_cast<const uint16_t *>(&b);
        if ((w & 0x7F80u) == 0x7F80u) w = __float_as_uint(v) >> 16;
        r.p[i] = (uint16_t)w;
        v -= __uint_as_float(w << 16);
    }
    return r;
}

// The pieces of a (low half) and b.  Up to the largest bf16 both are split at
// once and nothing can overflow: one by one, with the checks, router_dense_prep
// took 2 us longer at 31595 x 272 x 73 (40 us for the whole call) and 0.5 at
// 8192 x 2048 x 64.
__device__ __forceinline__ void split3x2(float a, float b, uint32_t (&o)[3]) {
    if (fabsf(a) <= 0x1.fep127f && fabsf(b) <= 0x1.fep127f) {
#pragma unroll
        for (int i = 0; i < 3; ++i) {
            o[i] = pack_bf16x2(a, b);
            a -= __uint_as_float(o[i] << 16);
            b -= __uint_as_float(o[i] & 0xFFFF0000u);
        }
        return;
    }
    const Pieces pa = split3(a), pb = split3(b);
#pragma unroll
    for (int i = 0; i < 3; ++i) o[i] = (uint32_t)pa.p[i] | ((uint32_t)pb.p[i] << 16);
}

constexpr int kPrepThreads = 256;
constexpr int kPrepTok = 64;  // tokens of a transposed block
constexpr int kPrepExp = 32;  // experts of a transposed block

// blockIdx.y < chunks: dl's pieces dlp[3][N][Tp] of 32 experts, the token
// blocks of 64 strided over blockIdx.x, and those tokens' sums in
// db_part[blockIdx.x][N].  The CTAs from there on: W's pieces wp[3][N][dp].
// Columns from T to Tp and from d to dp are zeros.
__global__ void __launch_bounds__(kPrepThreads)
router_dense_prep(int T, int64_t Tp, int N, int d, int dp, int chunks,
                  const float *__restrict__ dl, const float *__restrict__ w, uint16_t *__restrict__ dlp,
                  uint16_t *__restrict__ wp, float *__restrict__ db_part) {
    pdl_enter();
    __shared__ float tile[kPrepTok][kPrepExp + 1];
    if ((int)blockIdx.y >= chunks) {
        const int64_t cta = (int64_t)(blockIdx.y - chunks) * gridDim.x + blockIdx.x;
        const int64_t ctas = (int64_t)(gridDim.y - chunks) * gridDim.x;
        const int per = dp / 8;
        const int64_t n = (int64_t)N * per, plane = (int64_t)N * dp;
        for (int64_t i = cta * kPrepThreads + threadIdx.x; i < n; i += ctas * kPrepThreads) {
            const int64_t e = i / per;
            const int c = (int)(i % per) * 8;
            float f[8] = {0, 0, 0, 0, 0, 0, 0, 0};
            if (c < d) {
                const float4 *src = reinterpret_cast<const float4 *>(w + e * d + c);
                const float4 a = src[0], b = src[1];
                f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
                f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
            }
            uint32_t o[3][4];
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                uint32_t w3[3];
                split3x2(f[2 * q], f[2 * q + 1], w3);
#pragma unroll
                for (int p = 0; p < 3; ++p) o[p][q] = w3[p];
            }
#pragma unroll
            for (int p = 0; p < 3; ++p)
                *reinterpret_cast<uint4 *>(wp + p * plane + e * dp + c) =
                    make_uint4(o[p][0], o[p][1], o[p][2], o[p][3]);
        }
        return;
    }
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int e0 = blockIdx.y * kPrepExp;
    const int64_t plane = (int64_t)N * Tp;
    float sum[4] = {0.f, 0.f, 0.f, 0.f};
    for (int64_t t0 = (int64_t)blockIdx.x * kPrepTok; t0 < Tp; t0 += (int64_t)gridDim.x * kPrepTok) {
        // warp w loads tokens w, w + 8, ..., a lane per expert
#pragma unroll
        for (int i = 0; i < kPrepTok / 8; ++i) {
            const int64_t t = t0 + warp + 8 * i;
            tile[warp + 8 * i][lane] = t < T && e0 + lane < N ? dl[t * N + e0 + lane] : 0.f;
        }
        __syncthreads();
        // warp w writes experts 4 w .. 4 w + 3, a lane per pair of tokens
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int e = e0 + 4 * warp + i;
            const float a = tile[2 * lane][4 * warp + i], b = tile[2 * lane + 1][4 * warp + i];
            sum[i] += a + b;
            if (e >= N) continue;
            uint32_t w3[3];
            split3x2(a, b, w3);
#pragma unroll
            for (int p = 0; p < 3; ++p)
                *reinterpret_cast<uint32_t *>(dlp + p * plane + (int64_t)e * Tp + t0 + 2 * lane) = w3[p];
        }
        __syncthreads();
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float v = sum[i];
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, off);
        const int e = e0 + 4 * warp + i;
        if (lane == 0 && e < N) db_part[(int64_t)blockIdx.x * N + e] = v;
    }
}

// ------------------------------------------------------------ TMA and MMA --

__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap *map, uint32_t bar,
                                            int32_t x, int32_t y, int32_t z) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(bar)
        : "memory");
}

__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap *map, uint32_t bar,
                                            int32_t x, int32_t y, int32_t z, int32_t w) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(w), "r"(bar)
        : "memory");
}

// MN-major operand, 128-byte swizzle: K rows of 128 bytes (64 M/N elements),
// 8-row groups 1 KB apart, 64-element M/N blocks `block` bytes apart.
__device__ __forceinline__ uint64_t mnmajor_desc(uint32_t smem_addr, uint32_t block) {
    uint64_t d = 0;
    d |= (uint64_t)((smem_addr >> 4) & 0x3FFFu);
    d |= (uint64_t)(block >> 4) << 16;
    d |= (uint64_t)(1024u >> 4) << 32;
    d |= (uint64_t)1u << 46;
    d |= (uint64_t)2u << 61;
    return d;
}

// As idesc_bf16_f32, with each operand K-major (0) or MN-major (1).
__host__ __device__ constexpr uint32_t idesc_major(int M, int N, int a_mn, int b_mn) {
    return idesc_bf16_f32(M, N) | ((uint32_t)a_mn << 15) | ((uint32_t)b_mn << 16);
}

// Pieces [3][rows][inner] (inner a multiple of 64) as [3][inner / 64][rows][64]:
// one box of 64 x box_rows x 2 blocks x 3 pieces lands piece by piece, block by
// block, each block box_rows swizzled 128-byte rows.  Rows past the last read
// as zeros.
inline bool make_map_pieces_mn(CUtensorMap *m, const void *base, uint64_t inner, uint64_t rows,
                               uint32_t box_rows) {
    EncodeTiledFn fn = encode_fn();
    if (!fn) return false;
    const cuuint64_t dims[4] = {64, rows, inner / 64, 3};
    const cuuint64_t strides[3] = {inner * 2, 128, inner * rows * 2};
    const cuuint32_t box[4] = {64, box_rows, 2, 3};
    const cuuint32_t estr[4] = {1, 1, 1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void *>(base), dims, strides, box,
              estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
              CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Pieces [3][rows][inner] read along inner: box 64 x box_rows x 3 pieces.
inline bool make_map_pieces_k(CUtensorMap *m, const void *base, uint64_t inner, uint64_t rows,
                              uint32_t box_rows) {
    EncodeTiledFn fn = encode_fn();
    if (!fn) return false;
    const cuuint64_t dims[3] = {inner, rows, 3};
    const cuuint64_t strides[2] = {inner * 2, inner * rows * 2};
    const cuuint32_t box[3] = {64, box_rows, 3};
    const cuuint32_t estr[3] = {1, 1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(base), dims, strides, box,
              estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
              CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Row-major [rows, inner] fp32 in boxes of 32 x 32, 128-byte swizzle.
inline bool make_map_f32(CUtensorMap *m, const void *base, uint64_t inner, uint64_t rows) {
    EncodeTiledFn fn = encode_fn();
    if (!fn) return false;
    const cuuint64_t dims[2] = {inner, rows};
    const cuuint64_t strides[1] = {inner * 4};
    const cuuint32_t box[2] = {32, 32};
    const cuuint32_t estr[2] = {1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 2, const_cast<void *>(base), dims, strides, box,
              estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
              CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

constexpr int kGemmThreads = 64 + 256;  // producer warp, MMA warp, 8 epilogue warps
constexpr int kEpiWarps = 8;

// -------------------------------------------------------------- last sums --

struct Sums {
    int64_t n4;       // N * d / 4; 0: dw is not wanted
    int splits, lanes, N, groups;
    const float4 *part;
    const float *db_part;
    float4 *dw;
    float *dbias;     // NULL: not wanted
};

// The share of `unit` (of `units`, each of 256 threads) in dw = the sum of the
// splits, four columns a thread, and dbias = the sum of the prep CTAs, a warp
// per expert.  q.lanes (1, 2, 4 or 8) threads of a warp share a sum where there
// are fewer sums than threads: one thread for the 152 splits of 24 x 128 took
// 9 us longer than eight.
__device__ __forceinline__ void add_partials(const Sums &q, int unit, int units, int thread) {
    const int per = 32 / q.lanes, lane = thread & 31;
    const int64_t step = (int64_t)units * 8 * per;
    // all lanes of a warp take the same rounds
    for (int64_t w = ((int64_t)unit * 8 + (thread >> 5)) * per; w < q.n4; w += step) {
        const int64_t i = w + lane % per;
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
        if (i < q.n4) {
#pragma unroll 4
            for (int s = lane / per; s < q.splits; s += q.lanes) {
                const float4 p = q.part[s * q.n4 + i];
                v.x += p.x;
                v.y += p.y;
                v.z += p.z;
                v.w += p.w;
            }
        }
        for (int off = per; off < 32; off <<= 1) {
            v.x += __shfl_xor_sync(0xFFFFFFFFu, v.x, off);
            v.y += __shfl_xor_sync(0xFFFFFFFFu, v.y, off);
            v.z += __shfl_xor_sync(0xFFFFFFFFu, v.z, off);
            v.w += __shfl_xor_sync(0xFFFFFFFFu, v.w, off);
        }
        if (lane < per && i < q.n4) q.dw[i] = v;
    }
    if (!q.dbias) return;
    for (int e = unit * 8 + (thread >> 5); e < q.N; e += units * 8) {
        float v = 0.f;
#pragma unroll 4
        for (int g = thread & 31; g < q.groups; g += 32) v += q.db_part[(int64_t)g * q.N + e];
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, off);
        if ((thread & 31) == 0) q.dbias[e] = v;
    }
}

__global__ void __launch_bounds__(256) router_dense_sum(const Sums q) {
    pdl_enter();
    add_partials(q, blockIdx.x, gridDim.x, threadIdx.x);
}

// ---------------------------------------------------------------------- dx --
//
// Persistent CTAs, tiles of 128 tokens x 128 columns, columns fastest.  A
// k-block is 32 experts: the three pieces of dl (24 KB) and of W (24 KB), both
// MN-major, by one TMA request each.  An accumulator takes 128 of the 512
// tensor-memory columns, so four are in flight between the MMA thread and the
// epilogue.
//
// The tensor core cuts where an fp32 addition rounds, always towards zero, and
// each of the twelve MMAs of a k-block does: one accumulator for a whole tile
// was 5, 27 and 115 u (u = 2^-24) off in the 2-norm at 64, 256 and 1024
// experts, where an fp32 sum of the same length is 2.4, 4.8 and 9.6 u off.  A
// cut costs an ulp of the sum it is added to.  So
//   up to four k-blocks, each k-block has an accumulator of its own, the
//   smallest piece products first, and the epilogue adds the k-blocks in fp32
//   registers: 1.1 u at 64 experts, 1.2 at 128;
//   beyond them, all of a tile's small piece products (2^-8 of the sum and less)
//   go to one accumulator and the leading ones of every four k-blocks to
//   another, which leaves eight k-blocks in flight instead of four and a third
//   of the reads: 2 to 3 u from 256 to 1024.
// The whole call, us, with one accumulator a tile, with one a k-block and with
// the small products apart:
//   T =  8192, d = 2048, N = 64          40.8     41.5     41.9
//   T = 16384, d = 2048, N = 128         95       96       96.5
//   T =  9998, d = 2768, N = 152         96      103       95.5
//   T =  4096, d = 4096, N = 256         75       86       78
//   T =  4096, d = 2048, N = 512         78.5     87       81
//
// The epilogue's work is the traffic: each warp owns 32 tokens x 64 columns of
// a tile and SLOTS blocks of 4 KB in shared memory, through which it streams
// 32 x 32 blocks of dx_in (TMA load, SLOTS - 1 ahead), adds the accumulator in
// place and stores the block to dx (TMA store).  No warp waits for another's
// block, and 24 or 32 blocks of 4 KB cover the latency of the loads and stores.
//
// One k-block a tile (N <= 32) needs one operand stage and leaves room for four
// slots.  Up to four k-blocks the epilogue's traffic weighs more and takes three
// slots, beyond them the operands' latency does and takes three stages.  The
// whole call, us, with STAGES, SLOTS, while a tile had one accumulator:
//                                     <1, 4>   <2, 3>   <3, 2>   <2, 4>
//   T = 32768, d = 4096, N = 32         213      221      266      232
//   T =  8192, d = 2048, N = 64          45       41       49       41
//   T = 16384, d = 2048, N = 128        130       96       99       97
//   T =  4096, d = 4096, N = 256        115       82       76       82
constexpr int kDxPiece = 2 * 32 * 128;              // 128 columns or tokens x 32 experts: 8 KB
constexpr int kDxStageBytes = 2 * 3 * kDxPiece;     // 48 KB
constexpr int kDxBlk = 32 * 32 * 4;
constexpr int kDxAcc = 4;
// Declared for more threads than it has, which holds it to 128 registers: with
// the 166 that it would take, no CTA of the stream's next kernel finds registers
// beside one of these before it ends.  Calls in a row, us: T = 82, d = 624, N =
// 269 15.6 (16.9 with 166), 25 x 1064 x 418 18.3 (19.4), 64 x 4096 x 256 16.2
// (17.1), 31595 x 272 x 73 38.1 (38.6), larger ones within 1% either way.
constexpr int kDxBound = 512;
constexpr int kDxGroup = 4;  // k-blocks of leading products in an accumulator

template <int STAGES, int SLOTS>
struct Dx {
    // accumulators 0 and 1: the small products of two tiles; 2 and 3: the leading
    // ones.  Otherwise all four go from k-block to k-block.
    static constexpr bool small_apart = STAGES == 3;
    static constexpr int ring = small_apart ? 2 : kDxAcc;
    static constexpr int ring0 = small_apart ? 2 : 0;
    static constexpr int group = small_apart ? kDxGroup : 1;  // k-blocks of an accumulator of the ring
    struct alignas(8) Bars {
        uint64_t full[STAGES];
        uint64_t empty[STAGES];
        uint64_t tfull[kDxAcc];
        uint64_t tempty[kDxAcc];
        uint64_t in[kEpiWarps][SLOTS];
        uint32_t tmem_base;
        int abort;
    };
    static constexpr size_t smem =
        1024 + (size_t)STAGES * kDxStageBytes + (size_t)kEpiWarps * SLOTS * kDxBlk + sizeof(Bars);
};

template <int STAGES, int SLOTS>
__global__ void __launch_bounds__(kDxBound, 1)
router_dense_dx(const __grid_constant__ CUtensorMap tm_dl, const __grid_constant__ CUtensorMap tm_w,
                const __grid_constant__ CUtensorMap tm_in, const __grid_constant__ CUtensorMap tm_out,
                int T, int N, int d, int has_in, const Sums sums, int *status) {
    pdl_enter();
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
    uint8_t *blocks = smem + (size_t)STAGES * kDxStageBytes;
    using C = Dx<STAGES, SLOTS>;
    using Bars = typename C::Bars;
    Bars *bars = reinterpret_cast<Bars *>(blocks + (size_t)kEpiWarps * SLOTS * kDxBlk);
    volatile int *abort = &bars->abort;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int ntc = (d + 127) / 128, nk = (N + 31) / 32;
    const int total = (int)(((int64_t)T + 127) / 128) * ntc;

    if (threadIdx.x == 0) {
        for (int s = 0; s < STAGES; ++s) {
            mbar_init(smem_u32(&bars->full[s]), 1);
            mbar_init(smem_u32(&bars->empty[s]), 1);
        }
        for (int a = 0; a < kDxAcc; ++a) {
            mbar_init(smem_u32(&bars->tfull[a]), 1);
            mbar_init(smem_u32(&bars->tempty[a]), kEpiWarps);
        }
        for (int w = 0; w < kEpiWarps; ++w)
            for (int s = 0; s < SLOTS; ++s) mbar_init(smem_u32(&bars->in[w][s]), 1);
        bars->abort = 0;
        fence_mbar_init();
    }
    if (warp == 1) tmem_alloc(smem_u32(&bars->tmem_base), 512);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem_base = bars->tmem_base;

    if (warp == 0) {
        if (lane == 0) {
            int stage = 0, issued = 0;
            uint32_t phase = 0;
            bool ok = true;
            for (int g = blockIdx.x; g < total && ok; g += gridDim.x) {
                for (int kb = 0; kb < nk; ++kb) {
                    if (!mbar_wait(smem_u32(&bars->empty[stage]), phase ^ 1, status, abort)) {
                        ok = false;
                        break;
                    }
                    const uint32_t full = smem_u32(&bars->full[stage]);
                    const uint32_t sa = smem_u32(smem + (size_t)stage * kDxStageBytes);
                    mbar_arrive_expect_tx(full, kDxStageBytes);
                    tma_load_4d(sa, &tm_dl, full, 0, kb * 32, g / ntc * 2, 0);
                    tma_load_4d(sa + 3 * kDxPiece, &tm_w, full, 0, kb * 32, g % ntc * 2, 0);
                    ++issued;
                    if (++stage == STAGES) { stage = 0; phase ^= 1; }
                }
            }
            // the copies in flight land before the CTA leaves
            for (int i = max(0, issued - STAGES); i < issued; ++i) {
                volatile int no_abort = 0;
                mbar_wait(smem_u32(&bars->full[i % STAGES]), (uint32_t)(i / STAGES & 1), status,
                          &no_abort);
            }
        }
    } else if (warp == 1) {
        if (lane == 0) {
            constexpr uint32_t idesc = idesc_major(128, 128, 1, 1);
            // One k-block's piece products, the smallest first.  One thread issues
            // twelve MMAs of 64 cycles: with a descriptor built anew for each, the
            // issue took longer than the MMAs (T = 4096, d = 4096, N = 256: 102 us
            // against 90).  `two`: more than 16 experts; fresh: the accumulator's
            // first products.
            auto products = [&](uint32_t small, bool fresh_small, uint32_t lead, bool fresh_lead, int s,
                                bool two) {
                const uint32_t sa = smem_u32(smem + (size_t)s * kDxStageBytes);
                const uint64_t da = mnmajor_desc(sa, 4096), db = mnmajor_desc(sa + 3 * kDxPiece, 4096);
#pragma unroll
                for (int sum = 2; sum >= 0; --sum)
#pragma unroll
                    for (int pa = 0; pa <= sum; ++pa)
#pragma unroll
                        for (int kk = 0; kk < 2; ++kk) {
                            const bool fresh = kk == 0 && ((sum == 2 && pa == 0 && fresh_small) ||
                                                           (sum == 0 && fresh_lead));
                            if (kk == 0 || two)
                                tc_mma_bf16(sum > 0 ? small : lead, da + ((pa * kDxPiece + kk * 2048) >> 4),
                                            db + (((sum - pa) * kDxPiece + kk * 2048) >> 4), idesc, !fresh);
                        }
            };
            int stage = 0, acc = 0, tile = 0;
            uint32_t phase = 0, acc_phase = 0;
            bool ok = true;
            for (int g = blockIdx.x; g < total && ok; g += gridDim.x, ++tile) {
                const int sa = tile & 1;  // this tile's accumulator of small products
                if (C::small_apart &&
                    !mbar_wait(smem_u32(&bars->tempty[sa]), (uint32_t)(tile >> 1 & 1) ^ 1, status, abort))
                    break;
                for (int kb = 0; kb < nk; ++kb) {
                    const int at = C::ring0 + acc, in_group = kb % C::group;
                    if ((in_group == 0 &&
                         !mbar_wait(smem_u32(&bars->tempty[at]), acc_phase ^ 1, status, abort)) ||
                        !mbar_wait(smem_u32(&bars->full[stage]), phase, status, abort)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint32_t lead = tmem_base + (uint32_t)(at * 128);
                    if (C::small_apart)
                        products(tmem_base + (uint32_t)(sa * 128), kb == 0, lead, in_group == 0, stage,
                                 N - kb * 32 > 16);
                    else
                        products(lead, true, lead, false, stage, N - kb * 32 > 16);
                    tc_commit(smem_u32(&bars->empty[stage]));
                    if (++stage == STAGES) { stage = 0; phase ^= 1; }
                    if (in_group == C::group - 1 || kb == nk - 1) {
                        tc_commit(smem_u32(&bars->tfull[at]));
                        if (++acc == C::ring) { acc = 0; acc_phase ^= 1; }
                    }
                }
                if (C::small_apart && ok) tc_commit(smem_u32(&bars->tfull[sa]));
            }
        }
    } else {
        const int quad = warp & 3, half = (warp - 2) >> 2;
        uint8_t *mine = blocks + (size_t)(warp - 2) * SLOTS * kDxBlk;
        uint64_t *in = bars->in[warp - 2];
        // This warp's blocks: two per tile, those that start inside dx.  The
        // load cursor runs SLOTS - 1 blocks ahead of the one being added.
        auto block_at = [&](int g, int u, int &row, int &col) {
            row = g / ntc * 128 + quad * 32;
            col = g % ntc * 128 + half * 64 + u * 32;
            return row < T && col < d;
        };
        int lg = blockIdx.x, lu = 0, loaded = 0, used = 0;
        auto load_next = [&] {  // lane 0
            while (lg < total) {
                int row, col;
                const bool valid = block_at(lg, lu, row, col);
                if (++lu == 2) { lu = 0; lg += gridDim.x; }
                if (!valid) continue;
                const int s = loaded++ % SLOTS;
                const uint32_t bar = smem_u32(&in[s]);
                mbar_arrive_expect_tx(bar, kDxBlk);
                tma_load_2d(smem_u32(mine + s * kDxBlk), &tm_in, bar, col, row);
                return;
            }
        };
        if (has_in && lane == 0)
            for (int i = 0; i < SLOTS - 1; ++i) load_next();
        __syncwarp();
        add_partials(sums, blockIdx.x, gridDim.x, threadIdx.x - 64);
        const uint32_t tmem = tmem_base + ((uint32_t)(quad * 32) << 16) + (uint32_t)(half * 64);
        auto release = [&](int a) {  // this warp has read accumulator a
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&bars->tempty[a]));
        };
        // 32 columns of accumulator a
        auto columns = [&](int a, int c, uint32_t (&r)[2][16]) {
            tmem_ld16(tmem + (uint32_t)(a * 128 + c), r[0]);
            tmem_ld16(tmem + (uint32_t)(a * 128 + c + 16), r[1]);
            tmem_ld_wait();
            reg_fence(r[0]);
            reg_fence(r[1]);
        };
        auto pair = [](const uint32_t (&r)[2][16], int i) {
            return make_float2(__uint_as_float(r[i / 8][i % 8 * 2]), __uint_as_float(r[i / 8][i % 8 * 2 + 1]));
        };
        int acc = 0, tile = 0;
        uint32_t acc_phase = 0;
        bool ok = true;
        for (int g = blockIdx.x; g < total && ok; g += gridDim.x, ++tile) {
            // the sum of all accumulators of this tile but the last, in order
            float2 v[32];
#pragma unroll
            for (int i = 0; i < 32; ++i) v[i] = make_float2(0.f, 0.f);
            for (int kb = C::small_apart ? 0 : 1; kb < nk; kb += C::group) {
                const int a = C::ring0 + acc;
                if (!mbar_wait(smem_u32(&bars->tfull[a]), acc_phase, status, abort)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
#pragma unroll
                for (int c = 0; c < 64; c += 32) {
                    uint32_t r[2][16];
                    columns(a, c, r);
#pragma unroll
                    for (int i = 0; i < 16; ++i) v[c / 2 + i] = __fadd2_rn(v[c / 2 + i], pair(r, i));
                }
                release(a);
                if (++acc == C::ring) { acc = 0; acc_phase ^= 1; }
            }
            if (!ok) break;
            const int last = C::small_apart ? tile & 1 : acc;
            if (!mbar_wait(smem_u32(&bars->tfull[last]),
                           C::small_apart ? (uint32_t)(tile >> 1 & 1) : acc_phase, status, abort))
                break;
            if (!C::small_apart && ++acc == C::ring) { acc = 0; acc_phase ^= 1; }
            tc_fence_after();
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                int row, col;
                const bool valid = block_at(g, u, row, col);  // warp-uniform
                uint32_t r[2][16];
                columns(last, u * 32, r);
                if (u == 1) release(last);
                if (!valid) continue;
                const int s = used % SLOTS;
                uint8_t *blk = mine + s * kDxBlk;
                if (has_in) {
                    if (!mbar_wait(smem_u32(&in[s]), (uint32_t)(used / SLOTS & 1), status, abort)) {
                        ok = false;
                        break;
                    }
                } else {
                    if (lane == 0) bulk_wait_read<SLOTS - 1>();
                    __syncwarp();
                }
                ++used;
#pragma unroll
                for (int q = 0; q < 8; ++q) {
                    float4 *at4 = reinterpret_cast<float4 *>(blk + lane * 128 + ((q ^ (lane & 7)) * 16));
                    float2 lo = pair(r, 2 * q), hi = pair(r, 2 * q + 1);
                    if (STAGES > 1) {
                        lo = __fadd2_rn(v[16 * u + 2 * q], lo);
                        hi = __fadd2_rn(v[16 * u + 2 * q + 1], hi);
                    }
                    const float4 o = has_in ? *at4 : make_float4(0.f, 0.f, 0.f, 0.f);
                    *at4 = make_float4(o.x + lo.x, o.y + lo.y, o.z + hi.x, o.w + hi.y);
                }
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                __syncwarp();
                if (lane == 0) {
                    tma_store_2d(&tm_out, smem_u32(blk), col, row);
                    bulk_commit();
                    if (has_in) {
                        // the next load's block is the one stored before this
                        bulk_wait_read<1>();
                        load_next();
                    }
                }
            }
            if (!ok) break;
        }
        if (lane == 0) {
            for (; used < loaded; ++used) {  // after an abort: loads still in flight
                volatile int no_abort = 0;
                mbar_wait(smem_u32(&in[used % SLOTS]), (uint32_t)(used / SLOTS & 1), status,
                          &no_abort);
            }
            bulk_wait<0>();  // stores complete before the CTA ends
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem_base, 512);
    }
}

// ---------------------------------------------------------------------- dW --
//
// The transposed product dW^T = x^T dl: 128 or 256 columns of x as the rows of
// one or two MMAs (MN-major boxes of 64 columns x 64 tokens), the three pieces
// of NT experts side by side as their 3 NT columns, the tokens as K in blocks
// of 64.
// What limits a CTA is its shared memory, which the copies fill and every MMA
// reads: three MMAs of NT columns, one per piece, would read x's tile three
// times (61 us against 43 at T = 32768, d = 4096, N = 32).  The epilogue adds the
// three accumulators.  There are few output tiles, so the tokens are split
// over CTAs and the partial sums added by the last kernel.
//
// The tensor core's accumulator keeps fp32 but cuts where an fp32 addition
// rounds, so a long sum drifts; after every kDwGroup k-blocks (256 tokens) the
// epilogue adds the accumulator to fp32 registers while the next group runs in
// the other half of tensor memory.
constexpr int kDwGroup = 4;
constexpr int kDwBlk = 64 * 128;                 // 64 columns x 64 tokens: 8 KB

template <int NT>
struct Dw {
    static constexpr int mmas = NT == 32 ? 2 : 1;    // of 128 columns of x
    static constexpr int cols = 128 * mmas;
    static constexpr int stages = NT == 32 ? 4 : 5;
    static constexpr int a_bytes = cols / 64 * kDwBlk;
    static constexpr int stage_bytes = a_bytes + 3 * NT * 128;
    static constexpr int per_warp = NT / 2 * mmas;   // experts of an epilogue warp
    struct alignas(8) Bars {
        uint64_t full[stages];
        uint64_t empty[stages];
        uint64_t tfull[2];
        uint64_t tempty[2];
        uint32_t tmem_base;
        int abort;
    };
    static constexpr size_t smem = 1024 + (size_t)stages * stage_bytes + sizeof(Bars);
};

template <int NT>
__global__ void __launch_bounds__(kGemmThreads, 1)
router_dense_dw(const __grid_constant__ CUtensorMap tm_x, const __grid_constant__ CUtensorMap tm_dl,
                int T, int N, int d, float *__restrict__ part, int *status) {
    using C = Dw<NT>;
    pdl_enter();
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
    typename C::Bars *bars = reinterpret_cast<typename C::Bars *>(smem + (size_t)C::stages * C::stage_bytes);
    volatile int *abort = &bars->abort;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int c0 = blockIdx.x * C::cols, e0 = blockIdx.y * NT;
    const int nc = (int)(((int64_t)T + 63) / 64);
    const int k0 = (int)((int64_t)nc * blockIdx.z / gridDim.z);
    const int nk = (int)((int64_t)nc * (blockIdx.z + 1) / gridDim.z) - k0;

    if (threadIdx.x == 0) {
        for (int s = 0; s < C::stages; ++s) {
            mbar_init(smem_u32(&bars->full[s]), 1);
            mbar_init(smem_u32(&bars->empty[s]), 1);
        }
        for (int a = 0; a < 2; ++a) {
            mbar_init(smem_u32(&bars->tfull[a]), 1);
            mbar_init(smem_u32(&bars->tempty[a]), kEpiWarps);
        }
        bars->abort = 0;
        fence_mbar_init();
    }
    if (warp == 1) tmem_alloc(smem_u32(&bars->tmem_base), 512);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem_base = bars->tmem_base;

    if (warp == 0) {
        if (lane == 0) {
            int stage = 0, issued = 0;
            uint32_t phase = 0;
            for (int kb = 0; kb < nk; ++kb) {
                if (!mbar_wait(smem_u32(&bars->empty[stage]), phase ^ 1, status, abort)) break;
                const uint32_t full = smem_u32(&bars->full[stage]);
                const uint32_t sa = smem_u32(smem + (size_t)stage * C::stage_bytes);
                const int t = (k0 + kb) * 64;
                mbar_arrive_expect_tx(full, C::stage_bytes);
#pragma unroll
                for (int b = 0; b < C::cols / 64; ++b)
                    tma_load_2d(sa + b * kDwBlk, &tm_x, full, c0 + b * 64, t);
                tma_load_3d(sa + C::a_bytes, &tm_dl, full, t, e0, 0);
                ++issued;
                if (++stage == C::stages) { stage = 0; phase ^= 1; }
            }
            for (int i = max(0, issued - C::stages); i < issued; ++i) {
                volatile int no_abort = 0;
                mbar_wait(smem_u32(&bars->full[i % C::stages]), (uint32_t)(i / C::stages & 1), status,
                          &no_abort);
            }
        }
    } else if (warp == 1) {
        if (lane == 0) {
            constexpr uint32_t idesc = idesc_major(128, 3 * NT, 1, 0);
            int stage = 0, acc = 0;
            uint32_t phase = 0, acc_phase = 0;
            bool ok = true;
            for (int kb0 = 0; kb0 < nk && ok; kb0 += kDwGroup) {
                if (!mbar_wait(smem_u32(&bars->tempty[acc]), acc_phase ^ 1, status, abort)) break;
                tc_fence_after();
                const uint32_t d_tmem = tmem_base + (uint32_t)(acc * C::mmas * 3 * NT);
                for (int kb = kb0; kb < min(nk, kb0 + kDwGroup); ++kb) {
                    if (!mbar_wait(smem_u32(&bars->full[stage]), phase, status, abort)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint32_t sa = smem_u32(smem + (size_t)stage * C::stage_bytes);
                    const uint64_t da = mnmajor_desc(sa, kDwBlk);
                    const uint64_t db = sw128_kmajor_desc(sa + C::a_bytes);
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk)
#pragma unroll
                        for (int m = 0; m < C::mmas; ++m)
                            tc_mma_bf16(d_tmem + m * 3 * NT, da + ((m * 2 * kDwBlk + kk * 2048) >> 4),
                                        db + ((kk * 32) >> 4), idesc, kk > 0 || kb > kb0);
                    tc_commit(smem_u32(&bars->empty[stage]));
                    if (++stage == C::stages) { stage = 0; phase ^= 1; }
                }
                if (!ok) break;
                tc_commit(smem_u32(&bars->tfull[acc]));
                if (++acc == 2) { acc = 0; acc_phase ^= 1; }
            }
        }
    } else {
        // TMEM lane = column of x; four of the warps take the second MMA's
        // columns, or the second half of the experts
        const int quad = warp & 3, half = (warp - 2) >> 2;
        const int m = C::mmas == 2 ? half : 0, je = C::mmas == 2 ? 0 : half * C::per_warp;
        float sum[C::per_warp];
#pragma unroll
        for (int j = 0; j < C::per_warp; ++j) sum[j] = 0.f;
        int acc = 0;
        uint32_t acc_phase = 0;
        for (int kb0 = 0; kb0 < nk; kb0 += kDwGroup) {
            if (!mbar_wait(smem_u32(&bars->tfull[acc]), acc_phase, status, abort)) break;
            tc_fence_after();
            const uint32_t at = tmem_base + ((uint32_t)(quad * 32) << 16) +
                                (acc * C::mmas + m) * 3 * NT + je;
#pragma unroll
            for (int j = 0; j < C::per_warp; j += 16) {
                uint32_t r0[16], r1[16], r2[16];
                tmem_ld16(at + j, r0);
                tmem_ld16(at + NT + j, r1);
                tmem_ld16(at + 2 * NT + j, r2);
                tmem_ld_wait();
                reg_fence(r0);
                reg_fence(r1);
                reg_fence(r2);
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    sum[j + i] += __uint_as_float(r2[i]) + __uint_as_float(r1[i]) + __uint_as_float(r0[i]);
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&bars->tempty[acc]));
            if (++acc == 2) { acc = 0; acc_phase ^= 1; }
        }
        const int col = c0 + m * 128 + quad * 32 + lane;
        if (col < d) {
            float *o = part + ((int64_t)blockIdx.z * N + e0 + je) * d + col;
#pragma unroll
            for (int j = 0; j < C::per_warp; ++j)
                if (e0 + je + j < N) o[(int64_t)j * d] = sum[j];
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem_base, 512);
    }
}

// ------------------------------------------------------------------- host --

// How the work of one shape is split, and where the workspace holds what.
struct Plan {
    int64_t Tp;
    int dp, chunks, groups, nt, splits;
    size_t dlp, wp, db, part, bytes;
};

inline size_t align256(size_t v) { return (v + 255) & ~(size_t)255; }

Plan plan_of(const moe_shape *s) {
    Plan p;
    p.Tp = ((int64_t)s->T + 63) / 64 * 64;
    p.dp = (s->d + 63) / 64 * 64;
    p.chunks = (s->N + kPrepExp - 1) / kPrepExp;
    p.groups = (int)std::max<int64_t>(1, std::min<int64_t>(p.Tp / kPrepTok, 4 * kSms / p.chunks));
    p.nt = s->N <= 32 ? 32 : 64;
    const int cols = p.nt == 32 ? Dw<32>::cols : Dw<64>::cols;
    const int64_t tiles = (int64_t)((s->d + cols - 1) / cols) * ((s->N + p.nt - 1) / p.nt);
    p.splits = (int)std::max<int64_t>(1, std::min<int64_t>(p.Tp / 64, kSms / tiles));
    p.dlp = 256;
    p.wp = p.dlp + align256((size_t)3 * s->N * p.Tp * 2);
    p.db = p.wp + align256((size_t)3 * s->N * p.dp * 2);
    p.part = p.db + align256((size_t)p.groups * s->N * 4);
    p.bytes = p.part + align256((size_t)p.splits * s->N * s->d * 4);
    return p;
}

template <int STAGES, int SLOTS>
bool dx_attr() {
    static PerDeviceOnce smem_attr;
    return device_once(smem_attr, [] {
        return set_smem_limit(router_dense_dx<STAGES, SLOTS>, Dx<STAGES, SLOTS>::smem);
    });
}

template <int NT>
moe_status launch_dw(const CUtensorMap &mx, const CUtensorMap &mdl, const moe_shape *s, int splits,
                     float *part, int *status, cudaStream_t stream) {
    static PerDeviceOnce smem_attr;
    if (!device_once(smem_attr, [] { return set_smem_limit(router_dense_dw<NT>, Dw<NT>::smem); }))
        return MOE_ERR_CUDA;
    launch_pdl(router_dense_dw<NT>,
               dim3((s->d + Dw<NT>::cols - 1) / Dw<NT>::cols, (s->N + NT - 1) / NT, (unsigned)splits), kGemmThreads,
               Dw<NT>::smem, stream, mx, mdl, s->T, s->N, s->d, part, status);
    return launch_status();
}

}  // namespace
}  // namespace moe

using namespace moe;

MOE_API size_t moe_router_dense_backward_workspace_bytes(const moe_shape *s) {
    if (check_shape(s) != MOE_OK) return 0;
    return plan_of(s).bytes;
}

MOE_API moe_status moe_router_dense_backward(const moe_shape *s, const moe_bf16 *x,
                                             const float *w_router, const float *dlogits,
                                             const float *dx_in, float *dx, float *dw_router,
                                             float *dbias, void *ws, size_t ws_bytes,
                                             cudaStream_t stream) {
    moe_status r = check_shape(s);
    if (r != MOE_OK) return r;
    if (s->T > 0 && (!dlogits || (dx && !w_router) || (dw_router && !x) || (dx_in && !dx)))
        return MOE_ERR_INVALID_ARG;
    const void *ptrs[] = {x, w_router, dlogits, dx_in, dx, dw_router, dbias};
    for (const void *p : ptrs)
        if (!aligned16(p)) return MOE_ERR_ALIGNMENT;
    const Plan pl = plan_of(s);
    if (!ws || (reinterpret_cast<uintptr_t>(ws) & 255u) || ws_bytes < pl.bytes)
        return MOE_ERR_WORKSPACE;
    if (!dx && !dw_router && !dbias) return MOE_OK;
    const int T = s->T, N = s->N, d = s->d;
    uint8_t *base = static_cast<uint8_t *>(ws);
    int *status = static_cast<int *>(ws);
    uint16_t *dlp = reinterpret_cast<uint16_t *>(base + pl.dlp);
    uint16_t *wp = reinterpret_cast<uint16_t *>(base + pl.wp);
    float *db = reinterpret_cast<float *>(base + pl.db);
    float *part = reinterpret_cast<float *>(base + pl.part);
    // whatever can fail comes before the first launch
    const int blocks = (N + 31) / 32;  // k-blocks of a tile of dx
    CUtensorMap mx, mdl_k, mdl, mw, min_, mout;
    if (T > 0 && dw_router &&
        (!make_map(&mx, x, d, T, 64) || !make_map_pieces_k(&mdl_k, dlp, pl.Tp, N, pl.nt)))
        return MOE_ERR_CUDA;
    if (T > 0 && dx) {
        if (!(blocks == 1 ? dx_attr<1, 4>() : blocks <= 4 ? dx_attr<2, 3>() : dx_attr<3, 2>()) ||
            !make_map_pieces_mn(&mdl, dlp, pl.Tp, N, 32) || !make_map_pieces_mn(&mw, wp, pl.dp, N, 32) ||
            !make_map_f32(&min_, dx_in ? dx_in : dx, d, T) || !make_map_f32(&mout, dx, d, T))
            return MOE_ERR_CUDA;
    }
    if (T > 0) {
        // W's CTAs: eight columns a thread, or four CTAs an SM
        const int64_t wctas =
            std::min<int64_t>(((int64_t)N * pl.dp / 8 + kPrepThreads - 1) / kPrepThreads, 4 * kSms);
        const int rows = dx ? (int)((wctas + pl.groups - 1) / pl.groups) : 0;
        launch_pdl(router_dense_prep, dim3(pl.groups, pl.chunks + rows), kPrepThreads, 0, stream, T,
                   pl.Tp, N, d, pl.dp, pl.chunks, dlogits, w_router, dlp, wp, db);
        if (dw_router) {
            r = pl.nt == 32 ? launch_dw<32>(mx, mdl_k, s, pl.splits, part, status, stream)
                            : launch_dw<64>(mx, mdl_k, s, pl.splits, part, status, stream);
            if (r != MOE_OK) return r;
        }
    }
    Sums sums;
    sums.n4 = dw_router ? (int64_t)N * d / 4 : 0;
    sums.splits = T > 0 ? pl.splits : 0;
    sums.N = N;
    sums.groups = T > 0 ? pl.groups : 0;
    sums.part = reinterpret_cast<const float4 *>(part);
    sums.db_part = db;
    sums.dw = reinterpret_cast<float4 *>(dw_router);
    sums.dbias = dbias;
    sums.lanes = 1;  // by the shape alone, so that every call adds in the same order
    while (sums.lanes < 8 && 2 * sums.lanes <= sums.splits && 2 * sums.lanes * sums.n4 <= kSms * 256)
        sums.lanes *= 2;
    const int64_t adds =
        std::max<int64_t>((sums.n4 * sums.lanes + 255) / 256, dbias ? (N + 7) / 8 : 0);
    if (dx && T > 0) {
        // CTAs without a tile add partial sums
        const int64_t tiles = ((int64_t)T + 127) / 128 * ((d + 127) / 128);
        const unsigned grid = (unsigned)std::min<int64_t>(std::max(tiles, adds), num_sms());
        auto go = [&](auto *kern, size_t smem) {
            launch_pdl(kern, grid, kGemmThreads, smem, stream, mdl, mw, min_, mout, T, N, d,
                       dx_in ? 1 : 0, sums, status);
        };
        if (blocks == 1) go(router_dense_dx<1, 4>, Dx<1, 4>::smem);
        else if (blocks <= 4) go(router_dense_dx<2, 3>, Dx<2, 3>::smem);
        else go(router_dense_dx<3, 2>, Dx<3, 2>::smem);
    } else if (dw_router || dbias) {
        launch_pdl(router_dense_sum, (unsigned)std::min<int64_t>(adds, 4 * kSms), 256, 0, stream, sums);
    }
    return launch_status();
}

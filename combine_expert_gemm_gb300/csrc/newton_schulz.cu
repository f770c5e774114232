// Newton-Schulz orthogonalisation of batches of matrices and the Muon step built
// on it (include/moe_dense.h).  With X [m, n], m <= n (the matrix or its
// transpose), |X|_F = 1 at first, a step is
//
//   S = X X^T;  C = a I + b S + c S S;  X <- C X
//
// Three products a step, 2 m^2 n, 2 m^3 and 2 m^2 n operations; S and C are
// symmetric, so of their tiles only those on and above the diagonal are computed
// and each is stored twice.  a sits on C's diagonal, so the third product needs no
// epilogue of its own: its result is the next X.  Nor does the second one:
//   C = c (S + b / (2 c) I)^2 + (a - b^2 / (4 c)) I,
// so the first product's epilogue shifts S's diagonal and the second's reads nothing.
// (With S read for b S the second product of 64 matrices 1024 x 2048 took 259 us,
// its multiplications 147.)  A step with c = 0 takes C from the first product and has
// no second; only a c that is small beside b leaves S as it is and reads it.
//
// Precision.  A step multiplies a small singular value by a (3.4445), so a
// rounding error of the first step reaches the last one up to 485 times larger
// where M's singular values are small; 8 bits of mantissa would leave percents.
// The iterates are held as two fp16 pieces, v 2^10 = hi + lo, hi = fp16(v 2^10),
// lo = fp16(v 2^10 - hi): the difference is exact, |v| < 60 stays finite and lo
// loses nothing to fp16's smallest step (2^-24, or 2^-34 of 1) that matters
// beside hi's 2^-22.  A product takes three MMAs a k-step, lo hi, hi lo, hi hi
// (lo lo is 2^-22 of the product and random); a stage holds the four pieces, so
// the third MMA loads nothing.  The accumulators hold kGroup k-blocks and
// are added in fp32 registers (pair_gemm.cuh says why).
//
// Launches: two passes over the matrices (momentum and sums of squares; scaling,
// splitting and transposing), three products a step; the last product's epilogue
// writes the result or updates the weights.  The products have three forms: CTA
// pairs (pair_gemm.cuh); single SMs where one round of 128 x 128 tiles holds them
// (small_gemm.cuh); and one CTA a matrix for all steps where it fits an SM.
#include <cmath>

#include "../../include/moe_dense.h"
#include "small_gemm.cuh"

namespace moe {
namespace {

using namespace pair;

constexpr float kScale = 1024.0f;     // pieces hold 2^10 times the value
constexpr float kUnscale = 1.0f / kScale;
constexpr int kParts = 128;           // partial sums of squares of a matrix, at most
constexpr int kNormThreads = 256;

// Pieces of two values, each packed as a pair (a in the low half).
__device__ __forceinline__ void split2(float a, float b, uint32_t &hi, uint32_t &lo) {
    const __half2 h = __floats2half2_rn(a, b);
    const float2 f = __half22float2(h);
    const __half2 l = __floats2half2_rn(a - f.x, b - f.y);
    hi = *reinterpret_cast<const uint32_t *>(&h);
    lo = *reinterpret_cast<const uint32_t *>(&l);
}
__device__ __forceinline__ float2 join2(uint32_t hi, uint32_t lo) {
    const float2 a = __half22float2(*reinterpret_cast<const __half2 *>(&hi));
    const float2 b = __half22float2(*reinterpret_cast<const __half2 *>(&lo));
    return make_float2(a.x + b.x, a.y + b.y);
}

__device__ __forceinline__ float load_elem(const float *p, int64_t i) { return p[i]; }
__device__ __forceinline__ float load_elem(const uint16_t *p, int64_t i) {
    return __uint_as_float((uint32_t)p[i] << 16);
}

// ---------------------------------------------------------- first passes --

// A thread's sum of squares.  Groups of values whose squares stay in fp32 are added there,
// with the part that each addition cuts carried to the next (a chain of 4096 equal values
// is off by 6e-5 without it, and a matrix may have 2^32); the others in 64 bits, where
// nothing vanishes or overflows.  All of it in 64 bits took 4 us more for three
// matrices 1001 x 717: 16 cycles a warp for each addition.
struct Squares {
    float s = 0.0f, cut = 0.0f;
    double far = 0.0;
    template <int N>
    __device__ __forceinline__ void add(const float (&v)[N]) {
        float top = 0.0f;
#pragma unroll
        for (int i = 0; i < N; ++i) top = fmaxf(top, fabsf(v[i]));  // drops NaNs, which either sum keeps
        if (top == 0.0f || (top >= 0x1p-50f && top <= 0x1p45f)) {
            float t = 0.0f;
#pragma unroll
            for (int i = 0; i < N; ++i) t = fmaf(v[i], v[i], t);
            t -= cut;
            const float sum = s + t;
            cut = (sum - s) - t;
            s = sum;
        } else {
#pragma unroll 1
            for (int i = 0; i < N; ++i) far = fma((double)v[i], (double)v[i], far);
        }
    }
};

// Sums of squares of matrix blockIdx.y: part[y][x] over a strided share of it.
// With MUON the values are the update direction and the momentum is advanced.
template <bool MUON, typename TIN>
__global__ void __launch_bounds__(kNormThreads)
ns_norm(int64_t elems, const TIN *__restrict__ x, float *__restrict__ momentum, float mu, int nesterov,
        double *__restrict__ part) {
    pdl_enter();
    const int64_t base = (int64_t)blockIdx.y * elems;
    Squares sq;
    constexpr int U = 8;  // elements of a thread in flight
    const int64_t step = (int64_t)gridDim.x * kNormThreads;
    for (int64_t i = (int64_t)blockIdx.x * kNormThreads + threadIdx.x; i < elems; i += U * step) {
        float v[U], m[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const bool in = i + u * step < elems;
            v[u] = in ? load_elem(x, base + i + u * step) : 0.0f;
            if (MUON) m[u] = in ? momentum[base + i + u * step] : 0.0f;
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (MUON) {
                m[u] = fmaf(mu, m[u], v[u]);
                if (i + u * step < elems) momentum[base + i + u * step] = m[u];
                v[u] = nesterov ? fmaf(mu, m[u], v[u]) : m[u];
            }
        }
        sq.add(v);
    }
    __shared__ double red[kNormThreads / 32];
    if (__syncthreads_or(sq.far != 0.0)) {
        double t = sq.far + sq.s;
#pragma unroll
        for (int o = 16; o; o >>= 1) t += __shfl_xor_sync(0xFFFFFFFFu, t, o);
        if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = t;
    } else {
        float t = sq.s;
#pragma unroll
        for (int o = 16; o; o >>= 1) t += __shfl_xor_sync(0xFFFFFFFFu, t, o);
        if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = t;
    }
    __syncthreads();
    if (threadIdx.x == 0) {
        double t = 0.0;
        for (int i = 0; i < kNormThreads / 32; ++i) t += red[i];
        part[(int64_t)blockIdx.y * gridDim.x + blockIdx.x] = t;
    }
}

constexpr int kSplitTile = 64;

// The pieces of X_0 = M / (|M| + eps), or of its transpose: a 64 x 64 tile of
// M a CTA.  hi [B][m][ld], lo [B][m][ld] one plane group after the other.
template <bool MUON, typename TIN>
__global__ void __launch_bounds__(256)
ns_split(int rows, int cols, int tall, int64_t ld, const TIN *__restrict__ x, const float *__restrict__ momentum,
         float mu, int nesterov, float eps, const double *__restrict__ part, int parts, uint16_t *__restrict__ hi,
         uint16_t *__restrict__ lo) {
    pdl_enter();
    __shared__ float tile[kSplitTile][kSplitTile + 1];
    __shared__ float inv_s, pre_s;
    const int64_t b = blockIdx.z;
    const int r0 = blockIdx.y * kSplitTile, c0 = blockIdx.x * kSplitTile;
    const int64_t base = b * rows * cols;
    const int tx = threadIdx.x & 63, ty = threadIdx.x >> 6;
    float v[kSplitTile / 4];  // the tile is on its way while the norm is added up
#pragma unroll
    for (int r = 0; r < kSplitTile / 4; ++r) {
        const int row = r0 + 4 * r + ty;
        const int64_t i = base + (int64_t)row * cols + c0 + tx;
        const bool in = row < rows && c0 + tx < cols;
        v[r] = in ? (MUON && !nesterov ? momentum[i] : load_elem(x, i)) : 0.0f;
        if (MUON && nesterov && in) v[r] = fmaf(mu, momentum[i], v[r]);
    }
    if (threadIdx.x < 32) {
        double s = 0.0;
        for (int i = threadIdx.x; i < parts; i += 32) s += part[b * parts + i];
#pragma unroll
        for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, o);
        if (threadIdx.x == 0) {
            // v / (|M| + eps) as (v pre) inv, with a power of two that brings a sum of squares
            // outside fp32 into it (a 64-bit root and division took 3 us more)
            const bool large = s > 0x1p100, small = s < 0x1p-100;
            const float pre = large ? 0x1p-100f : 1.0f, up = small ? 0x1p80f : pre;
            const float root = sqrtf((float)(s * ((double)up * up)));
            inv_s = 1.0f / ((small ? root * 0x1p-80f : root) + eps * pre);
            pre_s = pre;
        }
    }
    __syncthreads();
    const float inv = inv_s, pre = pre_s;
    const int64_t out = b * (tall ? cols : rows) * ld;
#pragma unroll
    for (int r = 0; r < kSplitTile / 4; ++r) tile[4 * r + ty][tx] = v[r] * pre * inv * kScale;
    __syncthreads();
    // rows of the iterate: of M, or its columns
    const int orow0 = tall ? c0 : r0, ocol0 = tall ? r0 : c0;
    const int orows = tall ? cols : rows;
    for (int i = threadIdx.x; i < kSplitTile * (kSplitTile / 2); i += 256) {
        const int r = i / (kSplitTile / 2), c = 2 * (i % (kSplitTile / 2));
        if (orow0 + r >= orows || ocol0 + c >= ld) continue;
        uint32_t h, l;
        split2(tall ? tile[c][r] : tile[r][c], tall ? tile[c + 1][r] : tile[r][c + 1], h, l);
        const int64_t at = out + (int64_t)(orow0 + r) * ld + ocol0 + c;
        *reinterpret_cast<uint32_t *>(hi + at) = h;
        *reinterpret_cast<uint32_t *>(lo + at) = l;
    }
}

// ------------------------------------------------------------- products --

// NS_GRAM: r I + q X X^T.  NS_SQUARE: r I + q S S.  NS_POLY: r I + q S S + b S, for
// steps whose square cannot be completed.  NS_APPLY: C X.  NS_LAST: its last.
enum { NS_GRAM, NS_SQUARE, NS_POLY, NS_APPLY, NS_LAST };

struct NsArgs {
    CUtensorMap a, b;    // operands: planes [0, B) are hi, [B, 2 B) lo
    CUtensorMap o;       // pieces of the result
    int B, m, n, k;      // result [m, n], reduction k
    int mt, nt;
    float r, q, lin;     // of the symmetric products: diagonal, product, S
    const uint16_t *s;   // NS_POLY: the pieces of S, rows lds apart
    int64_t lds;
    // NS_LAST: out [B, rows, cols] or the weights' update
    int rows, cols, tall, out_f32;
    void *out;
    float *w;
    uint16_t *w_copy;
    const float *lr;
    float decay, factor;
    int *status;
};

// As store_block16, transposed: element (row lane, column i) of the block goes to
// row i of (x, y, z).
__device__ __forceinline__ void store_mirrored(Epi &e, const uint32_t (&w)[16], const CUtensorMap *map, int x,
                                               int y, int z) {
    uint8_t *blk = e.blk + (e.turn ^= 2048);
    if (e.lane == 0) bulk_wait_read<1>();
    __syncwarp();
    // row i at 64 i, its 16-byte chunk lane / 8 swizzled by (i / 2) % 4
    uint8_t *at = blk + (e.lane & 7) * 2;
#pragma unroll
    for (int i = 0; i < 32; ++i)
        *reinterpret_cast<uint16_t *>(at + i * 64 + (((e.lane >> 3) ^ ((i >> 1) & 3)) * 16)) =
            (uint16_t)(i & 1 ? w[i / 2] >> 16 : w[i / 2]);
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    __syncwarp();
    if (e.lane == 0) {
        tma_store_3d(map, smem_u32(blk), x, y, z);
        bulk_commit();
    }
}

template <int MODE, int N>
struct Ns {
    using Args = NsArgs;
    struct Regs {};
    static constexpr int kN = N, kStages = N == 256 ? 3 : 4;
    static constexpr int kStageBytes = 2 * OPERAND + 2 * b_bytes(N);  // hi and lo of A, hi and lo of B
    static constexpr int kGroup = 2;
    static constexpr int COLS = N / 2;
    static constexpr int kRows = 16;  // M's rows of a lane in flight in the last epilogue
    static constexpr bool kSym = MODE < NS_APPLY;
    static __device__ __forceinline__ int per_matrix(const Args &p) {
        // row m of the upper triangle has nt - m PM / N tiles
        return kSym ? p.mt * p.nt - p.mt * (p.mt - 1) / 2 * (PM / N) : p.mt * p.nt;
    }
    static __device__ __forceinline__ int count(const Args &p, int unit, int units) {
        return strided_count(p.B * per_matrix(p), unit, units);
    }
    static __device__ __forceinline__ Tile tile(const Args &p, int unit, int units, int i) {
        const int g = unit + i * units, per = per_matrix(p), z = g / per;
        int r = g - z * per, m = 0, n;
        if (kSym) {
            while (r >= p.nt - m * (PM / N)) r -= p.nt - PM / N * m++;
            n = m * (PM / N) + r;
        } else {
            band_tile(r, p.mt, p.nt, m, n);
        }
        return Tile{z, m * PM, n * N};
    }
    static __device__ __forceinline__ int k_blocks(const Args &p, const Tile &) { return (p.k + BK - 1) / BK; }
    static __device__ __forceinline__ void load(const Args &p, const Tile &t, int kb, uint32_t s, uint32_t bar,
                                                int rank) {
        const int k = kb * BK, row = t.m + rank * BM, col = t.n + rank * (N / 2);
        load_k(s, &p.a, bar, k, row, t.z);
        load_k(s + OPERAND, &p.a, bar, k, row, t.z + p.B);
        if (kSym) {
            load_k(s + 2 * OPERAND, &p.b, bar, k, col, t.z);
            load_k(s + 2 * OPERAND + b_bytes(N), &p.b, bar, k, col, t.z + p.B);
        } else {
            load_mn<N / 2>(s + 2 * OPERAND, &p.b, bar, col, k, t.z);
            load_mn<N / 2>(s + 2 * OPERAND + b_bytes(N), &p.b, bar, col, k, t.z + p.B);
        }
    }
    static __device__ __forceinline__ void mma(const Args &, const Tile &, uint32_t d, uint32_t s, bool first) {
        // the small products first: what they leave is cut least
        mma_block<0, N, false, !kSym>(d, s + OPERAND, s + 2 * OPERAND, first);
        mma_block<0, N, false, !kSym>(d, s, s + 2 * OPERAND + b_bytes(N), false);
        mma_block<0, N, false, !kSym>(d, s, s + 2 * OPERAND, false);
    }
    // The chunks of 32 columns one after the other in a loop, which picks its sums by
    // selections, as registers have no index: unrolled over the four chunks, the
    // epilogue's code comes through the instruction cache too slowly (the last
    // product of 64 matrices 1024 x 2048 took 1.4 ms where the others take 0.47; of
    // three matrices 1001 x 717, 42 us instead of 27).
    static __device__ __forceinline__ void finish(const Args &p, const Tile &t, Epi &e, int wrow,
                                                  const float (&sum)[COLS]) {
        const int row0 = t.m + wrow;
        if (row0 >= p.m) return;
        const int col0 = t.n + e.col, row = row0 + e.lane;
        float ahead[kRows];  // NS_LAST: the weights of the rows to come
        if constexpr (MODE == NS_LAST) fetch_w(p, t.z, row0, col0, 0, e.lane, ahead);
        uint4 s4[8];  // NS_POLY: S's pieces of the 32 columns to come
        if constexpr (MODE == NS_POLY) fetch_s(p, t.z, row, col0, s4);
#pragma unroll 1
        for (int c = 0; c < COLS / 32; ++c) {
            const int col = col0 + 32 * c;
            if (col >= p.n) break;
            float v[32];
            pick32(sum, c, v);
            if constexpr (MODE == NS_LAST) {
                last(p, t, e, row0, col, c + 1 < COLS / 32, v, ahead);
                continue;
            }
            uint32_t hi[16], lo[16];
            if constexpr (kSym) {
                const float q = p.q * kUnscale, r = p.r * kScale;
#pragma unroll
                for (int i = 0; i < 32; ++i) v[i] = fmaf(q, v[i], row == col + i ? r : 0.0f);
                if constexpr (MODE == NS_POLY) {
                    const uint32_t *sw = reinterpret_cast<const uint32_t *>(s4);
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        const float2 s = join2(sw[i], sw[16 + i]);
                        v[2 * i] = fmaf(p.lin, s.x, v[2 * i]);
                        v[2 * i + 1] = fmaf(p.lin, s.y, v[2 * i + 1]);
                    }
                    if (c + 1 < COLS / 32) fetch_s(p, t.z, row, col + 32, s4);
                }
            } else {
#pragma unroll
                for (int i = 0; i < 32; ++i) v[i] *= kUnscale;
            }
#pragma unroll
            for (int i = 0; i < 16; ++i) split2(v[2 * i], v[2 * i + 1], hi[i], lo[i]);
            store_block16(e, hi, &p.o, col, row0, t.z);
            store_block16(e, lo, &p.o, col, row0, t.z + p.B);
            if (kSym && t.n >= t.m + PM) {
                store_mirrored(e, hi, &p.o, row0, col, t.z);
                store_mirrored(e, lo, &p.o, row0, col, t.z + p.B);
            }
        }
    }
    // 32 columns of row `row` of S: hi in v[0..3], lo in v[4..7].
    static __device__ __forceinline__ void fetch_s(const Args &p, int z, int row, int col, uint4 (&v)[8]) {
        const uint16_t *sh = p.s + ((int64_t)z * p.m + row) * p.lds + col;
        const uint16_t *sl = sh + (int64_t)p.B * p.m * p.lds;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const bool in = row < p.m && col + 8 * i < p.lds;
            v[i] = in ? reinterpret_cast<const uint4 *>(sh)[i] : make_uint4(0, 0, 0, 0);
            v[4 + i] = in ? reinterpret_cast<const uint4 *>(sl)[i] : make_uint4(0, 0, 0, 0);
        }
    }
    // The weights of rows [i0, i0 + kRows) of the 32 x 32 block at (row0, col) of the
    // iterate, in M's orientation.
    static __device__ __forceinline__ void fetch_w(const Args &p, int z, int row0, int col, int i0, int lane,
                                                   float (&w)[kRows]) {
        if (!p.w) return;
        const int r = (p.tall ? col : row0) + i0, j = (p.tall ? row0 : col) + lane;
        const int n = j < p.cols ? p.rows - r : 0;
        const float *src = p.w + ((int64_t)z * p.rows + r) * p.cols + j;
#pragma unroll
        for (int i = 0; i < kRows; ++i, src += p.cols) w[i] = i < n ? *src : 0.0f;
    }
    // 32 x 32 values of the last iterate (rows row0.., columns col..) to M's own
    // layout, whatever its alignment is: through shared memory, so that the lanes run
    // along M's rows (the iterate's columns where M is tall) and the loop over M's rows is
    // short.  The weights of the kRows rows to come are on their way while kRows are
    // updated; `more`: another block of this tile follows.
    static __device__ __forceinline__ void last(const Args &p, const Tile &t, Epi &e, int row0, int col, bool more,
                                                const float (&v)[32], float (&ahead)[kRows]) {
        float *blk = reinterpret_cast<float *>(e.blk);  // row i of M: 32 columns, rotated by i
        __syncwarp();
        if (p.tall) {
#pragma unroll
            for (int i = 0; i < 32; ++i) blk[i * 32 + ((e.lane + i) & 31)] = v[i];
        } else {
#pragma unroll
            for (int i = 0; i < 32; ++i) blk[e.lane * 32 + ((i + e.lane) & 31)] = v[i];
        }
        __syncwarp();
        const int r = p.tall ? col : row0, j = (p.tall ? row0 : col) + e.lane;
        const int rows = min(32, p.rows - r);
        const bool in = j < p.cols;
        const int64_t step = p.cols;
        int64_t at = ((int64_t)t.z * p.rows + r) * p.cols + j;
        const float lr = p.w ? *p.lr : 0.0f, keep = 1.0f - lr * p.decay;
        const float f = p.w ? -lr * p.factor * (kUnscale * kUnscale) : kUnscale * kUnscale;
        uint16_t *const o16 = p.w ? p.w_copy : p.out_f32 ? nullptr : static_cast<uint16_t *>(p.out);
        float *const o32 = p.w ? p.w : p.out_f32 ? static_cast<float *>(p.out) : nullptr;
        // pairs of columns a lane, of every other row, where they are 4-byte aligned
        const bool pairs = (p.cols & 1) == 0 && (reinterpret_cast<uintptr_t>(o16) & 3) == 0;
#pragma unroll 1
        for (int i0 = 0; i0 < rows; i0 += kRows, at += kRows * step) {
            const int n = in ? rows - i0 : 0;
            float u[kRows];
#pragma unroll
            for (int i = 0; i < kRows; ++i) u[i] = ahead[i];
            const bool down = i0 + kRows < rows;
            if (down || more) fetch_w(p, t.z, row0, down ? col : col + 32, down ? i0 + kRows : 0, e.lane, ahead);
#pragma unroll
            for (int i = 0; i < kRows; ++i) {
                const float o = f * blk[(i0 + i) * 32 + ((e.lane + i0 + i) & 31)];
                u[i] = p.w ? fmaf(keep, u[i], o) : o;
            }
            if (o32) {
                float *dst = o32 + at;
#pragma unroll
                for (int i = 0; i < kRows; ++i, dst += step)
                    if (i < n) *dst = u[i];
            }
            if (!o16) continue;
            uint16_t *dst = o16 + at;
            if (pairs) {
                const int odd = e.lane & 1;
                if (odd) dst += step - 1;
#pragma unroll
                for (int i = 0; i < kRows; i += 2, dst += 2 * step) {
                    const float other = __shfl_xor_sync(0xFFFFFFFFu, odd ? u[i] : u[i + 1], 1);
                    const uint32_t w = odd ? pack_bf16x2(other, u[i + 1]) : pack_bf16x2(u[i], other);
                    if (i + odd < n) *reinterpret_cast<uint32_t *>(dst) = w;
                }
            } else {
#pragma unroll
                for (int i = 0; i < kRows; ++i, dst += step)
                    if (i < n) *reinterpret_cast<__nv_bfloat16 *>(dst) = __float2bfloat16_rn(u[i]);
            }
        }
    }
};

// ------------------------------------------------------------ few matrices --
//
// The same products for batches whose tiles do not fill the pairs (small_gemm.cuh).
// Of the symmetric products, tiles of 128 x 128 are computed on and above the diagonal
// only; narrower ones all, there being SMs for them.

struct SmallNsArgs {
    CUtensorMap a, b;  // features' and tokens' operand, planes as in NsArgs
    int B, T, F, nk, split, tt;  // result [T, F]
    float r, q, lin;
    const uint16_t *s; // NS_POLY
    uint16_t *o;       // pieces of the result, rows ld apart
    int64_t ld;
    void *out;         // NS_LAST: [B, T, F]
    int out_f32;
    float *w;
    uint16_t *w_copy;
    const float *lr;
    float decay, factor;
    int *status;
};

// NS_LAST with TALL: M's columns are the iterate's rows, so the features are C's rows and
// the tokens the iterate's columns.
template <int MODE, bool TALL, int N>
struct SmallNs {
    using Args = SmallNsArgs;
    static constexpr int kN = N;
    static constexpr bool kPairs = false, kEarly = false, kSym = MODE < NS_APPLY;
    static constexpr int kFmt = 0, kPieces = 2;
    static constexpr int kAMn = !kSym && !TALL, kBMn = !kSym && TALL;
    static constexpr bool kMirror = kSym && N == small::kM;
    static __device__ __forceinline__ void prefetch_maps(const Args &p) {
        tma_prefetch_desc(&p.a);
        tma_prefetch_desc(&p.b);
    }
    static __device__ __forceinline__ void load_a(const Args &p, uint32_t s, uint32_t bar, int kb, int f0, int z,
                                                  int q) {
        if (kAMn) {
            small::load_box(s, &p.a, bar, f0, kb * BK, z + q * p.B);
            small::load_box(s + BLK, &p.a, bar, f0 + 64, kb * BK, z + q * p.B);
        } else {
            small::load_box(s, &p.a, bar, kb * BK, f0, z + q * p.B);
        }
    }
    static __device__ __forceinline__ void load_b(const Args &p, uint32_t s, uint32_t bar, int kb, int t0, int z,
                                                  int q) {
        if (kBMn) {
#pragma unroll
            for (int i = 0; i < N / 64; ++i)
                small::load_box(s + i * BLK, &p.b, bar, t0 + 64 * i, kb * BK, z + q * p.B);
        } else {
            small::load_box(s, &p.b, bar, kb * BK, t0, z + q * p.B);
        }
    }
    struct In {
        float4 w;   // NS_LAST: the weights
        uint2 h, l; // NS_POLY: S
        float lr;
    };
    static __device__ __forceinline__ void fetch(const Args &p, int t, int f, int z, In &in) {
        if (f >= p.F) return;
        if (MODE == NS_LAST) {
            in.lr = p.w ? *p.lr : 0.0f;
            if (!p.w) return;
            const float *src = p.w + ((int64_t)z * p.T + t) * p.F + f;
            if ((p.F & 3) == 0 && (reinterpret_cast<uintptr_t>(p.w) & 15) == 0) {
                in.w = *reinterpret_cast<const float4 *>(src);
            } else {
                const int n = p.F - f;
                in.w = make_float4(src[0], n > 1 ? src[1] : 0.0f, n > 2 ? src[2] : 0.0f, n > 3 ? src[3] : 0.0f);
            }
        }
        if (MODE == NS_POLY) {
            const int64_t at = ((int64_t)z * p.T + t) * p.ld + f;
            in.h = *reinterpret_cast<const uint2 *>(p.s + at);
            in.l = *reinterpret_cast<const uint2 *>(p.s + (int64_t)p.B * p.T * p.ld + at);
        }
    }
    static __device__ __forceinline__ void emit(const Args &p, bool ok, int t, int f, int z, const float4 &a,
                                                const float4 &, const In &in) {
        if (!ok || f >= p.F) return;
        float v[4] = {a.x, a.y, a.z, a.w};
        if constexpr (MODE == NS_LAST) {
            const int64_t at = ((int64_t)z * p.T + t) * p.F + f;
            const int n = min(4, p.F - f);
            const float lr = in.lr, keep = 1.0f - lr * p.decay;
            const float c = p.w ? -lr * p.factor * (kUnscale * kUnscale) : kUnscale * kUnscale;
#pragma unroll
            for (int i = 0; i < 4; ++i) v[i] *= c;
            if (p.w) {
                v[0] = fmaf(keep, in.w.x, v[0]);
                v[1] = fmaf(keep, in.w.y, v[1]);
                v[2] = fmaf(keep, in.w.z, v[2]);
                v[3] = fmaf(keep, in.w.w, v[3]);
            }
            float *o32 = p.w ? p.w : p.out_f32 ? static_cast<float *>(p.out) : nullptr;
            uint16_t *o16 = p.w ? p.w_copy : p.out_f32 ? nullptr : static_cast<uint16_t *>(p.out);
            if (o32) {
                float *dst = o32 + at;
                if ((p.F & 3) == 0 && (reinterpret_cast<uintptr_t>(o32) & 15) == 0) {
                    *reinterpret_cast<float4 *>(dst) = make_float4(v[0], v[1], v[2], v[3]);
                } else {
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if (i < n) dst[i] = v[i];
                }
            }
            if (o16) {
                uint16_t *dst = o16 + at;
                if ((p.F & 3) == 0 && (reinterpret_cast<uintptr_t>(o16) & 7) == 0) {
                    *reinterpret_cast<uint2 *>(dst) = make_uint2(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]));
                } else {
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if (i < n) reinterpret_cast<__nv_bfloat16 *>(dst)[i] = __float2bfloat16_rn(v[i]);
                }
            }
        } else {
            const int64_t at = ((int64_t)z * p.T + t) * p.ld + f, plane = (int64_t)p.B * p.T * p.ld;
            if constexpr (kSym) {
                const float q = p.q * kUnscale, r = p.r * kScale;
#pragma unroll
                for (int i = 0; i < 4; ++i) v[i] = fmaf(q, v[i], t == f + i ? r : 0.0f);
                if constexpr (MODE == NS_POLY) {
                    const float2 s0 = join2(in.h.x, in.l.x), s1 = join2(in.h.y, in.l.y);
                    v[0] = fmaf(p.lin, s0.x, v[0]);
                    v[1] = fmaf(p.lin, s0.y, v[1]);
                    v[2] = fmaf(p.lin, s1.x, v[2]);
                    v[3] = fmaf(p.lin, s1.y, v[3]);
                }
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i) v[i] *= kUnscale;
            }
            uint2 hi, lo;
            split2(v[0], v[1], hi.x, lo.x);
            split2(v[2], v[3], hi.y, lo.y);
            // rows are padded to 8 elements, so four of them fit behind any column
            *reinterpret_cast<uint2 *>(p.o + at) = hi;
            *reinterpret_cast<uint2 *>(p.o + plane + at) = lo;
        }
    }
};

// ----------------------------------------------------- small matrices, fused --
//
// A matrix of at most 128 x 256 (its sides in either order) never leaves one SM: the
// pieces of X, [m][n] in blocks of 64 columns (128 rows of 128 swizzled bytes each),
// and those of S or C over each other, 192 KB in all; the sums in tensor memory.
// One image of X is both a K-major operand (for X X^T) and an MN-major one (for C X).
// A step is three products of 12 to 24 MMAs and three passes of the CTA over the
// sums; as launches of their own the same products took 4.6 us each, 15 of them and
// two passes before them 78 us for 8 matrices of 256 x 128.

constexpr int kFuseM = 128, kFuseN = 256;
constexpr int kFuseBlk = kFuseM * 128;  // 64 columns of a piece: 16 KB
constexpr int kFuseThreads = 512;

struct FuseStep {
    float gr, gq;        // the Gram matrix's: r I + q X X^T
    float pr, pq, plin;  // r I + q S S + lin S
    int poly;            // whether there is a second product
};

struct FuseArgs {
    int rows, cols, tall, m, n, nb;  // nb: blocks of 64 columns
    int steps;
    float eps;
    const void *x;       // the matrices, or the gradients
    float *momentum;
    float mu;
    int nesterov;
    void *out;
    int out_f32;
    float *w;
    uint16_t *w_copy;
    const float *lr;
    float decay, factor;
    FuseStep step[MOE_NS_MAX_STEPS];
    int *status;
};

inline size_t fuse_smem(int nb) { return 1024 + (size_t)(2 * nb + 4) * kFuseBlk + 64; }

// MN-major operand of blocks kFuseBlk apart.
__device__ __forceinline__ uint64_t fuse_mn_desc(uint32_t a) {
    return (pair::mn_desc(a) & ~((uint64_t)0x3FFF << 16)) | (uint64_t)(kFuseBlk >> 4) << 16;
}

template <bool MUON, typename TIN>
__global__ void __launch_bounds__(kFuseThreads, 1) ns_fused(const __grid_constant__ FuseArgs p) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem =
        reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
    uint8_t *xh = smem, *xl = xh + p.nb * kFuseBlk, *sh = xl + p.nb * kFuseBlk, *sl = sh + 2 * kFuseBlk;
    __shared__ uint64_t bar;
    __shared__ uint32_t tmem_base;
    __shared__ int abort;
    __shared__ float red[2][kFuseThreads / 32];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        mbar_init(smem_u32(&bar), 1);
        abort = 0;
        fence_mbar_init();
    }
    pdl_enter();
    if (warp == 0) tmem_alloc(smem_u32(&tmem_base), 512);

    const int elems = p.rows * p.cols;
    const int64_t base = (int64_t)blockIdx.x * elems;
    {
        // The update direction in registers: pairs of neighbouring columns of the iterate,
        // the lanes along M's rows, kBatch pairs of loads on their way at once.
        constexpr int kBatch = 8, kPairs = kFuseM * kFuseN / 2 / kFuseThreads;
        const TIN *x = static_cast<const TIN *>(p.x) + base;
        float *mom = MUON ? p.momentum + base : nullptr;
        const int np = 32 * p.nb;  // pairs of a row, padded
        const int next = p.tall ? p.cols : 1;
        float a[kPairs], b[kPairs];
        float top = 0.0f;
        auto place = [&](int u, int &r, int &c) {
            const int i = u * kFuseThreads + (int)threadIdx.x;
            r = p.tall ? i & (kFuseM - 1) : i / np;
            c = 2 * (p.tall ? i / kFuseM : i - r * np);
        };
#pragma unroll
        for (int u0 = 0; u0 < kPairs; u0 += kBatch) {
            if (u0 * kFuseThreads >= kFuseM * np) break;  // the same for all
            float ma[kBatch], mb[kBatch];
#pragma unroll
            for (int u = 0; u < kBatch; ++u) {
                int r, c;
                place(u0 + u, r, c);
                const int at = p.tall ? c * p.cols + r : r * p.cols + c;
                const bool in = r < p.m && c < p.n, in1 = r < p.m && c + 1 < p.n;
                a[u0 + u] = in ? load_elem(x, at) : 0.0f;
                b[u0 + u] = in1 ? load_elem(x, at + next) : 0.0f;
                if (MUON) {
                    ma[u] = in ? mom[at] : 0.0f;
                    mb[u] = in1 ? mom[at + next] : 0.0f;
                }
            }
#pragma unroll
            for (int u = 0; u < kBatch; ++u) {
                if (MUON) {
                    int r, c;
                    place(u0 + u, r, c);
                    const int at = p.tall ? c * p.cols + r : r * p.cols + c;
                    float &va = a[u0 + u], &vb = b[u0 + u];
                    ma[u] = fmaf(p.mu, ma[u], va);
                    mb[u] = fmaf(p.mu, mb[u], vb);
                    if (r < p.m && c < p.n) mom[at] = ma[u];
                    if (r < p.m && c + 1 < p.n) mom[at + next] = mb[u];
                    va = p.nesterov ? fmaf(p.mu, ma[u], va) : ma[u];
                    vb = p.nesterov ? fmaf(p.mu, mb[u], vb) : mb[u];
                }
                top = fmaxf(top, fmaxf(fabsf(a[u0 + u]), fabsf(b[u0 + u])));
            }
        }
#pragma unroll
        for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
        if (lane == 0) red[0][warp] = top;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kFuseThreads / 32; ++i) top = fmaxf(top, red[0][i]);
        // the largest entry's size is taken out first (a power of two, so no bit changes):
        // squares neither vanish nor overflow.  Below 2^-100, where eps is all that counts,
        // and from 2^126 on the power stays.
        const uint32_t size = min(max(__float_as_uint(top) >> 23, 27u), 253u);
        const float pre = __uint_as_float((254u - size) << 23);
        float s = 0.0f;
#pragma unroll
        for (int u = 0; u < kPairs; ++u) {
            if (u * kFuseThreads >= kFuseM * np) break;
            a[u] *= pre;
            b[u] *= pre;
            s = fmaf(a[u], a[u], s);
            s = fmaf(b[u], b[u], s);
        }
#pragma unroll
        for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, o);
        if (lane == 0) red[1][warp] = s;
        __syncthreads();
        float inv = 0.0f;
#pragma unroll
        for (int i = 0; i < kFuseThreads / 32; ++i) inv += red[1][i];
        inv = 1.0f / (sqrtf(inv) + p.eps * pre);
#pragma unroll
        for (int u = 0; u < kPairs; ++u) {
            if (u * kFuseThreads >= kFuseM * np) break;
            int r, c;
            place(u, r, c);
            uint32_t h, l;
            split2(a[u] * inv * kScale, b[u] * inv * kScale, h, l);
            const int at = (c >> 6) * kFuseBlk + r * 128 + ((((c >> 3) & 7) ^ (r & 7)) << 4) + (c & 7) * 2;
            *reinterpret_cast<uint32_t *>(xh + at) = h;
            *reinterpret_cast<uint32_t *>(xl + at) = l;
        }
    }
    const uint32_t tmem = tmem_base;

    uint32_t parity = 0;
    // What the threads wrote is seen by the tensor core; one thread issues the three
    // products of pieces of k-blocks [0, kb), each into an accumulator of its own, `stride`
    // columns apart; everyone waits.
    auto multiply = [&](uint8_t *ah, uint8_t *al, uint8_t *bh, uint8_t *bl, bool b_mn, int cols, int kb, int stride) {
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        tc_fence_before();
        __syncthreads();
        if (threadIdx.x == 0) {
            tc_fence_after();
            const uint32_t idesc = (1u << 4) | ((b_mn ? 1u : 0u) << 16) | ((uint32_t)(cols >> 3) << 17) |
                                   ((uint32_t)(kFuseM >> 4) << 24);
            for (int k = 0; k < kb; ++k) {
#pragma unroll 1
                for (int q = 0; q < 3; ++q) {  // lo hi, hi lo, hi hi
                    const uint32_t a = smem_u32(q == 0 ? al : ah) + k * kFuseBlk;
                    const uint32_t b = smem_u32(q == 1 ? bl : bh) + k * (b_mn ? 64 * 128 : kFuseBlk);
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk)
                        tc_mma_bf16(tmem + k * stride, sw128_kmajor_desc(a + kk * 32),
                                    b_mn ? fuse_mn_desc(b + kk * 2048) : sw128_kmajor_desc(b + kk * 32), idesc,
                                    (q | kk) != 0 ? 1u : 0u);
                }
            }
            tc_commit(smem_u32(&bar));
        }
        __syncwarp();
        mbar_wait(smem_u32(&bar), parity, p.status, &abort);
        parity ^= 1;
        tc_fence_after();
    };
    const int row = (warp & 3) * 32 + lane, part = warp >> 2;  // a quarter of the columns
    const uint32_t tlane = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    // 16 columns from c of this lane's row, the accumulators added
    auto sum16 = [&](int c, int kb, int stride, float (&v)[16]) {
        uint32_t t[16];
        tmem_ld16(tlane + c, t);
        tmem_ld_wait();
        reg_fence(t);
#pragma unroll
        for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(t[i]);
#pragma unroll 1
        for (int k = 1; k < kb; ++k) {
            tmem_ld16(tlane + k * stride + c, t);
            tmem_ld_wait();
            reg_fence(t);
#pragma unroll
            for (int i = 0; i < 16; ++i) v[i] += __uint_as_float(t[i]);
        }
    };
    auto put16 = [&](uint8_t *hi, uint8_t *lo, int c, const float (&v)[16]) {
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            uint32_t h[4], l[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) split2(v[8 * q + 2 * i], v[8 * q + 2 * i + 1], h[i], l[i]);
            const int at = (c >> 6) * kFuseBlk + row * 128 + (((((c >> 3) & 7) + q) ^ (row & 7)) << 4);
            *reinterpret_cast<uint4 *>(hi + at) = make_uint4(h[0], h[1], h[2], h[3]);
            *reinterpret_cast<uint4 *>(lo + at) = make_uint4(l[0], l[1], l[2], l[3]);
        }
    };
    const int kbm = (p.m + 63) / 64, scols = 64 * kbm, xcols = 64 * p.nb;
    // r I + q sum (+ lin S) into S's place: what lies past m stays 0
    auto symmetric = [&](int kb, float r, float q, float lin) {
#pragma unroll 1
        for (int c = part * (scols / 4); c < (part + 1) * (scols / 4); c += 16) {
            float v[16];
            sum16(c, kb, kFuseM, v);
#pragma unroll
            for (int i = 0; i < 16; ++i) v[i] = fmaf(q * kUnscale, v[i], row == c + i && row < p.m ? r * kScale : 0.0f);
            if (lin != 0.0f) {
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const int at = (c >> 6) * kFuseBlk + row * 128 + (((((c >> 3) & 7) + j) ^ (row & 7)) << 4);
                    const uint4 h = *reinterpret_cast<const uint4 *>(sh + at);
                    const uint4 l = *reinterpret_cast<const uint4 *>(sl + at);
                    const uint32_t hw[4] = {h.x, h.y, h.z, h.w}, lw[4] = {l.x, l.y, l.z, l.w};
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float2 s = join2(hw[i], lw[i]);
                        v[8 * j + 2 * i] = fmaf(lin, s.x, v[8 * j + 2 * i]);
                        v[8 * j + 2 * i + 1] = fmaf(lin, s.y, v[8 * j + 2 * i + 1]);
                    }
                }
            }
            put16(sh, sl, c, v);
        }
    };
#pragma unroll 1
    for (int k = 0; k < p.steps; ++k) {
        const FuseStep &t = p.step[k];
        multiply(xh, xl, xh, xl, false, scols, p.nb, kFuseM);
        symmetric(p.nb, t.gr, t.gq, 0.0f);
        if (t.poly) {
            multiply(sh, sl, sh, sl, false, scols, kbm, kFuseM);
            symmetric(kbm, t.pr, t.pq, t.plin);
        }
        multiply(sh, sl, xh, xl, true, xcols, kbm, kFuseN);
        if (k + 1 < p.steps) {
#pragma unroll 1
            for (int c = part * (xcols / 4); c < (part + 1) * (xcols / 4); c += 16) {
                float v[16];
                sum16(c, kbm, kFuseN, v);
#pragma unroll
                for (int i = 0; i < 16; ++i) v[i] *= kUnscale;
                put16(xh, xl, c, v);
            }
        }
    }
    // the last iterate to M's layout, 16 columns of this lane's row at a time
    const float lr = p.w ? *p.lr : 0.0f, keep = 1.0f - lr * p.decay;
    const float f = p.w ? -lr * p.factor * (kUnscale * kUnscale) : kUnscale * kUnscale;
    float *const o32 = p.w ? p.w + base : p.out_f32 ? static_cast<float *>(p.out) + base : nullptr;
    uint16_t *const o16 = p.w        ? (p.w_copy ? p.w_copy + base : nullptr)
                          : p.out_f32 ? nullptr
                                      : static_cast<uint16_t *>(p.out) + base;
    const int step = p.tall ? p.cols : 1;
#pragma unroll 1
    for (int c = part * (xcols / 4); c < (part + 1) * (xcols / 4); c += 16) {
        const int at = p.tall ? c * p.cols + row : row * p.cols + c;
        const int n = row < p.m ? min(16, p.n - c) : 0;
        float w[16], v[16];
        if (p.w) {
#pragma unroll
            for (int i = 0; i < 16; ++i) w[i] = i < n ? o32[at + i * step] : 0.0f;
        }
        sum16(c, kbm, kFuseN, v);
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            v[i] *= f;
            if (p.w) v[i] = fmaf(keep, w[i], v[i]);
            if (i < n) {
                if (o32) o32[at + i * step] = v[i];
                if (o16) reinterpret_cast<__nv_bfloat16 *>(o16)[at + i * step] = __float2bfloat16_rn(v[i]);
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 0) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

// -------------------------------------------------------------- host side --

inline size_t align256(size_t v) { return (v + 255) & ~(size_t)255; }

struct Layout {
    int m, n;
    int64_t ldx, lds;  // rows of the iterates and of S, C
    size_t part, x[2], s, c, bytes;
    Layout(int64_t B, int rows, int cols) {
        m = std::min(rows, cols);
        n = std::max(rows, cols);
        ldx = (n + 7) / 8 * 8;
        lds = (m + 7) / 8 * 8;
        const size_t xb = align256((size_t)(2 * B * m * ldx * 2)), sb = align256((size_t)(2 * B * m * lds * 2));
        part = 256;
        x[0] = part + align256((size_t)(B * kParts * 8));
        x[1] = x[0] + xb;
        s = x[1] + xb;
        c = s + sb;
        bytes = m <= kFuseM && n <= kFuseN ? 256 : c + sb;  // one CTA a matrix needs the status word only
    }
};

inline moe_status check_ns(int32_t B, int32_t rows, int32_t cols) {
    if (B < 0 || rows <= 0 || cols <= 0) return MOE_ERR_INVALID_ARG;
    if (rows > 65536 || cols > 65536 || B > 65535) return MOE_ERR_UNSUPPORTED;
    const int64_t mt = (rows + PM - 1) / PM, nt = (cols + PM - 1) / PM;
    if (B * mt * nt >= (int64_t)1 << 30) return MOE_ERR_UNSUPPORTED;
    return MOE_OK;
}

// One step's polynomial on singular values in [0, r]: the largest result, a little
// enlarged (1024 samples of a polynomial of degree 5; 2% and 1e-3 cover what lies
// between them), and whether it and the factor stay inside the pieces' range.
inline bool step_bound(double r, double a, double b, double c, double &next) {
    double most = 0.0, factor = 0.0;
    for (int i = 0; i <= 1024; ++i) {
        const double s = r * i / 1024, t = s * s, f = a + t * (b + c * t);
        factor = std::max(factor, std::fabs(f));
        most = std::max(most, std::fabs(s * f));
    }
    next = most * 1.02 + 1e-3;
    return factor <= 60.0 && most <= 7.5;
}

inline bool bounded(int steps, const float *coef) {
    double r = 1.001;
    for (int k = 0; k < steps; ++k)
        if (!step_bound(r, coef[3 * k], coef[3 * k + 1], coef[3 * k + 2], r)) return false;
    return true;
}

// A step's symmetric products: S' = gr I + gq X X^T, then, where there is a second one,
// C = pr I + pq S' S' + plin S'.  `most` is the bound of X's singular values, before and
// after.  The square is completed where the shift stays inside the pieces' range.
struct Products {
    double gr, gq, pr = 0.0, pq = 0.0, plin = 0.0;
    bool poly;
    Products(const float *coef, double &most) {
        const double a = coef[0], b = coef[1], c = coef[2];
        poly = c != 0.0;
        if (!poly) {
            gr = a;
            gq = b;
        } else {
            const double shift = b / (2 * c);
            // beyond four times S's size the squares' rounding would outgrow b S's
            const double size = std::max(1.0, most * most);
            const bool square = std::fabs(shift) <= std::min(8.0, 4.0 * size) && size + std::fabs(shift) < 60.0;
            gr = square ? shift : 0.0;
            gq = 1.0;
            pr = square ? a - b * b / (4 * c) : a;
            pq = c;
            plin = square ? 0.0 : b;
        }
        step_bound(most, a, b, c, most);
    }
};

constexpr float kDefault[3] = {3.4445f, -4.7750f, 2.0315f};

struct Update {  // NS_LAST
    void *out = nullptr;
    int out_f32 = 0;
    float *w = nullptr;
    uint16_t *w_copy = nullptr;
    const float *lr = nullptr;
    float decay = 0.0f, factor = 0.0f;
};

// Checks what both calls share; coef gets steps x 3 coefficients.
moe_status check_steps(int steps, const float *coefficients, float eps, float (&coef)[3 * MOE_NS_MAX_STEPS]) {
    if (steps < 1 || steps > MOE_NS_MAX_STEPS) return MOE_ERR_INVALID_ARG;
    if (!std::isfinite(eps) || eps < 1e-30f) return MOE_ERR_INVALID_ARG;
    for (int i = 0; i < 3 * steps; ++i) {
        coef[i] = coefficients ? coefficients[i] : kDefault[i % 3];
        if (!std::isfinite(coef[i])) return MOE_ERR_INVALID_ARG;
    }
    return bounded(steps, coef) ? MOE_OK : MOE_ERR_UNSUPPORTED;
}

template <int MODE>
moe_status launch_ns(const NsArgs &a, int columns, int64_t tiles, cudaStream_t st) {
    return columns == 128 ? launch<Ns<MODE, 128>>(a, tiles, st) : launch<Ns<MODE, 256>>(a, tiles, st);
}

template <int MODE, bool TALL>
moe_status launch_small(SmallNsArgs a, const uint16_t *pa, int64_t lda, int arows, int acols, const uint16_t *pb,
                        int64_t ldb, int brows, int bcols, cudaStream_t st) {
    constexpr bool kSym = MODE < NS_APPLY;
    constexpr bool a_mn = !kSym && !TALL, b_mn = !kSym && TALL;
    const int ft = (a.F + small::kM - 1) / small::kM;
    // as few tokens a tile as leave every tile an SM of its own (an MN-major operand
    // comes in blocks of 64)
    // (one tile of a symmetric product is best whole: it loads one operand)
    int n = 128;
    while (!(kSym && a.T <= small::kM) && n > (b_mn ? 64 : 32) && (int64_t)a.B * ft * ((a.T + n / 2 - 1) / (n / 2)) <= num_sms()) n /= 2;
    int tiles = ft;  // of a matrix and token tile, or of a triangle
    a.tt = (a.T + n - 1) / n;
    if (kSym && n == small::kM) {
        tiles = ft * (ft + 1) / 2;
        a.tt = 1;
    }
    a.split = small::split_for((int64_t)a.B * tiles * a.tt, a.nk, 1);
    const uint64_t planes = 2 * (uint64_t)a.B;
    if (!make_map_16(&a.a, pa, acols, arows, planes, lda, 64, a_mn ? 64 : small::kM) ||
        !make_map_16(&a.b, pb, bcols, brows, planes, ldb, 64, b_mn ? 64 : n))
        return MOE_ERR_CUDA;
    if constexpr (!b_mn)
        if (n == 32) return small::launch<SmallNs<MODE, TALL, 32>>(a, tiles, a.B, st);
    return n == 64 ? small::launch<SmallNs<MODE, TALL, 64>>(a, tiles, a.B, st)
                   : small::launch<SmallNs<MODE, TALL, 128>>(a, tiles, a.B, st);
}

template <bool MUON, typename TIN>
moe_status run(int B, int rows, int cols, const TIN *x, float *momentum, float mu, int nesterov, int steps,
               const float *coef, float eps, const Update &up, char *ws, cudaStream_t st) {
    const Layout at(B, rows, cols);
    const int m = at.m, n = at.n;
    const int tall = rows > cols;
    if (m <= kFuseM && n <= kFuseN) {
        FuseArgs a{};
        a.rows = rows;
        a.cols = cols;
        a.tall = tall;
        a.m = m;
        a.n = n;
        a.nb = (n + 63) / 64;
        a.steps = steps;
        a.eps = eps;
        a.x = x;
        a.momentum = momentum;
        a.mu = mu;
        a.nesterov = nesterov;
        a.out = up.out;
        a.out_f32 = up.out_f32;
        a.w = up.w;
        a.w_copy = up.w_copy;
        a.lr = up.lr;
        a.decay = up.decay;
        a.factor = up.factor;
        a.status = reinterpret_cast<int *>(ws);
        double most = 1.001;
        for (int k = 0; k < steps; ++k) {
            const Products t(coef + 3 * k, most);
            a.step[k] = FuseStep{(float)t.gr, (float)t.gq, (float)t.pr, (float)t.pq, (float)t.plin, t.poly};
        }
        static PerDeviceOnce attr;
        if (!device_once(attr, [] { return set_smem_limit(ns_fused<MUON, TIN>, fuse_smem(kFuseN / 64)); }))
            return MOE_ERR_CUDA;
        launch_pdl(ns_fused<MUON, TIN>, (unsigned)B, kFuseThreads, fuse_smem(a.nb), st, a);
        return launch_status();
    }
    uint16_t *xs[2] = {reinterpret_cast<uint16_t *>(ws + at.x[0]), reinterpret_cast<uint16_t *>(ws + at.x[1])};
    uint16_t *s = reinterpret_cast<uint16_t *>(ws + at.s), *c = reinterpret_cast<uint16_t *>(ws + at.c);
    NsArgs gram{}, poly{}, apply[2] = {};
    gram.B = B;
    gram.status = reinterpret_cast<int *>(ws);
    gram.m = gram.n = m;
    gram.k = n;
    gram.mt = (m + PM - 1) / PM;
    auto triangle = [&](int c) {  // tiles of c columns
        return (int64_t)B * (gram.mt * ((m + c - 1) / c) - gram.mt * (gram.mt - 1) / 2 * (PM / c));
    };
    const int sn = narrow(triangle(256), triangle(128)) ? 128 : 256;  // columns of the symmetric products' tiles
    gram.nt = (m + sn - 1) / sn;
    gram.lds = at.lds;
    poly = gram;
    poly.k = m;
    poly.s = s;
    apply[0] = gram;
    apply[0].n = n;
    apply[0].k = m;
    const int an = narrow((int64_t)B * gram.mt * ((n + 255) / 256), (int64_t)B * gram.mt * ((n + 127) / 128)) ? 128 : 256;
    apply[0].nt = (n + an - 1) / an;
    apply[0].rows = rows;
    apply[0].cols = cols;
    apply[0].tall = tall;
    apply[0].out = up.out;
    apply[0].out_f32 = up.out_f32;
    apply[0].w = up.w;
    apply[0].w_copy = up.w_copy;
    apply[0].lr = up.lr;
    apply[0].decay = up.decay;
    apply[0].factor = up.factor;
    apply[1] = apply[0];
    const uint64_t planes = 2 * (uint64_t)B;
    CUtensorMap xk[2], xb[2];  // X as the Gram product's two operands
    for (int i = 0; i < 2; ++i)
        if (!map_k(&xk[i], xs[i], n, m, planes, at.ldx) || !map_k(&xb[i], xs[i], n, m, planes, at.ldx, sn / 2) || !map_mn(&apply[i].b, xs[i], n, m, planes, at.ldx) ||
            !map_store(&apply[i].o, xs[1 - i], n, m, planes, at.ldx) || !map_k(&apply[i].a, c, m, m, planes, at.lds))
            return MOE_ERR_CUDA;
    CUtensorMap to_s, to_c;
    if (!map_store(&to_s, s, m, m, planes, at.lds) || !map_k(&poly.a, s, m, m, planes, at.lds) ||
        !map_k(&poly.b, s, m, m, planes, at.lds, sn / 2) || !map_store(&to_c, c, m, m, planes, at.lds))
        return MOE_ERR_CUDA;

    const int64_t elems = (int64_t)rows * cols;
    const int want = std::max(1, 8 * num_sms() / B);
    const int parts = (int)std::min<int64_t>(std::min(want, kParts), (elems + kNormThreads * 8 - 1) / (kNormThreads * 8));
    double *part = reinterpret_cast<double *>(ws + at.part);
    launch_pdl(ns_norm<MUON, TIN>, dim3(parts, B), kNormThreads, 0, st, elems, x, momentum, mu, nesterov, part);
    moe_status r = launch_status();
    if (r != MOE_OK) return r;
    launch_pdl(ns_split<MUON, TIN>,
               dim3((cols + kSplitTile - 1) / kSplitTile, (rows + kSplitTile - 1) / kSplitTile, B), 256, 0, st, rows,
               cols, tall, at.ldx, x, momentum, mu, nesterov, eps, part, parts, xs[0],
               xs[0] + (int64_t)B * m * at.ldx);
    if ((r = launch_status()) != MOE_OK) return r;
    const int64_t tri = triangle(sn), full = (int64_t)B * apply[0].mt * apply[0].nt;
    // Single SMs where one round of 128 x 128 tiles holds the products, and where m fits one
    // tile: half of a pair's rows would be padding (45 matrices of 1873 x 70: 375 us).
    const bool few = (m <= small::kM && (int64_t)B * ((n + 63) / 64) <= 65535) ||
                     (int64_t)B * ((m + small::kM - 1) / small::kM) * ((n + small::kM - 1) / small::kM) <= num_sms();
    SmallNsArgs sm{};
    sm.B = B;
    sm.status = gram.status;
    sm.out = up.out;
    sm.out_f32 = up.out_f32;
    sm.w = up.w;
    sm.w_copy = up.w_copy;
    sm.lr = up.lr;
    sm.decay = up.decay;
    sm.factor = up.factor;
    auto symmetric = [&](int mode, const uint16_t *in, int64_t ld, int k, uint16_t *o, double r0, double q,
                         double lin) -> moe_status {
        if (few) {
            SmallNsArgs a = sm;
            a.T = a.F = m;
            a.nk = (k + BK - 1) / BK;
            a.r = (float)r0;
            a.q = (float)q;
            a.lin = (float)lin;
            a.s = s;
            a.o = o;
            a.ld = at.lds;
            return mode == NS_GRAM     ? launch_small<NS_GRAM, false>(a, in, ld, m, k, in, ld, m, k, st)
                   : mode == NS_SQUARE ? launch_small<NS_SQUARE, false>(a, in, ld, m, k, in, ld, m, k, st)
                                       : launch_small<NS_POLY, false>(a, in, ld, m, k, in, ld, m, k, st);
        }
        NsArgs &a = mode == NS_GRAM ? gram : poly;
        a.r = (float)r0;
        a.q = (float)q;
        a.lin = (float)lin;
        a.o = o == s ? to_s : to_c;
        return mode == NS_GRAM     ? launch_ns<NS_GRAM>(a, sn, tri, st)
               : mode == NS_SQUARE ? launch_ns<NS_SQUARE>(a, sn, tri, st)
                                   : launch_ns<NS_POLY>(a, sn, tri, st);
    };
    double most = 1.001;  // of X's singular values
    for (int k = 0; k < steps; ++k) {
        const int cur = k & 1;
        const Products t(coef + 3 * k, most);
        gram.a = xk[cur];
        gram.b = xb[cur];
        r = symmetric(NS_GRAM, xs[cur], at.ldx, n, t.poly ? s : c, t.gr, t.gq, 0.0);
        if (r == MOE_OK && t.poly)
            r = symmetric(t.plin == 0.0 ? NS_SQUARE : NS_POLY, s, at.lds, m, c, t.pr, t.pq, t.plin);
        if (r != MOE_OK) return r;
        const bool last = k + 1 == steps;
        if (few) {
            SmallNsArgs a = sm;
            a.nk = (m + BK - 1) / BK;
            a.T = last && tall ? n : m;
            a.F = last && tall ? m : n;
            a.o = xs[1 - cur];
            a.ld = at.ldx;
            r = !last  ? launch_small<NS_APPLY, false>(a, xs[cur], at.ldx, m, n, c, at.lds, m, m, st)
                : tall ? launch_small<NS_LAST, true>(a, c, at.lds, m, m, xs[cur], at.ldx, m, n, st)
                       : launch_small<NS_LAST, false>(a, xs[cur], at.ldx, m, n, c, at.lds, m, m, st);
        } else {
            r = last ? launch_ns<NS_LAST>(apply[cur], an, full, st) : launch_ns<NS_APPLY>(apply[cur], an, full, st);
        }
        if (r != MOE_OK) return r;
    }
    return MOE_OK;
}

inline bool aligned(const void *p, size_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

}  // namespace
}  // namespace moe

using namespace moe;

MOE_API size_t moe_newton_schulz_workspace_bytes(int32_t B, int32_t rows, int32_t cols) {
    if (check_ns(B, rows, cols) != MOE_OK) return 0;
    return Layout(B, rows, cols).bytes;
}

MOE_API moe_status moe_newton_schulz(int32_t B, int32_t rows, int32_t cols, int32_t x_dtype, const void *x,
                                     int32_t out_dtype, void *out, int32_t steps, const float *coefficients,
                                     float eps, void *ws, size_t ws_bytes, cudaStream_t stream) {
    moe_status r = check_ns(B, rows, cols);
    if (r != MOE_OK) return r;
    if ((x_dtype != MOE_BF16 && x_dtype != MOE_FP32) || (out_dtype != MOE_BF16 && out_dtype != MOE_FP32))
        return MOE_ERR_INVALID_ARG;
    float coef[3 * MOE_NS_MAX_STEPS];
    if ((r = check_steps(steps, coefficients, eps, coef)) != MOE_OK) return r;
    if (!ws || ws_bytes < Layout(B, rows, cols).bytes || !aligned(ws, 256)) return MOE_ERR_WORKSPACE;
    if (B == 0) return MOE_OK;
    if (!x || !out || (x == out && x_dtype != out_dtype)) return MOE_ERR_INVALID_ARG;
    if (!aligned(x, x_dtype == MOE_FP32 ? 4 : 2) || !aligned(out, out_dtype == MOE_FP32 ? 4 : 2))
        return MOE_ERR_ALIGNMENT;
    Update up;
    up.out = out;
    up.out_f32 = out_dtype == MOE_FP32;
    if (x_dtype == MOE_FP32)
        return run<false>(B, rows, cols, static_cast<const float *>(x), nullptr, 0.0f, 0, steps, coef, eps, up,
                          static_cast<char *>(ws), stream);
    return run<false>(B, rows, cols, static_cast<const uint16_t *>(x), nullptr, 0.0f, 0, steps, coef, eps, up,
                      static_cast<char *>(ws), stream);
}

MOE_API moe_status moe_muon_step(int32_t B, int32_t rows, int32_t cols, float *w, moe_bf16 *w_copy,
                                 float *momentum, const float *grad, const float *lr, float mu,
                                 float weight_decay, float scale, int32_t nesterov, int32_t steps,
                                 const float *coefficients, float eps, void *ws, size_t ws_bytes,
                                 cudaStream_t stream) {
    moe_status r = check_ns(B, rows, cols);
    if (r != MOE_OK) return r;
    if (!std::isfinite(mu) || !std::isfinite(weight_decay) || !std::isfinite(scale)) return MOE_ERR_INVALID_ARG;
    float coef[3 * MOE_NS_MAX_STEPS];
    if ((r = check_steps(steps, coefficients, eps, coef)) != MOE_OK) return r;
    if (!ws || ws_bytes < Layout(B, rows, cols).bytes || !aligned(ws, 256)) return MOE_ERR_WORKSPACE;
    if (B == 0) return MOE_OK;
    if (!w || !momentum || !grad || !lr) return MOE_ERR_INVALID_ARG;
    if (w == momentum || w == grad || momentum == grad || lr == w || lr == momentum ||
        (const void *)w_copy == (const void *)w || (const void *)w_copy == (const void *)momentum ||
        (const void *)w_copy == (const void *)grad)
        return MOE_ERR_INVALID_ARG;
    if (!aligned(w, 4) || !aligned(momentum, 4) || !aligned(grad, 4) || !aligned(lr, 4) || !aligned(w_copy, 2))
        return MOE_ERR_ALIGNMENT;
    Update up;
    up.w = w;
    up.w_copy = reinterpret_cast<uint16_t *>(w_copy);
    up.lr = lr;
    up.decay = weight_decay;
    up.factor = scale;
    return run<true>(B, rows, cols, grad, momentum, mu, nesterov != 0, steps, coef, eps, up, static_cast<char *>(ws),
                     stream);
}

// ns.cuh - orthogonalisation of expert weight updates by Newton-Schulz
// products: for every matrix G of a batch, with m = min and n = max of its
// two sizes and X (m, n) = G or G^T,
//
//   X0 = G / (|G|_F + eps);   A = X X^T;   B = b A + c A A;   X <- a X + B X
//
// for a few steps with given (a, b, c), which drives the singular values of X
// towards one.
//
// Numerics. The products run on the fp16 tensor cores with fp32 accumulators:
// the values are bounded (singular values stay near one), so fp16's 11-bit
// significand costs nothing in range and is eight times finer than bf16's. Two
// things keep what fp16 rounds away below what rounding the result to bf16
// costs (1.7e-3 of the norm; all errors below are without that):
//   - X is held as hi + lo, two fp16 words (22 bits): the products read hi, the
//     term a X adds both. With hi alone the rounding of X is multiplied by a =
//     3.4 in every later step wherever a singular value is small: 9e-3 on a
//     matrix whose singular values fall to 1e-4.
//   - The diagonals of A and B stay in fp32. X comes near to orthogonal, so A
//     is near to a multiple of the identity, and the diagonal is where most of
//     its rounding error would be. With A = A' + diag(alpha), A' rounded once,
//       B = B' + diag(beta),  beta = b alpha + c alpha^2 + c (A' A')_rr,
//       B'_rs = c (A' A')_rs + (b + c (alpha_r + alpha_s)) A'_rs  off the diagonal
//     and X <- (a + beta_r) X + B' X, row by row. On random 64 x 1000 matrices
//     1.9e-3 falls to 2.5e-4, on 512 x 512 ones 1.5e-3 to 7e-4.
// Scales are powers of two: X 2^8 (a random 2048 x 7168 matrix starts with
// elements near 2^-12, fp16's normal range ends at 2^-14), lo 2^11 on top of
// X's, A' 2^10, B' 2^10 or as much less as the step's coefficients ask for.
// With singular values s <= 4 the elements of A are at most 16, but those of B
// up to the largest |b s^2 + c s^4|: 444 for the usual coefficients at s = 4,
// while 2^10 B' ends at 64. The host bounds s from step to step (s <= 1 at the
// start) and with it B. The smaller scale costs what small elements lose below
// fp16's normal range: an absolute error of B (at most 2^-27), beside the a of
// order one that it is added to.
//
// For the products a matrix is kept by rows alone, and read by rows or by columns
// (K-major or MN-major) as a product needs it. A = X X^T takes X by rows twice,
// B X takes X by columns: X^T is never written. X is held twice so, since the
// tiles of B X read what others replace. A and A A are symmetric: computed on
// and below the diagonal of 256 x 256 blocks, and a block of K above the
// diagonal is read by columns from below. Writing X^T as well took 253 us in
// place of 240 at (5, 1409, 577), 453 of 415 at (16, 512, 2048); writing both
// halves of A and B 199 in place of 189 at (2, 1024, 1024).
//
// Epilogue. A lane holds one row of the accumulator, so what it writes along
// the row lands in 32 different lines per store. What the epilogue reads itself,
// X as hi and lo and A for the next product, it keeps apart, in chunks of 32 x 32
// elements in the order in which the warp holds them, 16 bytes per lane and
// access, padded to whole chunks so that nothing is predicated; what the products
// read goes through shared memory and a TMA store. So hi and A are written twice,
// and a workspace holds four arrays of X's size (two by rows, hi, lo). Row-wise
// 16-byte accesses to one copy kept the load/store unit busy for 16 K cycles a
// tile against 8 K of MMAs, 2-byte accesses down the columns cost 1.6 us a chunk.
//
// Kernel: the CTA-pair pipeline of gemm2.cuh (tcgen05.mma.cta_group::2, one
// 256 x 256 tile per pair of SMs, six 32 KB stages of 64 fp16 columns, two
// accumulators in TMEM); warps 0-7 epilogue (a warp takes 32 lanes and half
// of the columns), warp 8 TMA, warp 9 MMA and TMEM. Both CTAs' loads count on
// the leader's barrier (TMA loads of cta_group::2), which its MMA thread waits
// on. Edges are filled with zeros by TMA (every matrix is its own plane of a
// rank-3 map) and cut off by the epilogue. At (4, 2048, 7168) A takes 100 us at
// 1.54 GHz, 1.35 PFLOP/s, 81 % of the tensor pipe, bound by power; B X 216 us, 1.11
// PFLOP/s (read and write of X beside the products); A A 39 us in two rounds of
// tiles. Small products are bound by their latency, 5 to 7 us a launch.
#pragma once

#include <type_traits>

#include <cuda_fp16.h>

#include "gemm2.cuh"

namespace mxq {
namespace ns {

constexpr int HALF = 128;              // rows of one CTA
constexpr int TILE = 2 * HALF;         // rows of a pair's tile; it has TN columns
constexpr int BK = 64;                 // fp16 elements per 128-byte row
constexpr int OP_BYTES = HALF * 128;   // row operand, one stage, one CTA
constexpr int EPI_WARPS = 8;
constexpr int THREADS = (EPI_WARPS + 2) * 32;
constexpr int ACC = 2;
constexpr int CHUNK = 32;              // an epilogue step: 32 rows x 32 columns per warp
constexpr int CHUNK_BYTES = CHUNK * CHUNK * 2;
constexpr int MAX_PARTS = 256;         // partial sums of squares per matrix

constexpr float SX = 256.0f;           // stored X  = X 2^8
constexpr float SA = 1024.0f;          // stored A' = A' 2^10, and B' unless its range asks for less
constexpr float SLO = 2048.0f;         // stored lo = (X 2^8 - hi) 2^11

template <int TN> struct __align__(1024) Smem {
    static constexpr int STAGES = TN == 256 ? 6 : (TN == 128 ? 8 : 9); // what 227 KB hold
    static constexpr int Q_BYTES = TN / 2 * 128; // column operand, one stage, one CTA
    uint8_t a[STAGES][OP_BYTES];
    uint8_t b[STAGES][Q_BYTES];
    uint8_t stage[EPI_WARPS][2][CHUNK_BYTES]; // row-major chunks on their way out
    uint64_t full[STAGES];  // the leader's: both CTAs' loads
    uint64_t empty[STAGES];
    uint64_t acc_full[ACC];
    uint64_t acc_empty[ACC];
    uint64_t mma_done;
    uint32_t tmem_base;
    int abort_flag;
};
template <int TN> constexpr size_t smem_bytes() { return sizeof(Smem<TN>) + 1024; }

// fp32 accumulator, f16 x f16, N = TN, M 256 (the pair)
template <int TN> constexpr uint32_t idesc()
{
    return (1u << 4) | ((uint32_t)(TN >> 3) << 17) | ((uint32_t)(TILE >> 4) << 24);
}

enum Mode { GRAM = 0, POLY = 1, STEP = 2, LAST = 3 };

struct Args {
    int E, m, n;          // batch, X is (m, n)
    float a, b, c;
    float pb, pc;         // b and c times the scale of B' over that of A'
    float unscale;        // one over the scale of B'
    uint16_t *hi, *lo;    // X as the epilogue keeps it: chunks of (m, n)
    uint16_t *a_own;      // A' as the epilogue keeps it: chunks of (m, m)
    float *alpha, *beta;  // (E, m): the diagonals of A and B
    uint16_t *out;        // LAST: bf16, (E, m, n) or, transposed, (E, n, m)
    int out_t, out_vec;
};

// An operand read by columns (MN-major): K runs down its rows, which lie W = 64
// or 128 bytes apart with the W-byte swizzle, eight rows a group; blocks of
// W / 2 columns follow at `block` bytes. The instruction is told by a bit.
template <int W> MXQ_DEV uint64_t smem_desc_columns(uint32_t addr, uint32_t block)
{
    return (uint64_t)((addr >> 4) & 0x3FFFu) | (uint64_t)(block >> 4) << 16 | (uint64_t(8 * W) >> 4) << 32 |
           (uint64_t(1) << 46) | (uint64_t(W == 128 ? 2 : 4) << 61);
}
constexpr uint32_t IDESC_A_COLUMNS = 1u << 15, IDESC_B_COLUMNS = 1u << 16;

template <uint32_t IDESC>
MXQ_DEV void mma_pair_f16(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t accumulate)
{
    asm volatile("{\n\t.reg .pred p;\n\t"
                 "setp.ne.b32 p, %3, 0;\n\t"
                 "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %4, p;\n\t}" ::"r"(d_tmem),
                 "l"(adesc), "l"(bdesc), "r"(accumulate), "r"(IDESC)
                 : "memory");
}

// chunks of 32 along `len`, and the first element of a chunk in the epilogue's
// own arrays: piece g (8 columns) of lane l follows at g * 256 + l * 8
__host__ __device__ constexpr int64_t chunks_of(int64_t len) { return (len + CHUNK - 1) / CHUNK; }
MXQ_DEV int64_t chunk_at(int e, int m, int n, int r0, int c0)
{
    return (((int64_t)e * chunks_of(m) + r0 / CHUNK) * chunks_of(n) + c0 / CHUNK) * (CHUNK * CHUNK);
}

// TMA load into this CTA's shared memory that counts on a barrier of the
// pair's leader (a shared::cluster address)
MXQ_DEV void load_pair(void *dst, const CUtensorMap *map, uint32_t bar, int x, int y, int z)
{
    asm volatile("cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2"
                 " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(smem_u32(dst)),
                 "l"(map), "r"(x), "r"(y), "r"(z), "r"(bar)
                 : "memory");
}

// a stage's operand of N rows or columns and 64 of K, by rows or by columns (in
// blocks of W bytes)
template <int N, int W, bool COLUMNS>
MXQ_DEV void load_operand(uint8_t *dst, const CUtensorMap *rows, const CUtensorMap *columns, uint32_t bar, int first,
                          int k, int e)
{
    if constexpr (COLUMNS) {
#pragma unroll
        for (int c = 0; c < N; c += W / 2)
            load_pair(dst + c * 2 * BK, columns, bar, first + c, k, e);
    } else {
        load_pair(dst, rows, bar, k, first, e);
    }
}

MXQ_DEV void prefetch_map(const CUtensorMap *map)
{
    asm volatile("prefetch.tensormap [%0];" ::"l"(map) : "memory");
}

MXQ_DEV uint32_t pack_half2(float lo, float hi)
{
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
MXQ_DEV uint32_t word_of(const uint4 &v, int i) { return i == 0 ? v.x : (i == 1 ? v.y : (i == 2 ? v.z : v.w)); }
MXQ_DEV float2 unpack_half2(uint32_t w) { return __half22float2(*reinterpret_cast<__half2 *>(&w)); }

// A warp's 32 x 32 chunk of 16-bit values, one row per lane (two columns per
// word), to shared memory: rows of 64 bytes, 16-byte pieces swizzled by the
// row as the 64-byte TMA swizzle does, so that no two lanes' stores share banks
MXQ_DEV void chunk_to_smem(uint8_t *st, const uint32_t (&h)[16])
{
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int g = 0; g < 4; ++g)
        sts_v4(smem_u32(st) + (uint32_t)(lane * 64 + ((g ^ ((lane >> 1) & 3)) << 4)),
               make_uint4(h[4 * g], h[4 * g + 1], h[4 * g + 2], h[4 * g + 3]));
}

// The chunk to rows of a row-major matrix (dst: its first element, n per row;
// `rows` and `cols` of it exist) through shared memory, so that a store covers
// whole lines: eight rows of four 16-byte pieces at a time with `vec`, else a
// row at a time, one element per lane.
MXQ_DEV void rows_out(uint8_t *st, const uint32_t (&h)[16], uint16_t *dst, int64_t n, int rows, int cols, int vec)
{
    const int lane = threadIdx.x & 31;
    chunk_to_smem(st, h);
    __syncwarp();
    if (vec && cols >= CHUNK) {
        const int g = lane & 3;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int y = 8 * i + (lane >> 2);
            const uint4 x = *reinterpret_cast<const uint4 *>(st + y * 64 + ((g ^ ((y >> 1) & 3)) << 4));
            if (y < rows)
                st_v4(dst + y * n + 8 * g, x.x, x.y, x.z, x.w);
        }
    } else if (lane < cols) {
#pragma unroll 8
        for (int y = 0; y < 32; ++y)
            if (y < rows)
                dst[y * n + lane] =
                    *reinterpret_cast<const uint16_t *>(st + y * 64 + (((lane >> 3) ^ ((y >> 1) & 3)) << 4) + (lane & 7) * 2);
    }
    __syncwarp();
}

// two neighbouring elements; `pair`: as one aligned word
MXQ_DEV float2 in_pair(const uint16_t *p, bool pair, bool second)
{
    if (pair) {
        const uint32_t w = *reinterpret_cast<const uint32_t *>(p);
        return make_float2(bf16_lo(w), bf16_hi(w));
    }
    return make_float2(__uint_as_float((uint32_t)p[0] << 16), second ? __uint_as_float((uint32_t)p[1] << 16) : 0.0f);
}
MXQ_DEV float2 in_pair(const float *p, bool pair, bool second)
{
    if (pair)
        return *reinterpret_cast<const float2 *>(p);
    return make_float2(p[0], second ? p[1] : 0.0f);
}

// the elements of one aligned 16-byte vector, eight (the last four zero for
// fp32)
MXQ_DEV void in_vec(const uint4 x, const uint16_t *, float (&v)[8])
{
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[2 * i] = bf16_lo(w[i]);
        v[2 * i + 1] = bf16_hi(w[i]);
    }
}
MXQ_DEV void in_vec(const uint4 x, const float *, float (&v)[8])
{
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[i] = __uint_as_float(w[i]);
        v[4 + i] = 0.0f;
    }
}

// Sum of squares of a slice of matrix blockIdx.y. Eight squares at a time are
// added in fp32 and the sums in fp64; where the eight leave the range in which
// fp32 squares are sound (values near 1e-18 or 1e19 and beyond) they are
// squared in fp64. `vec`: every matrix is whole 16-byte vectors. 77 us at (16,
// 2048, 7168) bf16, 0.94 of the measured copy rate.
template <typename T>
__global__ void __launch_bounds__(256)
    k_ns_sumsq(const T *__restrict__ g, int64_t size, int vec, double *__restrict__ part)
{
    constexpr int V = 16 / sizeof(T);
    let_next_kernel_start();
    const T *p = g + (int64_t)blockIdx.y * size;
    const int64_t per = ((size + gridDim.x - 1) / gridDim.x + 7) & ~int64_t(7);
    const int64_t lo = blockIdx.x * per, hi = lo + per < size ? lo + per : size;
    double t = 0.0;
    auto add = [&](const float (&v)[8]) {
        float s = 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i)
            s = fmaf(v[i], v[i], s);
        if (s > 0x1p-90f && s < 0x1p120f) {
            t += (double)s;
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                t = fma((double)v[i], (double)v[i], t);
        }
    };
    if (vec) {
        for (int64_t i = lo + V * threadIdx.x; i < hi; i += 4 * V * 256) {
            uint4 x[4];
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                x[u] = make_uint4(0u, 0u, 0u, 0u);
                if (i + u * V * 256 < hi)
                    x[u] = ld_stream_v4(p + i + u * V * 256);
            }
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                float v[8];
                in_vec(x[u], p, v);
                add(v);
            }
        }
    } else {
        for (int64_t i = lo + threadIdx.x; i < hi; i += 8 * 256) {
            float v[8];
#pragma unroll
            for (int u = 0; u < 8; ++u)
                v[u] = i + u * 256 < hi ? in_pair(p + i + u * 256, false, false).x : 0.0f;
            add(v);
        }
    }
    __shared__ double w[8];
#pragma unroll
    for (int o = 16; o; o >>= 1)
        t += __shfl_xor_sync(0xffffffffu, t, o);
    if ((threadIdx.x & 31) == 0)
        w[threadIdx.x >> 5] = t;
    __syncthreads();
    if (threadIdx.x == 0) {
        for (int i = 1; i < 8; ++i)
            t += w[i];
        part[(size_t)blockIdx.y * gridDim.x + blockIdx.x] = t;
    }
}

// 2^8 / norm as two fp32 factors, to be multiplied one after the other: either
// alone may leave fp32's range, an element times the first does not where it
// matters. A norm of zero gives zeros, NaN gives NaN.
MXQ_DEV void scale_factors(double norm, float &f0, float &f1)
{
    const double inv = norm > 0.0 ? (double)SX / norm : (norm == 0.0 ? 0.0 : norm);
    int ex = 0;
    const double fr = frexp(inv, &ex);
    const bool plain = inv == 0.0 || !(norm > 0.0) || isinf(norm);
    f0 = plain ? 1.0f : (float)ldexp(1.0, ex / 2);
    f1 = plain ? (float)inv : (float)ldexp(fr, ex - ex / 2);
}

// X0 from G (rows, cols) in 64 x 64 tiles. X is G, or with `tall` G^T: the
// tile as it is read, or its transpose, goes to X, and both halves to the
// epilogue's chunks. A thread moves pairs of neighbours. 380 us at (16, 2048,
// 7168) bf16, 1.9 GB (288 at the copy rate): loads, then stores, so residency
// counts, and eight CTAs per SM, with 48 to 60 bytes of spills a thread, took 495
// us where six took 585 (with X^T). No __restrict__ on part: it is written while
// this kernel already runs.
template <typename T>
__global__ void __launch_bounds__(256, 8)
    k_ns_init(const T *__restrict__ g, int rows, int cols, int pair, const double *part, int parts,
              double eps, int tall, uint16_t *__restrict__ xh, int ldx, uint16_t *__restrict__ hi,
              uint16_t *__restrict__ lo)
{
    __shared__ uint32_t tile[64][65];
    __shared__ float s_f[2];
    const int e = blockIdx.z, r0 = blockIdx.y * 64, c0 = blockIdx.x * 64;
    let_next_kernel_start();
    wait_for_previous_kernel();
    const T *p = g + (int64_t)e * rows * cols;
    const int64_t base_x = (int64_t)e * (tall ? cols : rows) * ldx;
    const int tx = 2 * (threadIdx.x & 31), ty = threadIdx.x >> 5;
    float2 v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int R = r0 + ty + 8 * i, C = c0 + tx;
        v[i] = R < rows && C < cols ? in_pair(p + (int64_t)R * cols + C, pair != 0, C + 1 < cols)
                                    : make_float2(0.0f, 0.0f);
    }
    if (threadIdx.x < 32) { // the norm, while the tile is on its way
        double s = 0.0;
        for (int i = threadIdx.x; i < parts; i += 32)
            s += part[(size_t)e * parts + i];
#pragma unroll
        for (int o = 16; o; o >>= 1)
            s += __shfl_xor_sync(0xffffffffu, s, o);
        if (threadIdx.x == 0) {
            scale_factors(sqrt(s) + eps, s_f[0], s_f[1]);
        }
    }
    __syncthreads();
    const float f0 = s_f[0], f1 = s_f[1];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int r = ty + 8 * i, R = r0 + r, C = c0 + tx;
        const float x = (v[i].x * f0) * f1, y = (v[i].y * f0) * f1;
        const uint32_t h = pack_half2(x, y);
        const float2 f = unpack_half2(h);
        const uint32_t l = pack_half2((x - f.x) * SLO, (y - f.y) * SLO);
        const uint32_t w0 = __byte_perm(h, l, 0x5410), w1 = __byte_perm(h, l, 0x7632);
        tile[r][tx] = w0;
        tile[r][tx + 1] = w1;
        if (!tall && R < rows && C < cols) // X's rows are padded to pairs
            *reinterpret_cast<uint32_t *>(xh + base_x + (int64_t)R * ldx + C) = h;
    }
    __syncthreads();
    if (tall) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int c = ty + 8 * i, C = c0 + c, R = r0 + tx;
            if (R < rows && C < cols)
                *reinterpret_cast<uint32_t *>(xh + base_x + (int64_t)C * ldx + R) =
                    __byte_perm(tile[tx][c], tile[tx + 1][c], 0x5410);
        }
    }
    // a warp per chunk and pair of pieces
    const int m = tall ? cols : rows, n = tall ? rows : cols;
    const int lane = threadIdx.x & 31, chunk = threadIdx.x >> 6, half = threadIdx.x >> 5 & 1;
    const int y = CHUNK * (chunk >> 1), x = CHUNK * (chunk & 1); // in the tile, along X's rows and columns
    const int xr = (tall ? c0 : r0) + y, xc = (tall ? r0 : c0) + x;
    if (xr < m && xc < n) {
        const int64_t at = chunk_at(e, m, n, xr, xc) + lane * 8;
#pragma unroll
        for (int g = 2 * half; g < 2 * half + 2; ++g) {
            uint32_t w[8], a[4], b[4];
#pragma unroll
            for (int i = 0; i < 8; ++i)
                w[i] = tall ? tile[x + 8 * g + i][y + lane] : tile[y + lane][x + 8 * g + i];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                a[i] = __byte_perm(w[2 * i], w[2 * i + 1], 0x5410);
                b[i] = __byte_perm(w[2 * i], w[2 * i + 1], 0x7632);
            }
            st_v4(hi + at + g * 256, a[0], a[1], a[2], a[3]);
            st_v4(lo + at + g * 256, b[0], b[1], b[2], b[3]);
        }
    }
}

// tiles of one matrix: row tile i of a symmetric product has the columns up to
// its diagonal block's end, of the others all
template <bool SYM, int TN> __host__ __device__ inline int64_t sym_or_all_tiles(int m, int n)
{
    const int64_t tm = (m + TILE - 1) / TILE, tn = ((SYM ? m : n) + TN - 1) / TN;
    if (!SYM)
        return tm * tn;
    // all but the last row tile end within the matrix
    return (TILE / TN) * (tm * (tm - 1) / 2) + tn;
}

// D = P Q^T (GRAM, POLY) or P Q (STEP, LAST) over K = 64 nkb for every matrix,
// with the epilogue of MODE. Maps of P and Q by rows (boxes of 128 and TN / 2
// rows) and by columns (64 rows and 64 columns, for Q and TN 64 32 columns with
// the 64-byte swizzle), of the result's row-major copy (X, A or B) in boxes of
// 32 x 32 with the 64-byte swizzle, unused by LAST. Grid: an even number of
// CTAs in clusters of two.
template <int MODE, int TN>
__global__ void __launch_bounds__(THREADS, 1)
    k_ns_gemm(const __grid_constant__ CUtensorMap tm_p, const __grid_constant__ CUtensorMap tm_pc,
              const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_qc,
              const __grid_constant__ CUtensorMap tm_o, const Args q, int nkb, uint64_t wait_ns)
{
    constexpr bool SYM = MODE == GRAM || MODE == POLY;
    constexpr int QW = TN == 64 ? 64 : 128; // bytes of a row of Q read by columns, in shared memory
    constexpr int STAGES = Smem<TN>::STAGES;
    constexpr int TMEM_COLS = ACC * TN;
    constexpr int RATIO = TILE / TN; // column tiles per row tile
    extern __shared__ uint8_t smem_raw[];
    Smem<TN> &sm = *reinterpret_cast<Smem<TN> *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = g2::cta_rank();
    const bool leader = rank == 0;

    let_next_kernel_start();
    if (threadIdx.x == 0) {
        prefetch_map(&tm_p);
        if (MODE != GRAM)
            prefetch_map(&tm_pc);
        if (SYM)
            prefetch_map(&tm_q);
        if (MODE != GRAM)
            prefetch_map(&tm_qc);
        if (MODE != LAST)
            prefetch_map(&tm_o);
        for (int s = 0; s < STAGES; ++s) {
            mbar_init(&sm.full[s], 1);
            mbar_init(&sm.empty[s], 1);
        }
        for (int i = 0; i < ACC; ++i) {
            mbar_init(&sm.acc_full[i], 1);
            mbar_init(&sm.acc_empty[i], 2 * EPI_WARPS);
        }
        mbar_init(&sm.mma_done, 1);
        sm.abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == EPI_WARPS + 1) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&sm.tmem_base)),
                     "r"(TMEM_COLS)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    }
    gm::tc_fence_before();
    g2::cluster_sync(); // barriers initialised and TMEM allocated in both CTAs
    gm::tc_fence_after();
    const uint32_t tmem = sm.tmem_base;
    wait_for_previous_kernel();

    const int64_t pair = blockIdx.x >> 1, npairs = gridDim.x >> 1;
    const int tm = (q.m + TILE - 1) / TILE, tn = ((SYM ? q.m : q.n) + TN - 1) / TN;
    const int64_t per = sym_or_all_tiles<SYM, TN>(q.m, q.n);
    const int64_t total = per * q.E;
    // tile t of a matrix: row tile i, column tile j; symmetric products take
    // the column tiles up to the diagonal's, the others run down the row tiles
    // first, so that the pairs at work share a column tile of X and all of B
    struct Item {
        int e, i, j;
    };
    auto item = [&](int64_t it) {
        Item w;
        w.e = (int)(it / per);
        int t = (int)(it - (int64_t)w.e * per);
        if (SYM) {
            w.i = 0;
            for (int c = min(RATIO, tn); t >= c; c = min(RATIO * (w.i + 1), tn)) {
                t -= c;
                ++w.i;
            }
            w.j = t;
        } else {
            w.j = t / tm;
            w.i = t - w.j * tm;
        }
        return w;
    };

    // the first of K's blocks for which P and Q are read by columns: a
    // symmetric operand behind the diagonal block of the tile's rows (P) or
    // columns (Q), X in B X always
    auto p_turn = [&](const Item &w) { return MODE == GRAM ? nkb : (w.i + 1) * (TILE / BK); };
    auto q_turn = [&](const Item &w) {
        return MODE == GRAM ? nkb : (MODE == POLY ? (w.j / RATIO + 1) * (TILE / BK) : 0);
    };

    if (warp == EPI_WARPS) {
        // ------------------------------------------------ TMA producer (both CTAs)
        if (lane == 0) {
            const uint32_t leader_full0 = g2::peer_addr(&sm.full[0], 0);
            int s = 0, filled = 0; // the next stage, stages filled so far (up to STAGES)
            uint32_t ph = 1;       // of the wait for it: passes at once in the first round
            for (int64_t it = pair; it < total && !gm::aborted(&sm.abort_flag); it += npairs) {
                const Item w = item(it);
                const int turn_p = p_turn(w), turn_q = q_turn(w);
                const int p0 = w.i * TILE + (int)rank * HALF, q0 = w.j * TN + (int)rank * (TN / 2);
                int kb = 0;
                bool ok = true;
                auto fill = [&](auto p_columns, auto q_columns) {
                    if (!mbar_wait(&sm.empty[s], ph, wait_ns)) {
                        *reinterpret_cast<volatile int *>(&sm.abort_flag) = 1;
                        ok = false;
                        return;
                    }
                    if (leader)
                        mbar_arrive_expect_tx(&sm.full[s], 2 * (OP_BYTES + Smem<TN>::Q_BYTES));
                    const uint32_t bar = leader_full0 + (uint32_t)(s * sizeof(uint64_t));
                    load_operand<HALF, 128, decltype(p_columns)::value>(sm.a[s], &tm_p, &tm_pc, bar, p0, kb * BK, w.e);
                    load_operand<TN / 2, QW, decltype(q_columns)::value>(sm.b[s], &tm_q, &tm_qc, bar, q0, kb * BK, w.e);
                    ++kb;
                    filled = min(filled + 1, STAGES);
                    ph ^= s + 1 == STAGES;
                    s = s + 1 == STAGES ? 0 : s + 1;
                };
                // a branch per block in place of these loops cost B X 10 %
                while (ok && kb < min(turn_q, nkb))
                    fill(std::false_type{}, std::false_type{});
                while (MODE != GRAM && ok && kb < min(turn_p, nkb)) // turn_q <= turn_p
                    fill(std::false_type{}, std::true_type{});
                while (MODE != GRAM && ok && kb < nkb)
                    fill(std::true_type{}, std::true_type{});
            }
            // drain: every issued fill, of both CTAs, has landed before the
            // leader goes to the closing barrier; the stages before s were
            // filled in this round (phase ph ^ 1), the others in the last
            if (leader)
                for (int j = 0; j < STAGES; ++j)
                    if (j < s || filled == STAGES)
                        mbar_wait(&sm.full[j], j < s ? ph ^ 1u : ph, wait_ns);
        }
    } else if (warp == EPI_WARPS + 1) {
        // ------------------------------------------------ leader: the pair's MMAs (one thread)
        if (leader && lane == 0) {
            int t = 0, s = 0;
            uint32_t ph = 0;
            bool issued = false;
            for (int64_t it = pair; it < total && !gm::aborted(&sm.abort_flag); it += npairs, ++t) {
                const int acc = t & 1;
                if (t >= ACC && !mbar_wait(&sm.acc_empty[acc], ((uint32_t)(t / ACC) & 1u) ^ 1u, wait_ns)) {
                    *reinterpret_cast<volatile int *>(&sm.abort_flag) = 1;
                    break;
                }
                gm::tc_fence_after();
                const uint32_t d = tmem + (uint32_t)(acc * TN);
                const Item w = item(it);
                const int turn_p = p_turn(w), turn_q = q_turn(w);
                bool ok = mbar_wait(&sm.full[s], ph, wait_ns);
                // one block of K; the next slot is waited on before this slot's
                // last MMA, so that the wait overlaps MMAs already in the pipe
                auto block = [&](int kb, auto p_columns, auto q_columns) {
                    constexpr bool PC = decltype(p_columns)::value, QC = decltype(q_columns)::value;
                    constexpr uint32_t ID = idesc<TN>() | (PC ? IDESC_A_COLUMNS : 0u) | (QC ? IDESC_B_COLUMNS : 0u);
                    constexpr int P_STEP = PC ? 128 : 2, Q_STEP = QC ? QW : 2; // 16 of K: 16 rows, or 32 bytes of a row
                    gm::tc_fence_after();
                    const uint32_t pa = smem_u32(sm.a[s]), qa = smem_u32(sm.b[s]);
                    const uint64_t ad = PC ? smem_desc_columns<128>(pa, 128 * BK) : gm::smem_desc_k128(pa);
                    const uint64_t bd = QC ? smem_desc_columns<QW>(qa, QW * BK) : gm::smem_desc_k128(qa);
#pragma unroll
                    for (int k = 0; k < 3; ++k)
                        mma_pair_f16<ID>(d, ad + P_STEP * k, bd + Q_STEP * k, (kb > 0 || k > 0) ? 1u : 0u);
                    const int s_next = s + 1 == STAGES ? 0 : s + 1;
                    const uint32_t ph_next = s + 1 == STAGES ? ph ^ 1u : ph;
                    if (kb + 1 < nkb)
                        ok = mbar_wait(&sm.full[s_next], ph_next, wait_ns);
                    mma_pair_f16<ID>(d, ad + P_STEP * 3, bd + Q_STEP * 3, 1u);
                    g2::commit_pair(&sm.empty[s], 0x3);
                    issued = true;
                    s = s_next;
                    ph = ph_next;
                };
                int kb = 0;
                for (; ok && kb < min(turn_q, nkb); ++kb)
                    block(kb, std::false_type{}, std::false_type{});
                for (; MODE != GRAM && ok && kb < min(turn_p, nkb); ++kb) // turn_q <= turn_p
                    block(kb, std::false_type{}, std::true_type{});
                for (; MODE != GRAM && ok && kb < nkb; ++kb)
                    block(kb, std::true_type{}, std::true_type{});
                if (!ok) {
                    *reinterpret_cast<volatile int *>(&sm.abort_flag) = 1;
                    break;
                }
                g2::commit_pair(&sm.acc_full[acc], 0x3);
            }
            if (issued) { // every issued MMA completes before TMEM is freed
                g2::commit_pair(&sm.mma_done, 0x1);
                mbar_wait(&sm.mma_done, 0u, wait_ns);
            }
        }
        __syncwarp();
    } else {
        // ------------------------------------------------ epilogue (both CTAs)
        const uint32_t leader_acc_empty0 = g2::peer_addr(&sm.acc_empty[0], 0);
        const int quad = warp & 3, part = warp >> 2;
        int t = 0, buf = 0;
        for (int64_t it = pair; it < total; it += npairs, ++t) {
            const Item w = item(it);
            const int acc = t & 1;
            const int r0 = w.i * TILE + (int)rank * HALF + 32 * quad; // the warp's rows, one per lane
            const int r = r0 + lane;
            const bool row_ok = r < q.m;
            const int cols = SYM ? q.m : q.n;
            const bool rows_full = r0 + 32 <= q.m; // the same in every lane
            const bool rows_any = r0 < q.m;
            // what the chunk adds to the product: X (hi and lo), or A
            uint4 old_h[4], old_l[MODE == POLY ? 1 : 4];
            float alpha_c = 0.0f; // POLY: alpha of the chunk's column `lane`
            auto load_old = [&](int c0) {
                if (MODE == POLY && c0 + lane < cols)
                    alpha_c = q.alpha[(int64_t)w.e * q.m + c0 + lane];
                if (rows_any && c0 < cols) {
                    const int64_t o = chunk_at(w.e, q.m, cols, r0, c0) + lane * 8;
#pragma unroll
                    for (int g = 0; g < 4; ++g) {
                        old_h[g] = *reinterpret_cast<const uint4 *>((MODE == POLY ? q.a_own : q.hi) + o + g * 256);
                        if constexpr (MODE != POLY)
                            old_l[g] = *reinterpret_cast<const uint4 *>(q.lo + o + g * 256);
                    }
                }
            };
            const int64_t diag_at = (int64_t)w.e * q.m + r;
            // this row's share of the diagonals: alpha_r, or a + beta_r
            float own = 0.0f;
            if (MODE != GRAM && row_ok)
                own = MODE == POLY ? q.alpha[diag_at] : q.a + q.beta[diag_at];
            if constexpr (MODE != GRAM)
                load_old(w.j * TN + CHUNK * part); // in flight while the product finishes
            bool ok = mbar_wait(&sm.acc_full[acc], (uint32_t)(t / ACC) & 1u, wait_ns);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok || gm::aborted(&sm.abort_flag)) {
                *reinterpret_cast<volatile int *>(&sm.abort_flag) = 1;
                break;
            }
            gm::tc_fence_after();
#pragma unroll 1
            for (int ch = part; ch < TN / CHUNK; ch += 2) {
                const int c0 = w.j * TN + CHUNK * ch;
                if (c0 >= cols)
                    break; // the same in every lane
                uint32_t d[CHUNK];
                gm::tc_ld32(tmem + (uint32_t)(acc * TN + CHUNK * ch) + ((uint32_t)(32 * quad) << 16), d);
                uint32_t h[CHUNK / 2], l[CHUNK / 2]; // pairs of the row, high and low words
                // in the chunk on the diagonal, element `lane` of the row stays
                // in fp32 and is zero in A' and B'
                const int dk = SYM && c0 == r0 ? lane : -1;
                float on_diag = 0.0f;
#pragma unroll
                for (int k = 0; k < CHUNK / 2; ++k) {
                    const float d0 = __uint_as_float(d[2 * k]), d1 = __uint_as_float(d[2 * k + 1]);
                    float v0, v1;
                    if constexpr (MODE == GRAM) {
                        v0 = d0 * (SA / (SX * SX));
                        v1 = d1 * (SA / (SX * SX));
                    } else {
                        const float2 oh = unpack_half2(word_of(old_h[k >> 2], k & 3));
                        if constexpr (MODE == POLY) {
                            const float a0 = own + __shfl_sync(0xffffffffu, alpha_c, 2 * k);
                            const float a1 = own + __shfl_sync(0xffffffffu, alpha_c, 2 * k + 1);
                            v0 = fmaf(q.pc * (1.0f / SA), d0, fmaf(q.pc, a0, q.pb) * oh.x);
                            v1 = fmaf(q.pc * (1.0f / SA), d1, fmaf(q.pc, a1, q.pb) * oh.y);
                        } else {
                            const float2 ol = unpack_half2(word_of(old_l[k >> 2], k & 3));
                            v0 = fmaf(own, fmaf(ol.x, 1.0f / SLO, oh.x), d0 * q.unscale);
                            v1 = fmaf(own, fmaf(ol.y, 1.0f / SLO, oh.y), d1 * q.unscale);
                        }
                    }
                    if constexpr (SYM) {
                        on_diag = dk == 2 * k ? d0 : (dk == 2 * k + 1 ? d1 : on_diag);
                        v0 = dk == 2 * k ? 0.0f : v0;
                        v1 = dk == 2 * k + 1 ? 0.0f : v1;
                    }
                    if constexpr (MODE == LAST) {
                        h[k] = gm::pack_bf16x2(v0 * (1.0f / SX), v1 * (1.0f / SX));
                    } else {
                        h[k] = pack_half2(v0, v1);
                        if constexpr (MODE == STEP) {
                            const float2 f = unpack_half2(h[k]);
                            l[k] = pack_half2((v0 - f.x) * SLO, (v1 - f.y) * SLO);
                        }
                    }
                }
                if (SYM && c0 == r0 && row_ok) { // the chunk on the diagonal
                    if constexpr (MODE == GRAM)
                        q.alpha[diag_at] = on_diag * (1.0f / (SX * SX));
                    else
                        q.beta[diag_at] = fmaf(fmaf(q.c, own, q.b), own, q.c * (on_diag * (1.0f / (SA * SA))));
                }
                if constexpr (MODE != GRAM) {
                    if (ch + 2 < TN / CHUNK && c0 + 2 * CHUNK < cols)
                        load_old(c0 + 2 * CHUNK);
                }
                // the epilogue's own copies
                if constexpr (MODE == STEP || MODE == GRAM) {
                    if (rows_any) {
                        const int64_t o = chunk_at(w.e, q.m, cols, r0, c0) + lane * 8;
#pragma unroll
                        for (int g = 0; g < 4; ++g) {
                            st_v4((MODE == GRAM ? q.a_own : q.hi) + o + g * 256, h[4 * g], h[4 * g + 1], h[4 * g + 2],
                                  h[4 * g + 3]);
                            if constexpr (MODE == STEP)
                                st_v4(q.lo + o + g * 256, l[4 * g], l[4 * g + 1], l[4 * g + 2], l[4 * g + 3]);
                        }
                    }
                }
                // G^T's update: down the columns (a matrix has less than 2^31
                // elements, so 32 bits hold its byte offsets)
                if (MODE == LAST && q.out_t) {
                    const uint32_t ld2 = (uint32_t)q.m * 2u;
                    uint32_t o = (uint32_t)c0 * ld2 + (uint32_t)r * 2u;
                    uint8_t *dst = reinterpret_cast<uint8_t *>(q.out + (int64_t)w.e * cols * q.m);
                    auto put = [&](int k) {
                        *reinterpret_cast<uint16_t *>(dst + o) = (uint16_t)(k & 1 ? h[k >> 1] >> 16 : h[k >> 1]);
                    };
                    if (rows_full && c0 + CHUNK <= cols) {
#pragma unroll
                        for (int k = 0; k < CHUNK; ++k, o += ld2)
                            put(k);
                    } else {
#pragma unroll
                        for (int k = 0; k < CHUNK; ++k, o += ld2)
                            if (row_ok && c0 + k < cols)
                                put(k);
                    }
                }
                // along the rows, through shared memory
                if (MODE != LAST || !q.out_t) {
                    uint8_t *st = sm.stage[warp][buf];
                    if constexpr (MODE != LAST) {
                        if (lane == 0)
                            bulk_wait_read<1>(); // the store before the last has read this buffer
                        __syncwarp();
                    }
                    if constexpr (MODE != LAST) {
                        chunk_to_smem(st, h);
                        fence_proxy_async_smem();
                        __syncwarp();
                        if (lane == 0 && r0 < q.m) {
                            tma_store_3d(&tm_o, st, c0, r0, w.e);
                            bulk_commit();
                        }
                    } else {
                        rows_out(st, h, q.out + ((int64_t)w.e * q.m + r0) * q.n + c0, q.n, q.m - r0, cols - c0,
                                 q.out_vec);
                    }
                    buf ^= 1;
                }
            }
            gm::tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                if (leader)
                    mbar_arrive(&sm.acc_empty[acc]);
                else
                    g2::arrive_remote(leader_acc_empty0 + (uint32_t)(acc * sizeof(uint64_t)));
            }
        }
        if (MODE != LAST && lane == 0)
            bulk_wait_read<0>(); // the stores have left shared memory; the kernel's end completes them
    }

    __syncwarp(); // the cluster barrier below is warp-aligned
    gm::tc_fence_before();
    g2::cluster_sync(); // the pair's MMAs and both epilogues are done
    gm::tc_fence_after();
    if (warp == EPI_WARPS + 1)
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(TMEM_COLS) : "memory");
}

} // namespace ns
} // namespace mxq

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
// significand costs nothing in range and is eight times finer than bf16's.
// X is held as a pair hi + lo of fp16 words (22 bits): the products read hi,
// the term a X adds both. Without lo the rounding of X would be multiplied by
// a = 3.4 in every later step wherever a singular value is small: on a matrix
// whose singular values fall to 1e-4 the result was off by 0.9% of its norm,
// with lo by 0.08%, half of what rounding the result to bf16 costs. A and B
// are rounded once each to fp16. Scales are powers of two: X 2^8 (a random
// 2048 x 7168 matrix starts with elements near 2^-12, fp16's normal range
// ends at 2^-14), A and B 2^10, lo 2^11 on top of X's.
//
// Every product is D = P Q^T with both operands K-major: A = X X^T, A A = A
// A^T (A is symmetric), B X = B (X^T)^T; the epilogue that writes X therefore
// writes X^T too. A and A A are computed on and below the diagonal of tiles
// and mirrored by the epilogue.
//
// Kernel: the CTA-pair pipeline of gemm2.cuh (tcgen05.mma.cta_group::2, one
// 256 x 256 tile per pair of SMs, six 32 KB stages of 64 fp16 columns, two
// accumulators in TMEM); warps 0-7 epilogue (a warp takes 32 lanes and half
// of the columns), warp 8 TMA, warp 9 MMA and TMEM, warp 10 passes its CTA's
// filled slots on to the leader. Edges are filled with zeros by TMA (every
// matrix is its own plane of a rank-3 map) and cut off by the epilogue.
#pragma once

#include <cuda_fp16.h>

#include "gemm2.cuh"

namespace mxq {
namespace ns {

constexpr int HALF = 128;
constexpr int TILE = 256;              // rows and columns of a pair's tile
constexpr int BK = 64;                 // fp16 elements per 128-byte row
constexpr int STAGES = 6;
constexpr int OP_BYTES = HALF * 128;   // one operand, one stage, one CTA
constexpr int EPI_WARPS = 8;
constexpr int THREADS = (EPI_WARPS + 3) * 32;
constexpr int ACC = 2;
constexpr int TMEM_COLS = ACC * TILE;
constexpr int MAX_PARTS = 64;          // partial sums of squares per matrix

constexpr float SX = 256.0f;           // stored X  = X 2^8
constexpr float SA = 1024.0f;          // stored A, B = A, B 2^10
constexpr float SLO = 2048.0f;         // stored lo = (X 2^8 - hi) 2^11

struct __align__(1024) Smem {
    uint8_t a[STAGES][OP_BYTES];
    uint8_t b[STAGES][OP_BYTES];
    uint64_t full[STAGES];
    uint64_t ready[STAGES];
    uint64_t empty[STAGES];
    uint64_t acc_full[ACC];
    uint64_t acc_empty[ACC];
    uint64_t mma_done;
    uint32_t tmem_base;
    int abort_flag;
};
constexpr size_t SMEM_BYTES = sizeof(Smem) + 1024;

// fp32 accumulator, f16 x f16, both K-major, N 256, M 256 (the pair)
constexpr uint32_t IDESC = (1u << 4) | ((uint32_t)(TILE >> 3) << 17) | ((uint32_t)(TILE >> 4) << 24);

enum Mode { GRAM = 0, POLY = 1, STEP = 2, LAST = 3 };

struct Args {
    int E, m, n;          // batch, X is (m, n)
    int ldx, ldt;         // row lengths of X (n up to 8) and of X^T, A, B (m up to 8)
    float a, b, c;
    __half *xh, *xl;      // (E, m, ldx)
    __half *xt;           // (E, n, ldt): written by STEP
    __half *A, *B;        // (E, m, ldt)
    uint16_t *out;        // LAST: bf16, (E, m, n) or, transposed, (E, n, m)
    int out_t, out_vec;
};

MXQ_DEV void mma_pair_f16(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t accumulate)
{
    asm volatile("{\n\t.reg .pred p;\n\t"
                 "setp.ne.b32 p, %3, 0;\n\t"
                 "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %4, p;\n\t}" ::"r"(d_tmem),
                 "l"(adesc), "l"(bdesc), "r"(accumulate), "r"(IDESC)
                 : "memory");
}

MXQ_DEV uint32_t pack_half2(float lo, float hi)
{
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
MXQ_DEV float2 unpack_half2(uint32_t w) { return __half22float2(*reinterpret_cast<__half2 *>(&w)); }

MXQ_DEV float in_value(const uint16_t *p, int64_t i) { return __uint_as_float((uint32_t)p[i] << 16); }
MXQ_DEV float in_value(const float *p, int64_t i) { return p[i]; }

// sum of squares of a slice of matrix blockIdx.y, in 64 bits: squares of fp32
// values leave fp32's range
template <typename T>
__global__ void __launch_bounds__(256) k_ns_sumsq(const T *__restrict__ g, int64_t size, double *__restrict__ part)
{
    const T *p = g + (int64_t)blockIdx.y * size;
    const int64_t per = (size + gridDim.x - 1) / gridDim.x;
    const int64_t lo = blockIdx.x * per, hi = lo + per < size ? lo + per : size;
    double s[4] = {0.0, 0.0, 0.0, 0.0};
    for (int64_t i = lo + threadIdx.x; i < hi; i += 4 * 256) {
        float v[4];
#pragma unroll
        for (int u = 0; u < 4; ++u)
            v[u] = i + u * 256 < hi ? in_value(p, i + u * 256) : 0.0f;
#pragma unroll
        for (int u = 0; u < 4; ++u)
            s[u] = fma((double)v[u], (double)v[u], s[u]);
    }
    double t = (s[0] + s[1]) + (s[2] + s[3]);
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

// X0 from G (rows, cols), 64 x 64 tiles: hi and lo of X and hi of X^T. With
// `tall` X is G^T, so the tile's transpose is X's and the tile itself X^T's.
template <typename T>
__global__ void __launch_bounds__(256)
    k_ns_init(const T *__restrict__ g, int rows, int cols, const double *__restrict__ part, int parts, double eps,
              int tall, __half *__restrict__ xh, __half *__restrict__ xl, int ldx, __half *__restrict__ xt, int ldt)
{
    __shared__ __half sh[64][66], sl[64][66];
    __shared__ double s_inv;
    const int e = blockIdx.z, r0 = blockIdx.y * 64, c0 = blockIdx.x * 64;
    if (threadIdx.x == 0) {
        double s = 0.0;
        for (int i = 0; i < parts; ++i)
            s += part[(size_t)e * parts + i];
        const double norm = sqrt(s) + eps;
        s_inv = norm > 0.0 ? (double)SX / norm : (norm == 0.0 ? 0.0 : norm);
    }
    __syncthreads();
    const double inv = s_inv;
    const T *p = g + (int64_t)e * rows * cols;
    const int64_t base_x = (int64_t)e * (tall ? cols : rows) * ldx;
    const int64_t base_t = (int64_t)e * (tall ? rows : cols) * ldt;
    const int tx = threadIdx.x & 63, ty = threadIdx.x >> 6;
#pragma unroll 4
    for (int r = ty; r < 64; r += 4) {
        const int R = r0 + r, C = c0 + tx;
        if (R < rows && C < cols) {
            const float x = (float)((double)in_value(p, (int64_t)R * cols + C) * inv);
            const __half h = __float2half_rn(x);
            const __half l = __float2half_rn((x - __half2float(h)) * SLO);
            sh[r][tx] = h;
            sl[r][tx] = l;
            if (tall) {
                xt[base_t + (int64_t)R * ldt + C] = h;
            } else {
                xh[base_x + (int64_t)R * ldx + C] = h;
                xl[base_x + (int64_t)R * ldx + C] = l;
            }
        }
    }
    __syncthreads();
#pragma unroll 4
    for (int c = ty; c < 64; c += 4) {
        const int C = c0 + c, R = r0 + tx;
        if (R < rows && C < cols) {
            if (tall) {
                xh[base_x + (int64_t)C * ldx + R] = sh[tx][c];
                xl[base_x + (int64_t)C * ldx + R] = sl[tx][c];
            } else {
                xt[base_t + (int64_t)C * ldt + R] = sh[tx][c];
            }
        }
    }
}

// D = P Q^T over K = 64 nkb columns for every matrix, with the epilogue of
// MODE. Grid: an even number of CTAs in clusters of two.
template <int MODE>
__global__ void __launch_bounds__(THREADS, 1)
    k_ns_gemm(const __grid_constant__ CUtensorMap tm_p, const __grid_constant__ CUtensorMap tm_q, const Args q,
              int nkb, uint64_t wait_ns)
{
    constexpr bool SYM = MODE == GRAM || MODE == POLY;
    extern __shared__ uint8_t smem_raw[];
    Smem &sm = *reinterpret_cast<Smem *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = g2::cta_rank();
    const bool leader = rank == 0;

    if (threadIdx.x == 0) {
        for (int s = 0; s < STAGES; ++s) {
            mbar_init(&sm.full[s], 1);
            mbar_init(&sm.ready[s], 2);
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

    const int64_t pair = blockIdx.x >> 1, npairs = gridDim.x >> 1;
    const int tm = (q.m + TILE - 1) / TILE, tn = (q.n + TILE - 1) / TILE;
    const int64_t per = SYM ? (int64_t)tm * (tm + 1) / 2 : (int64_t)tm * tn;
    const int64_t total = per * q.E;
    // tile t of a matrix: row tile i, column tile j; symmetric products take
    // j <= i, the others run down the row tiles first, so that the pairs at
    // work share a column tile of X^T and all of B
    struct Item {
        int e, i, j;
    };
    auto item = [&](int64_t it) {
        Item w;
        w.e = (int)(it / per);
        int t = (int)(it - (int64_t)w.e * per);
        if (SYM) {
            w.i = 0;
            while (t > w.i)
                t -= ++w.i;
            w.j = t;
        } else {
            w.j = t / tm;
            w.i = t - w.j * tm;
        }
        return w;
    };

    if (warp == EPI_WARPS) {
        // ------------------------------------------------ TMA producer (both CTAs)
        if (lane == 0) {
            int seq = 0;
            for (int64_t it = pair; it < total && !gm::aborted(&sm.abort_flag); it += npairs) {
                const Item w = item(it);
                for (int kb = 0; kb < nkb; ++kb, ++seq) {
                    const int s = seq % STAGES;
                    if (seq >= STAGES && !mbar_wait(&sm.empty[s], ((uint32_t)(seq / STAGES) & 1u) ^ 1u, wait_ns)) {
                        *reinterpret_cast<volatile int *>(&sm.abort_flag) = 1;
                        break;
                    }
                    mbar_arrive_expect_tx(&sm.full[s], 2 * OP_BYTES);
                    tma_load_3d(sm.a[s], &tm_p, &sm.full[s], kb * BK, w.i * TILE + (int)rank * HALF, w.e);
                    tma_load_3d(sm.b[s], &tm_q, &sm.full[s], kb * BK, w.j * TILE + (int)rank * HALF, w.e);
                }
            }
            // drain: every issued fill has landed before the CTA leaves
            for (int j = seq - STAGES; j < seq; ++j)
                if (j >= 0)
                    mbar_wait(&sm.full[j % STAGES], (uint32_t)(j / STAGES) & 1u, wait_ns);
        }
    } else if (warp == EPI_WARPS + 2) {
        // ------------------------------------------------ hand-off of filled slots (both CTAs)
        if (lane == 0) {
            const uint32_t leader_ready0 = g2::peer_addr(&sm.ready[0], 0);
            int s = 0;
            uint32_t ph = 0;
            bool ok = true;
            for (int64_t it = pair; ok && it < total && !gm::aborted(&sm.abort_flag); it += npairs)
                for (int kb = 0; kb < nkb; ++kb) {
                    ok = mbar_wait(&sm.full[s], ph, wait_ns);
                    if (!ok) {
                        *reinterpret_cast<volatile int *>(&sm.abort_flag) = 1;
                        break;
                    }
                    g2::arrive_remote(leader_ready0 + (uint32_t)(s * sizeof(uint64_t)));
                    if (++s == STAGES) {
                        s = 0;
                        ph ^= 1u;
                    }
                }
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
                const uint32_t d = tmem + (uint32_t)(acc * TILE);
                // the next slot is waited on before this slot's last MMA, so
                // that the wait overlaps MMAs already in the pipe
                bool ok = mbar_wait(&sm.ready[s], ph, wait_ns);
                for (int kb = 0; ok && kb < nkb; ++kb) {
                    gm::tc_fence_after();
                    const uint64_t ad = gm::smem_desc_k128(smem_u32(sm.a[s]));
                    const uint64_t bd = gm::smem_desc_k128(smem_u32(sm.b[s]));
#pragma unroll
                    for (int k = 0; k < 3; ++k) // 16 columns per MMA: 32 bytes
                        mma_pair_f16(d, ad + 2 * k, bd + 2 * k, (kb > 0 || k > 0) ? 1u : 0u);
                    const int s_next = s + 1 == STAGES ? 0 : s + 1;
                    const uint32_t ph_next = s + 1 == STAGES ? ph ^ 1u : ph;
                    if (kb + 1 < nkb)
                        ok = mbar_wait(&sm.ready[s_next], ph_next, wait_ns);
                    mma_pair_f16(d, ad + 6, bd + 6, 1u);
                    g2::commit_pair(&sm.empty[s], 0x3);
                    issued = true;
                    s = s_next;
                    ph = ph_next;
                }
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
        int t = 0;
        for (int64_t it = pair; it < total; it += npairs, ++t) {
            const Item w = item(it);
            const int acc = t & 1;
            bool ok = mbar_wait(&sm.acc_full[acc], (uint32_t)(t / ACC) & 1u, wait_ns);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok || gm::aborted(&sm.abort_flag)) {
                *reinterpret_cast<volatile int *>(&sm.abort_flag) = 1;
                break;
            }
            gm::tc_fence_after();
            const int r = w.i * TILE + (int)rank * HALF + 32 * quad + lane; // this thread's row
            const bool row_ok = r < q.m;
            const int64_t row_t = ((int64_t)w.e * q.m + r) * q.ldt, row_x = ((int64_t)w.e * q.m + r) * q.ldx;
            const int cols = SYM ? q.m : q.n, ld = SYM ? q.ldt : q.ldx;
#pragma unroll 1
            for (int ch = 0; ch < 4; ++ch) {
                const int c0 = w.j * TILE + part * HALF + 32 * ch;
                if (c0 >= cols)
                    break; // the same in every lane
                uint32_t d[32];
                gm::tc_ld32(tmem + (uint32_t)(acc * TILE + part * HALF + 32 * ch) + ((uint32_t)(32 * quad) << 16), d);
                uint32_t h[16]; // the chunk's result, two fp16 per word
#pragma unroll
                for (int g = 0; g < 4; ++g) {
                    const int c = c0 + 8 * g;
                    const bool in = row_ok && c < ld;
                    float v[8];
                    if constexpr (MODE == GRAM) {
#pragma unroll
                        for (int k = 0; k < 8; ++k)
                            v[k] = __uint_as_float(d[8 * g + k]) * (SA / (SX * SX));
                    } else if constexpr (MODE == POLY) {
                        uint4 x = make_uint4(0u, 0u, 0u, 0u);
                        if (in)
                            x = *reinterpret_cast<const uint4 *>(q.A + row_t + c);
                        const uint32_t xw[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            const float2 f = unpack_half2(xw[k]);
                            v[2 * k] = fmaf(q.c * (1.0f / SA), __uint_as_float(d[8 * g + 2 * k]), q.b * f.x);
                            v[2 * k + 1] = fmaf(q.c * (1.0f / SA), __uint_as_float(d[8 * g + 2 * k + 1]), q.b * f.y);
                        }
                    } else {
                        uint4 x = make_uint4(0u, 0u, 0u, 0u), y = x;
                        if (in) {
                            x = *reinterpret_cast<const uint4 *>(q.xh + row_x + c);
                            y = *reinterpret_cast<const uint4 *>(q.xl + row_x + c);
                        }
                        const uint32_t xw[4] = {x.x, x.y, x.z, x.w}, yw[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            const float2 f = unpack_half2(xw[k]), l = unpack_half2(yw[k]);
                            v[2 * k] = fmaf(q.a, fmaf(l.x, 1.0f / SLO, f.x),
                                            __uint_as_float(d[8 * g + 2 * k]) * (1.0f / SA));
                            v[2 * k + 1] = fmaf(q.a, fmaf(l.y, 1.0f / SLO, f.y),
                                                __uint_as_float(d[8 * g + 2 * k + 1]) * (1.0f / SA));
                        }
                    }
                    if constexpr (MODE == LAST) {
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            h[4 * g + k] = gm::pack_bf16x2(v[2 * k] * (1.0f / SX), v[2 * k + 1] * (1.0f / SX));
                    } else {
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            h[4 * g + k] = pack_half2(v[2 * k], v[2 * k + 1]);
                        if (in) {
                            __half *dst = MODE == GRAM ? q.A + row_t + c : MODE == POLY ? q.B + row_t + c : q.xh + row_x + c;
                            st_v4(dst, h[4 * g], h[4 * g + 1], h[4 * g + 2], h[4 * g + 3]);
                            if constexpr (MODE == STEP) {
                                uint32_t lo[4];
#pragma unroll
                                for (int k = 0; k < 4; ++k) {
                                    const float2 f = unpack_half2(h[4 * g + k]);
                                    lo[k] = pack_half2((v[2 * k] - f.x) * SLO, (v[2 * k + 1] - f.y) * SLO);
                                }
                                st_v4(q.xl + row_x + c, lo[0], lo[1], lo[2], lo[3]);
                            }
                        }
                    }
                }
                // the transpose: one column per store, neighbouring lanes
                // hold neighbouring rows
                if constexpr (MODE == LAST) {
                    if (q.out_t) {
                        uint16_t *dst = q.out + ((int64_t)w.e * q.n + c0) * q.m + r;
#pragma unroll
                        for (int k = 0; k < 32; ++k)
                            if (row_ok && c0 + k < cols)
                                dst[(int64_t)k * q.m] = (uint16_t)(k & 1 ? h[k >> 1] >> 16 : h[k >> 1]);
                    } else if (row_ok) {
                        uint16_t *dst = q.out + ((int64_t)w.e * q.m + r) * q.n + c0;
                        if (q.out_vec && c0 + 32 <= cols) {
#pragma unroll
                            for (int g = 0; g < 4; ++g)
                                st_v4(dst + 8 * g, h[4 * g], h[4 * g + 1], h[4 * g + 2], h[4 * g + 3]);
                        } else {
#pragma unroll
                            for (int k = 0; k < 32; ++k)
                                if (c0 + k < cols)
                                    dst[k] = (uint16_t)(k & 1 ? h[k >> 1] >> 16 : h[k >> 1]);
                        }
                    }
                } else if (!SYM || w.i != w.j) {
                    uint16_t *dst = reinterpret_cast<uint16_t *>(MODE == GRAM ? q.A : MODE == POLY ? q.B : q.xt) +
                                    ((int64_t)w.e * cols + c0) * q.ldt + r;
#pragma unroll
                    for (int k = 0; k < 32; ++k)
                        if (row_ok && c0 + k < cols)
                            dst[(int64_t)k * q.ldt] = (uint16_t)(k & 1 ? h[k >> 1] >> 16 : h[k >> 1]);
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

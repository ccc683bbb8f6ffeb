// ns_small.cuh - newton_schulz (see ns.cuh) for matrices whose smaller side is
// at most 128: all steps of a matrix in one launch, on chip.
//
// A CTA holds a slab of up to 256 columns of X (m <= 128 rows): hi of X as fp16
// in shared memory in the layout that tcgen05.mma reads, by rows for X X^T and
// by columns for B' X, X itself in fp32 in half of TMEM, so that it is never
// rounded; the other half takes the products, A and A A and then, both read,
// B' X.
// A matrix with more columns takes a cluster of up to sixteen CTAs: each
// multiplies its slab with itself, the partial 128 x 128 products are summed
// over distributed shared memory in rank order (every CTA sums some rows and
// sends them to all), and the rest is local to the slab.
//
// Per step: three products (K = 256, 128, 128; about 1.4 us of tensor time),
// three drains of TMEM by sixteen warps, two cluster barriers. What bounds it is
// the chain of barriers, TMEM loads and shared-memory stores, not bandwidth or
// the tensor pipe; against the general kernels' three launches per step it
// saves their launch, fill and drain (about 6 us each): (4, 96, 224) takes 39 us
// against 80, 5 a step and 12 to start; (8, 128, 1024) on four CTAs each 60
// against 112.
#pragma once

#include <cstddef>

#include "ns.cuh"

namespace mxq {
namespace ns {

constexpr int SM_M = 128;              // rows of X, at most
constexpr int SM_SLAB = 256;           // columns of X per CTA
constexpr int SM_MAX_CTAS = 16;        // CTAs per matrix; more than 8 where the device has such clusters
constexpr int SM_THREADS = 512;        // four warps per 32 rows, a quarter of the columns each
constexpr int MAX_STEPS = 64;

struct Coefs {
    float v[3 * MAX_STEPS];
    float pb[MAX_STEPS], pc[MAX_STEPS]; // b and c times the scale of B' over that of A'
    float unscale[MAX_STEPS];           // one over the scale of B'
};

struct __align__(1024) SmallSmem {
    uint8_t xh[SM_SLAB / 64][SM_M * 128];  // X: blocks of 64 columns, 128-byte rows
    uint8_t ab[SM_M / 64][SM_M * 128];     // A, then B
    float alpha[SM_M], beta[SM_M];         // the diagonals of A and B
    double warp_sum[SM_THREADS / 32];
    uint64_t bar;
    uint32_t tmem_base;
    float factor[2];
    alignas(16) float part[SM_M * SM_M];   // fp32 A of this slab (clusters only)
};
// one CTA per matrix needs no room for partial products
constexpr size_t small_smem_bytes(bool cluster)
{
    return (cluster ? sizeof(SmallSmem) : offsetof(SmallSmem, part)) + 1024;
}

// fp32 accumulator, f16 x f16, both K-major, M 128, N n (a multiple of 16)
MXQ_DEV uint32_t small_idesc(int n) { return (1u << 4) | ((uint32_t)(n >> 3) << 17) | ((uint32_t)(SM_M >> 4) << 24); }

MXQ_DEV void mma_f16(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc, uint32_t accumulate)
{
    asm volatile("{\n\t.reg .pred p;\n\t"
                 "setp.ne.b32 p, %4, 0;\n\t"
                 "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
                 "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
                 : "memory");
}

// 32 lanes x 32 columns of fp32 to TMEM
MXQ_DEV void tc_st32(uint32_t taddr, const uint32_t (&r)[32])
{
    asm volatile("tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
                 "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, "
                 "%17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};" ::"r"(taddr),
                 "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
                 "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]),
                 "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]),
                 "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
                 : "memory");
}
MXQ_DEV void tc_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// generic-proxy writes of shared memory, also by other CTAs of the cluster,
// before the async proxy (the tensor core's operand reads)
MXQ_DEV void fence_proxy_async_all() { asm volatile("fence.proxy.async;" ::: "memory"); }

MXQ_DEV float4 ld_cluster_v4(uint32_t addr)
{
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "r"(addr)
                 : "memory");
    return v;
}
MXQ_DEV void st_cluster_v2(uint32_t addr, uint32_t a, uint32_t b)
{
    asm volatile("st.shared::cluster.v2.u32 [%0], {%1, %2};" ::"r"(addr), "r"(a), "r"(b) : "memory");
}
MXQ_DEV void st_cluster_f32(uint32_t addr, float v)
{
    asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(addr), "f"(v) : "memory");
}
MXQ_DEV double ld_cluster_f64(uint32_t addr)
{
    double v;
    asm volatile("ld.shared::cluster.f64 %0, [%1];" : "=d"(v) : "r"(addr) : "memory");
    return v;
}

// element `dk` (none if negative) of the row that a lane holds: returned, and
// zero in v. By selects: a branch on the lane would put v into local memory.
MXQ_DEV float take_diagonal(uint32_t (&v)[32], int dk)
{
    uint32_t x = 0u;
#pragma unroll
    for (int k = 0; k < 32; ++k) {
        x = dk == k ? v[k] : x;
        v[k] = dk == k ? 0u : v[k];
    }
    return __uint_as_float(x);
}

// byte of column byte `b` (of 128) of row `r` in a block of 128-byte rows with
// the 128-byte swizzle
MXQ_DEV uint32_t swz(int r, int b) { return (uint32_t)(r * 128 + (b ^ ((r & 7) << 4))); }

// Grid: E * ctas CTAs in clusters of `ctas`. g (E, rows, cols); X = G, or with
// `tall` G^T.
template <typename T>
__global__ void __launch_bounds__(SM_THREADS, 1)
    k_ns_small(const T *__restrict__ g, int rows, int cols, int ctas, int tall, int steps,
               const __grid_constant__ Coefs co, double eps, uint16_t *__restrict__ out, int out_vec,
               uint64_t wait_ns)
{
    extern __shared__ uint8_t smem_raw[];
    SmallSmem &sm = *reinterpret_cast<SmallSmem *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int quad = warp & 3, part = warp >> 2;
    const int rank = (int)g2::cta_rank(), e = blockIdx.x / ctas;
    const int m = tall ? cols : rows, n = tall ? rows : cols;
    const int c_base = rank * SM_SLAB, ncol = min(SM_SLAB, n - c_base); // this slab's columns, at least one
    const int m16 = (m + 15) & ~15, n16 = (ncol + 15) & ~15;
    const int r = 32 * quad + lane;         // this thread's row of X
    const bool active = 32 * quad < m16;    // the warp has rows that a product reads

    if (warp == 0) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&sm.tmem_base)),
                     "r"(512u)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    if (tid == 0) {
        mbar_init(&sm.bar, 1);
        fence_mbar_init();
    }
    gm::tc_fence_before();
    __syncthreads();
    gm::tc_fence_after();
    const uint32_t lanes = sm.tmem_base + ((uint32_t)(32 * quad) << 16);
    const uint32_t d_x = 0, d_a = SM_SLAB, d_b = SM_SLAB + SM_M, d_y = SM_SLAB; // TMEM columns of X, A, A A, B' X

    // ---- G into TMEM, its sum of squares
    double sq = 0.0;
    if (active) {
        const T *p = g + (int64_t)e * rows * cols;
#pragma unroll 1
        for (int ch = part; 32 * ch < n16; ch += 4) {
            uint32_t v[32];
            float f[32];
            const int c0 = c_base + 32 * ch;
            if (tall) { // X(r, c) is G[c][r]: neighbouring lanes, neighbouring elements
                const T *q = p + (int64_t)c0 * cols + r;
#pragma unroll
                for (int k = 0; k < 32; ++k)
                    f[k] = r < m && 32 * ch + k < ncol ? in_pair(q + (int64_t)k * cols, false, false).x : 0.0f;
            } else { // a row at a time, turned over where X and A will be
                const T *q = p + (int64_t)(32 * quad) * cols + c0 + lane;
                const bool in = 32 * ch + lane < ncol;
#pragma unroll
                for (int k = 0; k < 32; ++k)
                    f[k] = in && 32 * quad + k < m ? in_pair(q + (int64_t)k * cols, false, false).x : 0.0f;
                float *st = reinterpret_cast<float *>(sm.xh[0]) + warp * (32 * 33);
#pragma unroll
                for (int k = 0; k < 32; ++k)
                    st[k * 33 + lane] = f[k];
                __syncwarp();
#pragma unroll
                for (int k = 0; k < 32; ++k)
                    f[k] = st[lane * 33 + k];
                __syncwarp();
            }
#pragma unroll
            for (int k = 0; k < 32; k += 8) {
                float s = 0.0f;
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    s = fmaf(f[k + i], f[k + i], s);
                if (s > 0x1p-90f && s < 0x1p120f) {
                    sq += (double)s;
                } else {
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        sq = fma((double)f[k + i], (double)f[k + i], sq);
                }
            }
#pragma unroll
            for (int k = 0; k < 32; ++k)
                v[k] = __float_as_uint(f[k]);
            tc_st32(lanes + d_x + 32 * ch, v);
        }
        tc_wait_st();
    }
#pragma unroll
    for (int o = 16; o; o >>= 1)
        sq += __shfl_xor_sync(0xffffffffu, sq, o);
    if (lane == 0)
        sm.warp_sum[warp] = sq;
    __syncwarp();
    g2::cluster_sync(); // every CTA of the cluster runs and has its sums
    if (warp == 0) { // a lane per CTA, then the lanes, in the same order everywhere
        double s = 0.0;
        if (lane < ctas) {
            double w[SM_THREADS / 32];
#pragma unroll
            for (int i = 0; i < SM_THREADS / 32; ++i)
                w[i] = ld_cluster_f64(g2::peer_addr(&sm.warp_sum[i], (uint32_t)lane));
#pragma unroll
            for (int i = 0; i < SM_THREADS / 32; ++i)
                s += w[i];
        }
#pragma unroll
        for (int o = 16; o; o >>= 1)
            s += __shfl_xor_sync(0xffffffffu, s, o);
        if (lane == 0)
            scale_factors(sqrt(s) + eps, sm.factor[0], sm.factor[1]);
    }
    __syncthreads();

    // hi of a chunk of X, times 2^8, to its place
    auto put_x = [&](int c0, const float (&x)[32]) {
        uint32_t h[16];
#pragma unroll
        for (int k = 0; k < 16; ++k)
            h[k] = pack_half2(x[2 * k], x[2 * k + 1]);
        uint8_t *row = sm.xh[c0 >> 6];
#pragma unroll
        for (int q = 0; q < 4; ++q)
            sts_v4(smem_u32(row) + swz(r, (c0 & 32) * 2 + 16 * q),
                   make_uint4(h[4 * q], h[4 * q + 1], h[4 * q + 2], h[4 * q + 3]));
    };
    if (active) {
        const float f0 = sm.factor[0], f1 = sm.factor[1];
#pragma unroll 1
        for (int ch = part; 32 * ch < n16; ch += 4) {
            uint32_t v[32];
            float x[32];
            gm::tc_ld32(lanes + d_x + 32 * ch, v);
#pragma unroll
            for (int k = 0; k < 32; ++k) {
                x[k] = (__uint_as_float(v[k]) * f0) * f1;
                v[k] = __float_as_uint(x[k]);
            }
            put_x(32 * ch, x);
            tc_st32(lanes + d_x + 32 * ch, v); // X 2^8
        }
        tc_wait_st();
    }

    uint32_t phase = 0;
    // everything that the tensor core will read is written: then one thread
    // multiplies P (128 x K) by Q^T (Q has N rows) or, by_columns, by Q (N
    // columns) into TMEM column d. Rows and columns of shared memory that were
    // never written reach only rows of the product that nothing reads.
    auto product = [&](uint32_t d, const uint8_t *P, const uint8_t *Q, bool by_columns, int N, int K) {
        fence_proxy_async_all();
        gm::tc_fence_before();
        __syncthreads();
        if (tid == 0) {
            gm::tc_fence_after();
            const uint32_t id = small_idesc(N) | (by_columns ? IDESC_B_COLUMNS : 0u);
            for (int k = 0; k < K; k += 16) {
                const uint64_t ad = gm::smem_desc_k128(smem_u32(P) + (k >> 6) * SM_M * 128) + 2 * ((k >> 4) & 3);
                const uint64_t bd = by_columns
                                        ? smem_desc_columns<128>(smem_u32(Q) + k * 128, SM_M * 128)
                                        : gm::smem_desc_k128(smem_u32(Q) + (k >> 6) * SM_M * 128) + 2 * ((k >> 4) & 3);
                mma_f16(sm.tmem_base + d, ad, bd, id, k > 0 ? 1u : 0u);
            }
            gm::tc_commit(&sm.bar);
        }
        __syncwarp();
        mbar_wait(&sm.bar, phase, wait_ns); // a wait that runs out is in the status; no CTA leaves the cluster
        phase ^= 1u;
        gm::tc_fence_after();
    };

#pragma unroll 1
    for (int s = 0; s < steps; ++s) {
        const float cb = co.v[3 * s + 1], cc = co.v[3 * s + 2];
        const float pb = co.pb[s], pc = co.pc[s];
        // ---- A = X X^T
        product(d_a, sm.xh[0], sm.xh[0], false, m16, n16);
        if (active) {
#pragma unroll 1
            for (int ch = part; 32 * ch < m16; ch += 4) {
                uint32_t v[32];
                gm::tc_ld32(lanes + d_a + 32 * ch, v);
                if (ctas == 1) {
                    const float on_diag = take_diagonal(v, ch == quad ? lane : -1); // to fp32, and out of A
                    if (ch == quad)
                        sm.alpha[r] = on_diag * (1.0f / (SX * SX));
#pragma unroll
                    for (int q = 0; q < 4; ++q)
                        if (32 * ch + 8 * q < m16) {
                            uint32_t h[4];
#pragma unroll
                            for (int k = 0; k < 4; ++k)
                                h[k] = pack_half2(__uint_as_float(v[8 * q + 2 * k]) * (SA / (SX * SX)),
                                                  __uint_as_float(v[8 * q + 2 * k + 1]) * (SA / (SX * SX)));
                            sts_v4(smem_u32(sm.ab[ch >> 1]) + swz(r, (ch & 1) * 64 + 16 * q),
                                   make_uint4(h[0], h[1], h[2], h[3]));
                        }
                } else {
                    // 16-byte chunks, swizzled by the row so that 32 rows'
                    // stores fall into different banks
#pragma unroll
                    for (int q = 0; q < 8; ++q)
                        sts_v4(smem_u32(sm.part) + (uint32_t)(r * 512 + (((8 * ch + q) ^ lane) << 4)),
                               make_uint4(v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]));
                }
            }
        }
        if (ctas > 1) {
            __syncwarp();
            g2::cluster_sync(); // every slab's product is in its CTA's shared memory
            const int per = (m16 + ctas - 1) / ctas, r0 = rank * per, nr = min(per, m16 - r0);
            for (int i = tid; i < nr * 32; i += SM_THREADS) {
                const int row = r0 + (i >> 5), ch = i & 31;
                if (4 * ch >= m16)
                    continue;
                const uint32_t at = (uint32_t)(row * 512 + ((ch ^ (row & 31)) << 4));
                float4 a = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                for (int p0 = 0; p0 < ctas; p0 += 8) { // eight loads in flight, then their sum in rank order
                    float4 b[8];
#pragma unroll
                    for (int p = 0; p < 8; ++p)
                        if (p0 + p < ctas)
                            b[p] = ld_cluster_v4(g2::peer_addr(sm.part, (uint32_t)(p0 + p)) + at);
#pragma unroll
                    for (int p = 0; p < 8; ++p)
                        if (p0 + p < ctas)
                            a.x += b[p].x, a.y += b[p].y, a.z += b[p].z, a.w += b[p].w;
                }
                if (ch == row >> 2) { // the diagonal: to fp32 in every CTA, and out of A
                    const int i = row & 3;
                    const float x = i == 0 ? a.x : (i == 1 ? a.y : (i == 2 ? a.z : a.w));
                    for (int p = 0; p < ctas; ++p)
                        st_cluster_f32(g2::peer_addr(&sm.alpha[row], (uint32_t)p), x * (1.0f / (SX * SX)));
                    a.x = i == 0 ? 0.0f : a.x, a.y = i == 1 ? 0.0f : a.y;
                    a.z = i == 2 ? 0.0f : a.z, a.w = i == 3 ? 0.0f : a.w;
                }
                constexpr float F = SA / (SX * SX);
                const uint32_t h0 = pack_half2(a.x * F, a.y * F), h1 = pack_half2(a.z * F, a.w * F);
                const uint32_t to = (uint32_t)((ch >> 4) * SM_M * 128) + swz(row, (ch & 15) * 8);
                for (int p = 0; p < ctas; ++p)
                    st_cluster_v2(g2::peer_addr(sm.ab[0], (uint32_t)p) + to, h0, h1);
            }
            fence_proxy_async_all();
            __syncwarp();
            g2::cluster_sync(); // A is whole in every CTA
        }
        // ---- B' from A' and alpha, in A's place, and beta
        product(d_b, sm.ab[0], sm.ab[0], false, m16, m16);
        if (active) {
#pragma unroll 1
            for (int ch = part; 32 * ch < m16; ch += 4) {
                uint32_t v[32];
                gm::tc_ld32(lanes + d_b + 32 * ch, v);
                const float alpha_r = sm.alpha[r];
                const float on_diag = take_diagonal(v, ch == quad ? lane : -1); // A' is zero there, so B' will be
                if (ch == quad)
                    sm.beta[r] = fmaf(fmaf(cc, alpha_r, cb), alpha_r, cc * (on_diag * (1.0f / (SA * SA))));
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    if (32 * ch + 8 * q < m16) {
                        uint8_t *p = sm.ab[ch >> 1] + swz(r, (ch & 1) * 64 + 16 * q);
                        const uint4 a = *reinterpret_cast<const uint4 *>(p);
                        const uint32_t w[4] = {a.x, a.y, a.z, a.w};
                        uint32_t h[4];
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            const float2 f = unpack_half2(w[k]);
                            const float2 ac = *reinterpret_cast<const float2 *>(&sm.alpha[32 * ch + 8 * q + 2 * k]);
                            h[k] = pack_half2(fmaf(pc * (1.0f / SA), __uint_as_float(v[8 * q + 2 * k]),
                                                   fmaf(pc, alpha_r + ac.x, pb) * f.x),
                                              fmaf(pc * (1.0f / SA), __uint_as_float(v[8 * q + 2 * k + 1]),
                                                   fmaf(pc, alpha_r + ac.y, pb) * f.y));
                        }
                        *reinterpret_cast<uint4 *>(p) = make_uint4(h[0], h[1], h[2], h[3]);
                    }
            }
        }
        // ---- X = (a + beta) X + B' X
        product(d_y, sm.ab[0], sm.xh[0], true, n16, m16);
        if (active) {
            const float scale = co.v[3 * s] + sm.beta[r], unscale = co.unscale[s];
#pragma unroll 1
            for (int ch = part; 32 * ch < n16; ch += 4) {
                uint32_t v[32], y[32];
                float x[32];
                gm::tc_ld32_nowait(lanes + d_x + 32 * ch, v);
                gm::tc_ld32_nowait(lanes + d_y + 32 * ch, y);
                gm::tc_wait_ld();
#pragma unroll
                for (int k = 0; k < 32; ++k) // behind n16 no product was written, and X is zero
                    x[k] = fmaf(scale, __uint_as_float(v[k]),
                                32 * ch + (k & 16) < n16 ? __uint_as_float(y[k]) * unscale : 0.0f);
                const int c0 = 32 * ch;
                if (s + 1 < steps) {
                    put_x(c0, x);
#pragma unroll
                    for (int k = 0; k < 32; ++k)
                        v[k] = __float_as_uint(x[k]);
                    tc_st32(lanes + d_x + c0, v);
                } else {
                    uint32_t h[16];
#pragma unroll
                    for (int k = 0; k < 16; ++k)
                        h[k] = gm::pack_bf16x2(x[2 * k] * (1.0f / SX), x[2 * k + 1] * (1.0f / SX));
                    uint16_t *dst = out + (int64_t)e * rows * cols;
                    if (tall) {
                        dst += (int64_t)(c_base + c0) * m + r;
#pragma unroll
                        for (int k = 0; k < 32; ++k)
                            if (r < m && c0 + k < ncol)
                                dst[(int64_t)k * m] = (uint16_t)(k & 1 ? h[k >> 1] >> 16 : h[k >> 1]);
                    } else { // turned over where hi was: its last product is done
                        rows_out(sm.xh[0] + warp * CHUNK_BYTES, h, dst + (int64_t)(32 * quad) * n + c_base + c0, n,
                                 m - 32 * quad, ncol - c0, out_vec);
                    }
                }
            }
            tc_wait_st();
        }
    }

    __syncwarp();
    gm::tc_fence_before();
    g2::cluster_sync(); // no CTA's shared memory goes while another may read it
    gm::tc_fence_after();
    if (warp == 0)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(sm.tmem_base), "r"(512u) : "memory");
}

} // namespace ns
} // namespace mxq

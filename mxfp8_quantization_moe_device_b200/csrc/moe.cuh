// moe.cuh - the operators that surround the experts' grouped GEMMs: the
// router (softmax, k best experts, per-expert counts, balance loss, and their
// gradient), the order of the tokens by expert, and the movement of the token
// rows into that order and back.
//
//   route      p = softmax(logits[t]); ids = the k largest logits, ties to the
//              lowest index; w_j = p[id_j], or divided by their sum
//              loss = E sum_e (c_e / (k n)) (1/n sum_t p_te), c_e the number
//              of times expert e was chosen, n the number of valid tokens
//   plan       pos[t][j] = place of entry (t, j) in the stable order by expert
//   dispatch   xs[pos[t][j]] = x[t]
//   combine    out[t] = sum_j w[t][j] y[pos[t][j]]
//
// An expert with logit -inf is never chosen; a slot for which no expert is
// left has id -1 and weight 0, and its pos is -1. Every sum is taken in a
// fixed order, so results do not change from run to run.
#pragma once

#include "common.cuh"

namespace mxq {
namespace moe {

constexpr int MAX_E = 1024;
constexpr int MAX_K = 32;

// bf16 or fp32 element access; V elements (V * size a power of two up to 16
// bytes) move as one word or vector
template <typename T> struct Elem;
template <> struct Elem<uint16_t> {
    static MXQ_DEV float get(uint16_t v) { return __uint_as_float((uint32_t)v << 16); }
    static MXQ_DEV uint16_t put(float f)
    {
        uint16_t r;
        asm("cvt.rn.bf16.f32 %0, %1;" : "=h"(r) : "f"(f));
        return r;
    }
};
template <> struct Elem<float> {
    static MXQ_DEV float get(float v) { return v; }
    static MXQ_DEV float put(float f) { return f; }
};

template <typename T, int V> struct alignas(sizeof(T) * V) Vec {
    T v[V];
};

template <typename T, int V> MXQ_DEV Vec<T, V> ld_vec(const T *p) { return *reinterpret_cast<const Vec<T, V> *>(p); }
template <typename T, int V> MXQ_DEV void st_vec(T *p, const Vec<T, V> &x) { *reinterpret_cast<Vec<T, V> *>(p) = x; }

// unsigned key in the order of the float (-inf lowest; the caller has turned
// -0 into +0 and has no NaN)
MXQ_DEV uint32_t order_key(float f)
{
    const uint32_t b = __float_as_uint(f);
    return b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
}
MXQ_DEV float key_value(uint32_t k) { return __uint_as_float(k ^ ((uint32_t)((int32_t)~k >> 31) | 0x80000000u)); }

template <int LPT> MXQ_DEV uint32_t group_max(uint32_t x)
{
    if constexpr (LPT == 32) {
        return __reduce_max_sync(0xffffffffu, x);
    } else {
#pragma unroll
        for (int o = 1; o < LPT; o <<= 1)
            x = max(x, __shfl_xor_sync(0xffffffffu, x, o));
        return x;
    }
}
template <int LPT> MXQ_DEV float group_sum(float x)
{
#pragma unroll
    for (int o = 1; o < LPT; o <<= 1)
        x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}

// a token's logits: lane i of its LPT lanes holds experts [i EPL, (i+1) EPL);
// experts from E on read as -inf
template <typename T, int EPL> MXQ_DEV void load_logits(const T *row, int e0, int E, bool vec, float (&v)[EPL])
{
    if (vec && e0 + EPL <= E) {
        constexpr int V = 16 / sizeof(T);
#pragma unroll
        for (int i = 0; i < EPL; i += V) {
            const Vec<T, V> x = ld_vec<T, V>(row + e0 + i);
#pragma unroll
            for (int j = 0; j < V; ++j)
                v[i + j] = Elem<T>::get(x.v[j]);
        }
    } else {
#pragma unroll
        for (int i = 0; i < EPL; ++i)
            v[i] = e0 + i < E ? Elem<T>::get(row[e0 + i]) : -INFINITY;
    }
}

// softmax over the token's lanes: v becomes p, returns the largest logit.
// A row of -inf alone has p = 0. A row with a NaN or +inf has p = NaN.
// `bad` is the same in all lanes of the token.
template <int LPT, int EPL> MXQ_DEV float softmax(float (&v)[EPL], bool live, bool &bad, float &rz)
{
    const int lane = threadIdx.x & 31;
    float m = v[0];
    bool odd = !(v[0] < INFINITY);
#pragma unroll
    for (int i = 1; i < EPL; ++i) {
        m = fmaxf(m, v[i]);
        odd |= !(v[i] < INFINITY);
    }
    const uint32_t group = LPT == 32 ? 0xffffffffu : ((1u << LPT) - 1u) << (lane & ~(LPT - 1));
    // every lane takes part in the vote and in the maxima, whatever its row
    const uint32_t odd_lanes = __ballot_sync(0xffffffffu, odd);
    bad = live && (odd_lanes & group) != 0;
    m = key_value(group_max<LPT>(order_key(m + 0.0f)));
    const bool some = live && m > -INFINITY && !bad;
    const float base = some ? m : 0.0f;
    float z = 0.0f;
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
        v[i] = some ? expf(v[i] - base) : 0.0f;
        z += v[i];
    }
    z = group_sum<LPT>(z);
    rz = bad ? NAN : (some ? __fdiv_rn(1.0f, z) : 0.0f);
#pragma unroll
    for (int i = 0; i < EPL; ++i)
        v[i] = bad ? NAN : v[i] * rz;
    return m;
}

constexpr int ROUTE_THREADS = 256;
constexpr int ROUTE_WARPS = ROUTE_THREADS / 32;

// bytes of the ids and weights that a CTA stages before it stores them
__host__ __device__ constexpr size_t route_stage_bytes(int tpw, int k) { return (size_t)ROUTE_WARPS * tpw * k * 8; }

// what the CTAs leave for the finishing kernel: rows of E sums of p and of
// choice counts per CTA, the valid tokens per CTA, partial losses, a ticket
struct RoutePart {
    float *p;       // (R, E)
    int *c;         // (R, E)
    int *n;         // (R)
    double *loss;   // (ceil(E / 32))
    int *ticket;
};

// loss = f sum_e c_e P_e with P_e the sum of p_te over the tokens and
// f = E / (k n^2); its derivative by p_te is f c_e for every token
MXQ_DEV double loss_factor(int E, int k, double n) { return n > 0.0 ? (double)E / ((double)k * n * n) : 0.0; }

} // namespace moe

// Router forward: a token on LPT lanes with EPL experts each, 32 / LPT tokens
// per warp at a time.
template <typename T, int LPT, int EPL>
__global__ void __launch_bounds__(moe::ROUTE_THREADS)
    k_moe_route(const T *__restrict__ logits, int64_t tokens, int E, int64_t ld, const uint8_t *__restrict__ valid,
                int k, int renorm, int vec, float *__restrict__ weights, int32_t *__restrict__ ids,
                moe::RoutePart part, int32_t *counts, float *loss, float *loss_grad)
{
    using namespace moe;
    constexpr int TPW = 32 / LPT;
    extern __shared__ __align__(16) uint8_t smem[];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int sub = lane / LPT, li = lane % LPT, e0 = li * EPL;
    int *s_ids = reinterpret_cast<int *>(smem) + (size_t)warp * TPW * k;
    float *s_w = reinterpret_cast<float *>(smem + route_stage_bytes(TPW, k) / 2) + (size_t)warp * TPW * k;
    float *s_p = reinterpret_cast<float *>(smem + route_stage_bytes(TPW, k)); // (warps, E)
    int *s_c = reinterpret_cast<int *>(s_p + (size_t)ROUTE_WARPS * E);        // E
    __shared__ int s_n;
    for (int e = tid; e < E; e += ROUTE_THREADS)
        s_c[e] = 0;
    if (tid == 0)
        s_n = 0;
    __syncthreads();

    float acc[EPL];
#pragma unroll
    for (int i = 0; i < EPL; ++i)
        acc[i] = 0.0f;
    int nvalid = 0;
    const int64_t step = (int64_t)gridDim.x * ROUTE_WARPS * TPW;
    for (int64_t t0 = ((int64_t)blockIdx.x * ROUTE_WARPS + warp) * TPW; t0 < tokens; t0 += step) {
        const int64_t t = t0 + sub;
        const bool in = t < tokens;
        const bool live = in && (!valid || valid[t]);
        float v[EPL];
        if (in)
            load_logits<T, EPL>(logits + t * ld, e0, E, vec, v);
        else
#pragma unroll
            for (int i = 0; i < EPL; ++i)
                v[i] = -INFINITY;
        // selection keys: the logit's order; for 16-bit logits the index in
        // the low half, so that one maximum gives both
        uint32_t c[EPL];
#pragma unroll
        for (int i = 0; i < EPL; ++i) {
            const bool can = live && v[i] > -INFINITY;
            const uint32_t key = order_key(v[i] + 0.0f);
            c[i] = !can ? 0u : (sizeof(T) == 2 ? ((key & 0xFFFF0000u) | (0xFFFFu - (uint32_t)(e0 + i))) : key);
        }
        bool bad;
        float rz;
        const float m = softmax<LPT, EPL>(v, live, bad, rz);
#pragma unroll
        for (int i = 0; i < EPL; ++i)
            acc[i] += v[i];
        nvalid += live && li == 0;
        float ssum = 0.0f;
        for (int j = 0; j < k; ++j) {
            uint32_t best = c[0];
#pragma unroll
            for (int i = 1; i < EPL; ++i)
                best = max(best, c[i]);
            uint32_t g = group_max<LPT>(best);
            g = bad ? 0u : g;
            int e = -1;
            float val = 0.0f;
            if (sizeof(T) == 2) {
                if (g) {
                    e = (int)(0xFFFFu - (g & 0xFFFFu));
                    // a negative value's key has its cleared low half inverted
                    val = key_value((g & 0x80000000u) ? (g & 0xFFFF0000u) : (g | 0xFFFFu));
                }
#pragma unroll
                for (int i = 0; i < EPL; ++i)
                    c[i] = c[i] == g ? 0u : c[i];
            } else {
                // the first lane with the largest key, then its first expert
                const uint32_t group = LPT == 32 ? 0xffffffffu : ((1u << LPT) - 1u) << (lane & ~(LPT - 1));
                const uint32_t who = __ballot_sync(0xffffffffu, best == g) & group;
                const int src = __ffs(who) - 1;
                int mine = 0;
#pragma unroll
                for (int i = EPL - 1; i >= 0; --i)
                    mine = c[i] == g ? i : mine;
                if (lane == src)
#pragma unroll
                    for (int i = 0; i < EPL; ++i)
                        c[i] = i == mine ? 0u : c[i];
                const int eo = __shfl_sync(0xffffffffu, e0 + mine, src < 0 ? lane : src);
                if (g) {
                    e = eo;
                    val = key_value(g);
                }
            }
            const float w = bad ? NAN : (e >= 0 ? expf(val - m) : 0.0f);
            ssum += w;
            if (li == 0) {
                s_ids[sub * k + j] = e;
                s_w[sub * k + j] = w;
                if (e >= 0)
                    atomicAdd(&s_c[e], 1);
            }
        }
        const float scale = renorm ? (ssum > 0.0f ? __fdiv_rn(1.0f, ssum) : (bad ? NAN : 0.0f)) : rz;
        __syncwarp();
        for (int j = li; j < k; j += LPT)
            s_w[sub * k + j] *= scale;
        __syncwarp();
        const int64_t left = (tokens - t0 < TPW ? tokens - t0 : TPW) * k;
        for (int i = lane; i < left; i += 32) {
            ids[t0 * k + i] = s_ids[i];
            weights[t0 * k + i] = s_w[i];
        }
        __syncwarp();
    }
    // the warp's tokens of one expert, then the CTA's warps in order
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
#pragma unroll
        for (int o = LPT; o < 32; o <<= 1)
            acc[i] += __shfl_xor_sync(0xffffffffu, acc[i], o);
        if (sub == 0 && e0 + i < E)
            s_p[(size_t)warp * E + e0 + i] = acc[i];
    }
    for (int o = 16; o; o >>= 1)
        nvalid += __shfl_xor_sync(0xffffffffu, nvalid, o);
    if (lane == 0)
        atomicAdd(&s_n, nvalid);
    __syncthreads();
    for (int e = tid; e < E; e += ROUTE_THREADS) {
        float p = 0.0f;
#pragma unroll
        for (int w = 0; w < ROUTE_WARPS; ++w)
            p += s_p[(size_t)w * E + e];
        s_p[e] = p; // row 0, which this thread alone reads from here on
        part.p[(size_t)blockIdx.x * E + e] = p;
        part.c[(size_t)blockIdx.x * E + e] = s_c[e];
    }
    if (tid == 0) {
        part.n[blockIdx.x] = s_n;
        if (blockIdx.x == 0)
            *part.ticket = 0;
    }
    if (gridDim.x == 1) { // one CTA saw every token: it finishes alone
        __shared__ double s_loss[ROUTE_WARPS];
        const double f = loss_factor(E, k, (double)s_n);
        double sum = 0.0;
        for (int e = tid; e < E; e += ROUTE_THREADS) {
            const int c = s_c[e];
            counts[e] = c;
            if (loss_grad)
                loss_grad[e] = (float)(f * c);
            sum += (double)s_p[e] * c;
        }
        for (int o = 16; o; o >>= 1)
            sum += __shfl_xor_sync(0xffffffffu, sum, o);
        if (lane == 0)
            s_loss[warp] = sum;
        __syncthreads();
        if (tid == 0) {
            for (int w = 1; w < ROUTE_WARPS; ++w)
                sum += s_loss[w];
            *loss = (float)(f * sum);
        }
    }
}

// Sums over the CTAs: a CTA of 32 warps takes 32 experts (one per lane), warp
// w the rows w, w + 32, ...; the last CTA to finish adds the partial losses
// in order.
__global__ void __launch_bounds__(1024)
    k_moe_route_finish(moe::RoutePart part, int R, int E, int k, int32_t *counts, float *loss, float *loss_grad)
{
    using namespace moe;
    __shared__ double s_p[32][33];
    __shared__ int s_c[32][33];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int e = blockIdx.x * 32 + lane;
    double p = 0.0;
    int c = 0;
    if (e < E) {
#pragma unroll 8
        for (int r = warp; r < R; r += 32) {
            p += (double)part.p[(size_t)r * E + e];
            c += part.c[(size_t)r * E + e];
        }
    }
    s_p[warp][lane] = p;
    s_c[warp][lane] = c;
    __syncthreads();
    if (warp)
        return;
    long long n = 0;
    for (int r = lane; r < R; r += 32)
        n += part.n[r];
    p = 0.0;
    c = 0;
#pragma unroll
    for (int w = 0; w < 32; ++w) {
        p += s_p[w][lane];
        c += s_c[w][lane];
    }
    for (int o = 16; o; o >>= 1)
        n += __shfl_xor_sync(0xffffffffu, n, o);
    const double f = loss_factor(E, k, (double)n);
    double sum = 0.0;
    if (e < E) {
        counts[e] = c;
        if (loss_grad)
            loss_grad[e] = (float)(f * c);
        sum = p * c;
    }
    for (int o = 16; o; o >>= 1)
        sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if (lane == 0) {
        part.loss[blockIdx.x] = sum;
        __threadfence();
        if (atomicAdd(part.ticket, 1) == (int)gridDim.x - 1) {
            __threadfence();
            double s = 0.0;
            for (unsigned b = 0; b < gridDim.x; ++b)
                s += reinterpret_cast<volatile double *>(part.loss)[b];
            *loss = (float)(f * s);
        }
    }
}

// Router backward. With G = sum_j g_j w_j and b_e = grad_loss * loss_grad[e]
//   dl_e = p_e (b_e - sum p b) + { w_j g_j where e = id_j, - p_e G    plain
//                                { w_j (g_j - G) where e = id_j       renormalized
template <typename T, int LPT, int EPL>
__global__ void __launch_bounds__(moe::ROUTE_THREADS)
    k_moe_route_bwd(const T *__restrict__ logits, int64_t tokens, int E, int64_t ld, const uint8_t *__restrict__ valid,
                    int k, int renorm, int vec, const float *__restrict__ weights, const int32_t *__restrict__ ids,
                    const float *__restrict__ loss_grad, const float *__restrict__ gw, const float *__restrict__ gl,
                    T *__restrict__ out)
{
    using namespace moe;
    constexpr int TPW = 32 / LPT;
    extern __shared__ __align__(16) uint8_t smem[];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int sub = lane / LPT, li = lane % LPT, e0 = li * EPL;
    float *s_q = reinterpret_cast<float *>(smem) + (size_t)warp * 32 * EPL + sub * (LPT * EPL);
    float b[EPL];
    const float g_loss = gl ? *gl : 0.0f;
#pragma unroll
    for (int i = 0; i < EPL; ++i)
        b[i] = gl && e0 + i < E ? g_loss * loss_grad[e0 + i] : 0.0f;
    const int64_t step = (int64_t)gridDim.x * ROUTE_WARPS * TPW;
    for (int64_t t0 = ((int64_t)blockIdx.x * ROUTE_WARPS + warp) * TPW; t0 < tokens; t0 += step) {
        const int64_t t = t0 + sub;
        const bool in = t < tokens;
        const bool live = in && (!valid || valid[t]);
        float v[EPL];
        if (in)
            load_logits<T, EPL>(logits + t * ld, e0, E, vec, v);
        else
#pragma unroll
            for (int i = 0; i < EPL; ++i)
                v[i] = -INFINITY;
#pragma unroll
        for (int i = 0; i < EPL; ++i)
            s_q[e0 + i] = 0.0f;
        __syncwarp();
        bool bad;
        float rz;
        softmax<LPT, EPL>(v, live, bad, rz);
        float G = 0.0f;
        if (gw) {
            if (live && !bad)
                for (int j = li; j < k; j += LPT)
                    if (ids[t * k + j] >= 0)
                        G = fmaf(gw[t * k + j], weights[t * k + j], G);
            G = group_sum<LPT>(G);
            if (live && !bad)
                for (int j = li; j < k; j += LPT) {
                    const int e = ids[t * k + j];
                    if (e >= 0 && e < E) {
                        const float g = gw[t * k + j];
                        atomicAdd(&s_q[e], weights[t * k + j] * (renorm ? g - G : g));
                    }
                }
        }
        __syncwarp();
        float pb = 0.0f;
#pragma unroll
        for (int i = 0; i < EPL; ++i)
            pb = fmaf(v[i], b[i], pb);
        pb = group_sum<LPT>(pb) + (renorm ? 0.0f : G);
        float d[EPL];
#pragma unroll
        for (int i = 0; i < EPL; ++i)
            d[i] = fmaf(v[i], b[i] - pb, s_q[e0 + i]);
        if (in) {
            T *row = out + t * E;
            if (vec && e0 + EPL <= E) {
                constexpr int V = 16 / sizeof(T);
#pragma unroll
                for (int i = 0; i < EPL; i += V) {
                    Vec<T, V> x;
#pragma unroll
                    for (int j = 0; j < V; ++j)
                        x.v[j] = Elem<T>::put(d[i + j]);
                    st_vec<T, V>(row + e0 + i, x);
                }
            } else {
#pragma unroll
                for (int i = 0; i < EPL; ++i)
                    if (e0 + i < E)
                        row[e0 + i] = Elem<T>::put(d[i]);
            }
        }
        __syncwarp();
    }
}

// ---------------------------------------------------------------------------
// Order by expert. The n = tokens * k entries are cut into C chunks of whole
// tiles; pass 1 counts each chunk's entries per expert, pass 2 adds the counts
// of smaller experts and of earlier chunks and ranks the chunk's entries:
// a warp owns a run of a tile's entries, ranks 32 of them at a time among
// their equals (match.any), and the warps' counters are then summed in order.
// One chunk needs no pass 1. No atomics across CTAs, nothing to clear.
namespace moe {
constexpr int PLAN_THREADS = 1024;
constexpr int PLAN_WARPS = PLAN_THREADS / 32;
constexpr int PLAN_R = 8;                                // entries per thread and tile
constexpr int PLAN_TILE = PLAN_THREADS * PLAN_R;         // 8192
constexpr int PLAN_MAX_CHUNKS = 64;

// expert of entry i: -1 outside [0, E) and behind the end
MXQ_DEV int entry_expert(const int32_t *ids, int64_t i, int64_t end, int E)
{
    if (i >= end)
        return -1;
    const int e = ids[i];
    if (e >= E)
        set_status(MXQ_ERR_BAD_INDEX);
    return e < 0 || e >= E ? -1 : e;
}
} // namespace moe

__global__ void __launch_bounds__(moe::PLAN_THREADS)
    k_moe_plan_count(const int32_t *__restrict__ ids, int64_t n, int E, int64_t chunk, int *__restrict__ hist)
{
    using namespace moe;
    extern __shared__ int s_h[];
    for (int e = threadIdx.x; e < E; e += PLAN_THREADS)
        s_h[e] = 0;
    __syncthreads();
    const int64_t lo = blockIdx.x * chunk, hi = lo + chunk < n ? lo + chunk : n;
    for (int64_t i0 = lo; i0 < hi; i0 += PLAN_TILE) {
        int e[PLAN_R];
#pragma unroll
        for (int r = 0; r < PLAN_R; ++r)
            e[r] = entry_expert(ids, i0 + r * PLAN_THREADS + threadIdx.x, hi, E);
#pragma unroll
        for (int r = 0; r < PLAN_R; ++r)
            if (e[r] >= 0)
                atomicAdd(&s_h[e[r]], 1);
    }
    __syncthreads();
    for (int e = threadIdx.x; e < E; e += PLAN_THREADS)
        hist[(size_t)blockIdx.x * E + e] = s_h[e];
}

// hist (C, E) of pass 1, or NULL when the grid is one CTA over one tile
__global__ void __launch_bounds__(moe::PLAN_THREADS)
    k_moe_plan_rank(const int32_t *__restrict__ ids, int64_t n, int E, int64_t chunk, const int *__restrict__ hist,
                    int C, int32_t *__restrict__ pos, int32_t *__restrict__ offs)
{
    using namespace moe;
    extern __shared__ int smem_i[];
    int *base = smem_i;                                              // E: next position of each expert
    uint16_t *cnt = reinterpret_cast<uint16_t *>(smem_i + MAX_E);    // (warps, E)
    __shared__ int s_scan[PLAN_WARPS];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int64_t lo = blockIdx.x * chunk, hi = lo + chunk < n ? lo + chunk : n;

    // exclusive sum over the experts of `total`, plus `before`; the last
    // thread's inclusive sums are the group ends
    auto set_base = [&](int total, int before) {
        int x = total;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, x, o);
            if (lane >= o)
                x += y;
        }
        if (lane == 31)
            s_scan[warp] = x;
        __syncthreads();
        if (warp == 0) {
            int s = s_scan[lane];
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int y = __shfl_up_sync(0xffffffffu, s, o);
                if (lane >= o)
                    s += y;
            }
            s_scan[lane] = s;
        }
        __syncthreads();
        x += warp ? s_scan[warp - 1] : 0;
        if (tid < E) {
            base[tid] = x - total + before;
            if (blockIdx.x == 0)
                offs[tid] = x;
        }
        __syncthreads();
    };

    if (hist) {
        int total = 0, before = 0;
        if (tid < E) {
#pragma unroll 16
            for (int c = 0; c < C; ++c) {
                const int h = hist[(size_t)c * E + tid];
                total += h;
                before += c < (int)blockIdx.x ? h : 0;
            }
        }
        set_base(total, before);
    }
    for (int64_t i0 = lo; i0 < hi || i0 == 0; i0 += PLAN_TILE) {
        for (int e = tid; e < PLAN_WARPS * E; e += PLAN_THREADS)
            cnt[e] = 0;
        __syncthreads();
        uint16_t *mine = cnt + (size_t)warp * E;
        int e[PLAN_R], rank[PLAN_R];
#pragma unroll
        for (int r = 0; r < PLAN_R; ++r)
            e[r] = entry_expert(ids, i0 + (int64_t)warp * (32 * PLAN_R) + r * 32 + lane, hi, E);
#pragma unroll
        for (int r = 0; r < PLAN_R; ++r) {
            const uint32_t peers = __match_any_sync(0xffffffffu, e[r]);
            const int before = e[r] >= 0 ? mine[e[r]] : 0;
            rank[r] = before + __popc(peers & ((1u << lane) - 1u));
            __syncwarp();
            if (e[r] >= 0 && lane == __ffs(peers) - 1)
                mine[e[r]] = (uint16_t)(before + __popc(peers));
            __syncwarp();
        }
        __syncthreads();
        // the warps' counters become each warp's first rank within the tile
        int tile_total = 0;
        if (tid < E) {
#pragma unroll 8
            for (int w = 0; w < PLAN_WARPS; ++w) {
                const int c = cnt[(size_t)w * E + tid];
                cnt[(size_t)w * E + tid] = (uint16_t)tile_total;
                tile_total += c;
            }
        }
        if (!hist)
            set_base(tile_total, 0); // the only tile
        __syncthreads();
#pragma unroll
        for (int r = 0; r < PLAN_R; ++r) {
            const int64_t i = i0 + (int64_t)warp * (32 * PLAN_R) + r * 32 + lane;
            if (i < hi)
                pos[i] = e[r] >= 0 ? base[e[r]] + mine[e[r]] + rank[r] : -1;
        }
        __syncthreads();
        if (tid < E)
            base[tid] += tile_total;
    }
}

// ---------------------------------------------------------------------------
// Row movement. A warp moves a segment of 32 * U vectors of V elements of one
// row; pos of up to 32 slots sits in the warp's lanes.
namespace moe {
constexpr int ROW_THREADS = 256;
constexpr int ROW_WARPS = ROW_THREADS / 32;

// a slot's row: -1 when dropped; a place outside [0, M) is reported
MXQ_DEV int64_t slot_row(const int32_t *pos, int64_t i, int64_t M)
{
    const int p = pos[i];
    if (p >= M)
        set_status(MXQ_ERR_BAD_INDEX);
    return p < 0 || p >= M ? -1 : p;
}
} // namespace moe

// xs[pos[t][j]] = x[t]; rows from offs[E-1] to M are zero
template <typename T, int V, int U>
__global__ void __launch_bounds__(moe::ROW_THREADS)
    k_moe_dispatch(const T *__restrict__ x, int64_t tokens, int64_t K, int64_t ld, const int32_t *__restrict__ pos,
                   int k, const int32_t *__restrict__ offs, int E, T *__restrict__ out, int64_t M)
{
    using namespace moe;
    const int lane = threadIdx.x & 31;
    const int64_t nvec = K / V, segs = (nvec + 32 * U - 1) / (32 * U);
    const int64_t end = max(0, offs[E - 1]);
    const int64_t copies = tokens * segs, all = copies + (end < M ? (M - end) * segs : 0);
    for (int64_t w = (int64_t)blockIdx.x * ROW_WARPS + (threadIdx.x >> 5); w < all;
         w += (int64_t)gridDim.x * ROW_WARPS) {
        if (w < copies) {
            const int64_t t = w / segs, v0 = (w - t * segs) * (32 * U) + lane;
            const int64_t row = lane < k ? slot_row(pos, t * k + lane, M) : -1;
            Vec<T, V> r[U];
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (v0 + 32 * u < nvec)
                    r[u] = ld_vec<T, V>(x + t * ld + (v0 + 32 * u) * V);
            for (int j = 0; j < k; ++j) {
                const int64_t d = __shfl_sync(0xffffffffu, row, j);
                if (d < 0)
                    continue;
#pragma unroll
                for (int u = 0; u < U; ++u)
                    if (v0 + 32 * u < nvec)
                        st_vec<T, V>(out + d * K + (v0 + 32 * u) * V, r[u]);
            }
        } else {
            const int64_t z = w - copies, d = end + z / segs, v0 = (z % segs) * (32 * U) + lane;
            Vec<T, V> zero = {};
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (v0 + 32 * u < nvec)
                    st_vec<T, V>(out + d * K + (v0 + 32 * u) * V, zero);
        }
    }
}

// out[t] = sum_j w[t][j] y[pos[t][j]] (w NULL: ones), slots in order, fp32
template <typename T, int V, int U>
__global__ void __launch_bounds__(moe::ROW_THREADS)
    k_moe_combine(const T *__restrict__ y, int64_t M, int64_t K, int64_t ld, const int32_t *__restrict__ pos,
                  const float *__restrict__ weights, int64_t tokens, int k, T *__restrict__ out)
{
    using namespace moe;
    const int lane = threadIdx.x & 31;
    const int64_t nvec = K / V, segs = (nvec + 32 * U - 1) / (32 * U), all = tokens * segs;
    for (int64_t w = (int64_t)blockIdx.x * ROW_WARPS + (threadIdx.x >> 5); w < all;
         w += (int64_t)gridDim.x * ROW_WARPS) {
        const int64_t t = w / segs, v0 = (w - t * segs) * (32 * U) + lane;
        const int64_t row = lane < k ? slot_row(pos, t * k + lane, M) : -1;
        const float wl = lane < k ? (weights ? weights[t * k + lane] : 1.0f) : 0.0f;
        float acc[U][V];
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int i = 0; i < V; ++i)
                acc[u][i] = 0.0f;
        for (int j0 = 0; j0 < k; j0 += 4) {
            Vec<T, V> r[4][U];
            int64_t s[4];
            float wj[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) { // lanes from k on hold -1
                s[j] = __shfl_sync(0xffffffffu, row, (j0 + j) & 31);
                wj[j] = __shfl_sync(0xffffffffu, wl, (j0 + j) & 31);
                if (j0 + j >= k)
                    s[j] = -1;
#pragma unroll
                for (int u = 0; u < U; ++u)
                    if (s[j] >= 0 && v0 + 32 * u < nvec)
                        r[j][u] = ld_vec<T, V>(y + s[j] * ld + (v0 + 32 * u) * V);
            }
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (s[j] >= 0)
#pragma unroll
                    for (int u = 0; u < U; ++u)
#pragma unroll
                        for (int i = 0; i < V; ++i)
                            acc[u][i] = fmaf(wj[j], Elem<T>::get(r[j][u].v[i]), acc[u][i]);
        }
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (v0 + 32 * u < nvec) {
                Vec<T, V> o;
#pragma unroll
                for (int i = 0; i < V; ++i)
                    o.v[i] = Elem<T>::put(acc[u][i]);
                st_vec<T, V>(out + t * K + (v0 + 32 * u) * V, o);
            }
    }
}

// dy[pos[t][j]] = w[t][j] dout[t] and dw[t][j] = <dout[t], y[pos[t][j]]>, a
// warp per entry; rows of dy from offs[E-1] to M are zero. dy or dw may be
// NULL.
template <typename T, int V, int U>
__global__ void __launch_bounds__(moe::ROW_THREADS)
    k_moe_combine_bwd(const T *__restrict__ dout, int64_t ldd, const T *__restrict__ y, int64_t ldy, int64_t M,
                      int64_t K, const int32_t *__restrict__ pos, const float *__restrict__ weights, int64_t tokens,
                      int k, const int32_t *__restrict__ offs, int E, T *__restrict__ dy, float *__restrict__ dw)
{
    using namespace moe;
    const int lane = threadIdx.x & 31;
    const int64_t nvec = K / V, n = tokens * k;
    const int64_t end = max(0, offs[E - 1]);
    const int64_t all = n + (dy && end < M ? M - end : 0);
    for (int64_t w = (int64_t)blockIdx.x * ROW_WARPS + (threadIdx.x >> 5); w < all;
         w += (int64_t)gridDim.x * ROW_WARPS) {
        if (w >= n) {
            Vec<T, V> zero = {};
            T *d = dy + (end + w - n) * K;
            for (int64_t v = lane; v < nvec; v += 32)
                st_vec<T, V>(d + v * V, zero);
            continue;
        }
        const int64_t s = slot_row(pos, w, M);
        if (s < 0) {
            if (dw && lane == 0)
                dw[w] = 0.0f;
            continue;
        }
        const T *g = dout + (w / k) * ldd;
        const float wt = weights ? weights[w] : 1.0f;
        float acc = 0.0f;
        for (int64_t v0 = lane; v0 < nvec; v0 += 32 * U) {
            Vec<T, V> a[U], b[U];
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (v0 + 32 * u < nvec) {
                    a[u] = ld_vec<T, V>(g + (v0 + 32 * u) * V);
                    if (dw)
                        b[u] = ld_vec<T, V>(y + s * ldy + (v0 + 32 * u) * V);
                }
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (v0 + 32 * u < nvec) {
                    Vec<T, V> o;
#pragma unroll
                    for (int i = 0; i < V; ++i) {
                        const float f = Elem<T>::get(a[u].v[i]);
                        if (dw)
                            acc = fmaf(f, Elem<T>::get(b[u].v[i]), acc);
                        o.v[i] = Elem<T>::put(wt * f);
                    }
                    if (dy)
                        st_vec<T, V>(dy + s * K + (v0 + 32 * u) * V, o);
                }
        }
        if (dw) {
#pragma unroll
            for (int o = 16; o; o >>= 1)
                acc += __shfl_xor_sync(0xffffffffu, acc, o);
            if (lane == 0)
                dw[w] = acc;
        }
    }
}

} // namespace mxq

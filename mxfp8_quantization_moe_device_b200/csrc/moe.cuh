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

#include <type_traits>

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

MXQ_DEV uint32_t pack_bf16(float lo, float hi)
{
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

template <typename T, int V> struct alignas(sizeof(T) * V) Vec {
    T v[V];
};

template <typename T, int V> MXQ_DEV Vec<T, V> ld_vec(const T *p) { return *reinterpret_cast<const Vec<T, V> *>(p); }
template <typename T, int V> MXQ_DEV void st_vec(T *p, const Vec<T, V> &x) { *reinterpret_cast<Vec<T, V> *>(p) = x; }

// Load of one vector that stays where it is written: left to itself the
// compiler moves a batch of loads down to their uses, one at a time.
template <typename T, int V> MXQ_DEV Vec<T, V> ld_now(const T *p)
{
    Vec<T, V> x;
    if constexpr (sizeof(T) * V == 16) {
        const uint4 w = ld_stream_v4(p);
        memcpy(&x, &w, 16);
    } else if constexpr (sizeof(T) * V == 4) {
        uint32_t w;
        asm volatile("ld.global.nc.u32 %0, [%1];" : "=r"(w) : "l"(p));
        memcpy(&x, &w, 4);
    } else {
        uint16_t w;
        asm volatile("ld.global.nc.u16 %0, [%1];" : "=h"(w) : "l"(p));
        memcpy(&x, &w, 2);
    }
    return x;
}

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

// A token's logits as raw words: lane i of its LPT lanes holds experts [i EPL,
// (i + 1) EPL); experts from E on read as -inf.
template <typename T, int EPL> struct Raw {
    static constexpr int W = EPL * (int)sizeof(T) / 4;
    static constexpr uint32_t NONE = sizeof(T) == 2 ? 0xFF80FF80u : 0xFF800000u; // -inf
    uint32_t w[W];

    MXQ_DEV void none()
    {
#pragma unroll
        for (int i = 0; i < W; ++i)
            w[i] = NONE;
    }
    MXQ_DEV void load(const T *row, int e0, int E, bool vec)
    {
        if (vec && e0 + EPL <= E) {
#pragma unroll
            for (int i = 0; i < W; i += 4) {
                const uint4 x = ld_stream_v4(reinterpret_cast<const uint32_t *>(row + e0) + i);
                w[i] = x.x, w[i + 1] = x.y, w[i + 2] = x.z, w[i + 3] = x.w;
            }
        } else {
#pragma unroll
            for (int i = 0; i < EPL; ++i) {
                if constexpr (sizeof(T) == 2) {
                    const uint32_t h = e0 + i < E ? (uint32_t)row[e0 + i] : 0xFF80u;
                    w[i >> 1] = i & 1 ? w[i >> 1] | (h << 16) : h;
                } else {
                    w[i] = e0 + i < E ? __float_as_uint(row[e0 + i]) : NONE;
                }
            }
        }
    }
    MXQ_DEV float get(int i) const
    {
        if constexpr (sizeof(T) == 2)
            return i & 1 ? bf16_hi(w[i >> 1]) : bf16_lo(w[i >> 1]);
        else
            return __uint_as_float(w[i]);
    }
};

// 2^x by ex2.approx (2 ulp)
MXQ_DEV float exp2_fast(float x)
{
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
constexpr float LOG2E = 1.4426950408889634f;

// exp(v - m) as 2^(v log2(e) - c) with c = m log2(e): one instruction to the
// exponent, and c's own rounding is a factor of all of a token's values, which
// cancels. Where |m| is so large (2^20) that this factor is no small one, the
// token takes 2^((v - m) log2(e)); the other tokens of its warp keep theirs, so
// that a token's results are the same bits beside any others.
struct Shift {
    float m, c; // one of them is zero
    bool far;   // a token of the warp is far (the same in every lane)

    MXQ_DEV explicit Shift(float largest)
    {
        const bool mine = fabsf(largest) > 0x1p20f && largest != -INFINITY;
        m = mine ? largest : 0.0f;
        c = mine || largest == -INFINITY ? 0.0f : largest * LOG2E;
        far = __any_sync(0xffffffffu, mine);
    }
    MXQ_DEV float exp(float v) const { return exp2_fast(fmaf(v - m, LOG2E, -c)); }
};

// a token's logits in its lanes become exp(v - m), rz the reciprocal of their
// sum. A row of -inf alone gives zeros and rz 0; a row with a NaN or +inf gives
// rz NaN (m - m is NaN there) and returns true.
template <int LPT, int EPL> MXQ_DEV bool exponentials(float (&v)[EPL], const Shift &shift, float &rz)
{
    float z = 0.0f;
    if (shift.far) {
#pragma unroll
        for (int i = 0; i < EPL; ++i)
            v[i] = shift.exp(v[i]);
    } else { // m is zero
#pragma unroll
        for (int i = 0; i < EPL; ++i)
            v[i] = exp2_fast(fmaf(v[i], LOG2E, -shift.c));
    }
#pragma unroll
    for (int i = 0; i < EPL; ++i)
        z += v[i];
    z = group_sum<LPT>(z);
    rz = z == 0.0f ? 0.0f : __fdiv_rn(1.0f, z);
    return !(z == z);
}

// selection keys of a pair of bf16 logits (x low, y high): the order of the
// value above, the complement of the expert's index below. -0 becomes +0 by
// adding zero; a negative value's bits are all turned over, a positive one's
// sign is set.
MXQ_DEV void pair_keys(uint32_t w, uint32_t code, uint32_t &x, uint32_t &y)
{
    uint32_t z;
    asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(z) : "r"(w), "r"(0x3F803F80u), "r"(0u)); // w * 1 + 0
    const uint32_t neg = ((z >> 15) & 0x00010001u) * 0xFFFFu;
    const uint32_t k = z ^ (neg | 0x80008000u);
    x = __byte_perm(k, code, 0x1054);     // key of the low half over code
    y = __byte_perm(k, code - 1, 0x3254); // of the high half over the next index's
}

// Batcher's odd-even merge sort of N registers, descending: sort both halves,
// then merge the elements R apart from LO on
template <int LO, int N, int R, int S, typename K> MXQ_DEV void merge_descending(K (&c)[S])
{
    auto exchange = [&](int i, int j) {
        const K a = c[i], b = c[j];
        c[i] = a > b ? a : b;
        c[j] = a > b ? b : a;
    };
    if constexpr (2 * R < N) {
        merge_descending<LO, N, 2 * R>(c);
        merge_descending<LO + R, N, 2 * R>(c);
#pragma unroll
        for (int i = LO + R; i + R < LO + N; i += 2 * R)
            exchange(i, i + R);
    } else {
        exchange(LO, LO + R);
    }
}
template <int LO, int N, int S, typename K> MXQ_DEV void sort_descending(K (&c)[S])
{
    if constexpr (N > 1) {
        sort_descending<LO, N / 2>(c);
        sort_descending<LO + N / 2, N / 2>(c);
        merge_descending<LO, N, 1>(c);
    }
}

constexpr int ROUTE_THREADS = 512;
constexpr int ROUTE_WARPS = ROUTE_THREADS / 32;
constexpr int ROUTE_BWD_THREADS = 256;
constexpr int ROUTE_BWD_WARPS = ROUTE_BWD_THREADS / 32;
constexpr int ROUTE_ROWS = 8;          // warps' sums of p side by side in shared memory

// slots that a lane keeps: slot j of a token sits in its lane j % LPT
template <int LPT, int EPL> constexpr int lane_slots() { return (LPT * EPL < MAX_K ? LPT * EPL : MAX_K) / LPT; }

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
// per warp at a time. A lane sorts its logits' keys once; the k best are then
// the largest of the lanes' heads, k times, the winner's lane moving its list
// up (a maximum over all of a lane's keys in every round cost three times the
// instructions). Keys: the logit's order; 16-bit logits leave room for the
// complement of the index below, so that one maximum gives value and index and
// equal logits go to the lowest index; 32-bit ones carry it in a second word.
// The next token's logits are loaded while this one is worked on. A lane's sums
// of p are one fp32 chain of its n tokens (all terms positive: off by n 2^-24 at
// most, 14 at 65536 tokens of 256 experts), the CTAs' are added in fp64. 65536
// tokens, 256 experts, k = 8, bf16: 39 us, bound by the ALU pipe (2.9
// instructions a cycle), where reading the 34 MB would take 5. fp32 logits, with
// keys of 64 bits, take 70 with the finishing kernel; above 512 experts they
// spill (576 bytes a thread): 130 at 16384 x 1024.
template <typename T, int LPT, int EPL>
__global__ void __launch_bounds__(moe::ROUTE_THREADS)
    k_moe_route(const T *__restrict__ logits, int64_t tokens, int E, int64_t ld, const uint8_t *__restrict__ valid,
                int k, int renorm, int vec, float *__restrict__ weights, int32_t *__restrict__ ids,
                moe::RoutePart part, int32_t *counts, float *loss, float *loss_grad)
{
    using namespace moe;
    using Key = std::conditional_t<sizeof(T) == 2, uint32_t, uint64_t>;
    constexpr int TPW = 32 / LPT, SLOTS = lane_slots<LPT, EPL>();
    constexpr uint32_t FIRST = 0x00800000u; // keys below belong to -inf
    constexpr int STEP = LPT < 8 ? LPT : 8;  // rounds unrolled
    extern __shared__ __align__(16) uint8_t smem[];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int sub = lane / LPT, li = lane % LPT, e0 = li * EPL;
    float *s_p = reinterpret_cast<float *>(smem);                     // (ROUTE_ROWS, E)
    int *s_c = reinterpret_cast<int *>(s_p + (size_t)ROUTE_ROWS * E); // E
    __shared__ int s_n;
    let_next_kernel_start();
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
    int64_t t = ((int64_t)blockIdx.x * ROUTE_WARPS + warp) * TPW + sub; // this lane's token
    const T *row = logits + t * ld;
    float *w_out = weights + t * k + li;
    int32_t *id_out = ids + t * k + li;
    Raw<T, EPL> next;
    bool next_live = false;
    auto fetch = [&](int64_t at, const T *p) {
        next.none();
        next_live = false;
        if (at < tokens) {
            next.load(p, e0, E, vec);
            next_live = !valid || valid[at] != 0;
        }
    };
    fetch(t, row);
    for (; t - sub < tokens; t += step, w_out += step * k, id_out += step * k) {
        Raw<T, EPL> raw = next;
        const bool live = next_live;
        row += step * ld;
        fetch(t + step, row);
        if (!live)
            raw.none();
        float v[EPL];
        Key c[EPL];
#pragma unroll
        for (int i = 0; i < EPL; ++i) {
            v[i] = raw.get(i);
            if constexpr (sizeof(T) == 4)
                c[i] = ((uint64_t)order_key(v[i] + 0.0f) << 32) | (uint32_t)~(e0 + i);
            else if (i & 1)
                pair_keys(raw.w[i >> 1], 0xFFFFu - (uint32_t)(e0 + i - 1), c[i - 1], c[i]);
        }
        sort_descending<0, EPL>(c);
        uint32_t top; // the token's largest key, without the index
        if constexpr (sizeof(T) == 2) {
            top = group_max<LPT>(c[0]);
            top = top & 0x80000000u ? top & 0xFFFF0000u : top | 0xFFFFu; // a negative value's key ends in ones
        } else {
            top = group_max<LPT>((uint32_t)(c[0] >> 32));
        }
        const Shift shift(key_value(top));
        float rz;
        const bool bad = exponentials<LPT, EPL>(v, shift, rz);
#pragma unroll
        for (int i = 0; i < EPL; ++i)
            acc[i] = fmaf(v[i], rz, acc[i]);
        nvalid += live && li == 0;

        uint32_t best[SLOTS], who[SLOTS]; // this lane's slots: key and, for 32-bit logits, expert
#pragma unroll
        for (int s = 0; s < SLOTS; ++s) {
            best[s] = 0u;
            who[s] = 0u;
#pragma unroll 1
            for (int j0 = 0; j0 < LPT && s * LPT + j0 < k; j0 += STEP)
#pragma unroll
                for (int jj = j0; jj < j0 + STEP; ++jj) {
                    if (s * LPT + jj >= k)
                        break;
                    bool pop;
                    if constexpr (sizeof(T) == 2) {
                        const uint32_t g = group_max<LPT>(c[0]);
                        best[s] = li == jj ? g : best[s];
                        pop = c[0] == g;
                    } else {
                        // the first lane with the largest key: its experts come first
                        const uint32_t head = (uint32_t)(c[0] >> 32);
                        const uint32_t g = group_max<LPT>(head);
                        const uint32_t group = LPT == 32 ? 0xffffffffu : ((1u << (LPT & 31)) - 1u) << (lane & ~(LPT - 1));
                        const uint32_t eq = __ballot_sync(0xffffffffu, head == g) & group;
                        const int src = __ffs(eq) - 1; // a lane of this token holds its maximum
                        const uint32_t e = __shfl_sync(0xffffffffu, ~(uint32_t)c[0], src);
                        best[s] = li == jj ? g : best[s];
                        who[s] = li == jj ? e : who[s];
                        pop = lane == src;
                    }
#pragma unroll
                    for (int i = 0; i + 1 < EPL; ++i) // by select: some lane always pops
                        c[i] = pop ? c[i + 1] : c[i];
                    c[EPL - 1] = pop ? 0 : c[EPL - 1];
                }
        }
        float w[SLOTS], sum = 0.0f;
        int id[SLOTS];
#pragma unroll
        for (int s = 0; s < SLOTS; ++s) {
            const uint32_t g = best[s];
            const bool got = !bad && g >= FIRST;
            const uint32_t key = sizeof(T) == 4 ? g : (g & 0x80000000u ? g & 0xFFFF0000u : g | 0xFFFFu);
            id[s] = !got ? -1 : (sizeof(T) == 2 ? (int)(0xFFFFu - (g & 0xFFFFu)) : (int)who[s]);
            w[s] = got ? shift.exp(key_value(key)) : 0.0f;
            sum += w[s];
        }
        float scale = rz;
        if (renorm) {
            sum = group_sum<LPT>(sum);
            scale = sum == 0.0f ? 0.0f : __fdiv_rn(1.0f, sum);
        }
        if (bad)
            scale = NAN;
#pragma unroll
        for (int s = 0; s < SLOTS; ++s) {
            if (s * LPT + li < k && t < tokens) {
                id_out[s * LPT] = id[s];
                w_out[s * LPT] = w[s] * scale;
                if (id[s] >= 0)
                    atomicAdd(&s_c[id[s]], 1);
            }
        }
    }
    // the warp's tokens of one expert, then the CTA's warps in order
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
#pragma unroll
        for (int o = LPT; o < 32; o <<= 1)
            acc[i] += __shfl_xor_sync(0xffffffffu, acc[i], o);
        if (warp < ROUTE_ROWS && sub == 0 && e0 + i < E)
            s_p[(size_t)warp * E + e0 + i] = acc[i];
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < EPL; ++i)
        if (warp >= ROUTE_ROWS && sub == 0 && e0 + i < E)
            s_p[(size_t)(warp - ROUTE_ROWS) * E + e0 + i] += acc[i];
    for (int o = 16; o; o >>= 1)
        nvalid += __shfl_xor_sync(0xffffffffu, nvalid, o);
    if (lane == 0)
        atomicAdd(&s_n, nvalid);
    __syncthreads();
    for (int e = tid; e < E; e += ROUTE_THREADS) {
        float p = 0.0f;
#pragma unroll
        for (int w = 0; w < ROUTE_ROWS; ++w)
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
// in order. 296 CTAs' rows of 256 experts: about 5 us behind the kernel above.
__global__ void __launch_bounds__(1024)
    k_moe_route_finish(moe::RoutePart part, int R, int E, int k, int32_t *counts, float *loss, float *loss_grad)
{
    using namespace moe;
    __shared__ double s_p[32][33];
    __shared__ int s_c[32][33];
    __shared__ long long s_n[32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int e = blockIdx.x * 32 + lane;
    wait_for_previous_kernel();
    double p = 0.0;
    int c = 0;
    if (e < E) {
#pragma unroll 8
        for (int r = warp; r < R; r += 32) {
            p += (double)part.p[(size_t)r * E + e];
            c += part.c[(size_t)r * E + e];
        }
    }
    long long n = 0;
    for (int r = threadIdx.x; r < R; r += 1024)
        n += part.n[r];
#pragma unroll
    for (int o = 16; o; o >>= 1)
        n += __shfl_xor_sync(0xffffffffu, n, o);
    if (lane == 0)
        s_n[warp] = n;
    s_p[warp][lane] = p;
    s_c[warp][lane] = c;
    __syncthreads();
    if (warp)
        return;
    p = 0.0;
    c = 0;
#pragma unroll
    for (int w = 0; w < 32; ++w) {
        p += s_p[w][lane];
        c += s_c[w][lane];
    }
    n = s_n[lane];
#pragma unroll
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
#pragma unroll
    for (int o = 16; o; o >>= 1)
        sum += __shfl_xor_sync(0xffffffffu, sum, o);
    int last = 0;
    if (lane == 0) {
        part.loss[blockIdx.x] = sum;
        __threadfence();
        last = atomicAdd(part.ticket, 1) == (int)gridDim.x - 1;
        __threadfence();
    }
    if (__shfl_sync(0xffffffffu, last, 0)) { // at most 32 CTAs
        sum = lane < (int)gridDim.x ? __ldcg(part.loss + lane) : 0.0;
#pragma unroll
        for (int o = 16; o; o >>= 1)
            sum += __shfl_xor_sync(0xffffffffu, sum, o);
        if (lane == 0)
            *loss = (float)(f * sum);
    }
}

// Router backward. With G = sum_j g_j w_j and b_e = grad_loss * loss_grad[e]
//   dl_e = p_e (b_e - sum p b) + { w_j g_j where e = id_j, - p_e G    plain
//                                { w_j (g_j - G) where e = id_j       renormalized
// The chosen experts' terms meet the dense ones in shared memory, one row per
// token. 25 us at 65536 x 256, k = 8, bf16 (70 MB: 11), bound by instructions.
template <typename T, int LPT, int EPL>
__global__ void __launch_bounds__(moe::ROUTE_BWD_THREADS)
    k_moe_route_bwd(const T *__restrict__ logits, int64_t tokens, int E, int64_t ld, const uint8_t *__restrict__ valid,
                    int k, int renorm, int vec, const float *__restrict__ weights, const int32_t *__restrict__ ids,
                    const float *__restrict__ loss_grad, const float *__restrict__ gw, const float *__restrict__ gl,
                    T *__restrict__ out)
{
    using namespace moe;
    constexpr int TPW = 32 / LPT, SLOTS = lane_slots<LPT, EPL>();
    extern __shared__ __align__(16) uint8_t smem[];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int sub = lane / LPT, li = lane % LPT, e0 = li * EPL;
    // the token's row of terms at the chosen experts
    float *s_q = reinterpret_cast<float *>(smem) + (size_t)warp * 32 * EPL + sub * (LPT * EPL);
    float4 *mine = reinterpret_cast<float4 *>(s_q + e0);
    float b[EPL];
    const float g_loss = gl ? *gl : 0.0f;
#pragma unroll
    for (int i = 0; i < EPL; ++i)
        b[i] = gl && e0 + i < E ? g_loss * loss_grad[e0 + i] : 0.0f;
    const int64_t step = (int64_t)gridDim.x * ROUTE_BWD_WARPS * TPW;
    int64_t t = ((int64_t)blockIdx.x * ROUTE_BWD_WARPS + warp) * TPW + sub;
    Raw<T, EPL> next;
    bool next_live = false;
    int next_id[SLOTS];
    float next_w[SLOTS], next_g[SLOTS];
    const T *row = logits + t * ld;
    T *out_row = out + t * E + e0;
    int64_t slot0 = t * k + li;
    auto fetch = [&](int64_t at) {
        next.none();
        next_live = false;
        const bool in = at < tokens;
        if (in) {
            next.load(row, e0, E, vec);
            next_live = !valid || valid[at] != 0;
        }
#pragma unroll
        for (int s = 0; s < SLOTS; ++s) {
            const bool slot = in && gw && s * LPT + li < k;
            next_id[s] = slot ? ids[slot0 + s * LPT] : -1;
            next_w[s] = slot ? weights[slot0 + s * LPT] : 0.0f;
            next_g[s] = slot ? gw[slot0 + s * LPT] : 0.0f;
        }
    };
    fetch(t);
    for (; t - sub < tokens; t += step, out_row += step * E) {
        Raw<T, EPL> raw = next;
        const bool live = next_live;
        int id[SLOTS];
        float w[SLOTS], g[SLOTS], G = 0.0f;
#pragma unroll
        for (int s = 0; s < SLOTS; ++s) {
            id[s] = live && next_id[s] < E ? next_id[s] : -1;
            w[s] = next_w[s];
            g[s] = next_g[s];
            G = id[s] >= 0 ? fmaf(g[s], w[s], G) : G;
        }
        row += step * ld;
        slot0 += step * k;
        fetch(t + step);
        if (!live)
            raw.none();
#pragma unroll
        for (int i = 0; i < EPL / 4; ++i)
            mine[i] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        float v[EPL];
        v[0] = raw.get(0);
        float m = v[0];
#pragma unroll
        for (int i = 1; i < EPL; ++i) {
            v[i] = raw.get(i);
            m = fmaxf(m, v[i]); // a NaN shows in the sum of the exponentials
        }
        m = key_value(group_max<LPT>(order_key(m)));
        float rz;
        exponentials<LPT, EPL>(v, Shift(m), rz);
#pragma unroll
        for (int i = 0; i < EPL; ++i)
            v[i] *= rz;
        G = group_sum<LPT>(G);
        __syncwarp();
#pragma unroll
        for (int s = 0; s < SLOTS; ++s)
            if (id[s] >= 0) // a token's experts are distinct
                s_q[id[s]] = w[s] * (renorm ? g[s] - G : g[s]);
        __syncwarp();
        float pb = 0.0f;
#pragma unroll
        for (int i = 0; i < EPL; ++i)
            pb = fmaf(v[i], b[i], pb);
        pb = group_sum<LPT>(pb) + (renorm ? 0.0f : G);
        float d[EPL];
#pragma unroll
        for (int i = 0; i < EPL / 4; ++i) {
            const float4 q = mine[i];
            d[4 * i] = fmaf(v[4 * i], b[4 * i] - pb, q.x);
            d[4 * i + 1] = fmaf(v[4 * i + 1], b[4 * i + 1] - pb, q.y);
            d[4 * i + 2] = fmaf(v[4 * i + 2], b[4 * i + 2] - pb, q.z);
            d[4 * i + 3] = fmaf(v[4 * i + 3], b[4 * i + 3] - pb, q.w);
        }
        if (!live) // padding, whatever the incoming gradients hold
#pragma unroll
            for (int i = 0; i < EPL; ++i)
                d[i] = 0.0f;
        if (t < tokens) {
            if (vec && e0 + EPL <= E) {
#pragma unroll
                for (int i = 0; i < EPL; i += 16 / (int)sizeof(T)) {
                    if constexpr (sizeof(T) == 2)
                        st_v4(out_row + i, pack_bf16(d[i], d[i + 1]), pack_bf16(d[i + 2], d[i + 3]),
                              pack_bf16(d[i + 4], d[i + 5]), pack_bf16(d[i + 6], d[i + 7]));
                    else
                        st_v4(out_row + i, __float_as_uint(d[i]), __float_as_uint(d[i + 1]),
                              __float_as_uint(d[i + 2]), __float_as_uint(d[i + 3]));
                }
            } else {
#pragma unroll
                for (int i = 0; i < EPL; ++i)
                    if (e0 + i < E)
                        out_row[i] = Elem<T>::put(d[i]);
            }
        }
        __syncwarp();
    }
}

// ---------------------------------------------------------------------------
// Order by expert. The n = tokens * k entries are cut into C chunks of whole
// tiles; pass 1 counts each chunk's entries per expert, pass 2 adds the counts
// of smaller experts and of earlier chunks and ranks the chunk's entries: a
// warp owns a run of a tile's entries, ranks 32 of them at a time among their
// equals (match.any), and the warps' counters are then summed in order. One
// tile needs no pass 1. No atomics across CTAs, nothing to clear. match.any
// bounds the ranking, so tiles are small and spread over the SMs: 131072
// entries of 64 experts take 7.8 us, in tiles of 8192 they took 19.9.
namespace moe {
constexpr int PLAN_THREADS = 512;
constexpr int PLAN_WARPS = PLAN_THREADS / 32;
constexpr int PLAN_R = 4;                                // entries per thread and tile
constexpr int PLAN_TILE = PLAN_THREADS * PLAN_R;         // 2048
constexpr int PLAN_MAX_CHUNKS = 128;
constexpr int PLAN_SELF_CHUNKS = 4;                      // up to here every CTA counts all entries itself:
                                                         // 9.0 us at 8192 entries against 8 for two kernels,
                                                         // and a launch less on the host; 14 at 16000

// dynamic shared memory of the ranking kernel: first positions, sums over the
// chunks, and the warps' counters
__host__ __device__ constexpr size_t plan_smem(int E) { return (size_t)E * 12 + (size_t)PLAN_WARPS * E * 2; }

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
    let_next_kernel_start();
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

// hist (C, E) of pass 1, or NULL when the grid is one CTA over one tile, or
// few enough that each counts the entries before and behind its own (a launch
// less). No __restrict__ on hist: it is written while this kernel already runs.
__global__ void __launch_bounds__(moe::PLAN_THREADS)
    k_moe_plan_rank(const int32_t *__restrict__ ids, int64_t n, int E, int64_t chunk, const int *hist,
                    int C, int32_t *__restrict__ pos, int32_t *__restrict__ offs)
{
    using namespace moe;
    extern __shared__ int smem_i[];
    int *base = smem_i;                                         // E: next position of each expert
    int *total = smem_i + E, *before = smem_i + 2 * E;          // E each: all chunks', earlier chunks' counts
    uint16_t *cnt = reinterpret_cast<uint16_t *>(smem_i + 3 * E); // (warps, E)
    __shared__ int s_scan[PLAN_WARPS];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int64_t lo = blockIdx.x * chunk, hi = lo + chunk < n ? lo + chunk : n;

    // base from `total` and `before`: an exclusive sum over the experts, two
    // neighbours per thread (E <= 1024); the inclusive sums are the group ends
    auto set_base = [&]() {
        const int a = 2 * tid < E ? total[2 * tid] : 0, b = 2 * tid + 1 < E ? total[2 * tid + 1] : 0;
        int x = a + b;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, x, o);
            if (lane >= o)
                x += y;
        }
        if (lane == 31)
            s_scan[warp] = x;
        __syncthreads();
        for (int w = 0; w < warp; ++w)
            x += s_scan[w];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int e = 2 * tid + i, end = i ? x : x - b;
            if (e < E) {
                base[e] = end - (i ? b : a) + before[e];
                if (blockIdx.x == 0)
                    offs[e] = end;
            }
        }
        __syncthreads();
    };

    for (int e = tid; e < E; e += PLAN_THREADS) {
        total[e] = 0;
        before[e] = 0;
    }
    __syncthreads();
    if (hist) {
        wait_for_previous_kernel();
        // the chunks' rows, 32 experts per warp at a time
        const int groups = (E + 31) / 32;
        for (int u = warp; u < groups * 4; u += PLAN_WARPS) { // a quarter of the chunks each
            const int e = (u >> 2) * 32 + lane, c0 = (u & 3) * ((C + 3) / 4), c1 = min(C, c0 + (C + 3) / 4);
            int all = 0, early = 0;
            if (e < E) {
#pragma unroll 16
                for (int c = c0; c < c1; ++c) {
                    const int h = hist[(size_t)c * E + e];
                    all += h;
                    early += c < (int)blockIdx.x ? h : 0;
                }
                atomicAdd(&total[e], all); // integers: the order does not matter
                atomicAdd(&before[e], early);
            }
        }
        __syncthreads();
        set_base();
    }
    if (!hist && C > 1) {
        auto count = [&](int64_t from, int64_t to, int *into) {
            for (int64_t i0 = from; i0 < to; i0 += 8 * PLAN_THREADS) {
                int e[8];
#pragma unroll
                for (int u = 0; u < 8; ++u)
                    e[u] = entry_expert(ids, i0 + u * PLAN_THREADS + tid, to, E);
#pragma unroll
                for (int u = 0; u < 8; ++u) {
                    // a warp of one expert adds once; others' equals queue at the address
                    const int first = __shfl_sync(0xffffffffu, e[u], 0);
                    if (__all_sync(0xffffffffu, e[u] == first)) {
                        if (lane == 0 && first >= 0)
                            atomicAdd(&into[first], 32);
                    } else if (e[u] >= 0) {
                        atomicAdd(&into[e[u]], 1);
                    }
                }
            }
        };
        count(0, lo, before);
        count(lo, n, total);
        __syncthreads();
        for (int e = tid; e < E; e += PLAN_THREADS)
            total[e] += before[e];
        __syncthreads();
        set_base();
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
            const int earlier = e[r] >= 0 ? mine[e[r]] : 0;
            rank[r] = earlier + __popc(peers & ((1u << lane) - 1u));
            __syncwarp();
            if (e[r] >= 0 && lane == __ffs(peers) - 1)
                mine[e[r]] = (uint16_t)(earlier + __popc(peers));
            __syncwarp();
        }
        __syncthreads();
        // the warps' counters become each warp's first rank within the tile
        for (int x = tid; x < E; x += PLAN_THREADS) {
            int sum = 0;
#pragma unroll
            for (int w = 0; w < PLAN_WARPS; ++w) {
                const int c = cnt[(size_t)w * E + x];
                cnt[(size_t)w * E + x] = (uint16_t)sum;
                sum += c;
            }
            total[x] = sum; // from here on the tile's counts
        }
        __syncthreads();
        if (C == 1)
            set_base(); // the only tile
#pragma unroll
        for (int r = 0; r < PLAN_R; ++r) {
            const int64_t i = i0 + (int64_t)warp * (32 * PLAN_R) + r * 32 + lane;
            if (i < hi)
                pos[i] = e[r] >= 0 ? base[e[r]] + mine[e[r]] + rank[r] : -1;
        }
        __syncthreads();
        for (int x = tid; x < E; x += PLAN_THREADS)
            base[x] += total[x];
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

// xs[pos[t][j]] = x[t]; rows from offs[E-1] to M are zero. A row is read once
// and written k times; HBM bounds it: 182 us at 16384 x 4 rows of 7168 bf16, 0.98
// of the measured copy rate, 196 at 16384 x 8 rows of 4096.
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

// out[t] = sum_j w[t][j] y[pos[t][j]] (w NULL: ones), slots in order, fp32. A
// warp takes one of `parts` runs of `run` vectors of a token's row and walks it
// 32 * U vectors at a time (one run per row when there are tokens enough: the
// slots are then looked up once a row). The loads of J slots are issued
// together: a branch that is the same for the whole warp leaves out a dropped
// slot, a lane behind the run's end reads the run's last vector and stores
// nothing. HBM bounds it on aligned rows: 174 to 182 us at 16384 x 4 rows of
// 7168 bf16 (180 at the measured copy rate); loads in flight on others: 45 at
// 5003 x 6 rows of 1419 fp32, a tenth of them dropped (28).
template <typename T, int V, int U, int J>
__global__ void __launch_bounds__(moe::ROW_THREADS, V * sizeof(T) == 16 ? 4 : 5)
    k_moe_combine(const T *__restrict__ y, int64_t M, int64_t K, int64_t ld, const int32_t *__restrict__ pos,
                  const float *__restrict__ weights, uint32_t tokens, uint32_t parts, uint32_t run, int k,
                  T *__restrict__ out)
{
    using namespace moe;
    const int lane = threadIdx.x & 31;
    const uint32_t nvec = (uint32_t)(K / V), all = tokens * parts, stride = gridDim.x * ROW_WARPS;
    for (uint32_t w = blockIdx.x * ROW_WARPS + (threadIdx.x >> 5); w < all; w += stride) {
        const uint32_t t = w / parts, v_lo = (w - t * parts) * run, v_hi = min(v_lo + run, nvec);
        const T *row = nullptr; // lane j: slot j's row and weight
        float wl = 0.0f;
        if (lane < k) {
            const int64_t i = (int64_t)t * k + lane, r = slot_row(pos, i, M);
            if (r >= 0) {
                row = y + r * ld;
                wl = weights ? weights[i] : 1.0f;
            }
        }
        const uint32_t there = __ballot_sync(0xffffffffu, row != nullptr);
        T *dst = out + (int64_t)t * K;
#pragma unroll 1
        for (uint32_t v0 = v_lo + lane; v0 - lane < v_hi; v0 += 32 * U) {
            float acc[U][V];
#pragma unroll
            for (int u = 0; u < U; ++u)
#pragma unroll
                for (int i = 0; i < V; ++i)
                    acc[u][i] = 0.0f;
            uint32_t at[U];
#pragma unroll
            for (int u = 0; u < U; ++u)
                at[u] = min(v0 + 32 * u, v_hi - 1) * V;
#pragma unroll 1
            for (int j0 = 0; j0 < k; j0 += J) {
                const uint32_t on = there >> j0; // bit j: slot j0 + j has a row
                Vec<T, V> r[J][U];
#pragma unroll
                for (int j = 0; j < J; ++j)
                    if (on >> j & 1u) {
                        const T *p = reinterpret_cast<const T *>(
                            __shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(row), j0 + j));
#pragma unroll
                        for (int u = 0; u < U; ++u)
                            r[j][u] = ld_now<T, V>(p + at[u]);
                    }
#pragma unroll
                for (int j = 0; j < J; ++j)
                    if (on >> j & 1u) {
                        const float wj = __shfl_sync(0xffffffffu, wl, j0 + j);
#pragma unroll
                        for (int u = 0; u < U; ++u)
#pragma unroll
                            for (int i = 0; i < V; ++i)
                                acc[u][i] = fmaf(wj, Elem<T>::get(r[j][u].v[i]), acc[u][i]);
                    }
            }
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (v0 + 32 * u < v_hi) {
                    Vec<T, V> o;
#pragma unroll
                    for (int i = 0; i < V; ++i)
                        o.v[i] = Elem<T>::put(acc[u][i]);
                    st_vec<T, V>(dst + (int64_t)(v0 + 32 * u) * V, o);
                }
        }
    }
}

// dy[pos[t][j]] = w[t][j] dout[t] and dw[t][j] = <dout[t], y[pos[t][j]]>, a
// warp per entry; rows of dy from offs[E-1] to M are zero. dy or dw may be
// NULL. 331 us at 16384 x 4 rows of 7168 bf16, bound by HBM (324 at the measured
// copy rate, dout's row re-read from L2), 66 at 5003 x 6 rows of 1419 fp32, a
// tenth of them dropped (54).
template <typename T, int V, int U>
__global__ void __launch_bounds__(moe::ROW_THREADS)
    k_moe_combine_bwd(const T *__restrict__ dout, int64_t ldd, const T *__restrict__ y, int64_t ldy, int64_t M,
                      int64_t K, const int32_t *__restrict__ pos, const float *__restrict__ weights, int64_t tokens,
                      int k, const int32_t *__restrict__ offs, int E, T *__restrict__ dy, float *__restrict__ dw)
{
    using namespace moe;
    const int lane = threadIdx.x & 31;
    const uint32_t nvec = (uint32_t)(K / V);
    const int64_t n = tokens * k, end = max(0, offs[E - 1]);
    const int64_t all = n + (dy && end < M ? M - end : 0);
    for (int64_t w = (int64_t)blockIdx.x * ROW_WARPS + (threadIdx.x >> 5); w < all;
         w += (int64_t)gridDim.x * ROW_WARPS) {
        if (w >= n) {
            Vec<T, V> zero = {};
            T *d = dy + (end + w - n) * K;
            for (uint32_t v = lane; v < nvec; v += 32)
                st_vec<T, V>(d + (int64_t)v * V, zero);
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
        const T *yr = y + s * ldy;
        T *out = dy + s * K;
        // 32 * U vectors from v0 on: with FULL all of them exist, and a lane's
        // lie at fixed distances; else a lane behind the end reads the last one
        auto block = [&](uint32_t v0, auto full) {
            constexpr bool FULL = decltype(full)::value;
            uint32_t at[U];
#pragma unroll
            for (int u = 0; u < U; ++u)
                at[u] = (FULL ? v0 + lane + 32 * u : min(v0 + lane + 32 * u, nvec - 1)) * V;
            Vec<T, V> a[U], b[U];
            const T *ga = g + at[0], *ya = yr + at[0];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                a[u] = ld_now<T, V>(FULL ? ga + 32 * u * V : ga + (at[u] - at[0]));
                if (dw)
                    b[u] = ld_now<T, V>(FULL ? ya + 32 * u * V : ya + (at[u] - at[0]));
            }
            T *d = out + at[0];
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (FULL || v0 + lane + 32 * u < nvec) {
                    Vec<T, V> o;
#pragma unroll
                    for (int i = 0; i < V; ++i) {
                        const float f = Elem<T>::get(a[u].v[i]);
                        if (dw)
                            acc = fmaf(f, Elem<T>::get(b[u].v[i]), acc);
                        o.v[i] = Elem<T>::put(wt * f);
                    }
                    if (dy)
                        st_vec<T, V>(d + 32 * u * V, o);
                }
        };
        uint32_t v0 = 0;
#pragma unroll 1
        for (; v0 + 32 * U <= nvec; v0 += 32 * U)
            block(v0, std::true_type{});
        if (v0 < nvec)
            block(v0, std::false_type{});
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

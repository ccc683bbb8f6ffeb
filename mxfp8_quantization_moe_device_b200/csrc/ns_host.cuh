// ns_host.cuh - host side of newton_schulz (ns.cuh): argument checks,
// workspace layout, the launches of a call. Included at the end of mxq.cu.
#pragma once

namespace {

struct NsPlan {
    int64_t m, n, ldx, ldt;
    int tall, parts;
    size_t xh[2], hi, lo, A, B, a_own, alpha, beta, part, bytes;
};

NsPlan ns_plan(int64_t E, int64_t rows, int64_t cols, int32_t steps)
{
    NsPlan p = {};
    p.tall = rows > cols;
    p.m = std::min(rows, cols);
    p.n = std::max(rows, cols);
    p.ldx = (p.n + 7) / 8 * 8;
    p.ldt = (p.m + 7) / 8 * 8;
    p.parts = (int)std::min<int64_t>(ns::MAX_PARTS, (rows * cols + 8191) / 8192);
    size_t o = 0;
    auto take = [&](size_t bytes) {
        const size_t at = o;
        o = round_up(o + bytes, 256);
        return at;
    };
    p.xh[0] = take((size_t)E * p.m * p.ldx * 2);
    p.xh[1] = steps > 1 ? take((size_t)E * p.m * p.ldx * 2) : p.xh[0];
    p.hi = take((size_t)E * ns::chunks_of(p.m) * ns::chunks_of(p.n) * ns::CHUNK_BYTES);
    p.lo = take((size_t)E * ns::chunks_of(p.m) * ns::chunks_of(p.n) * ns::CHUNK_BYTES);
    p.a_own = take((size_t)E * ns::chunks_of(p.m) * ns::chunks_of(p.m) * ns::CHUNK_BYTES);
    p.A = take((size_t)E * p.m * p.ldt * 2);
    p.B = take((size_t)E * p.m * p.ldt * 2);
    p.alpha = take((size_t)E * p.m * 4);
    p.beta = take((size_t)E * p.m * 4);
    p.part = take((size_t)E * p.parts * 8);
    p.bytes = o;
    return p;
}

int ns_check(int64_t E, int64_t rows, int64_t cols, int32_t steps)
{
    if (E < 0 || rows < 0 || cols < 0 || steps < 1)
        return MXQ_ERR_SHAPE;
    if (E > 65535 || rows > 65536 || cols > 65536 || steps > 64)
        return MXQ_ERR_UNSUPPORTED;
    // the kernels address a matrix with 32-bit byte offsets
    if (std::max(rows, cols) * ((std::min(rows, cols) + 7) / 8 * 8) >= (int64_t(1) << 31))
        return MXQ_ERR_UNSUPPORTED;
    return MXQ_OK;
}

// The largest |a s + b s^3 + c s^5| (what a step makes of a singular value s)
// and |b s^2 + c s^4| (B) for s in [0, r], at the end or where the derivative is
// zero.
double ns_largest_x(double a, double b, double c, double r)
{
    const auto at = [&](double u) { return std::fabs(std::sqrt(u) * (a + u * (b + u * c))); };
    double most = at(r * r);
    const double disc = 9.0 * b * b - 20.0 * a * c; // a + 3 b u + 5 c u^2 = 0
    if (disc >= 0.0) {
        const double q = -0.5 * (3.0 * b + std::copysign(std::sqrt(disc), b));
        for (const double u : {q / (5.0 * c), a / q})
            if (u > 0.0 && u < r * r)
                most = std::max(most, at(u));
    }
    return most;
}
double ns_largest_b(double b, double c, double r)
{
    const auto at = [&](double u) { return std::fabs(u * (b + u * c)); };
    const double u = -b / (2.0 * c);
    return u > 0.0 && u < r * r ? std::max(at(r * r), at(u)) : at(r * r);
}

// The coefficients with the scale of B' over that of A' in every step, false
// where the scheme does not carry them. The singular values are bounded by 1 at
// the start, then by what a step makes of them, and by 4 by the caller's word;
// 2^-8 more for what rounding adds, and B stays a factor of two from fp16's end.
// Coefficients of up to 16 leave the scale of B at 4 or more. Larger ones (a
// schedule's first steps, (8.2, -22.9, 16.5) say) are taken where the bound
// alone keeps the step's result within 4; at 256 the scale of B would be 1/4.
constexpr double NS_LARGEST = 4.0;
bool ns_coefs(const float *coefficients, int32_t steps, ns::Coefs &co)
{
    double r = 1.0 + 0x1p-8;
    for (int s = 0; s < steps; ++s) {
        const float a = coefficients[3 * s], b = coefficients[3 * s + 1], c = coefficients[3 * s + 2];
        const float size = std::max(std::fabs(a), std::max(std::fabs(b), std::fabs(c)));
        if (!std::isfinite(a) || !std::isfinite(b) || !std::isfinite(c) || size > 256.0f)
            return false;
        const double next = ns_largest_x(a, b, c, r) * (1.0 + 0x1p-8);
        if (size > 16.0f && next > NS_LARGEST)
            return false;
        const double most = ns_largest_b(b, c, r) * ns::SA;
        float part = 1.0f;
        while (most * part > 32752.0)
            part *= 0.5f;
        co.v[3 * s] = a;
        co.v[3 * s + 1] = b;
        co.v[3 * s + 2] = c;
        co.pb[s] = b * part;
        co.pc[s] = c * part;
        co.unscale[s] = 1.0f / (ns::SA * part);
        r = std::min(NS_LARGEST, next);
    }
    return true;
}

// how a product reads or writes a matrix: boxes of width x rows elements, the
// operands' with 128-byte rows and swizzle, but for narrow column tiles' 32 x 64,
// which has the 64-byte one as the epilogue's stores
enum NsBox { NS_STORE, NS_64x128, NS_64x64, NS_64x32, NS_32x64, NS_NUM_BOXES };
constexpr struct {
    int width, rows;
    CUtensorMapSwizzle swizzle;
} NS_BOXES[NS_NUM_BOXES] = {{ns::CHUNK, ns::CHUNK, CU_TENSOR_MAP_SWIZZLE_64B},
                            {64, 128, CU_TENSOR_MAP_SWIZZLE_128B},
                            {64, 64, CU_TENSOR_MAP_SWIZZLE_128B},
                            {64, 32, CU_TENSOR_MAP_SWIZZLE_128B},
                            {32, 64, CU_TENSOR_MAP_SWIZZLE_64B}};

// one operand of the products: fp16 matrices by rows, a plane each, with their
// inner length and row length, and the maps that the call has made so far
struct NsOperand {
    const void *p;
    int64_t inner, ld, rows, E;
    CUtensorMap maps[NS_NUM_BOXES];
    bool made[NS_NUM_BOXES];

    int map(NsBox i, const CUtensorMap **out)
    {
        if (!made[i]) {
            const uint64_t d[3] = {(uint64_t)inner, (uint64_t)rows, (uint64_t)E};
            const uint64_t s[2] = {(uint64_t)ld * 2, (uint64_t)ld * 2 * (uint64_t)rows};
            const uint32_t box[3] = {(uint32_t)NS_BOXES[i].width, (uint32_t)NS_BOXES[i].rows, 1};
            const int rc = make_map(&maps[i], CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3, p, d, s, box, NS_BOXES[i].swizzle);
            if (rc != MXQ_OK)
                return rc;
            made[i] = true;
        }
        *out = &maps[i];
        return MXQ_OK;
    }
};

// co-resident CTA pairs on the current device; the four products differ in
// the epilogue's code alone
template <int MODE, int TN> int ns_pairs(int *out)
{
    static std::atomic<uint64_t> set[2];
    static std::atomic<int> pairs[128];
    const int rc = allow_smem(ns::k_ns_gemm<MODE, TN>, (int)ns::smem_bytes<TN>(), set);
    if (rc != MXQ_OK)
        return rc;
    int d = 0;
    if (cudaGetDevice(&d) != cudaSuccess || d < 0 || d >= 128)
        return MXQ_ERR_CUDA;
    int np = pairs[d].load(std::memory_order_relaxed);
    if (np == 0) {
        if (max_pairs(ns::k_ns_gemm<MODE, TN>, dim3(ns::THREADS), ns::smem_bytes<TN>(), &np) != MXQ_OK || np < 1)
            return MXQ_ERR_CUDA;
        pairs[d].store(np, std::memory_order_relaxed);
    }
    *out = np;
    return MXQ_OK;
}

template <int MODE, int TN>
int ns_launch(NsOperand &p, NsOperand &q, NsOperand &o, const ns::Args &a, int pairs, cudaStream_t stream)
{
    constexpr bool sym = MODE == ns::GRAM || MODE == ns::POLY;
    constexpr NsBox rows = TN == 256 ? NS_64x128 : (TN == 128 ? NS_64x64 : NS_64x32);
    constexpr NsBox columns = TN == 64 ? NS_32x64 : NS_64x64;
    const CUtensorMap *mp, *mpc, *mq, *mqc, *mo;
    int rc;
    if ((rc = p.map(NS_64x128, &mp)) != MXQ_OK || (rc = p.map(NS_64x64, &mpc)) != MXQ_OK ||
        (rc = q.map(rows, &mq)) != MXQ_OK || (rc = q.map(columns, &mqc)) != MXQ_OK ||
        (rc = o.map(NS_STORE, &mo)) != MXQ_OK)
        return rc;
    const int64_t grid = std::min<int64_t>(a.E * ns::sym_or_all_tiles<sym, TN>(a.m, a.n), pairs);
    return launch_chained(ns::k_ns_gemm<MODE, TN>, dim3((unsigned)(2 * grid)), dim3(ns::THREADS), ns::smem_bytes<TN>(),
                          stream, true, *mp, *mpc, *mq, *mqc, *mo, a, (int)((p.inner + ns::BK - 1) / ns::BK), wait_ns());
}

// Tile width, by estimated time in units of a hundredth of one 64-column block
// of a 256 x 256 tile (about 4 ns): a block of a 256 x 128 tile takes about 88
// (half the products, three quarters of the loads), of a 256 x 64 tile 75;
// draining a tile takes about 1100, 550 and 275, hidden under the next tile's
// blocks but for the last round. The narrow tiles win where they spread the
// work over more pairs or where draining bounds: 226 us against 253 at (5, 1409,
// 577), 101 against 138 at (4, 256, 256); the wide one at 343 against 408 at (8,
// 1024, 1024), 394 against 436 at (16, 512, 2048).
template <int MODE, int TN>
int ns_estimate(const ns::Args &a, int64_t blocks, int64_t block_cost, int64_t drain, int *pairs, int64_t *time)
{
    const int rc = ns_pairs<MODE, TN>(pairs);
    if (rc != MXQ_OK)
        return rc;
    const int64_t tiles = a.E * ns::sym_or_all_tiles<MODE == ns::GRAM || MODE == ns::POLY, TN>(a.m, a.n);
    *time = (tiles + *pairs - 1) / *pairs * std::max(blocks * block_cost, drain) + drain;
    const int force = g_ns_tile.load();
    if (force)
        *time = force == TN ? 0 : INT64_MAX;
    return MXQ_OK;
}

template <int MODE>
int ns_product(NsOperand &p, NsOperand &q, NsOperand &o, const ns::Args &a, cudaStream_t stream)
{
    const int64_t blocks = (p.inner + ns::BK - 1) / ns::BK;
    int pairs[3], rc;
    int64_t t[3];
    if ((rc = ns_estimate<MODE, 256>(a, blocks, 100, 1100, &pairs[0], &t[0])) != MXQ_OK ||
        (rc = ns_estimate<MODE, 128>(a, blocks, 88, 550, &pairs[1], &t[1])) != MXQ_OK ||
        (rc = ns_estimate<MODE, 64>(a, blocks, 75, 275, &pairs[2], &t[2])) != MXQ_OK)
        return rc;
    if (t[2] < t[1] && t[2] < t[0])
        return ns_launch<MODE, 64>(p, q, o, a, pairs[2], stream);
    if (t[1] < t[0])
        return ns_launch<MODE, 128>(p, q, o, a, pairs[1], stream);
    return ns_launch<MODE, 256>(p, q, o, a, pairs[0], stream);
}

template <typename T>
int ns_start(const T *g, int64_t E, int64_t rows, int64_t cols, const NsPlan &p, double eps, uint8_t *ws,
             cudaStream_t stream)
{
    double *part = reinterpret_cast<double *>(ws + p.part);
    const int rc = launch(ns::k_ns_sumsq<T>, dim3((unsigned)p.parts, (unsigned)E), dim3(256), 0, stream, false, g,
                          rows * cols, (int)(aligned(g, 16) && rows * cols * sizeof(T) % 16 == 0), part);
    if (rc != MXQ_OK)
        return rc;
    return launch_chained(ns::k_ns_init<T>,
                          dim3((unsigned)((cols + 63) / 64), (unsigned)((rows + 63) / 64), (unsigned)E), dim3(256), 0,
                          stream, false, g, (int)rows, (int)cols, (int)(aligned(g, 2 * sizeof(T)) && cols % 2 == 0),
                  (const double *)part, p.parts, eps, p.tall, reinterpret_cast<uint16_t *>(ws + p.xh[0]),
                  (int)p.ldx, reinterpret_cast<uint16_t *>(ws + p.hi), reinterpret_cast<uint16_t *>(ws + p.lo));
}

// a launch of k_ns_small with `ctas` CTAs per matrix
void ns_small_config(cudaLaunchConfig_t *cfg, cudaLaunchAttribute *attr, int64_t E, int ctas, cudaStream_t stream)
{
    cfg->gridDim = dim3((unsigned)(E * ctas));
    cfg->blockDim = dim3(ns::SM_THREADS);
    cfg->dynamicSmemBytes = ns::small_smem_bytes(ctas > 1);
    cfg->stream = stream;
    attr->id = cudaLaunchAttributeClusterDimension;
    attr->val.clusterDim.x = (unsigned)ctas;
    attr->val.clusterDim.y = 1;
    attr->val.clusterDim.z = 1;
    cfg->attrs = attr;
    cfg->numAttrs = 1;
}

template <typename T> int ns_small_attributes()
{
    static std::atomic<uint64_t> set[2];
    int d = 0;
    if (cudaGetDevice(&d) != cudaSuccess || d < 0 || d >= 128)
        return MXQ_ERR_CUDA;
    if (set[d >> 6].load(std::memory_order_acquire) >> (d & 63) & 1)
        return MXQ_OK;
    if (cudaFuncSetAttribute(ns::k_ns_small<T>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             (int)ns::small_smem_bytes(true)) != cudaSuccess ||
        cudaFuncSetAttribute(ns::k_ns_small<T>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) != cudaSuccess) {
        (void)cudaGetLastError();
        return MXQ_ERR_CUDA;
    }
    set[d >> 6].fetch_or(uint64_t(1) << (d & 63), std::memory_order_release);
    return MXQ_OK;
}

// whether the current device runs clusters of SM_MAX_CTAS CTAs of k_ns_small
bool ns_large_clusters()
{
    static std::atomic<int> known[128]; // 0 unknown, 1 no, 2 yes
    int d = 0;
    if (cudaGetDevice(&d) != cudaSuccess || d < 0 || d >= 128) {
        (void)cudaGetLastError();
        return false;
    }
    int k = known[d].load(std::memory_order_relaxed);
    if (k == 0) {
        cudaLaunchConfig_t cfg = {};
        cudaLaunchAttribute attr[1];
        int n = 0, m = 0;
        ns_small_config(&cfg, attr, 1, ns::SM_MAX_CTAS, nullptr);
        const bool yes = ns_small_attributes<uint16_t>() == MXQ_OK && ns_small_attributes<float>() == MXQ_OK &&
                         cudaOccupancyMaxActiveClusters(&n, ns::k_ns_small<uint16_t>, &cfg) == cudaSuccess &&
                         cudaOccupancyMaxActiveClusters(&m, ns::k_ns_small<float>, &cfg) == cudaSuccess && n > 0 &&
                         m > 0;
        (void)cudaGetLastError();
        k = yes ? 2 : 1;
        known[d].store(k, std::memory_order_relaxed);
    }
    return k == 2;
}

// One launch for all steps: the smaller side fits a tile, the larger one a
// cluster, of eight CTAs (any device) or sixteen: 245 us by the general
// kernels at (3, 90, 4000).
bool ns_is_small(int64_t rows, int64_t cols)
{
    const int64_t ctas = (std::max(rows, cols) + ns::SM_SLAB - 1) / ns::SM_SLAB;
    return g_ns_tile.load() == 0 && std::min(rows, cols) <= ns::SM_M &&
           (ctas <= 8 || (ctas <= ns::SM_MAX_CTAS && ns_large_clusters()));
}

template <typename T>
int ns_small(const T *g, int64_t E, int64_t rows, int64_t cols, int32_t steps, const ns::Coefs &co, double eps,
             uint16_t *out, cudaStream_t stream)
{
    const int rc = ns_small_attributes<T>();
    if (rc != MXQ_OK)
        return rc;
    const int ctas = (int)((std::max(rows, cols) + ns::SM_SLAB - 1) / ns::SM_SLAB);
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    ns_small_config(&cfg, attr, E, ctas, stream);
    if (cudaLaunchKernelEx(&cfg, ns::k_ns_small<T>, g, (int)rows, (int)cols, ctas, (int)(rows > cols), (int)steps, co,
                           eps, out, (int)(cols % 8 == 0 && aligned(out, 16)), wait_ns()) != cudaSuccess) {
        (void)cudaGetLastError();
        return MXQ_ERR_LAUNCH;
    }
    return MXQ_OK;
}

} // namespace

extern "C" {

size_t newton_schulz_workspace_bytes(int64_t batch, int64_t rows, int64_t cols, int32_t steps)
{
    if (ns_check(batch, rows, cols, steps) != MXQ_OK || batch == 0 || rows == 0 || cols == 0 ||
        ns_is_small(rows, cols))
        return 0;
    return ns_plan(batch, rows, cols, steps).bytes;
}

int newton_schulz(const void *g, int32_t dtype, int64_t batch, int64_t rows, int64_t cols, int32_t steps,
                  const float *coefficients, double eps, void *out, void *workspace, size_t workspace_bytes,
                  cudaStream_t stream)
{
    int rc = ns_check(batch, rows, cols, steps);
    if (rc != MXQ_OK)
        return rc;
    if (!dtype_ok(dtype))
        return MXQ_ERR_UNSUPPORTED;
    if (!coefficients)
        return MXQ_ERR_NULL;
    if (!(eps >= 0.0) || eps > 1e30)
        return MXQ_ERR_UNSUPPORTED;
    ns::Coefs co = {};
    if (!ns_coefs(coefficients, steps, co))
        return MXQ_ERR_UNSUPPORTED;
    if (batch == 0 || rows == 0 || cols == 0)
        return MXQ_OK;
    if (!g || !out)
        return MXQ_ERR_NULL;
    if (!aligned(g, dtype_size(dtype)) || !aligned(out, 2))
        return MXQ_ERR_ALIGN;
    if (ns_is_small(rows, cols))
        return dtype == MXQ_BF16 ? ns_small(static_cast<const uint16_t *>(g), batch, rows, cols, steps, co, eps,
                                            static_cast<uint16_t *>(out), stream)
                                 : ns_small(static_cast<const float *>(g), batch, rows, cols, steps, co, eps,
                                            static_cast<uint16_t *>(out), stream);
    const NsPlan p = ns_plan(batch, rows, cols, steps);
    if (!workspace || workspace_bytes < p.bytes)
        return MXQ_ERR_WORKSPACE;
    if (!aligned(workspace, 256))
        return MXQ_ERR_ALIGN;
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    NsOperand A = {ws + p.A, p.m, p.ldt, p.m, batch, {}, {}}, B = {ws + p.B, p.m, p.ldt, p.m, batch, {}, {}};
    NsOperand xs[2] = {{ws + p.xh[0], p.n, p.ldx, p.m, batch, {}, {}}, {ws + p.xh[1], p.n, p.ldx, p.m, batch, {}, {}}};
    rc = dtype == MXQ_BF16 ? ns_start(static_cast<const uint16_t *>(g), batch, rows, cols, p, eps, ws, stream)
                           : ns_start(static_cast<const float *>(g), batch, rows, cols, p, eps, ws, stream);
    if (rc != MXQ_OK)
        return rc;
    ns::Args a = {};
    a.E = (int)batch;
    a.m = (int)p.m;
    a.n = (int)p.n;
    a.hi = reinterpret_cast<uint16_t *>(ws + p.hi);
    a.lo = reinterpret_cast<uint16_t *>(ws + p.lo);
    a.a_own = reinterpret_cast<uint16_t *>(ws + p.a_own);
    a.alpha = reinterpret_cast<float *>(ws + p.alpha);
    a.beta = reinterpret_cast<float *>(ws + p.beta);
    a.out = static_cast<uint16_t *>(out);
    a.out_t = p.tall;
    a.out_vec = cols % 8 == 0 && aligned(out, 16);
    for (int s = 0; s < steps; ++s) {
        a.a = co.v[3 * s];
        a.b = co.v[3 * s + 1];
        a.c = co.v[3 * s + 2];
        a.pb = co.pb[s];
        a.pc = co.pc[s];
        a.unscale = co.unscale[s];
        NsOperand &x = xs[s & 1], &next = xs[(s + 1) & 1];
        if ((rc = ns_product<ns::GRAM>(x, x, A, a, stream)) != MXQ_OK ||
            (rc = ns_product<ns::POLY>(A, A, B, a, stream)) != MXQ_OK ||
            (rc = s + 1 < steps ? ns_product<ns::STEP>(B, x, next, a, stream)
                                : ns_product<ns::LAST>(B, x, next, a, stream)) != MXQ_OK)
            return rc;
    }
    return MXQ_OK;
}

} // extern "C"

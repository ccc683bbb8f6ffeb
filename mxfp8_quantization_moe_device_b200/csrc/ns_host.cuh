// ns_host.cuh - host side of newton_schulz (ns.cuh): argument checks,
// workspace layout, the launches of a call. Included at the end of mxq.cu.
#pragma once

namespace {

struct NsPlan {
    int64_t m, n, ldx, ldt;
    int tall, parts;
    size_t xh, xl, xt[2], A, B, part, bytes;
};

NsPlan ns_plan(int64_t E, int64_t rows, int64_t cols, int32_t steps)
{
    NsPlan p = {};
    p.tall = rows > cols;
    p.m = std::min(rows, cols);
    p.n = std::max(rows, cols);
    p.ldx = (p.n + 7) / 8 * 8;
    p.ldt = (p.m + 7) / 8 * 8;
    p.parts = (int)std::min<int64_t>(ns::MAX_PARTS, (rows * cols + 32767) / 32768);
    size_t o = 0;
    auto take = [&](size_t bytes) {
        const size_t at = o;
        o = round_up(o + bytes, 256);
        return at;
    };
    p.xh = take((size_t)E * p.m * p.ldx * 2);
    p.xl = take((size_t)E * p.m * p.ldx * 2);
    p.xt[0] = take((size_t)E * p.n * p.ldt * 2);
    p.xt[1] = steps > 1 ? take((size_t)E * p.n * p.ldt * 2) : p.xt[0];
    p.A = take((size_t)E * p.m * p.ldt * 2);
    p.B = take((size_t)E * p.m * p.ldt * 2);
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
    return MXQ_OK;
}

// map of one fp16 matrix per plane: boxes of 64 elements x 128 rows
int ns_map(CUtensorMap *map, const void *p, int64_t inner, int64_t ld, int64_t rows, int64_t E)
{
    const uint64_t d[3] = {(uint64_t)inner, (uint64_t)rows, (uint64_t)E};
    const uint64_t s[2] = {(uint64_t)ld * 2, (uint64_t)ld * 2 * (uint64_t)rows};
    const uint32_t box[3] = {ns::BK, ns::HALF, 1};
    return make_map(map, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3, p, d, s, box, CU_TENSOR_MAP_SWIZZLE_128B);
}

template <int MODE>
int ns_product(const CUtensorMap &p, const CUtensorMap &q, const ns::Args &a, int64_t K, cudaStream_t stream)
{
    static std::atomic<uint64_t> set[2];
    const int rc = allow_smem(ns::k_ns_gemm<MODE>, (int)ns::SMEM_BYTES, set);
    if (rc != MXQ_OK)
        return rc;
    static std::atomic<int> pairs[128]; // per device: co-resident CTA pairs
    int d = 0;
    if (cudaGetDevice(&d) != cudaSuccess || d < 0 || d >= 128)
        return MXQ_ERR_CUDA;
    int np = pairs[d].load(std::memory_order_relaxed);
    if (np == 0) {
        if (max_pairs(ns::k_ns_gemm<MODE>, dim3(ns::THREADS), ns::SMEM_BYTES, &np) != MXQ_OK || np < 1)
            return MXQ_ERR_CUDA;
        pairs[d].store(np, std::memory_order_relaxed);
    }
    const int64_t tm = (a.m + ns::TILE - 1) / ns::TILE, tn = (a.n + ns::TILE - 1) / ns::TILE;
    const int64_t items = a.E * (MODE == ns::GRAM || MODE == ns::POLY ? tm * (tm + 1) / 2 : tm * tn);
    const int64_t grid = std::min<int64_t>(items, np);
    return launch_pairs(ns::k_ns_gemm<MODE>, dim3((unsigned)(2 * grid)), dim3(ns::THREADS), ns::SMEM_BYTES, stream, p, q,
                        a, (int)((K + ns::BK - 1) / ns::BK), wait_ns());
}

template <typename T>
int ns_start(const T *g, int64_t E, int64_t rows, int64_t cols, const NsPlan &p, double eps, uint8_t *ws,
             cudaStream_t stream)
{
    double *part = reinterpret_cast<double *>(ws + p.part);
    const int rc = launch(ns::k_ns_sumsq<T>, dim3((unsigned)p.parts, (unsigned)E), dim3(256), 0, stream, false, g,
                          rows * cols, part);
    if (rc != MXQ_OK)
        return rc;
    return launch(ns::k_ns_init<T>, dim3((unsigned)((cols + 63) / 64), (unsigned)((rows + 63) / 64), (unsigned)E),
                  dim3(256), 0, stream, false, g, (int)rows, (int)cols, (const double *)part, p.parts, eps, p.tall,
                  reinterpret_cast<__half *>(ws + p.xh), reinterpret_cast<__half *>(ws + p.xl), (int)p.ldx,
                  reinterpret_cast<__half *>(ws + p.xt[0]), (int)p.ldt);
}

} // namespace

extern "C" {

size_t newton_schulz_workspace_bytes(int64_t batch, int64_t rows, int64_t cols, int32_t steps)
{
    if (ns_check(batch, rows, cols, steps) != MXQ_OK || batch == 0 || rows == 0 || cols == 0)
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
    // larger coefficients would leave fp16's range in B
    for (int i = 0; i < 3 * steps; ++i)
        if (!(coefficients[i] >= -16.0f && coefficients[i] <= 16.0f))
            return MXQ_ERR_UNSUPPORTED;
    if (batch == 0 || rows == 0 || cols == 0)
        return MXQ_OK;
    if (!g || !out)
        return MXQ_ERR_NULL;
    if (!aligned(g, dtype_size(dtype)) || !aligned(out, 2))
        return MXQ_ERR_ALIGN;
    const NsPlan p = ns_plan(batch, rows, cols, steps);
    if (!workspace || workspace_bytes < p.bytes)
        return MXQ_ERR_WORKSPACE;
    if (!aligned(workspace, 256))
        return MXQ_ERR_ALIGN;
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    CUtensorMap mx, mt[2], ma, mb;
    if ((rc = ns_map(&mx, ws + p.xh, p.n, p.ldx, p.m, batch)) != MXQ_OK ||
        (rc = ns_map(&mt[0], ws + p.xt[0], p.m, p.ldt, p.n, batch)) != MXQ_OK ||
        (rc = ns_map(&mt[1], ws + p.xt[1], p.m, p.ldt, p.n, batch)) != MXQ_OK ||
        (rc = ns_map(&ma, ws + p.A, p.m, p.ldt, p.m, batch)) != MXQ_OK ||
        (rc = ns_map(&mb, ws + p.B, p.m, p.ldt, p.m, batch)) != MXQ_OK)
        return rc;
    rc = dtype == MXQ_BF16 ? ns_start(static_cast<const uint16_t *>(g), batch, rows, cols, p, eps, ws, stream)
                           : ns_start(static_cast<const float *>(g), batch, rows, cols, p, eps, ws, stream);
    if (rc != MXQ_OK)
        return rc;
    ns::Args a = {};
    a.E = (int)batch;
    a.m = (int)p.m;
    a.n = (int)p.n;
    a.ldx = (int)p.ldx;
    a.ldt = (int)p.ldt;
    a.xh = reinterpret_cast<__half *>(ws + p.xh);
    a.xl = reinterpret_cast<__half *>(ws + p.xl);
    a.A = reinterpret_cast<__half *>(ws + p.A);
    a.B = reinterpret_cast<__half *>(ws + p.B);
    a.out = static_cast<uint16_t *>(out);
    a.out_t = p.tall;
    a.out_vec = cols % 8 == 0 && aligned(out, 16);
    for (int s = 0; s < steps; ++s) {
        a.a = coefficients[3 * s];
        a.b = coefficients[3 * s + 1];
        a.c = coefficients[3 * s + 2];
        a.xt = reinterpret_cast<__half *>(ws + p.xt[(s + 1) & 1]);
        if ((rc = ns_product<ns::GRAM>(mx, mx, a, p.n, stream)) != MXQ_OK ||
            (rc = ns_product<ns::POLY>(ma, ma, a, p.m, stream)) != MXQ_OK ||
            (rc = s + 1 < steps ? ns_product<ns::STEP>(mb, mt[s & 1], a, p.m, stream)
                                : ns_product<ns::LAST>(mb, mt[s & 1], a, p.m, stream)) != MXQ_OK)
            return rc;
    }
    return MXQ_OK;
}

} // extern "C"

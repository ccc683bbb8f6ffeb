// moe_host.cuh - host side of the operators in moe.cuh: argument checks,
// choice of the variant, launches. Included at the end of mxq.cu.
#pragma once

namespace {

using namespace mxq;

// lanes per token: eight experts per lane until a warp is full
#define MXQ_ROUTE_VARIANTS(X, T) X(T, 1, 8) X(T, 2, 8) X(T, 4, 8) X(T, 8, 8) X(T, 16, 8) X(T, 32, 8) X(T, 32, 16) X(T, 32, 32)

struct RouteShape {
    int lpt, epl;
};

RouteShape route_shape(int64_t E)
{
    int lpt = 1;
    while (lpt < 32 && lpt * 8 < E)
        lpt *= 2;
    const int epl = E <= 256 ? 8 : (E <= 512 ? 16 : 32);
    return {lpt, epl};
}

// CTAs of the router: one for few tokens (it then needs no second launch),
// else a warp for every group of tokens up to two CTAs per SM, which then take
// the groups in turn
int64_t route_grid(int64_t T, int64_t E, int sms)
{
    const int64_t per_cta = (int64_t)moe::ROUTE_WARPS * (32 / route_shape(E).lpt);
    const int64_t want = (T + per_cta - 1) / per_cta;
    if (want <= 2)
        return 1;
    return std::min<int64_t>(want, (int64_t)sms * 2);
}

constexpr int64_t ROUTE_MAX_CTAS = 4096; // bound of the workspace, any device

size_t route_part_layout(int64_t R, int64_t E, moe::RoutePart *part, void *ws)
{
    uint8_t *p = static_cast<uint8_t *>(ws);
    size_t o = 0;
    auto take = [&](size_t bytes) {
        uint8_t *q = p + o;
        o = round_up(o + bytes, 256);
        return q;
    };
    uint8_t *a = take((size_t)R * E * 4), *b = take((size_t)R * E * 4), *c = take((size_t)R * 4);
    uint8_t *d = take((size_t)((E + 31) / 32) * 8), *e = take(4);
    if (part)
        *part = {reinterpret_cast<float *>(a), reinterpret_cast<int *>(b), reinterpret_cast<int *>(c),
                 reinterpret_cast<double *>(d), reinterpret_cast<int *>(e)};
    return o;
}

bool dtype_ok(int32_t dtype) { return dtype == MXQ_BF16 || dtype == MXQ_FP32; }
int dtype_size(int32_t dtype) { return dtype == MXQ_BF16 ? 2 : 4; }

int route_check(const void *logits, int32_t dtype, int64_t T, int64_t E, int64_t ld, int32_t k)
{
    if (T < 0 || E < 1 || k < 1 || k > E || (T > 0 && ld < E))
        return MXQ_ERR_SHAPE;
    if (!dtype_ok(dtype) || E > moe::MAX_E || k > moe::MAX_K || T >= (int64_t(1) << 31) / k)
        return MXQ_ERR_UNSUPPORTED;
    if (T > 0 && !logits)
        return MXQ_ERR_NULL;
    if (T > 0 && !aligned(logits, dtype_size(dtype)))
        return MXQ_ERR_ALIGN;
    return MXQ_OK;
}

bool rows_vec16(const void *p, int64_t ld, int size) { return aligned(p, 16) && ld * size % 16 == 0; }

template <typename T>
int route_forward(const void *logits, int64_t tokens, int64_t E, int64_t ld, const uint8_t *valid, int k, int renorm,
                  float *weights, int32_t *ids, const moe::RoutePart &part, int64_t grid, int32_t *counts,
                  float *loss, float *loss_grad, cudaStream_t stream)
{
    const RouteShape s = route_shape(E);
    // at most 36 KB (1024 experts), below what needs a function attribute
    const size_t smem = (size_t)(moe::ROUTE_ROWS + 1) * E * 4;
    const int vec = E % (16 / sizeof(T)) == 0 && rows_vec16(logits, ld, sizeof(T));
    const T *l = static_cast<const T *>(logits);
#define MXQ_ROUTE_CASE(TT, LPT, EPL)                                                                                 \
    if (s.lpt == LPT && s.epl == EPL)                                                                                \
        return launch(k_moe_route<TT, LPT, EPL>, dim3((unsigned)grid), dim3(moe::ROUTE_THREADS), smem, stream,       \
                      false, l, tokens, (int)E, ld, valid, k, renorm, vec, weights, ids, part, counts, loss,         \
                      loss_grad);
    MXQ_ROUTE_VARIANTS(MXQ_ROUTE_CASE, T)
#undef MXQ_ROUTE_CASE
    return MXQ_ERR_UNSUPPORTED;
}

template <typename T>
int route_backward(const void *logits, int64_t tokens, int64_t E, int64_t ld, const uint8_t *valid, int k, int renorm,
                   const float *weights, const int32_t *ids, const float *loss_grad, const float *gw,
                   const float *gl, void *out, int sms, cudaStream_t stream)
{
    const RouteShape s = route_shape(E);
    const int vec = E % (16 / sizeof(T)) == 0 && rows_vec16(logits, ld, sizeof(T)) && aligned(out, 16);
    const int64_t per_cta = (int64_t)moe::ROUTE_BWD_WARPS * (32 / s.lpt);
    const int64_t grid = std::min<int64_t>((tokens + per_cta - 1) / per_cta, (int64_t)sms * 8);
    const size_t smem = (size_t)moe::ROUTE_BWD_WARPS * 32 * s.epl * 4;
    const T *l = static_cast<const T *>(logits);
#define MXQ_ROUTE_CASE(TT, LPT, EPL)                                                                                 \
    if (s.lpt == LPT && s.epl == EPL)                                                                                \
        return launch(k_moe_route_bwd<TT, LPT, EPL>, dim3((unsigned)grid), dim3(moe::ROUTE_BWD_THREADS), smem, stream,   \
                      false, l, tokens, (int)E, ld, valid, k, renorm, vec, weights, ids, loss_grad, gw, gl,          \
                      static_cast<TT *>(out));
    MXQ_ROUTE_VARIANTS(MXQ_ROUTE_CASE, T)
#undef MXQ_ROUTE_CASE
    return MXQ_ERR_UNSUPPORTED;
}

// chunks of whole tiles for the order by expert
void plan_chunks(int64_t n, int64_t *chunks, int64_t *chunk)
{
    const int64_t tiles = std::max<int64_t>(1, (n + moe::PLAN_TILE - 1) / moe::PLAN_TILE);
    const int64_t per = (tiles + moe::PLAN_MAX_CHUNKS - 1) / moe::PLAN_MAX_CHUNKS;
    *chunks = (tiles + per - 1) / per;
    *chunk = per * moe::PLAN_TILE;
}

// elements that move as one vector: 16 bytes when every row of every operand
// starts on a 16-byte boundary, else 4 bytes, else one element
struct RowOperand {
    const void *p;
    int64_t ld;
};
int row_vector(std::initializer_list<RowOperand> ops, int64_t K, int size)
{
    for (int bytes = 16; bytes > size; bytes = bytes == 16 ? 4 : size) {
        bool ok = K * size % bytes == 0;
        for (const RowOperand &o : ops)
            ok = ok && aligned(o.p, bytes) && o.ld * size % bytes == 0;
        if (ok)
            return bytes / size;
    }
    return 1;
}

// Vectors of V elements, and how many of them a lane has in flight: U of one
// row where one row is read, U4 of each of up to four slots, U8 of each of J8
// slots where there are more (more in flight costs residency: at 16384 x 4 rows
// of 7168 bf16, U4 = 2 with four CTAs per SM, 24 bytes of spills a thread, sums in
// 186 us, with two CTAs and twice the loads in 197, with five CTAs and more spills
// in 235). Single elements want more of both: at 5003 x 6 rows of 1419 fp32, U8 =
// 4 of three slots with five CTAs per SM sums in 51 us, of four slots with four in
// 55; the backward takes 78 us with U = 12 and 82 with 8 (nothing dropped).
#define MXQ_ROW_VARIANTS(X) X(MXQ_BF16, uint16_t, 8, 4, 2, 8, 1) X(MXQ_BF16, uint16_t, 2, 8, 4, 4, 4) X(MXQ_BF16, uint16_t, 1, 12, 4, 3, 4) X(MXQ_FP32, float, 4, 4, 2, 8, 1) X(MXQ_FP32, float, 1, 12, 4, 3, 4)

unsigned row_grid(int64_t warps, int sms)
{
    return (unsigned)std::max<int64_t>(1, std::min<int64_t>((warps + moe::ROW_WARPS - 1) / moe::ROW_WARPS,
                                                            (int64_t)sms * 32));
}

int rows_check(int32_t dtype, int64_t T, int32_t k, int64_t K, int64_t M, int64_t ld)
{
    if (T < 0 || K < 0 || M < 0 || k < 1 || ld < K)
        return MXQ_ERR_SHAPE;
    if (!dtype_ok(dtype) || k > moe::MAX_K || K >= (int64_t(1) << 31) || M >= (int64_t(1) << 31) ||
        T >= (int64_t(1) << 31) / k)
        return MXQ_ERR_UNSUPPORTED;
    return MXQ_OK;
}

} // namespace

extern "C" {

size_t moe_route_workspace_bytes(int64_t tokens, int64_t experts)
{
    if (tokens < 0 || experts < 1 || experts > moe::MAX_E)
        return 0;
    const DevInfo *di = nullptr;
    const int64_t R = device_info(&di) == MXQ_OK ? route_grid(tokens, experts, di->sms) : ROUTE_MAX_CTAS;
    return route_part_layout(R, experts, nullptr, nullptr);
}

int moe_route(const void *logits, int32_t dtype, int64_t tokens, int64_t experts, int64_t row_stride,
              const uint8_t *valid, int32_t top_k, int32_t renormalize, float *weights, int32_t *ids,
              int32_t *counts, float *loss, float *loss_grad, void *workspace, size_t workspace_bytes,
              cudaStream_t stream)
{
    int rc = route_check(logits, dtype, tokens, experts, row_stride, top_k);
    if (rc != MXQ_OK)
        return rc;
    if (!counts || !loss || (tokens > 0 && (!weights || !ids)))
        return MXQ_ERR_NULL;
    if (!aligned(weights, 4) || !aligned(ids, 4) || !aligned(counts, 4) || !aligned(loss, 4) ||
        !aligned(loss_grad, 4))
        return MXQ_ERR_ALIGN;
    const DevInfo *di = nullptr;
    rc = device_info(&di);
    if (rc != MXQ_OK)
        return rc;
    const int64_t R = route_grid(tokens, experts, di->sms);
    if (!workspace || workspace_bytes < route_part_layout(R, experts, nullptr, nullptr))
        return MXQ_ERR_WORKSPACE;
    if (!aligned(workspace, 256))
        return MXQ_ERR_ALIGN;
    moe::RoutePart part;
    route_part_layout(R, experts, &part, workspace);
    rc = dtype == MXQ_BF16
             ? route_forward<uint16_t>(logits, tokens, experts, row_stride, valid, top_k, renormalize != 0, weights,
                                       ids, part, R, counts, loss, loss_grad, stream)
             : route_forward<float>(logits, tokens, experts, row_stride, valid, top_k, renormalize != 0, weights, ids,
                                    part, R, counts, loss, loss_grad, stream);
    if (rc != MXQ_OK || R == 1)
        return rc;
    return launch_chained(k_moe_route_finish, dim3((unsigned)((experts + 31) / 32)), dim3(1024), 0, stream, false,
                          part, (int)R, (int)experts, (int)top_k, counts, loss, loss_grad);
}

int moe_route_backward(const void *logits, int32_t dtype, int64_t tokens, int64_t experts, int64_t row_stride,
                       const uint8_t *valid, int32_t top_k, int32_t renormalize, const float *weights,
                       const int32_t *ids, const float *loss_grad, const float *grad_weights, const float *grad_loss,
                       void *grad_logits, cudaStream_t stream)
{
    int rc = route_check(logits, dtype, tokens, experts, row_stride, top_k);
    if (rc != MXQ_OK)
        return rc;
    if (tokens == 0)
        return MXQ_OK;
    if (!grad_logits || (grad_weights && (!weights || !ids)) || (grad_loss && !loss_grad))
        return MXQ_ERR_NULL;
    if (!aligned(weights, 4) || !aligned(ids, 4) || !aligned(loss_grad, 4) || !aligned(grad_weights, 4) ||
        !aligned(grad_loss, 4) || !aligned(grad_logits, dtype_size(dtype)))
        return MXQ_ERR_ALIGN;
    const DevInfo *di = nullptr;
    rc = device_info(&di);
    if (rc != MXQ_OK)
        return rc;
    return dtype == MXQ_BF16
               ? route_backward<uint16_t>(logits, tokens, experts, row_stride, valid, top_k, renormalize != 0,
                                          weights, ids, loss_grad, grad_weights, grad_loss, grad_logits, di->sms,
                                          stream)
               : route_backward<float>(logits, tokens, experts, row_stride, valid, top_k, renormalize != 0, weights,
                                       ids, loss_grad, grad_weights, grad_loss, grad_logits, di->sms, stream);
}

size_t moe_dispatch_plan_workspace_bytes(int64_t entries, int64_t experts)
{
    if (entries < 0 || experts < 1 || experts > moe::MAX_E)
        return 0;
    int64_t chunks, chunk;
    plan_chunks(entries, &chunks, &chunk);
    return chunks <= moe::PLAN_SELF_CHUNKS ? 0 : (size_t)chunks * experts * 4;
}

int moe_dispatch_plan(const int32_t *ids, int64_t entries, int64_t experts, int32_t *pos, int32_t *offs,
                      void *workspace, size_t workspace_bytes, cudaStream_t stream)
{
    if (entries < 0 || experts < 1)
        return MXQ_ERR_SHAPE;
    if (experts > moe::MAX_E || entries >= (int64_t(1) << 31))
        return MXQ_ERR_UNSUPPORTED;
    if (!offs || (entries > 0 && (!ids || !pos)))
        return MXQ_ERR_NULL;
    if (!aligned(ids, 4) || !aligned(pos, 4) || !aligned(offs, 4))
        return MXQ_ERR_ALIGN;
    int64_t chunks, chunk;
    plan_chunks(entries, &chunks, &chunk);
    const size_t need = moe_dispatch_plan_workspace_bytes(entries, experts);
    if (need && (!workspace || workspace_bytes < need))
        return MXQ_ERR_WORKSPACE;
    if (need && !aligned(workspace, 4))
        return MXQ_ERR_ALIGN;
    int *hist = need ? static_cast<int *>(workspace) : nullptr;
    if (hist) {
        const int rc = launch(k_moe_plan_count, dim3((unsigned)chunks), dim3(moe::PLAN_THREADS), (size_t)experts * 4,
                              stream, false, ids, entries, (int)experts, chunk, hist);
        if (rc != MXQ_OK)
            return rc;
    }
    // at most 44 KB (1024 experts), below what needs a function attribute
    const size_t smem = moe::plan_smem((int)experts);
    const dim3 grid((unsigned)chunks), block(moe::PLAN_THREADS);
    if (!hist)
        return launch(k_moe_plan_rank, grid, block, smem, stream, false, ids, entries, (int)experts, chunk,
                      (const int *)nullptr, (int)chunks, pos, offs);
    return launch_chained(k_moe_plan_rank, grid, block, smem, stream, false, ids, entries, (int)experts, chunk,
                          (const int *)hist, (int)chunks, pos, offs);
}

int moe_dispatch(const void *x, int32_t dtype, int64_t tokens, int64_t cols, int64_t row_stride, const int32_t *pos,
                 int32_t top_k, const int32_t *offs, int32_t num_groups, void *out, int64_t out_rows,
                 cudaStream_t stream)
{
    int rc = rows_check(dtype, tokens, top_k, cols, out_rows, row_stride);
    if (rc != MXQ_OK)
        return rc;
    if (num_groups < 1)
        return MXQ_ERR_SHAPE;
    if (out_rows == 0 || cols == 0)
        return MXQ_OK;
    if (!offs || !out || (tokens > 0 && (!x || !pos)))
        return MXQ_ERR_NULL;
    const int size = dtype_size(dtype);
    if (!aligned(x, size) || !aligned(out, size) || !aligned(pos, 4) || !aligned(offs, 4))
        return MXQ_ERR_ALIGN;
    const DevInfo *di = nullptr;
    rc = device_info(&di);
    if (rc != MXQ_OK)
        return rc;
    const int v = row_vector({{x, row_stride}, {out, cols}}, cols, size);
#define MXQ_ROW_CASE(D, T, V, U, U4, J8, U8)                                                                         \
    if (dtype == D && v == V) {                                                                                      \
        const int64_t segs = (cols / V + 32 * U - 1) / (32 * U);                                                     \
        return launch(k_moe_dispatch<T, V, U>, dim3(row_grid((tokens + 16) * segs, di->sms)),                        \
                      dim3(moe::ROW_THREADS), 0, stream, false, static_cast<const T *>(x), tokens, cols, row_stride, \
                      pos, (int)top_k, offs, (int)num_groups, static_cast<T *>(out), out_rows);                      \
    }
    MXQ_ROW_VARIANTS(MXQ_ROW_CASE)
#undef MXQ_ROW_CASE
    return MXQ_ERR_UNSUPPORTED;
}

int moe_combine(const void *y, int32_t dtype, int64_t rows, int64_t cols, int64_t row_stride, const int32_t *pos,
                const float *weights, int64_t tokens, int32_t top_k, void *out, cudaStream_t stream)
{
    int rc = rows_check(dtype, tokens, top_k, cols, rows, row_stride);
    if (rc != MXQ_OK)
        return rc;
    if (tokens == 0 || cols == 0)
        return MXQ_OK;
    if ((rows > 0 && !y) || !pos || !out)
        return MXQ_ERR_NULL;
    const int size = dtype_size(dtype);
    if (!aligned(y, size) || !aligned(out, size) || !aligned(pos, 4) || !aligned(weights, 4))
        return MXQ_ERR_ALIGN;
    const DevInfo *di = nullptr;
    rc = device_info(&di);
    if (rc != MXQ_OK)
        return rc;
    const int v = row_vector({{y, row_stride}, {out, cols}}, cols, size);
    // runs of a row: one when the tokens alone give every resident warp eight
    const int64_t want = std::max<int64_t>(1, (int64_t)di->sms * 32 * 8 / tokens);
#define MXQ_ROW_LAUNCH(T, V, U, J)                                                                                   \
    {                                                                                                                \
        const int64_t width = 32 * U, steps = (cols / V + width - 1) / width, split = std::min(steps, want);         \
        const int64_t run = (steps + split - 1) / split * width, parts = (cols / V + run - 1) / run;                 \
        return launch(k_moe_combine<T, V, U, J>, dim3(row_grid(tokens * parts, di->sms)), dim3(moe::ROW_THREADS), 0, \
                      stream, false, static_cast<const T *>(y), rows, cols, row_stride, pos, weights,                \
                      (uint32_t)tokens, (uint32_t)parts, (uint32_t)run, (int)top_k, static_cast<T *>(out));          \
    }
#define MXQ_ROW_CASE(D, T, V, U, U4, J8, U8)                                                                         \
    if (dtype == D && v == V && top_k <= 4)                                                                          \
        MXQ_ROW_LAUNCH(T, V, U4, 4)                                                                                  \
    if (dtype == D && v == V)                                                                                        \
        MXQ_ROW_LAUNCH(T, V, U8, J8)
    MXQ_ROW_VARIANTS(MXQ_ROW_CASE)
#undef MXQ_ROW_CASE
#undef MXQ_ROW_LAUNCH
    return MXQ_ERR_UNSUPPORTED;
}

int moe_combine_backward(const void *grad_out, int64_t grad_row_stride, const void *y, int64_t row_stride,
                         int32_t dtype, int64_t rows, int64_t cols, const int32_t *pos, const float *weights,
                         int64_t tokens, int32_t top_k, const int32_t *offs, int32_t num_groups, void *grad_y,
                         float *grad_weights, cudaStream_t stream)
{
    int rc = rows_check(dtype, tokens, top_k, cols, rows, std::min(row_stride, grad_row_stride));
    if (rc != MXQ_OK)
        return rc;
    if (num_groups < 1)
        return MXQ_ERR_SHAPE;
    if ((!grad_y || rows == 0 || cols == 0) && (!grad_weights || tokens == 0))
        return MXQ_OK;
    if (!offs || (tokens > 0 && (!pos || (cols > 0 && !grad_out))) || (grad_weights && rows > 0 && cols > 0 && !y))
        return MXQ_ERR_NULL;
    const int size = dtype_size(dtype);
    if (!aligned(y, size) || !aligned(grad_out, size) || !aligned(grad_y, size) || !aligned(pos, 4) ||
        !aligned(weights, 4) || !aligned(grad_weights, 4) || !aligned(offs, 4))
        return MXQ_ERR_ALIGN;
    const DevInfo *di = nullptr;
    rc = device_info(&di);
    if (rc != MXQ_OK)
        return rc;
    const int v = row_vector({{grad_out, grad_row_stride}, {grad_weights ? y : nullptr, grad_weights ? row_stride : 0},
                              {grad_y, cols}},
                             cols, size);
#define MXQ_ROW_CASE(D, T, V, U, U4, J8, U8)                                                                         \
    if (dtype == D && v == V)                                                                                        \
        return launch(k_moe_combine_bwd<T, V, U>, dim3(row_grid(tokens * top_k + 16, di->sms)),                      \
                      dim3(moe::ROW_THREADS), 0, stream, false, static_cast<const T *>(grad_out), grad_row_stride,   \
                      static_cast<const T *>(y), row_stride, rows, cols, pos, weights, tokens, (int)top_k, offs,     \
                      (int)num_groups, static_cast<T *>(grad_y), grad_weights);
    MXQ_ROW_VARIANTS(MXQ_ROW_CASE)
#undef MXQ_ROW_CASE
    return MXQ_ERR_UNSUPPORTED;
}

} // extern "C"

// moe_autograd.cpp - the differentiable router, dispatch and combine as C++
// autograd nodes over libmxq's C ABI (module _torch_ops, used by autograd.py).
//
// Why not Python functions as for the grouped matmuls: a training call here is
// 10 to 50 us of GPU work at ordinary sizes, and a Python node costs 120 us a
// forward and backward on the host (tensor allocations through Python, the
// interpreter taken again in the engine's thread); these cost half of that.
// Nothing is computed here: checks, torch allocations on the current stream,
// the library's calls, and what the backward keeps.
#include <ATen/cuda/CUDAContext.h>
#include <c10/cuda/CUDAGuard.h>
#include <torch/csrc/autograd/functions/basic_ops.h>
#include <torch/extension.h>

#include "mxq.h"

namespace {

using at::Tensor;
using torch::autograd::AutogradContext;
using torch::autograd::variable_list;

// a status other than MXQ_OK as binding.MXQError
void check(const char *fn, int rc)
{
    if (rc == MXQ_OK)
        return;
    pybind11::gil_scoped_acquire gil;
    const auto binding = pybind11::module_::import("mxfp8_quantization_moe_device_b200.binding");
    const pybind11::object error = binding.attr("MXQError");
    PyErr_SetObject(error.ptr(), error(fn, rc).ptr());
    throw pybind11::error_already_set();
}

const void *ptr(const Tensor &t) { return t.defined() ? t.const_data_ptr() : nullptr; }
void *out_ptr(const Tensor &t) { return t.defined() ? t.mutable_data_ptr() : nullptr; }
template <typename T> const T *ptr_as(const Tensor &t) { return static_cast<const T *>(ptr(t)); }
template <typename T> T *out_as(const Tensor &t) { return static_cast<T *>(out_ptr(t)); }

// bf16 or fp32 rows that are contiguous and do not overlap
struct Rows {
    int32_t dtype;
    int64_t rows, cols, stride;
};
Rows rows_of(const Tensor &t, const char *name)
{
    TORCH_CHECK_TYPE(t.is_cuda(), name, " must be a CUDA tensor");
    TORCH_CHECK_TYPE(t.dim() == 2 && (t.scalar_type() == at::kBFloat16 || t.scalar_type() == at::kFloat), name,
                     " must be a 2-D bfloat16 or float32 tensor");
    Rows r{t.scalar_type() == at::kBFloat16 ? MXQ_BF16 : MXQ_FP32, t.size(0), t.size(1), t.size(1)};
    TORCH_CHECK_TYPE((r.cols <= 1 || t.stride(1) == 1) && (r.rows <= 1 || t.stride(0) >= r.cols), name,
                     " must have contiguous rows that do not overlap");
    if (r.rows > 1)
        r.stride = t.stride(0);
    return r;
}

void array(const Tensor &t, const char *name, at::ScalarType type, at::IntArrayRef shape, const at::Device &dev)
{
    TORCH_CHECK_TYPE(t.is_cuda() && t.scalar_type() == type && t.sizes() == shape && t.is_contiguous() &&
                         t.device() == dev,
                     name, " must be a contiguous ", type, " tensor of shape ", shape, " on ", dev);
}

Tensor empty(at::IntArrayRef shape, at::ScalarType type, const at::Device &dev)
{
    return at::empty(shape, at::TensorOptions().dtype(type).device(dev));
}
Tensor workspace(size_t bytes, const at::Device &dev)
{
    return bytes ? empty({(int64_t)bytes}, at::kByte, dev) : Tensor();
}
cudaStream_t stream(const at::Device &dev) { return at::cuda::getCurrentCUDAStream(dev.index()).stream(); }

// Gradients that carry no graph of their own: differentiating them again, where
// the caller keeps a graph (create_graph), raises instead of giving zeros.
variable_list once(variable_list grads)
{
    if (!at::GradMode::is_enabled())
        return grads;
    variable_list given;
    for (Tensor &g : grads)
        if (g.defined())
            given.push_back(g.detach().set_requires_grad(true));
    const auto error = std::make_shared<torch::autograd::DelayedError>(
        "the gradients of the expert router, dispatch and combine cannot be differentiated again",
        (int)given.size());
    variable_list marked = (*error)(std::move(given));
    size_t i = 0;
    for (Tensor &g : grads)
        if (g.defined())
            g = marked[i++];
    return grads;
}

// ------------------------------------------------------------------ router
struct MoERoute : torch::autograd::Function<MoERoute> {
    static variable_list forward(AutogradContext *ctx, const Tensor &logits, int64_t k,
                                 const std::optional<Tensor> &mask, bool renormalize)
    {
        const Tensor valid = mask.value_or(Tensor());
        const Rows l = rows_of(logits, "logits");
        const at::Device dev = logits.device();
        TORCH_CHECK_VALUE(k >= 1 && k <= l.cols, "top_k must lie in [1, experts]");
        if (valid.defined())
            array(valid, "valid", valid.scalar_type() == at::kByte ? at::kByte : at::kBool, {l.rows}, dev);
        const c10::cuda::CUDAGuard guard(dev);
        Tensor weights = empty({l.rows, k}, at::kFloat, dev), ids = empty({l.rows, k}, at::kInt, dev);
        Tensor counts = empty({l.cols}, at::kInt, dev), loss = empty({}, at::kFloat, dev);
        Tensor loss_grad = empty({l.cols}, at::kFloat, dev);
        const size_t bytes = moe_route_workspace_bytes(l.rows, l.cols);
        const Tensor ws = workspace(bytes, dev);
        check("moe_route", moe_route(ptr(logits), l.dtype, l.rows, l.cols, l.stride, ptr_as<uint8_t>(valid), (int)k,
                                     renormalize, out_as<float>(weights), out_as<int32_t>(ids),
                                     out_as<int32_t>(counts), out_as<float>(loss), out_as<float>(loss_grad),
                                     out_ptr(ws), bytes, stream(dev)));
        ctx->set_materialize_grads(false);
        ctx->mark_non_differentiable({ids, counts});
        ctx->save_for_backward({logits, weights, ids, loss_grad, valid});
        ctx->saved_data["renormalize"] = renormalize;
        return {weights, ids, counts, loss};
    }

    static variable_list backward(AutogradContext *ctx, variable_list grads)
    {
        Tensor gw = grads[0], gl = grads[3];
        if (!gw.defined() && !gl.defined())
            return {Tensor(), Tensor(), Tensor(), Tensor()};
        const auto saved = ctx->get_saved_variables();
        const Tensor &logits = saved[0], &weights = saved[1], &ids = saved[2], &loss_grad = saved[3], &valid = saved[4];
        const Rows l = rows_of(logits, "logits");
        const at::Device dev = logits.device();
        const c10::cuda::CUDAGuard guard(dev);
        if (gw.defined())
            gw = gw.contiguous();
        Tensor out = empty({l.rows, l.cols}, logits.scalar_type(), dev);
        check("moe_route_backward",
              moe_route_backward(ptr(logits), l.dtype, l.rows, l.cols, l.stride, ptr_as<uint8_t>(valid),
                                 (int)ids.size(1), ctx->saved_data["renormalize"].toBool(), ptr_as<float>(weights),
                                 ptr_as<int32_t>(ids), ptr_as<float>(loss_grad), ptr_as<float>(gw),
                                 ptr_as<float>(gl), out_ptr(out), stream(dev)));
        return once({out, Tensor(), Tensor(), Tensor()});
    }
};

// ------------------------------------------------------------------ rows
// out (tokens, cols) = sum over the slots of weights (undefined: ones) * y
Tensor combine(const Tensor &y, const Rows &r, const Tensor &pos, const Tensor &weights)
{
    const at::Device dev = y.device();
    Tensor out = empty({pos.size(0), r.cols}, y.scalar_type(), dev);
    check("moe_combine", moe_combine(ptr(y), r.dtype, r.rows, r.cols, r.stride, ptr_as<int32_t>(pos),
                                     ptr_as<float>(weights), pos.size(0), (int)pos.size(1), out_ptr(out),
                                     stream(dev)));
    return out;
}

struct MoEDispatch : torch::autograd::Function<MoEDispatch> {
    static variable_list forward(AutogradContext *ctx, const Tensor &x, const Tensor &ids, int64_t num_experts)
    {
        const Rows r = rows_of(x, "x");
        const at::Device dev = x.device();
        TORCH_CHECK_TYPE(ids.dim() == 2, "ids must be a (tokens, top_k) int32 tensor");
        array(ids, "ids", at::kInt, {r.rows, ids.size(1)}, dev);
        TORCH_CHECK_VALUE(num_experts >= 1, "num_experts must be positive");
        TORCH_CHECK_VALUE(ids.size(1) >= 1, "ids must have at least one slot per token");
        const c10::cuda::CUDAGuard guard(dev);
        const cudaStream_t s = stream(dev);
        const int64_t entries = ids.numel(), rows = (entries + 15) / 16 * 16;
        Tensor pos = empty(ids.sizes(), at::kInt, dev), offs = empty({num_experts}, at::kInt, dev);
        const size_t bytes = moe_dispatch_plan_workspace_bytes(entries, num_experts);
        const Tensor ws = workspace(bytes, dev);
        check("moe_dispatch_plan", moe_dispatch_plan(ptr_as<int32_t>(ids), entries, num_experts, out_as<int32_t>(pos),
                                                     out_as<int32_t>(offs), out_ptr(ws), bytes, s));
        Tensor out = empty({rows, r.cols}, x.scalar_type(), dev);
        check("moe_dispatch", moe_dispatch(ptr(x), r.dtype, r.rows, r.cols, r.stride, ptr_as<int32_t>(pos),
                                           (int)ids.size(1), ptr_as<int32_t>(offs), (int)num_experts, out_ptr(out),
                                           rows, s));
        ctx->set_materialize_grads(false);
        ctx->mark_non_differentiable({pos, offs});
        ctx->save_for_backward({pos});
        return {out, pos, offs};
    }

    static variable_list backward(AutogradContext *ctx, variable_list grads)
    {
        if (!grads[0].defined())
            return {Tensor(), Tensor(), Tensor()};
        const Tensor pos = ctx->get_saved_variables()[0], g = grads[0].contiguous();
        const c10::cuda::CUDAGuard guard(g.device());
        return once({combine(g, rows_of(g, "the gradient"), pos, Tensor()), Tensor(), Tensor()});
    }
};

struct MoECombine : torch::autograd::Function<MoECombine> {
    static variable_list forward(AutogradContext *ctx, const Tensor &y, const Tensor &pos, const Tensor &weights,
                                 const Tensor &offs)
    {
        const Rows r = rows_of(y, "y");
        const at::Device dev = y.device();
        TORCH_CHECK_TYPE(pos.dim() == 2, "pos must be a (tokens, top_k) int32 tensor");
        array(pos, "pos", at::kInt, pos.sizes(), dev);
        array(weights, "weights", at::kFloat, pos.sizes(), dev);
        TORCH_CHECK_TYPE(offs.dim() == 1 && offs.numel() >= 1, "offs must be a 1-D int32 tensor of group ends");
        array(offs, "offs", at::kInt, offs.sizes(), dev);
        TORCH_CHECK_VALUE(pos.size(1) >= 1, "pos must have at least one slot per token");
        const c10::cuda::CUDAGuard guard(dev);
        ctx->set_materialize_grads(false);
        ctx->save_for_backward({y, pos, weights, offs});
        return {combine(y, r, pos, weights)};
    }

    static variable_list backward(AutogradContext *ctx, variable_list grads)
    {
        if (!grads[0].defined())
            return {Tensor(), Tensor(), Tensor(), Tensor()};
        const auto saved = ctx->get_saved_variables();
        const Tensor &y = saved[0], &pos = saved[1], &weights = saved[2], &offs = saved[3];
        const Tensor g = grads[0].contiguous();
        const Rows r = rows_of(y, "y");
        const at::Device dev = y.device();
        const c10::cuda::CUDAGuard guard(dev);
        Tensor dy, dw;
        if (ctx->needs_input_grad(0))
            dy = empty({r.rows, r.cols}, y.scalar_type(), dev);
        if (ctx->needs_input_grad(2))
            dw = empty(pos.sizes(), at::kFloat, dev);
        check("moe_combine_backward",
              moe_combine_backward(ptr(g), r.cols, ptr(y), r.stride, r.dtype, r.rows, r.cols, ptr_as<int32_t>(pos),
                                   ptr_as<float>(weights), pos.size(0), (int)pos.size(1), ptr_as<int32_t>(offs),
                                   (int)offs.numel(), out_ptr(dy), out_as<float>(dw), stream(dev)));
        return once({dy, Tensor(), dw, Tensor()});
    }
};

std::tuple<Tensor, Tensor, Tensor, Tensor> route(const Tensor &logits, int64_t top_k,
                                                 const std::optional<Tensor> &valid, bool renormalize)
{
    const variable_list o = MoERoute::apply(logits, top_k, valid, renormalize);
    return {o[0], o[1], o[2], o[3]};
}
std::tuple<Tensor, Tensor, Tensor> dispatch(const Tensor &x, const Tensor &ids, int64_t num_experts)
{
    const variable_list o = MoEDispatch::apply(x, ids, num_experts);
    return {o[0], o[1], o[2]};
}
Tensor combine_rows(const Tensor &y, const Tensor &pos, const Tensor &weights, const Tensor &offs)
{
    return MoECombine::apply(y, pos, weights, offs)[0];
}

} // namespace

PYBIND11_MODULE(TORCH_EXTENSION_NAME, m)
{
    m.def("moe_route", &route);
    m.def("moe_dispatch", &dispatch);
    m.def("moe_combine", &combine_rows);
}

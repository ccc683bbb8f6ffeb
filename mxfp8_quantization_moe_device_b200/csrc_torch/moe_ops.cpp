// moe_ops.cpp - the router, dispatch and combine of libmxq's C ABI for torch
// tensors, and their C++ autograd nodes (module _torch_ops, used by binding.py
// and autograd.py).
//
// Why C++ and not ctypes and Python functions as for the quantization ops: a
// call here is 3 to 50 us of GPU work at ordinary sizes, and through Python it
// cost the host 26 us (router) to 30 us (dispatch with its plan) forward, 120
// us and more forward and backward (tensor allocations, the interpreter taken
// again in the engine's thread); here 10, 12 and 60 to 75. Nothing is computed
// here: checks, torch allocations on the current stream, the library's calls,
// and what the backward keeps.
#include <ATen/cuda/CUDAContext.h>
#include <c10/cuda/CUDAGraphsC10Utils.h>
#include <c10/cuda/CUDAGuard.h>
#include <torch/csrc/autograd/functions/basic_ops.h>
#include <torch/csrc/autograd/graph_task.h>
#include <torch/extension.h>

#include <unordered_set>
#include <vector>

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
using Given = std::optional<Tensor>; // an output that the caller may have
Tensor output(const Given &t, const char *name, at::ScalarType type, at::IntArrayRef shape, const at::Device &dev)
{
    if (!t || !t->defined())
        return empty(shape, type, dev);
    array(*t, name, type, shape, dev);
    return *t;
}

// Whether `out`, contiguous, shares a byte with `t`: contiguous, or rows of
// contiguous elements that do not overlap (the gaps between them count as free).
bool overlaps(const Tensor &out, const Tensor &t)
{
    if (out.numel() == 0 || t.numel() == 0)
        return false;
    const auto at = [](const Tensor &x) { return reinterpret_cast<intptr_t>(x.const_data_ptr()); };
    const int64_t size = t.element_size(), lo = at(out) - at(t), hi = lo + (int64_t)out.nbytes();
    if (t.is_contiguous())
        return lo < (int64_t)t.nbytes() && hi > 0;
    // rows [i step, i step + row): the first that ends behind lo must begin before hi
    const int64_t row = t.size(1) * size, step = t.stride(0) * size;
    const int64_t i = lo < row ? 0 : (lo - row) / step + 1;
    return i < t.size(0) && i * step < hi;
}
// The kernels read some rows while others are written, so a given output
// overlaps no input, nor another output.
using Tensors = std::initializer_list<std::reference_wrapper<const Tensor>>;
void apart(const Given &out, const char *name, Tensors inputs, Tensors outputs = {})
{
    if (!out || !out->defined())
        return;
    for (const Tensor &i : inputs)
        TORCH_CHECK_VALUE(!i.defined() || !overlaps(*out, i), name, " must not overlap an input");
    for (const Tensor &o : outputs)
        TORCH_CHECK_VALUE(!o.defined() || !overlaps(*out, o), name, " must not overlap another output");
}
Tensor given(const Given &t) { return t.value_or(Tensor()); }
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

// A backward pass runs every node on the stream of its forward. During a
// stream capture, a leaf or node whose own stream is the default one (a graph
// that was built before the capture and still lives) would have the captured
// pass wait on that stream, which breaks the capture and can end the process.
// The forward refuses such an input, the backward such a node anywhere behind it.
bool capturing(const at::Device &dev)
{
    const c10::cuda::CUDAGuard guard(dev);
    return c10::cuda::currentStreamCaptureStatusMayInitCtx() != c10::cuda::CaptureStatus::None;
}
bool on_default_stream(torch::autograd::Node &node)
{
    const auto at = node.stream();
    return at && at->device_type() == at::kCUDA && *at == c10::cuda::getDefaultCUDAStream(at->device_index()).unwrap();
}
constexpr const char *LIVING = " belongs to an autograd graph built on the default stream before this capture; free that"
                               " graph first (and warm up on a side stream), or capture without gradients";

void check_capture(const Tensor &t, const char *name)
{
    if (!at::GradMode::is_enabled() || !t.requires_grad() || !t.is_cuda() || !capturing(t.device()))
        return;
    const auto node = t.grad_fn() ? t.grad_fn() : torch::autograd::impl::try_get_grad_accumulator(t);
    TORCH_CHECK(!node || !on_default_stream(*node), name, LIVING);
}

// in a node's backward: the nodes that this pass reaches through it
void check_captured_pass(const at::Device &dev)
{
    if (!capturing(dev))
        return;
    const auto *runs = torch::autograd::get_current_graph_task_exec_info(); // empty: all do
    std::unordered_set<torch::autograd::Node *> seen;
    std::vector<torch::autograd::Node *> open{torch::autograd::get_current_node().get()};
    while (!open.empty()) {
        torch::autograd::Node *const node = open.back();
        open.pop_back();
        for (const auto &edge : node->next_edges()) {
            torch::autograd::Node *const next = edge.function.get();
            if (!next || !seen.insert(next).second)
                continue;
            if (runs && !runs->empty()) {
                const auto at = runs->find(next);
                if (at == runs->end() || !at->second.should_execute())
                    continue;
            }
            TORCH_CHECK(!on_default_stream(*next), next->name(), LIVING);
            open.push_back(next);
        }
    }
}

// ------------------------------------------------------------------ calls
void check_valid(const Tensor &valid, int64_t tokens, const at::Device &dev)
{
    if (valid.defined())
        array(valid, "valid", valid.scalar_type() == at::kByte ? at::kByte : at::kBool, {tokens}, dev);
}

std::tuple<Tensor, Tensor, Tensor, Tensor> route(const Tensor &logits, int64_t k, const Given &mask, bool renormalize,
                                                 const Given &weights_, const Given &ids_, const Given &counts_,
                                                 const Given &loss_, const Given &loss_grad_)
{
    const Rows l = rows_of(logits, "logits");
    const at::Device dev = logits.device();
    TORCH_CHECK_VALUE(k >= 1 && k <= l.cols, "top_k must lie in [1, experts]");
    const Tensor valid = given(mask), loss_grad = given(loss_grad_);
    check_valid(valid, l.rows, dev);
    if (loss_grad.defined())
        array(loss_grad, "loss_grad", at::kFloat, {l.cols}, dev);
    const c10::cuda::CUDAGuard guard(dev);
    const Tensor weights = output(weights_, "weights", at::kFloat, {l.rows, k}, dev);
    const Tensor ids = output(ids_, "ids", at::kInt, {l.rows, k}, dev);
    const Tensor counts = output(counts_, "counts", at::kInt, {l.cols}, dev);
    const Tensor loss = output(loss_, "loss", at::kFloat, {}, dev);
    apart(weights_, "weights", {logits, valid}, {ids, counts, loss, loss_grad});
    apart(ids_, "ids", {logits, valid}, {counts, loss, loss_grad});
    apart(counts_, "counts", {logits, valid}, {loss, loss_grad});
    apart(loss_, "loss", {logits, valid}, {loss_grad});
    apart(loss_grad_, "loss_grad", {logits, valid});
    const size_t bytes = moe_route_workspace_bytes(l.rows, l.cols);
    const Tensor ws = workspace(bytes, dev);
    check("moe_route", moe_route(ptr(logits), l.dtype, l.rows, l.cols, l.stride, ptr_as<uint8_t>(valid),
                                 (int)std::min<int64_t>(k, INT32_MAX), renormalize, out_as<float>(weights),
                                 out_as<int32_t>(ids), out_as<int32_t>(counts), out_as<float>(loss),
                                 out_as<float>(loss_grad), out_ptr(ws), bytes, stream(dev)));
    return {weights, ids, counts, loss};
}

Tensor route_backward(const Tensor &logits, const Tensor &weights, const Tensor &ids, const Given &loss_grad_,
                      const Given &grad_weights, const Given &grad_loss, const Given &mask, bool renormalize,
                      const Given &out_)
{
    const Rows l = rows_of(logits, "logits");
    const at::Device dev = logits.device();
    TORCH_CHECK_TYPE(ids.dim() == 2 && ids.size(1) >= 1 && ids.size(1) <= l.cols,
                     "ids must be a (tokens, top_k) int32 tensor");
    const int64_t k = ids.size(1);
    const Tensor gw = given(grad_weights), gl = given(grad_loss), loss_grad = given(loss_grad_), valid = given(mask);
    array(ids, "ids", at::kInt, {l.rows, k}, dev);
    array(weights, "weights", at::kFloat, {l.rows, k}, dev);
    check_valid(valid, l.rows, dev);
    if (gw.defined())
        array(gw, "grad_weights", at::kFloat, {l.rows, k}, dev);
    if (gl.defined()) {
        array(gl, "grad_loss", at::kFloat, {}, dev);
        TORCH_CHECK_TYPE(loss_grad.defined(), "loss_grad is needed with grad_loss");
        array(loss_grad, "loss_grad", at::kFloat, {l.cols}, dev);
    }
    const c10::cuda::CUDAGuard guard(dev);
    const Tensor out = output(out_, "out", logits.scalar_type(), {l.rows, l.cols}, dev);
    apart(out_, "out", {logits, valid, weights, ids, loss_grad, gw, gl});
    check("moe_route_backward",
          moe_route_backward(ptr(logits), l.dtype, l.rows, l.cols, l.stride, ptr_as<uint8_t>(valid), (int)k,
                             renormalize, ptr_as<float>(weights), ptr_as<int32_t>(ids), ptr_as<float>(loss_grad),
                             ptr_as<float>(gw), ptr_as<float>(gl), out_ptr(out), stream(dev)));
    return out;
}

std::tuple<Tensor, Tensor> plan(const Tensor &ids, int64_t experts, const Given &pos_, const Given &offs_)
{
    TORCH_CHECK_TYPE(ids.is_cuda(), "ids must be a CUDA tensor");
    TORCH_CHECK_TYPE(ids.dim() == 2, "ids must be a (tokens, top_k) int32 tensor");
    const at::Device dev = ids.device();
    array(ids, "ids", at::kInt, ids.sizes(), dev);
    TORCH_CHECK_VALUE(experts >= 1, "num_experts must be positive");
    const c10::cuda::CUDAGuard guard(dev);
    const Tensor pos = output(pos_, "pos", at::kInt, ids.sizes(), dev);
    const Tensor offs = output(offs_, "offs", at::kInt, {experts}, dev);
    apart(pos_, "pos", {ids}, {offs});
    apart(offs_, "offs", {ids}, {pos});
    const size_t bytes = moe_dispatch_plan_workspace_bytes(ids.numel(), experts);
    const Tensor ws = workspace(bytes, dev);
    check("moe_dispatch_plan", moe_dispatch_plan(ptr_as<int32_t>(ids), ids.numel(), experts, out_as<int32_t>(pos),
                                                 out_as<int32_t>(offs), out_ptr(ws), bytes, stream(dev)));
    return {pos, offs};
}

// places (tokens, top_k >= 1) of `tokens` tokens (-1: any number)
void check_pos(const Tensor &pos, int64_t tokens, const at::Device &dev)
{
    TORCH_CHECK_TYPE(pos.dim() == 2, "pos must be a (tokens, top_k) int32 tensor");
    array(pos, "pos", at::kInt, {tokens < 0 ? pos.size(0) : tokens, pos.size(1)}, dev);
    TORCH_CHECK_VALUE(pos.size(1) >= 1, "pos must have at least one slot per token");
}
void check_offs(const Tensor &offs, const at::Device &dev)
{
    TORCH_CHECK_TYPE(offs.dim() == 1 && offs.numel() >= 1, "offs must be a 1-D int32 tensor of group ends");
    array(offs, "offs", at::kInt, offs.sizes(), dev);
}

Tensor dispatch(const Tensor &x, const Tensor &pos, const Tensor &offs, const Given &out_)
{
    const Rows r = rows_of(x, "x");
    const at::Device dev = x.device();
    check_pos(pos, r.rows, dev);
    check_offs(offs, dev);
    const bool mine = !out_ || !out_->defined();
    TORCH_CHECK_TYPE(mine || out_->dim() == 2, "out must be a (rows, cols) tensor");
    const int64_t rows = mine ? (pos.numel() + 15) / 16 * 16 : out_->size(0);
    const c10::cuda::CUDAGuard guard(dev);
    const Tensor out = output(out_, "out", x.scalar_type(), {rows, r.cols}, dev);
    apart(out_, "out", {x, pos, offs});
    check("moe_dispatch", moe_dispatch(ptr(x), r.dtype, r.rows, r.cols, r.stride, ptr_as<int32_t>(pos),
                                       (int)std::min<int64_t>(pos.size(1), INT32_MAX), ptr_as<int32_t>(offs),
                                       (int)offs.numel(), out_ptr(out), rows, stream(dev)));
    return out;
}

Tensor combine(const Tensor &y, const Tensor &pos, const Given &weights_, const Given &out_)
{
    const Rows r = rows_of(y, "y");
    const at::Device dev = y.device();
    check_pos(pos, -1, dev);
    const Tensor weights = given(weights_);
    if (weights.defined())
        array(weights, "weights", at::kFloat, pos.sizes(), dev);
    const c10::cuda::CUDAGuard guard(dev);
    const Tensor out = output(out_, "out", y.scalar_type(), {pos.size(0), r.cols}, dev);
    apart(out_, "out", {y, pos, weights});
    check("moe_combine", moe_combine(ptr(y), r.dtype, r.rows, r.cols, r.stride, ptr_as<int32_t>(pos),
                                     ptr_as<float>(weights), pos.size(0),
                                     (int)std::min<int64_t>(pos.size(1), INT32_MAX), out_ptr(out), stream(dev)));
    return out;
}

std::tuple<Given, Given> combine_backward(const Tensor &grad_out, const Tensor &y, const Tensor &pos,
                                          const Given &weights_, const Tensor &offs, bool need_y, bool need_weights,
                                          const Given &grad_y_, const Given &grad_weights_)
{
    const Rows r = rows_of(y, "y"), g = rows_of(grad_out, "grad_out");
    const at::Device dev = y.device();
    check_pos(pos, g.rows, dev);
    check_offs(offs, dev);
    TORCH_CHECK_TYPE(g.dtype == r.dtype && g.cols == r.cols && grad_out.device() == dev,
                     "grad_out must have y's type, columns and device");
    const Tensor weights = given(weights_);
    if (weights.defined())
        array(weights, "weights", at::kFloat, pos.sizes(), dev);
    const c10::cuda::CUDAGuard guard(dev);
    Tensor dy, dw;
    if (need_y)
        dy = output(grad_y_, "grad_y", y.scalar_type(), {r.rows, r.cols}, dev);
    if (need_weights)
        dw = output(grad_weights_, "grad_weights", at::kFloat, pos.sizes(), dev);
    if (need_y)
        apart(grad_y_, "grad_y", {y, grad_out, pos, weights, offs}, {dw});
    if (need_weights)
        apart(grad_weights_, "grad_weights", {y, grad_out, pos, weights, offs}, {dy});
    check("moe_combine_backward",
          moe_combine_backward(ptr(grad_out), g.stride, ptr(y), r.stride, r.dtype, r.rows, r.cols,
                               ptr_as<int32_t>(pos), ptr_as<float>(weights), pos.size(0),
                               (int)std::min<int64_t>(pos.size(1), INT32_MAX), ptr_as<int32_t>(offs),
                               (int)offs.numel(), out_ptr(dy), out_as<float>(dw), stream(dev)));
    return {need_y ? Given(dy) : Given(), need_weights ? Given(dw) : Given()};
}

// ------------------------------------------------------------------ autograd
struct MoERoute : torch::autograd::Function<MoERoute> {
    static variable_list forward(AutogradContext *ctx, const Tensor &logits, int64_t k, const Given &valid,
                                 bool renormalize)
    {
        const Rows l = rows_of(logits, "logits");
        Tensor loss_grad = empty({l.cols}, at::kFloat, logits.device());
        auto [weights, ids, counts, loss] = route(logits, k, valid, renormalize, {}, {}, {}, {}, loss_grad);
        ctx->set_materialize_grads(false);
        ctx->mark_non_differentiable({ids, counts});
        ctx->save_for_backward({logits, weights, ids, loss_grad, given(valid)});
        ctx->saved_data["renormalize"] = renormalize;
        return {weights, ids, counts, loss};
    }

    static variable_list backward(AutogradContext *ctx, variable_list grads)
    {
        Tensor gw = grads[0], gl = grads[3];
        if (!gw.defined() && !gl.defined())
            return {Tensor(), Tensor(), Tensor(), Tensor()};
        if (gw.defined())
            gw = gw.contiguous();
        const auto saved = ctx->get_saved_variables();
        check_captured_pass(saved[0].device());
        const Tensor out = route_backward(saved[0], saved[1], saved[2], saved[3], gw, gl, saved[4],
                                          ctx->saved_data["renormalize"].toBool(), {});
        return once({out, Tensor(), Tensor(), Tensor()});
    }
};

struct MoEDispatch : torch::autograd::Function<MoEDispatch> {
    static variable_list forward(AutogradContext *ctx, const Tensor &x, const Tensor &ids, int64_t num_experts)
    {
        rows_of(x, "x");
        auto [pos, offs] = plan(ids, num_experts, {}, {});
        const Tensor out = dispatch(x, pos, offs, {});
        ctx->set_materialize_grads(false);
        ctx->mark_non_differentiable({pos, offs});
        ctx->save_for_backward({pos});
        return {out, pos, offs};
    }

    static variable_list backward(AutogradContext *ctx, variable_list grads)
    {
        if (!grads[0].defined())
            return {Tensor(), Tensor(), Tensor()};
        const Tensor pos = ctx->get_saved_variables()[0];
        check_captured_pass(pos.device());
        return once({combine(grads[0].contiguous(), pos, {}, {}), Tensor(), Tensor()});
    }
};

struct MoECombine : torch::autograd::Function<MoECombine> {
    static variable_list forward(AutogradContext *ctx, const Tensor &y, const Tensor &pos, const Tensor &weights,
                                 const Tensor &offs)
    {
        const Tensor out = combine(y, pos, weights, {});
        check_offs(offs, y.device());
        ctx->set_materialize_grads(false);
        ctx->save_for_backward({y, pos, weights, offs});
        return {out};
    }

    static variable_list backward(AutogradContext *ctx, variable_list grads)
    {
        if (!grads[0].defined())
            return {Tensor(), Tensor(), Tensor(), Tensor()};
        const auto saved = ctx->get_saved_variables();
        check_captured_pass(saved[0].device());
        auto [dy, dw] = combine_backward(grads[0].contiguous(), saved[0], saved[1], saved[2], saved[3],
                                         ctx->needs_input_grad(0), ctx->needs_input_grad(2), {}, {});
        return once({given(dy), Tensor(), given(dw), Tensor()});
    }
};

std::tuple<Tensor, Tensor, Tensor, Tensor> grad_route(const Tensor &logits, int64_t top_k, const Given &valid,
                                                      bool renormalize)
{
    check_capture(logits, "logits");
    const variable_list o = MoERoute::apply(logits, top_k, valid, renormalize);
    return {o[0], o[1], o[2], o[3]};
}
std::tuple<Tensor, Tensor, Tensor> grad_dispatch(const Tensor &x, const Tensor &ids, int64_t num_experts)
{
    check_capture(x, "x");
    const variable_list o = MoEDispatch::apply(x, ids, num_experts);
    return {o[0], o[1], o[2]};
}
Tensor grad_combine(const Tensor &y, const Tensor &pos, const Tensor &weights, const Tensor &offs)
{
    check_capture(y, "y");
    check_capture(weights, "weights");
    return MoECombine::apply(y, pos, weights, offs)[0];
}

} // namespace

PYBIND11_MODULE(TORCH_EXTENSION_NAME, m)
{
    m.def("overlaps", &overlaps);
    m.def("moe_route", &route);
    m.def("moe_route_backward", &route_backward);
    m.def("moe_dispatch_plan", &plan);
    m.def("moe_dispatch", &dispatch);
    m.def("moe_combine", &combine);
    m.def("moe_combine_backward", &combine_backward);
    m.def("grad_route", &grad_route);
    m.def("grad_dispatch", &grad_dispatch);
    m.def("grad_combine", &grad_combine);
}

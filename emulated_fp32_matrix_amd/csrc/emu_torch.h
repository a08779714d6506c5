// What the differentiable operators' torch bindings share (block_torch.cpp,
// attention_torch.cpp): a C status as an exception, the device and stream of a
// call, checks of tensors and of what autograd may do with them, and
// workspaces.  Host code only.
#pragma once

#include <ATen/hip/impl/HIPStreamMasqueradingAsCUDA.h>
#include <c10/core/impl/TorchDispatchModeTLS.h>
#include <hip/hip_runtime_api.h>
#include <torch/csrc/jit/frontend/tracer.h>
#include <torch/extension.h>

#include <stdexcept>
#include <unordered_set>

#include "emu_sgemm.h"

namespace emu_torch {

using at::Tensor;
using std::optional;
using torch::autograd::AutogradContext;
using torch::autograd::Function;
using torch::autograd::variable_list;

// A C-ABI status other than success; Python sees EmuError.
struct EmuFailure : std::runtime_error {
    int status;
    std::string where;
    EmuFailure(int s, std::string w)
        : std::runtime_error(w + ": " + emu_status_string((emu_status_t)s)), status(s), where(std::move(w))
    {
    }
};

inline void done(emu_status_t s, const char* where)
{
    if (s != EMU_STATUS_SUCCESS) throw EmuFailure((int)s, where);
}

// The device of a tensor made current, and its current stream.
struct OnDevice {
    c10::DeviceGuard guard;
    hipStream_t stream;
    explicit OnDevice(const Tensor& t)
        : guard(t.device()), stream(c10::hip::getCurrentHIPStreamMasqueradingAsCUDA(t.device().index()).stream())
    {
    }
};

inline const Tensor* given(const optional<Tensor>& t) { return t.has_value() ? &*t : nullptr; }

// Refuses to read tensors for something that would have to see the kernels,
// which write to memory that torch only saw being allocated: the output would
// lack its tangent (forward-mode derivatives), or a recorded program would
// return that memory without what is written to it.  (Called for every tensor
// of a call from outside, and for the gradients that a backward pass is given.)
inline void check_readable(std::initializer_list<const Tensor*> ts)
{
    using c10::impl::TorchDispatchModeKey;
    using c10::impl::TorchDispatchModeTLS;
    TORCH_CHECK_NOT_IMPLEMENTED(!torch::jit::tracer::isTracing(), "the block operators cannot be traced by torch.jit");
    if (TorchDispatchModeTLS::any_modes_set()) {
        for (const auto key : {TorchDispatchModeKey::FAKE, TorchDispatchModeKey::PROXY, TorchDispatchModeKey::FUNCTIONAL})
            TORCH_CHECK_NOT_IMPLEMENTED(!TorchDispatchModeTLS::get_mode(key).has_value(),
                                        "the block operators cannot be traced: their kernels are no torch operators");
    }
    constexpr c10::DispatchKeySet wrappers({c10::DispatchKey::Python, c10::DispatchKey::Functionalize,
                                            c10::DispatchKey::FuncTorchGradWrapper, c10::DispatchKey::FuncTorchBatched});
    for (const Tensor* t : ts) {
        if (t == nullptr || !t->defined()) continue;
        TORCH_CHECK_NOT_IMPLEMENTED(!t->key_set().has_any(wrappers),
                                    "the block operators take plain tensors, not those of a tracer, of a torch.func "
                                    "transform or of a subclass with its own dispatch");
        TORCH_CHECK_NOT_IMPLEMENTED(!t->_fw_grad(0).defined(), "the block operators have no forward-mode derivative");
    }
}

inline void check(const Tensor& t, const char* name)
{
    TORCH_CHECK_TYPE(t.defined() && t.scalar_type() == at::kFloat && t.is_cuda(), name, " must be a float32 CUDA tensor");
}

inline void check_like(const Tensor& t, const char* name, const Tensor& other)
{
    check(t, name);
    TORCH_CHECK_VALUE(t.device() == other.device(), name, " must be on ", other.device(), ", not ", t.device());
}

// A tensor as a matrix of rows of `width` with unit stride: a view where its
// strides allow one, otherwise a copy (and of a view that stands for its
// negative, as the imaginary part of a conjugate does).
struct Rows {
    Tensor keep;
    int64_t n, width, ld;
    const float* data() const { return keep.numel() ? keep.const_data_ptr<float>() : nullptr; }
    Rows(const Tensor& given, int64_t w) : keep(given.is_neg() ? given.resolve_neg() : given), width(w)
    {
        const Tensor t = keep;
        n = 1;
        ld = std::max<int64_t>(w, 1);
        // one distance between rows, over the dimensions of more than one
        // element from the last but one on: the innermost's, if the others'
        // strides are what the rows before them take
        bool one = w <= 1 || t.stride(t.dim() - 1) == 1;
        int64_t step = 0;
        for (int64_t d = t.dim() - 2; d >= 0; --d) {
            if (t.size(d) > 1) {
                if (n == 1)
                    step = t.stride(d);
                else
                    one = one && t.stride(d) == step * n;
            }
            n *= t.size(d);
        }
        if (n > 1 && one && step >= w)
            ld = std::max<int64_t>(step, 1);
        else if (!t.is_contiguous() && (n > 1 || !one))
            keep = t.contiguous();
    }
};

// An optional vector of length n.
inline Tensor vector_of(const optional<Tensor>& t, const char* name, int64_t n, const Tensor& like)
{
    if (!t.has_value() || !t->defined()) return {};
    check_like(*t, name, like);
    TORCH_CHECK_VALUE(t->dim() == 1 && t->size(0) == n, name, " must be a vector of length ", n);
    return t->resolve_neg().contiguous();
}

inline const float* ptr(const Tensor& t) { return t.defined() ? t.const_data_ptr<float>() : nullptr; }
inline float* out_ptr(const Tensor& t) { return t.defined() ? t.mutable_data_ptr<float>() : nullptr; }

inline Tensor empty_rows(int64_t rows, int64_t cols, const Tensor& like) { return at::empty({rows, cols}, like.options()); }

struct Workspace {
    Tensor t;
    void* p = nullptr;
    size_t bytes;
    Workspace(size_t n, const Tensor& like) : bytes(n)
    {
        if (n > 0) {
            t = at::empty({(int64_t)n}, like.options().dtype(at::kByte));
            p = t.mutable_data_ptr();
        }
    }
};

inline bool wants_grad(std::initializer_list<const Tensor*> ts)
{
    if (!at::GradMode::is_enabled()) return false;
    for (const Tensor* t : ts)
        if (t->defined() && t->requires_grad()) return true;
    return false;
}

// Refuses a differentiable call captured in a graph whose inputs come from
// outside of the capture.  A gradient node keeps the stream of the call that
// made it (a leaf's, of the first call that used the leaf, as long as any
// result of it lives); a captured backward pass that reaches the node would
// make that stream wait for the captured one, and ending such a capture ends
// the process.  Every node that the inputs lead to has to be on a stream of
// this capture.
inline void claim_leaves(const OnDevice& on, std::initializer_list<const Tensor*> ts)
{
    const auto capture_of = [](hipStream_t s) -> unsigned long long {
        hipStreamCaptureStatus status = hipStreamCaptureStatusNone;
        unsigned long long id = 0;
        // (the default stream is never captured, and asking it may fail)
        if (s == nullptr) return 0;
        if (hipStreamGetCaptureInfo(s, &status, &id) != hipSuccess) {
            (void)hipGetLastError();   // (must not surface in a later launch check)
            return 0;
        }
        return status == hipStreamCaptureStatusActive ? id : 0;
    };
    const unsigned long long capture = capture_of(on.stream);
    if (capture == 0) return;
    std::unordered_set<torch::autograd::Node*> seen;
    std::vector<std::shared_ptr<torch::autograd::Node>> todo;
    const auto visit = [&](std::shared_ptr<torch::autograd::Node> node) {
        if (node && seen.insert(node.get()).second) todo.push_back(std::move(node));
    };
    for (const Tensor* t : ts)
        if (t->defined() && t->requires_grad())
            visit(t->is_leaf() ? torch::autograd::impl::try_get_grad_accumulator(*t) : t->grad_fn());
    while (!todo.empty()) {
        const auto node = std::move(todo.back());
        todo.pop_back();
        const auto stream = node->stream();
        if (stream.has_value()) {
            const hipStream_t s = c10::hip::HIPStreamMasqueradingAsCUDA(*stream).stream();
            TORCH_CHECK(s == on.stream || capture_of(s) == capture,
                        "capturing a differentiable call whose parameters or inputs still belong to the results of an "
                        "earlier call on another stream: release those results (or detach the inputs) first, or make "
                        "the earlier call on the capturing stream");
        }
        for (const auto& edge : node->next_edges()) visit(edge.function);
    }
}

// out, connected to a tensor it was made from by a derivative that raises: a
// gradient taken through it never goes missing silently.
struct Refuse : Function<Refuse> {
    static Tensor forward(AutogradContext* ctx, const Tensor& out, const Tensor&)
    {
        ctx->mark_dirty({out});   // (out itself, not a view of it, which could not be changed in place)
        return out;
    }
    static variable_list backward(AutogradContext*, variable_list)
    {
        TORCH_CHECK(false, "the block operators are differentiable twice: a third derivative is not implemented");
    }
};

// The outputs of a derivative that has none of its own.
inline void last_derivative(variable_list& outs, const variable_list& grads, const variable_list& saved)
{
    if (!at::GradMode::is_enabled()) return;
    for (const variable_list* l : {&grads, &saved})
        for (const Tensor& t : *l)
            if (t.defined() && t.requires_grad())
                for (Tensor& o : outs)
                    if (o.defined()) o = Refuse::apply(o, t);
}

}  // namespace emu_torch

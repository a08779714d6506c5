// The attention operators (include/emu_attention.h) as differentiable
// functions of torch tensors, as block_torch.cpp has the block operators:
// argument checks, outputs and workspaces from torch's allocator, and the
// derivatives up to the second (rotary positions and dropout, being linear,
// have them all).  Host code only; the Python face is
// emulated_fp32_matrix_amd/attention.py.
#include <cmath>

#include "emu_attention.h"
#include "emu_torch.h"

namespace {

using namespace emu_torch;

// A tensor of [batch][token][head][dim] with unit stride along dim, otherwise
// a copy (and of a view that stands for its negative).
Tensor heads_tensor(const Tensor& given)
{
    Tensor t = given.is_neg() ? given.resolve_neg() : given;
    return t.size(3) > 1 && t.stride(3) != 1 ? t.contiguous() : t;
}

emu_heads_t heads_of(const Tensor& t)
{
    if (!t.defined()) return {};
    return {t.numel() ? t.const_data_ptr<float>() : nullptr, t.stride(0), t.stride(1), t.stride(2)};
}

Tensor dense_like(const Tensor& t) { return at::empty(t.sizes(), t.options()); }

// ---- attention --------------------------------------------------------------------

// The tensors of a call that its derivatives keep.
struct Call {
    Tensor q, k, v, bias, mask, lengths;
    double scale;

    emu_attention_t sizes() const
    {
        emu_attention_t a{};
        a.batch = q.size(0);
        a.queries = q.size(1);
        a.keys = k.size(1);
        a.heads = (int32_t)q.size(2);
        a.kv_heads = (int32_t)k.size(2);
        a.dim = (int32_t)q.size(3);
        a.scale = (float)scale;
        if (bias.defined() && bias.numel()) {
            a.key_bias = bias.const_data_ptr<float>();
            a.key_bias_batch = bias.stride(0);
            a.key_bias_key = bias.stride(1);
        }
        if (mask.defined() && mask.numel()) {
            a.key_mask = reinterpret_cast<const uint8_t*>(mask.const_data_ptr<bool>());
            a.key_mask_batch = mask.stride(0);
            a.key_mask_key = mask.stride(1);
        }
        if (lengths.defined() && lengths.numel()) {
            a.lengths = lengths.const_data_ptr();
            a.lengths_64 = lengths.scalar_type() == at::kLong;
        }
        return a;
    }
    variable_list list() const { return {q, k, v, bias, mask, lengths}; }
    static Call from(const variable_list& l, double scale) { return {l[0], l[1], l[2], l[3], l[4], l[5], scale}; }
    // with arrays as the kernels read them
    Call ready() const
    {
        return {heads_tensor(q), heads_tensor(k), heads_tensor(v), bias.defined() && bias.is_neg() ? bias.resolve_neg() : bias,
                mask, lengths, scale};
    }
};

Tensor attention_forward(const Call& given, Tensor* stats)
{
    const Call c = given.ready();
    const emu_attention_t a = c.sizes();
    Tensor out = dense_like(c.q);
    if (stats) *stats = at::empty({a.batch, a.queries, a.heads, 2}, c.q.options());
    OnDevice on(c.q);
    size_t bytes = 0;
    done(emu_cross_attention_workspace(&a, &bytes), "emu_cross_attention_workspace");
    Workspace ws(bytes, c.q);
    done(emu_cross_attention(&a, heads_of(c.q), heads_of(c.k), heads_of(c.v), out_ptr(out),
                             stats ? out_ptr(*stats) : nullptr, ws.p, ws.bytes, on.stream), "emu_cross_attention");
    return out;
}

// (dq, dk, dv, dbias), those that `want` names (bits 0 to 3), else undefined.
variable_list attention_backward(const Call& given, const Tensor& gy, const Tensor& out, const Tensor& stats, int64_t want)
{
    const Call c = given.ready();
    const emu_attention_t a = c.sizes();
    const Tensor g = heads_tensor(gy);
    variable_list r(4);
    if (want & 1) r[0] = dense_like(c.q);
    if (want & 2) r[1] = dense_like(c.k);
    if (want & 4) r[2] = dense_like(c.v);
    if (want & 8) r[3] = dense_like(c.bias);
    OnDevice on(c.q);
    size_t bytes = 0;
    done(emu_cross_attention_backward_workspace(&a, &bytes), "emu_cross_attention_backward_workspace");
    Workspace ws(bytes, c.q);
    done(emu_cross_attention_backward(&a, heads_of(g), heads_of(c.q), heads_of(c.k), heads_of(c.v), ptr(out), ptr(stats),
                                      out_ptr(r[0]), out_ptr(r[1]), out_ptr(r[2]), out_ptr(r[3]), ws.p, ws.bytes,
                                      on.stream), "emu_cross_attention_backward");
    return r;
}

optional<Tensor> some(const Tensor& t) { return t.defined() ? optional<Tensor>(t) : std::nullopt; }

// The backward pass as a function of its own: gradients of gy, q, k, v and
// bias go through all of it (out and stats are what the inputs make them).
struct AttentionBackward : Function<AttentionBackward> {
    static variable_list forward(AutogradContext* ctx, const Tensor& gy, const Tensor& q, const Tensor& k,
                                 const Tensor& v, const optional<Tensor>& bias, const optional<Tensor>& mask,
                                 const optional<Tensor>& lengths, const Tensor& out, const Tensor& stats, double scale,
                                 int64_t want)
    {
        ctx->set_materialize_grads(false);
        ctx->saved_data["scale"] = scale;
        ctx->saved_data["want"] = want;
        const Call c{q, k, v, bias.value_or(Tensor()), mask.value_or(Tensor()), lengths.value_or(Tensor()), scale};
        variable_list keep = c.list();
        keep.insert(keep.end(), {gy, out, stats});
        ctx->save_for_backward(keep);
        variable_list r;
        for (const Tensor& t : attention_backward(c, gy, out, stats, want))
            if (t.defined()) r.push_back(t);
        return r;
    }

    static variable_list backward(AutogradContext* ctx, variable_list grads)
    {
        const auto saved = ctx->get_saved_variables();
        const int64_t want = ctx->saved_data["want"].toInt();
        const Call c = Call::from(saved, ctx->saved_data["scale"].toDouble()).ready();
        size_t at_grad = 0;
        const auto next = [&](int64_t bit) { return want & bit ? grads[at_grad++] : Tensor(); };
        const auto heads = [](const Tensor& t) { return t.defined() ? heads_tensor(t) : t; };
        const Tensor vq_in = next(1), vk_in = next(2), vv_in = next(4), vb_in = next(8);
        check_readable({&vq_in, &vk_in, &vv_in, &vb_in});
        variable_list out(11);
        if (!vq_in.defined() && !vk_in.defined() && !vv_in.defined() && !vb_in.defined()) return out;
        const Tensor vq = heads(vq_in), vk = heads(vk_in), vv = heads(vv_in);
        const Tensor vb = vb_in.defined() && vb_in.is_neg() ? vb_in.resolve_neg() : vb_in;
        const Tensor gy = heads_tensor(saved[6]);
        if (ctx->needs_input_grad(0)) out[0] = dense_like(c.q);
        if (ctx->needs_input_grad(1)) out[1] = dense_like(c.q);
        if (ctx->needs_input_grad(2)) out[2] = dense_like(c.k);
        if (ctx->needs_input_grad(3)) out[3] = dense_like(c.v);
        if (c.bias.defined() && ctx->needs_input_grad(4)) out[4] = dense_like(c.bias);
        {
            const emu_attention_t a = c.sizes();
            OnDevice on(c.q);
            size_t bytes = 0;
            done(emu_cross_attention_backward2_workspace(&a, &bytes), "emu_cross_attention_backward2_workspace");
            Workspace ws(bytes, c.q);
            done(emu_cross_attention_backward2(&a, heads_of(vq), heads_of(vk), heads_of(vv), ptr(vb),
                                               vb.defined() ? vb.stride(0) : 0, vb.defined() ? vb.stride(1) : 0,
                                               heads_of(gy), heads_of(c.q), heads_of(c.k), heads_of(c.v), ptr(saved[7]),
                                               ptr(saved[8]), out_ptr(out[0]), out_ptr(out[1]), out_ptr(out[2]),
                                               out_ptr(out[3]), out_ptr(out[4]), ws.p, ws.bytes, on.stream),
                 "emu_cross_attention_backward2");
        }
        last_derivative(out, grads, {saved[0], saved[1], saved[2], saved[3], saved[6]});
        return out;
    }
};

struct Attention : Function<Attention> {
    static Tensor forward(AutogradContext* ctx, const Tensor& q, const Tensor& k, const Tensor& v,
                          const optional<Tensor>& bias, const optional<Tensor>& mask, const optional<Tensor>& lengths,
                          double scale)
    {
        const Call c{q, k, v, bias.value_or(Tensor()), mask.value_or(Tensor()), lengths.value_or(Tensor()), scale};
        Tensor stats;
        Tensor out = attention_forward(c, &stats);
        variable_list keep = c.list();
        keep.insert(keep.end(), {out, stats});
        ctx->save_for_backward(keep);
        ctx->saved_data["scale"] = scale;
        return out;
    }

    static variable_list backward(AutogradContext* ctx, variable_list grads)
    {
        const auto saved = ctx->get_saved_variables();
        const Call c = Call::from(saved, ctx->saved_data["scale"].toDouble());
        const Tensor &gy = grads[0], &stats = saved[7];
        variable_list out(7);
        check_readable({&gy});
        int64_t want = 0;
        for (int i = 0; i < (c.bias.defined() ? 4 : 3); ++i)
            if (ctx->needs_input_grad(i)) want |= (int64_t)1 << i;
        if (!gy.defined() || want == 0) return out;
        if (at::GradMode::is_enabled()) {
            const variable_list g = AttentionBackward::apply(gy, c.q, c.k, c.v, some(c.bias), some(c.mask), some(c.lengths),
                                                             saved[6].detach(), stats, c.scale, want);
            size_t n = 0;
            for (int i = 0; i < 4; ++i)
                if (want >> i & 1) out[i] = g[n++];
            return out;
        }
        const variable_list g = attention_backward(c, gy, saved[6], stats, want);
        for (int i = 0; i < 4; ++i) out[i] = g[i];
        return out;
    }
};

Tensor cross_attention(const Tensor& q, const Tensor& k, const Tensor& v, const optional<Tensor>& bias_in,
                       const optional<Tensor>& mask_in, const optional<Tensor>& lengths_in, optional<double> scale_in)
{
    check_readable({&q, &k, &v, given(bias_in), given(mask_in), given(lengths_in)});
    check(q, "q");
    check_like(k, "k", q);
    check_like(v, "v", q);
    TORCH_CHECK_VALUE(q.dim() == 4 && k.dim() == 4 && v.dim() == 4, "q, k and v must be [batch, tokens, heads, dim]");
    const int64_t batch = q.size(0), keys = k.size(1), heads = q.size(2), kv_heads = k.size(2), dim = q.size(3);
    TORCH_CHECK_VALUE(k.sizes() == v.sizes(), "k and v must have one shape, not ", k.sizes(), " and ", v.sizes());
    TORCH_CHECK_VALUE(k.size(0) == batch && k.size(3) == dim, "k must have the batch and head width of q: ", k.sizes(),
                      " and ", q.sizes());
    TORCH_CHECK_VALUE(dim >= 1 && dim <= EMU_ATTENTION_MAX_DIM, "heads must be 1 to ", EMU_ATTENTION_MAX_DIM, " wide, not ", dim);
    TORCH_CHECK_VALUE(heads == 0 ? kv_heads == 0 : kv_heads >= 1 && heads % kv_heads == 0,
                      "the heads of q must be a multiple of those of k: ", heads, " and ", kv_heads);
    Call c{q, k, v, {}, {}, {}, 0.0};
    if (bias_in.has_value() && bias_in->defined()) {
        check_like(*bias_in, "key_bias", q);
        TORCH_CHECK_VALUE(bias_in->dim() == 2 && bias_in->size(0) == batch && bias_in->size(1) == keys,
                          "key_bias must be [batch, keys], not ", bias_in->sizes());
        c.bias = *bias_in;
    }
    if (mask_in.has_value() && mask_in->defined()) {
        TORCH_CHECK_TYPE(mask_in->scalar_type() == at::kBool && mask_in->is_cuda(), "key_mask must be a bool CUDA tensor");
        TORCH_CHECK_VALUE(mask_in->device() == q.device(), "key_mask must be on ", q.device(), ", not ", mask_in->device());
        TORCH_CHECK_VALUE(mask_in->dim() == 2 && mask_in->size(0) == batch && mask_in->size(1) == keys,
                          "key_mask must be [batch, keys], not ", mask_in->sizes());
        c.mask = *mask_in;
    }
    if (lengths_in.has_value() && lengths_in->defined()) {
        TORCH_CHECK_TYPE((lengths_in->scalar_type() == at::kInt || lengths_in->scalar_type() == at::kLong) && lengths_in->is_cuda(),
                         "lengths must be an int32 or int64 CUDA tensor");
        TORCH_CHECK_VALUE(lengths_in->device() == q.device(), "lengths must be on ", q.device(), ", not ", lengths_in->device());
        TORCH_CHECK_VALUE(lengths_in->dim() == 1 && lengths_in->size(0) == batch, "lengths must be [batch], not ", lengths_in->sizes());
        c.lengths = lengths_in->contiguous();
    }
    c.scale = scale_in.value_or(1.0 / std::sqrt((double)dim));
    TORCH_CHECK_VALUE(std::isfinite((float)c.scale), "scale must be finite");
    if (wants_grad({&q, &k, &v, &c.bias})) {
        claim_leaves(OnDevice(q), {&q, &k, &v, &c.bias});
        return Attention::apply(q, k, v, some(c.bias), some(c.mask), some(c.lengths), c.scale);
    }
    return attention_forward(c, nullptr);
}

// ---- rotary positions ---------------------------------------------------------------

Tensor rotary_forward(const Tensor& x, const Tensor& positions, const Tensor& turns, int64_t layout, double magnitude,
                      bool inverse)
{
    Tensor y = dense_like(x);
    const int64_t t = x.size(-3), h = x.size(-2), d = x.size(-1);
    int64_t b = 1;
    for (int64_t i = 0; i + 3 < x.dim(); ++i) b *= x.size(i);
    if (y.numel() == 0) return y;
    const Tensor x4 = heads_tensor(x.is_neg() ? x.resolve_neg().reshape({b, t, h, d}) : x.reshape({b, t, h, d}));
    OnDevice on(x);
    done(emu_rotary(b, t, h, d, heads_of(x4), positions.const_data_ptr<int64_t>(), positions.stride(0), positions.stride(1),
                    reinterpret_cast<const uint64_t*>(turns.const_data_ptr<int64_t>()), turns.size(0),
                    (emu_rotary_layout_t)layout, (float)magnitude, inverse, out_ptr(y), on.stream), "emu_rotary");
    return y;
}

struct Rotary : Function<Rotary> {
    static Tensor forward(AutogradContext* ctx, const Tensor& x, const Tensor& positions, const Tensor& turns,
                          int64_t layout, double magnitude, bool inverse)
    {
        ctx->save_for_backward({positions, turns});
        ctx->saved_data["layout"] = layout;
        ctx->saved_data["magnitude"] = magnitude;
        ctx->saved_data["inverse"] = inverse;
        return rotary_forward(x, positions, turns, layout, magnitude, inverse);
    }
    static variable_list backward(AutogradContext* ctx, variable_list grads)
    {
        const auto saved = ctx->get_saved_variables();
        const Tensor& g = grads[0];
        variable_list out(6);
        check_readable({&g});
        if (!g.defined() || !ctx->needs_input_grad(0)) return out;
        const int64_t layout = ctx->saved_data["layout"].toInt();
        const double magnitude = ctx->saved_data["magnitude"].toDouble();
        const bool inverse = !ctx->saved_data["inverse"].toBool();
        out[0] = wants_grad({&g}) ? Rotary::apply(g, saved[0], saved[1], layout, magnitude, inverse)
                                  : rotary_forward(g, saved[0], saved[1], layout, magnitude, inverse);
        return out;
    }
};

Tensor rotary(const Tensor& x, const Tensor& positions_in, const Tensor& turns_in, int64_t layout, double magnitude)
{
    check_readable({&x, &positions_in, &turns_in});
    check(x, "x");
    TORCH_CHECK_VALUE(x.dim() >= 3, "x must be [..., tokens, heads, dim], not ", x.sizes());
    TORCH_CHECK_TYPE((positions_in.scalar_type() == at::kLong || positions_in.scalar_type() == at::kInt) && positions_in.is_cuda(),
                     "positions must be an int32 or int64 CUDA tensor");
    TORCH_CHECK_TYPE(turns_in.scalar_type() == at::kLong && turns_in.is_cuda(), "turns must be an int64 CUDA tensor");
    TORCH_CHECK_VALUE(positions_in.device() == x.device() && turns_in.device() == x.device(),
                      "positions and turns must be on ", x.device());
    TORCH_CHECK_VALUE(turns_in.dim() == 1 && 2 * turns_in.size(0) <= x.size(-1), "x has heads of ", x.size(-1),
                      ", too narrow for ", 2 * turns_in.size(0), " rotated elements");
    TORCH_CHECK_VALUE(std::isfinite((float)magnitude), "magnitude must be finite");
    const auto lead = x.sizes().slice(0, x.dim() - 2);
    const bool whole = positions_in.sizes() == lead;
    TORCH_CHECK_VALUE(whole || (positions_in.dim() == 1 && positions_in.size(0) == x.size(-3)),
                      "positions must be [tokens] or have x's shape up to its tokens, not ", positions_in.sizes());
    int64_t b = 1;
    for (int64_t i = 0; i + 3 < x.dim(); ++i) b *= x.size(i);
    const Tensor p = positions_in.to(at::kLong);
    const Tensor positions = whole ? p.reshape({b, x.size(-3)}) : p.unsqueeze(0).expand({b, x.size(-3)});
    const Tensor turns = turns_in.contiguous();
    if (wants_grad({&x})) {
        claim_leaves(OnDevice(x), {&x});
        return Rotary::apply(x, positions, turns, layout, magnitude, false);
    }
    return rotary_forward(x, positions, turns, layout, magnitude, false);
}

// ---- dropout -------------------------------------------------------------------------

Tensor dropout_forward(const Tensor& x, const Tensor* residual, const Tensor& seed, double p)
{
    Tensor y = dense_like(x);
    if (y.numel() == 0) return y;
    const int64_t cols = x.dim() ? x.size(-1) : 1;
    const Tensor flat = x.dim() ? x : x.unsqueeze(0);
    const Rows r(flat, cols);
    OnDevice on(x);
    if (residual != nullptr) {
        const Rows s(residual->dim() ? *residual : residual->unsqueeze(0), cols);
        done(emu_dropout(r.n, cols, r.data(), r.ld, p, seed.const_data_ptr<int64_t>(), s.data(), s.ld, out_ptr(y), cols,
                         on.stream), "emu_dropout");
        return y;
    }
    done(emu_dropout(r.n, cols, r.data(), r.ld, p, seed.const_data_ptr<int64_t>(), nullptr, 0, out_ptr(y), cols, on.stream),
         "emu_dropout");
    return y;
}

struct Dropout : Function<Dropout> {
    static Tensor forward(AutogradContext* ctx, const Tensor& x, const optional<Tensor>& residual, const Tensor& seed, double p)
    {
        ctx->save_for_backward({seed});
        ctx->saved_data["p"] = p;
        ctx->saved_data["residual"] = residual.has_value();
        return dropout_forward(x, residual.has_value() ? &*residual : nullptr, seed, p);
    }
    static variable_list backward(AutogradContext* ctx, variable_list grads)
    {
        const auto saved = ctx->get_saved_variables();
        const Tensor& g = grads[0];
        const double p = ctx->saved_data["p"].toDouble();
        variable_list out(4);
        check_readable({&g});
        if (!g.defined()) return out;
        if (ctx->needs_input_grad(0))
            out[0] = wants_grad({&g}) ? Dropout::apply(g, std::nullopt, saved[0], p) : dropout_forward(g, nullptr, saved[0], p);
        if (ctx->saved_data["residual"].toBool() && ctx->needs_input_grad(1)) out[1] = g;
        return out;
    }
};

Tensor dropout(const Tensor& x, double p, const Tensor& seed_in, const optional<Tensor>& residual_in)
{
    check_readable({&x, &seed_in, given(residual_in)});
    check(x, "x");
    TORCH_CHECK_VALUE(p >= 0.0 && p <= 1.0, "p must be between 0 and 1, not ", p);
    TORCH_CHECK_TYPE(seed_in.scalar_type() == at::kLong && seed_in.is_cuda(), "seed must be an int64 CUDA tensor");
    TORCH_CHECK_VALUE(seed_in.device() == x.device(), "seed must be on ", x.device(), ", not ", seed_in.device());
    TORCH_CHECK_VALUE(seed_in.dim() == 1 && seed_in.size(0) == 2, "seed must hold two numbers, not ", seed_in.sizes());
    const Tensor residual = residual_in.value_or(Tensor());
    if (residual.defined()) {
        check_like(residual, "residual", x);
        TORCH_CHECK_VALUE(residual.sizes() == x.sizes(), "residual must have the shape of x, not ", residual.sizes());
    }
    const Tensor seed = seed_in.contiguous();
    if (wants_grad({&x, &residual})) {
        claim_leaves(OnDevice(x), {&x, &residual});
        return Dropout::apply(x, some(residual), seed, p);
    }
    return dropout_forward(x, residual.defined() ? &residual : nullptr, seed, p);
}

}  // namespace

void register_attention(py::module_& m)
{
    using gil = py::call_guard<py::gil_scoped_release>;
    m.def("cross_attention", &cross_attention, gil());
    m.def("rotary", &rotary, gil());
    m.def("dropout", &dropout, gil());
}

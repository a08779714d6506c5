// The transformer-block operators (include/emu_block.h) as differentiable
// functions of torch tensors: argument checks, outputs and workspaces from
// torch's allocator, and the derivatives up to the second.  Host code only;
// the Python face is emulated_fp32_matrix_amd/block.py.
//
// Native rather than Python functions because a small call is host-bound: a
// layer norm of one atom's 32 tokens takes the device 3 us, its Python
// binding took 13, and a training step's functions ran through the
// interpreter on autograd's thread (163 us for a layer norm's, forward and
// backward).
//
// Every function is differentiable twice, as training on forces needs
// ("Unlocking Tensor Core Performance for Machine Learning Interatomic
// Potentials", section "TF32x3 on Ampere GPUs"); a third derivative raises.
// In a backward pass that nothing differentiates (no create_graph) the
// kernels are called directly, and the activation's backward pass may run
// inside the weight gradient.  Forward-mode derivatives and tracing are
// refused.
#include "emu_block.h"
#include "emu_torch.h"

namespace {

using namespace emu_torch;

// ---- kernels ---------------------------------------------------------------------

int op_of(bool trans) { return trans ? EMU_OP_T : EMU_OP_N; }

// An array of the rows of `like`, `cols` wide, in the shape of `like`.  (Made in
// its shape: autograd lets no view that a Function returns be changed in place.)
Tensor empty_shaped(const Tensor& like, int64_t cols)
{
    if (like.dim() == 2) return empty_rows(like.size(0), cols, like);
    auto shape = like.sizes().vec();
    shape.back() = cols;
    return at::empty(shape, like.options());
}

// act(a @ op(w) + bias) + residual, in the shape of `like`; z receives the
// pre-activation when defined.  planes: op(w) split beforehand, or null.
Tensor product(const Rows& a, const Rows& w, bool trans, const Tensor& bias, int act, const Rows* residual,
               const Tensor& z, int mode, const void* planes, const Tensor& like)
{
    const int64_t M = a.n, K = a.width, N = trans ? w.n : w.width;
    Tensor c = empty_shaped(like, N);
    const int64_t ldn = std::max<int64_t>(N, 1);
    OnDevice on(a.keep);
    size_t bytes = 0;
    done(emu_sgemm_act_workspace((emu_op_t)op_of(trans), M, N, K, a.data(), a.ld, planes != nullptr, (emu_mode_t)mode,
                                 &bytes), "emu_sgemm_act_workspace");
    Workspace ws(bytes, a.keep);
    done(emu_sgemm_act((emu_op_t)op_of(trans), M, N, K, a.data(), a.ld, w.data(), w.ld, planes, ptr(bias),
                       (emu_act_t)act, out_ptr(z), ldn, residual ? residual->data() : nullptr,
                       residual ? residual->ld : ldn, out_ptr(c), ldn, (emu_mode_t)mode, ws.p, ws.bytes, on.stream),
         "emu_sgemm_act");
    return c;
}

Tensor gated(const Rows& a, const Rows& w, const Tensor& bias, int act, const Tensor& z, int mode, const void* planes,
             const Tensor& like)
{
    const int64_t M = a.n, K = a.width, F = w.n / 2;
    Tensor c = empty_shaped(like, F);
    OnDevice on(a.keep);
    size_t bytes = 0;
    done(emu_sgemm_gated_workspace(M, F, K, a.data(), a.ld, planes != nullptr, (emu_mode_t)mode, &bytes),
         "emu_sgemm_gated_workspace");
    Workspace ws(bytes, a.keep);
    done(emu_sgemm_gated(M, F, K, a.data(), a.ld, w.data(), w.ld, planes, ptr(bias), (emu_act_t)act, out_ptr(z),
                         std::max<int64_t>(2 * F, 1), out_ptr(c), std::max<int64_t>(F, 1), (emu_mode_t)mode, ws.p,
                         ws.bytes, on.stream), "emu_sgemm_gated");
    return c;
}

struct WeightGrads {
    Tensor dw, db, dz;
};

// In the place of a weight gradient's x where only db is wanted: its rows, no
// columns.
Tensor no_columns(const Rows& x) { return at::empty({x.n, 0}, x.keep.options()); }

// Rows as the weight gradient takes them: at most 16,777,088 elements apart
// (include/emu_block.h), as a slice of a large tensor may not have them.
Rows near_rows(const Rows& r)
{
    return r.n > 1 && r.ld > 16777088 && r.ld > r.width ? Rows(r.keep.contiguous(), r.width) : r;
}

WeightGrads weight_grad(const Rows& far_dz, const Rows& far_x, bool want_db)
{
    const Rows dz = near_rows(far_dz), x = near_rows(far_x);
    const int64_t rows = dz.n, M = dz.width, N = x.width;
    WeightGrads g;
    g.dw = empty_rows(M, N, dz.keep);
    if (want_db) g.db = at::empty({M}, dz.keep.options());
    OnDevice on(dz.keep);
    size_t bytes = 0;
    done(emu_wgrad_workspace(rows, M, N, &bytes), "emu_wgrad_workspace");
    Workspace ws(bytes, dz.keep);
    done(emu_wgrad(rows, M, N, dz.data(), dz.ld, x.data(), x.ld, out_ptr(g.dw), std::max<int64_t>(N, 1), out_ptr(g.db),
                   ws.p, ws.bytes, on.stream), "emu_wgrad");
    return g;
}

// The same with the activation's (or the gated product's) backward pass
// inside, which also gives dz.
WeightGrads weight_grad_from(const Rows& far_dy, const Rows& z, int act, const Rows& far_x, bool want_db, bool is_gated)
{
    const Rows dy = near_rows(far_dy), x = near_rows(far_x);
    const int64_t rows = dy.n, M = dy.width, N = x.width, wide = z.width;
    WeightGrads g;
    g.dz = empty_rows(rows, wide, dy.keep);
    g.dw = empty_rows(wide, N, dy.keep);
    if (want_db) g.db = at::empty({wide}, dy.keep.options());
    OnDevice on(dy.keep);
    size_t bytes = 0;
    done(is_gated ? emu_wgrad_gated_workspace(rows, M, N, &bytes) : emu_wgrad_workspace(rows, M, N, &bytes),
         "emu_wgrad_workspace");
    Workspace ws(bytes, dy.keep);
    const int64_t ldw = std::max<int64_t>(wide, 1), ldn = std::max<int64_t>(N, 1);
    if (is_gated)
        done(emu_wgrad_gated(rows, M, N, dy.data(), dy.ld, z.data(), z.ld, (emu_act_t)act, out_ptr(g.dz), ldw, x.data(),
                             x.ld, out_ptr(g.dw), ldn, out_ptr(g.db), ws.p, ws.bytes, on.stream), "emu_wgrad_gated");
    else
        done(emu_wgrad_act(rows, M, N, dy.data(), dy.ld, z.data(), z.ld, (emu_act_t)act, out_ptr(g.dz), ldw, x.data(),
                           x.ld, out_ptr(g.dw), ldn, out_ptr(g.db), ws.p, ws.bytes, on.stream), "emu_wgrad_act");
    return g;
}

// Whether the activation's backward pass runs inside the weight gradient:
// every 256 columns of x repeat it, which pays where there is one such tile
// (552,960 x 256 -> 2 x 512, silu: 3,230 us apart, 2,530 inside; 6,144 x 1024
// -> 4096, gelu, training step: 1,277 apart, 1,719 inside).
bool fuse_act(int64_t in_features) { return in_features <= 256; }

Tensor act_backward(const Rows& dy, const Rows& z, int act, bool is_gated)
{
    Tensor out = empty_rows(z.n, z.width, z.keep);
    OnDevice on(z.keep);
    const int64_t ld = std::max<int64_t>(z.width, 1);
    if (is_gated)
        done(emu_gated_backward(z.n, dy.width, dy.data(), dy.ld, z.data(), z.ld, (emu_act_t)act, out_ptr(out), ld,
                                on.stream), "emu_gated_backward");
    else
        done(emu_act_backward(z.n, z.width, dy.data(), dy.ld, z.data(), z.ld, (emu_act_t)act, out_ptr(out), ld,
                              on.stream), "emu_act_backward");
    return out;
}

Tensor norm_forward(const Rows& x, const Tensor& weight, const Tensor& bias, double eps, Tensor* stats, const Tensor& like)
{
    Tensor y = empty_shaped(like, x.width);
    if (stats) *stats = at::empty({2, x.n}, x.keep.options());
    OnDevice on(x.keep);
    float* s = stats ? out_ptr(*stats) : nullptr;
    done(emu_layer_norm(x.n, x.width, x.data(), x.ld, ptr(weight), ptr(bias), (float)eps, out_ptr(y), x.width, s,
                        s ? s + x.n : nullptr, on.stream), "emu_layer_norm");
    return y;
}

struct NormGrads {
    Tensor dx, dw, db;
};

NormGrads norm_backward(const Rows& dy, const Rows& x, const Tensor& weight, const Tensor& stats, bool want_x,
                        bool want_w, bool want_b, const Tensor& like)
{
    NormGrads g;
    const auto opt = x.keep.options();
    if (want_x) g.dx = empty_shaped(like, x.width);
    if (want_w) g.dw = at::empty({x.width}, opt);
    if (want_b) g.db = at::empty({x.width}, opt);
    OnDevice on(x.keep);
    size_t bytes = 0;
    if (want_w || want_b)
        done(emu_layer_norm_backward_workspace(x.n, x.width, &bytes), "emu_layer_norm_backward_workspace");
    Workspace ws(bytes, x.keep);
    const float* s = ptr(stats);
    done(emu_layer_norm_backward(x.n, x.width, dy.data(), dy.ld, x.data(), x.ld, ptr(weight), s, s ? s + x.n : s,
                                 out_ptr(g.dx), x.width, out_ptr(g.dw), out_ptr(g.db), ws.p, ws.bytes, on.stream),
         "emu_layer_norm_backward");
    return g;
}

// ---- differentiable pieces ------------------------------------------------------------

struct WeightGrad;

// a @ op(w), op(w) = w^T (trans) or w, differentiable.
struct Product : Function<Product> {
    static Tensor forward(AutogradContext* ctx, const Tensor& a, const Tensor& w, bool trans, int64_t mode)
    {
        ctx->save_for_backward({a, w});
        ctx->saved_data["trans"] = trans;
        ctx->saved_data["mode"] = mode;
        return product(Rows(a, a.size(1)), Rows(w, w.size(1)), trans, {}, 0, nullptr, {}, (int)mode, nullptr, a);
    }
    static variable_list backward(AutogradContext* ctx, variable_list grads);
};

// Skips autograd where nothing is recorded.
Tensor product_of(const Tensor& a, const Tensor& w, bool trans, int64_t mode)
{
    if (wants_grad({&a, &w})) return Product::apply(a, w, trans, mode);
    return product(Rows(a, a.size(1)), Rows(w, w.size(1)), trans, {}, 0, nullptr, {}, (int)mode, nullptr, a);
}

// (dz^T x, column sums of dz): with P and q the gradients of the two, dz gets
// x P^T + q and x gets dz P.
struct WeightGrad : Function<WeightGrad> {
    static variable_list forward(AutogradContext* ctx, const Tensor& dz, const Tensor& x, bool want_db, int64_t mode)
    {
        ctx->save_for_backward({dz, x});
        ctx->saved_data["mode"] = mode;
        ctx->set_materialize_grads(false);
        WeightGrads g = weight_grad(Rows(dz, dz.size(1)), Rows(x, x.size(1)), want_db);
        return want_db ? variable_list{g.dw, g.db} : variable_list{g.dw};
    }
    static variable_list backward(AutogradContext* ctx, variable_list grads)
    {
        const auto saved = ctx->get_saved_variables();
        const Tensor &dz = saved[0], &x = saved[1], &P = grads[0];
        const Tensor q = grads.size() > 1 ? grads[1] : Tensor();
        check_readable({&P, &q});
        const int64_t mode = ctx->saved_data["mode"].toInt();
        Tensor gdz, gx;
        if (ctx->needs_input_grad(0)) {
            if (P.defined()) gdz = product_of(x, P, true, mode);
            if (q.defined()) gdz = gdz.defined() ? gdz + q : q.expand({dz.size(0), q.size(0)});
        }
        if (ctx->needs_input_grad(1) && P.defined()) gx = product_of(dz, P, false, mode);
        return {gdz, gx, Tensor(), Tensor()};
    }
};

variable_list Product::backward(AutogradContext* ctx, variable_list grads)
{
    const auto saved = ctx->get_saved_variables();
    const Tensor &a = saved[0], &w = saved[1], &g = grads[0];
    check_readable({&g});
    const bool trans = ctx->saved_data["trans"].toBool();
    const int64_t mode = ctx->saved_data["mode"].toInt();
    Tensor ga, gw;
    if (ctx->needs_input_grad(0)) ga = product_of(g, w, !trans, mode);
    if (ctx->needs_input_grad(1)) {
        const Tensor &l = trans ? g : a, &r = trans ? a : g;
        gw = wants_grad({&l, &r}) ? WeightGrad::apply(l, r, false, mode)[0]
                                  : weight_grad(Rows(l, l.size(1)), Rows(r, r.size(1)), false).dw;
    }
    return {ga, gw, Tensor(), Tensor()};
}

// dz from dy and the pre-activations z (gated: Z).
struct ActBackward : Function<ActBackward> {
    static Tensor forward(AutogradContext* ctx, const Tensor& dy, const Tensor& z, int64_t act, bool is_gated)
    {
        ctx->save_for_backward({dy, z});
        ctx->saved_data["act"] = act;
        ctx->saved_data["gated"] = is_gated;
        return act_backward(Rows(dy, dy.size(1)), Rows(z, z.size(1)), (int)act, is_gated);
    }
    static variable_list backward(AutogradContext* ctx, variable_list grads)
    {
        const auto saved = ctx->get_saved_variables();
        const emu_act_t act = (emu_act_t)ctx->saved_data["act"].toInt();
        const Tensor &dy_t = saved[0], &z_t = saved[1], &v_t = grads[0];
        check_readable({&v_t});
        const Rows dy(dy_t, dy_t.size(1)), z(z_t, z_t.size(1)), v(v_t, v_t.size(1));
        variable_list out(4);
        if (ctx->needs_input_grad(0)) out[0] = empty_rows(dy.n, dy.width, dy.keep);
        if (ctx->needs_input_grad(1)) out[1] = empty_rows(z.n, z.width, z.keep);
        {
            OnDevice on(z_t);
            const int64_t ldy = std::max<int64_t>(dy.width, 1), ldz = std::max<int64_t>(z.width, 1);
            if (ctx->saved_data["gated"].toBool())
                done(emu_gated_backward2(z.n, dy.width, v.data(), v.ld, dy.data(), dy.ld, z.data(), z.ld, act,
                                         out_ptr(out[0]), ldy, out_ptr(out[1]), ldz, on.stream), "emu_gated_backward2");
            else
                done(emu_act_backward2(z.n, z.width, v.data(), v.ld, dy.data(), dy.ld, z.data(), z.ld, act,
                                       out_ptr(out[0]), ldy, out_ptr(out[1]), ldz, on.stream), "emu_act_backward2");
        }
        last_derivative(out, grads, saved);
        return out;
    }
};

// ---- linear layer and gated projection ---------------------------------------------------

// y = act(x W^T + b) + residual, or h = act(g) u.  The pre-activation z is an
// output of its own, so that the backward pass, which reads it, can be
// differentiated.
struct Layer : Function<Layer> {
    static variable_list forward(AutogradContext* ctx, const Tensor& x, const Tensor& weight,
                                 const optional<Tensor>& bias, const optional<Tensor>& residual, int64_t act,
                                 int64_t mode, bool is_gated, int64_t planes)
    {
        ctx->set_materialize_grads(false);
        ctx->saved_data["act"] = act;
        ctx->saved_data["mode"] = mode;
        ctx->saved_data["gated"] = is_gated;
        ctx->saved_data["bias"] = bias.has_value();
        ctx->saved_data["residual"] = residual.has_value();
        const Rows x2(x, weight.size(1)), w2(weight, weight.size(1));
        const void* pl = reinterpret_cast<const void*>(planes);
        Tensor z, y;
        if (is_gated || act != EMU_ACT_IDENTITY) z = empty_rows(x2.n, w2.n, x);
        const Tensor b = bias.value_or(Tensor());
        if (is_gated) {
            y = gated(x2, w2, b, (int)act, z, (int)mode, pl, x);
        } else if (residual.has_value()) {
            const Rows r(*residual, w2.n);
            y = product(x2, w2, true, b, (int)act, &r, z, (int)mode, pl, x);
        } else {
            y = product(x2, w2, true, b, (int)act, nullptr, z, (int)mode, pl, x);
        }
        ctx->save_for_backward({x, weight, z});
        return z.defined() ? variable_list{y, z} : variable_list{y};
    }

    static variable_list backward(AutogradContext* ctx, variable_list grads)
    {
        const auto saved = ctx->get_saved_variables();
        const Tensor &x = saved[0], &weight = saved[1], &z = saved[2], &gy = grads[0];
        const Tensor gz = grads.size() > 1 ? grads[1] : Tensor();
        const int64_t act = ctx->saved_data["act"].toInt(), mode = ctx->saved_data["mode"].toInt();
        const bool is_gated = ctx->saved_data["gated"].toBool(), has_bias = ctx->saved_data["bias"].toBool();
        const bool has_res = ctx->saved_data["residual"].toBool();
        variable_list out(8);
        check_readable({&gy, &gz});
        if (!gy.defined() && !gz.defined()) return out;
        const bool want_x = ctx->needs_input_grad(0), want_w = ctx->needs_input_grad(1);
        const bool want_b = has_bias && ctx->needs_input_grad(2);
        if (has_res && ctx->needs_input_grad(has_bias ? 3 : 2)) out[3] = gy;
        if (!want_x && !want_w && !want_b) return out;
        const int64_t K = weight.size(1), N = is_gated ? weight.size(0) / 2 : weight.size(0);
        const Rows x2(x, K);
        Tensor dz;
        if (!at::GradMode::is_enabled()) {
            // nothing is differentiated again
            if (z.defined() && !gz.defined() && want_w && fuse_act(K)) {
                WeightGrads g = weight_grad_from(Rows(gy, N), Rows(z, z.size(1)), (int)act, x2, want_b, is_gated);
                dz = g.dz;
                out[1] = g.dw;
                out[2] = g.db;
            } else {
                if (gy.defined())
                    dz = z.defined() ? act_backward(Rows(gy, N), Rows(z, z.size(1)), (int)act, is_gated) : gy;
                if (gz.defined()) dz = dz.defined() ? dz + gz : gz;
                if (want_w || want_b) {
                    WeightGrads g = weight_grad(Rows(dz, weight.size(0)), want_w ? x2 : Rows(no_columns(x2), 0), want_b);
                    if (want_w) out[1] = g.dw;
                    out[2] = g.db;
                }
            }
            if (want_x)
                out[0] = product(Rows(dz, weight.size(0)), Rows(weight, K), false, {}, 0, nullptr, {}, (int)mode, nullptr, x);
            return out;
        }
        const auto flat = [](const Tensor& t, int64_t n, int64_t width) { return t.dim() == 2 ? t : t.reshape({n, width}); };
        if (gy.defined()) {
            const Tensor g2 = flat(gy, x2.n, N);
            dz = z.defined() ? ActBackward::apply(g2, z, act, is_gated) : g2;
        }
        if (gz.defined()) dz = dz.defined() ? dz + gz : gz;
        if (want_x) out[0] = Product::apply(dz, weight, false, mode).view(x.sizes());
        if (want_w || want_b) {
            variable_list g = WeightGrad::apply(dz, want_w ? flat(x, x2.n, K) : no_columns(x2), want_b, mode);
            if (want_w) out[1] = g[0];
            if (want_b) out[2] = g[1];
        }
        return out;
    }
};

Tensor layer_call(const Tensor& x, const Tensor& weight, const optional<Tensor>& bias_in,
                  const optional<Tensor>& residual_in, int64_t act, int64_t mode, bool is_gated,
                  const optional<Tensor>& planes)
{
    check_readable({&x, &weight, given(bias_in), given(residual_in)});
    check(x, "x");
    check_like(weight, "weight", x);
    TORCH_CHECK_VALUE(weight.dim() == 2, "weight must be 2-D");
    const int64_t wide = weight.size(0), K = weight.size(1);
    TORCH_CHECK_VALUE(x.dim() >= 1 && x.size(-1) == K, "x must end in ", K, " features, not ", x.sizes());
    TORCH_CHECK_VALUE(!is_gated || wide % 2 == 0, "weight must hold as many gate rows as up rows");
    const Tensor bias = vector_of(bias_in, "bias", wide, x);
    const Tensor residual = residual_in.value_or(Tensor());
    if (residual.defined()) {
        check_like(residual, "residual", x);
        bool same = residual.dim() == x.dim() && residual.size(-1) == wide;
        for (int64_t d = 0; same && d + 1 < x.dim(); ++d) same = residual.size(d) == x.size(d);
        TORCH_CHECK_VALUE(same, "residual must have the output's shape, not ", residual.sizes());
    }
    if (planes.has_value())
        TORCH_CHECK_VALUE(planes->device() == x.device(), "the planes must be on ", x.device());
    const void* pl = planes.has_value() ? planes->const_data_ptr() : nullptr;
    const auto some = [](const Tensor& t) { return t.defined() ? optional<Tensor>(t) : std::nullopt; };
    if (wants_grad({&x, &weight, &bias, &residual})) {
        claim_leaves(OnDevice(x), {&x, &weight, &bias, &residual});
        return Layer::apply(x, weight, some(bias), some(residual), act, mode, is_gated, (int64_t)(uintptr_t)pl)[0];
    }
    const Rows x2(x, K), w2(weight, K);
    if (is_gated) return gated(x2, w2, bias, (int)act, {}, (int)mode, pl, x);
    if (!residual.defined()) return product(x2, w2, true, bias, (int)act, nullptr, {}, (int)mode, pl, x);
    const Rows r(residual, wide);
    return product(x2, w2, true, bias, (int)act, &r, {}, (int)mode, pl, x);
}

Tensor linear_act(const Tensor& x, const Tensor& weight, const optional<Tensor>& bias,
                  const optional<Tensor>& residual, int64_t act, int64_t mode, const optional<Tensor>& planes)
{
    return layer_call(x, weight, bias, residual, act, mode, false, planes);
}

Tensor gated_linear(const Tensor& x, const Tensor& weight, const optional<Tensor>& bias, int64_t act, int64_t mode,
                    const optional<Tensor>& planes)
{
    return layer_call(x, weight, bias, std::nullopt, act, mode, true, planes);
}

// ---- layer norm ------------------------------------------------------------------------------

// (dx, dweight, dbias), those that `want` names (bits 0, 1, 2); its gradient
// with respect to x is the whole one, through the mean and deviation too.
struct LayerNormBackward : Function<LayerNormBackward> {
    static variable_list forward(AutogradContext* ctx, const Tensor& gy, const Tensor& x,
                                 const optional<Tensor>& weight, const Tensor& stats, int64_t want)
    {
        ctx->set_materialize_grads(false);
        ctx->saved_data["want"] = want;
        ctx->saved_data["weight"] = weight.has_value();
        const Tensor w = weight.value_or(Tensor());
        ctx->save_for_backward({gy, x, w, stats});
        const int64_t cols = x.size(-1);
        NormGrads g = norm_backward(Rows(gy, cols), Rows(x, cols), w, stats, want & 1, want & 2, want & 4, x);
        variable_list out;
        if (want & 1) out.push_back(g.dx);
        if (want & 2) out.push_back(g.dw);
        if (want & 4) out.push_back(g.db);
        return out;
    }

    static variable_list backward(AutogradContext* ctx, variable_list grads)
    {
        const auto saved = ctx->get_saved_variables();
        const int64_t want = ctx->saved_data["want"].toInt();
        const bool has_w = ctx->saved_data["weight"].toBool();
        size_t at_grad = 0;
        const auto next = [&](int64_t bit) { return want & bit ? grads[at_grad++] : Tensor(); };
        const Tensor v = next(1), p_in = next(2), q_in = next(4);
        const int64_t cols = saved[1].size(-1);
        const Rows gy(saved[0], cols), x(saved[1], cols);
        const Tensor &w = saved[2], &stats = saved[3];
        check_readable({&v, &p_in, &q_in});
        const auto plain = [](const Tensor& t) { return t.defined() ? t.resolve_neg().contiguous() : t; };
        const Tensor p = plain(p_in), q = plain(q_in);
        variable_list out(5);
        if (ctx->needs_input_grad(0)) out[0] = at::empty(saved[1].sizes(), x.keep.options());
        if (ctx->needs_input_grad(1)) out[1] = at::empty(saved[1].sizes(), x.keep.options());
        if (has_w && ctx->needs_input_grad(2)) out[2] = at::empty({cols}, x.keep.options());
        {
            OnDevice on(x.keep);
            size_t bytes = 0;
            if (out[2].defined())
                done(emu_layer_norm_backward_workspace(x.n, cols, &bytes), "emu_layer_norm_backward_workspace");
            Workspace ws(bytes, x.keep);
            const float* s = ptr(stats);
            const Rows v2(v.defined() ? v : saved[0], cols);
            done(emu_layer_norm_backward2(x.n, cols, v.defined() ? v2.data() : nullptr, v2.ld, ptr(p), ptr(q),
                                          gy.data(), gy.ld, x.data(), x.ld, ptr(w), s, s ? s + x.n : s, out_ptr(out[0]),
                                          cols, out_ptr(out[1]), cols, out_ptr(out[2]), ws.p, ws.bytes, on.stream),
                 "emu_layer_norm_backward2");
        }
        last_derivative(out, grads, saved);
        return out;
    }
};

struct LayerNorm : Function<LayerNorm> {
    static Tensor forward(AutogradContext* ctx, const Tensor& x, const optional<Tensor>& weight,
                          const optional<Tensor>& bias, double eps)
    {
        const Tensor w = weight.value_or(Tensor());
        Tensor stats;
        Tensor y = norm_forward(Rows(x, x.size(-1)), w, bias.value_or(Tensor()), eps, &stats, x);
        ctx->save_for_backward({x, w, stats});
        ctx->saved_data["weight"] = weight.has_value();
        ctx->saved_data["bias"] = bias.has_value();
        return y;
    }

    static variable_list backward(AutogradContext* ctx, variable_list grads)
    {
        const auto saved = ctx->get_saved_variables();
        const Tensor &x = saved[0], &w = saved[1], &stats = saved[2], &gy = grads[0];
        const bool has_w = ctx->saved_data["weight"].toBool(), has_b = ctx->saved_data["bias"].toBool();
        const bool want_x = ctx->needs_input_grad(0), want_w = has_w && ctx->needs_input_grad(1);
        const bool want_b = has_b && ctx->needs_input_grad(has_w ? 2 : 1);
        variable_list out(4);
        check_readable({&gy});
        if (!gy.defined() || !(want_x || want_w || want_b)) return out;
        if (at::GradMode::is_enabled()) {
            const int64_t want = (want_x ? 1 : 0) | (want_w ? 2 : 0) | (want_b ? 4 : 0);
            variable_list g = LayerNormBackward::apply(gy, x, has_w ? optional<Tensor>(w) : std::nullopt, stats, want);
            size_t k = 0;
            if (want_x) out[0] = g[k++];
            if (want_w) out[1] = g[k++];
            if (want_b) out[2] = g[k++];
            return out;
        }
        const int64_t cols = x.size(-1);
        NormGrads g = norm_backward(Rows(gy, cols), Rows(x, cols), w, stats, want_x, want_w, want_b, x);
        out[0] = g.dx;
        out[1] = g.dw;
        out[2] = g.db;
        return out;
    }
};

Tensor layer_norm(const Tensor& x, const optional<Tensor>& weight_in, const optional<Tensor>& bias_in, double eps)
{
    check_readable({&x, given(weight_in), given(bias_in)});
    check(x, "x");
    TORCH_CHECK_VALUE(x.dim() >= 1 && x.size(-1) >= 1 && x.size(-1) <= EMU_LAYER_NORM_MAX_COLS,
                      "layer_norm takes 1 to ", EMU_LAYER_NORM_MAX_COLS, " features, not ", x.sizes());
    TORCH_CHECK_VALUE(eps >= 0.0, "eps must not be negative");
    const int64_t cols = x.size(-1);
    const Tensor weight = vector_of(weight_in, "weight", cols, x), bias = vector_of(bias_in, "bias", cols, x);
    if (wants_grad({&x, &weight, &bias})) {
        claim_leaves(OnDevice(x), {&x, &weight, &bias});
        const auto some = [](const Tensor& t) { return t.defined() ? optional<Tensor>(t) : std::nullopt; };
        return LayerNorm::apply(x, some(weight), some(bias), eps);
    }
    return norm_forward(Rows(x, cols), weight, bias, eps, nullptr, x);
}

// ---- the pieces on their own -------------------------------------------------------------------

std::tuple<Tensor, optional<Tensor>> wgrad(const Tensor& dz, const Tensor& x, bool want_db)
{
    check_readable({&dz, &x});
    check(dz, "dz");
    check_like(x, "x", dz);
    TORCH_CHECK_VALUE(dz.dim() == 2 && x.dim() == 2, "dz and x must be 2-D");
    TORCH_CHECK_VALUE(dz.size(0) == x.size(0), "row counts differ: ", dz.size(0), " vs ", x.size(0));
    if (wants_grad({&dz, &x})) {
        claim_leaves(OnDevice(dz), {&dz, &x});
        variable_list g = WeightGrad::apply(dz, x, want_db, (int64_t)EMU_MODE_AUTO);
        return {g[0], want_db ? optional<Tensor>(g[1]) : std::nullopt};
    }
    WeightGrads g = weight_grad(Rows(dz, dz.size(1)), Rows(x, x.size(1)), want_db);
    return {g.dw, want_db ? optional<Tensor>(g.db) : std::nullopt};
}

// dz = dy act'(z) for matrices, differentiable once.
Tensor act_grad(const Tensor& dy, const Tensor& z, int64_t act)
{
    check_readable({&dy, &z});
    check(dy, "dy");
    check_like(z, "z", dy);
    TORCH_CHECK_VALUE(dy.dim() == 2 && dy.sizes() == z.sizes(), "dy and z must be matrices of one shape");
    if (wants_grad({&dy, &z})) claim_leaves(OnDevice(dy), {&dy, &z});
    return ActBackward::apply(dy, z, act, false);
}

Tensor presplit_gated(const Tensor& w, int64_t mode)
{
    check_readable({&w});
    check(w, "weight");
    TORCH_CHECK_VALUE(w.dim() == 2 && w.size(0) % 2 == 0, "weight must hold as many gate rows as up rows");
    const Rows r(w, w.size(1));
    size_t bytes = 0;
    done(emu_presplit_gated_bytes(r.n / 2, r.width, (emu_mode_t)mode, &bytes), "emu_presplit_gated_bytes");
    Tensor planes = at::empty({std::max<int64_t>((int64_t)bytes, 1)}, w.options().dtype(at::kByte));
    OnDevice on(w);
    done(emu_presplit_gated(r.n / 2, r.width, r.data(), r.ld, (emu_mode_t)mode, planes.mutable_data_ptr(), on.stream),
         "emu_presplit_gated");
    return planes;
}

}  // namespace

void register_attention(py::module_& m);   // attention_torch.cpp

PYBIND11_MODULE(TORCH_EXTENSION_NAME, m)
{
    py::register_exception_translator([](std::exception_ptr p) {
        try {
            if (p) std::rethrow_exception(p);
        } catch (const EmuFailure& e) {
            const py::object cls = py::module_::import("emulated_fp32_matrix_amd").attr("EmuError");
            PyErr_SetObject(cls.ptr(), cls(e.status, e.where).ptr());
        }
    });
    using gil = py::call_guard<py::gil_scoped_release>;
    m.def("layer_norm", &layer_norm, gil());
    m.def("linear_act", &linear_act, gil());
    m.def("gated_linear", &gated_linear, gil());
    m.def("wgrad", &wgrad, gil());
    m.def("act_grad", &act_grad, gil());
    m.def("presplit_gated", &presplit_gated, gil());
    register_attention(m);
}

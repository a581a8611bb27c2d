// The expert operators for torch: argument checks, outputs and autograd nodes
// over the C ABI of lapsum_experts.h.  Every step runs in liblapsum.so; this
// module only marshals.  It is C++ because a small training step is bound by
// the host: an autograd node written in Python runs in the engine's own thread
// and takes the interpreter lock back and forth (dispatch with its gradient,
// 1000 rows: 91 us so, 46 us here, of which the GPU works 10).
#include "lapsum_torch.h"

using namespace lapsum_torch;

namespace {

// ---- the calls ------------------------------------------------------------------

std::tuple<Tensor, Tensor, Tensor> topk_call(const Tensor& p, int64_t m, double floor, bool normalize) {
    check(p, "p", at::kFloat, 2);
    const int64_t tokens = p.size(0), experts = p.size(1);
    TORCH_CHECK_VALUE(experts >= 1 && experts <= LAPSUM_MAX_EXPERTS, "p must have between 1 and ", LAPSUM_MAX_EXPERTS,
                      " experts (got ", experts, ")");
    TORCH_CHECK_VALUE(m >= 1 && m <= std::min<int64_t>(experts, LAPSUM_MAX_SLOTS),
                      "m must be between 1 and min(experts, ", LAPSUM_MAX_SLOTS, ") (got ", m, ")");
    TORCH_CHECK_VALUE(floor == floor, "floor must not be NaN");
    const On on(p);
    Tensor ids = at::empty({tokens, m}, p.options().dtype(at::kInt)), w = at::empty({tokens, m}, p.options()), sums;
    if (normalize) sums = at::empty({tokens}, p.options());
    check_ok(lapsum_expert_topk(ptr<float>(p), tokens, experts, m, (float)floor, normalize, ptr<int32_t>(ids),
                                ptr<float>(w), ptr<float>(sums), on.stream),
             "lapsum_expert_topk");
    return {ids, w, sums};
}

Tensor topk_vjp(const Tensor& ids, const Tensor& w, const Tensor& dw, int64_t experts,
                const std::optional<Tensor>& sums_) {
    const Tensor sums = sums_.value_or(Tensor());
    check(ids, "ids", at::kInt, 2);
    check(w, "w", at::kFloat, 2, &ids);
    check(dw, "dw", at::kFloat, 2, &ids);
    check_shape(w, "w", ids.sizes());
    check_shape(dw, "dw", ids.sizes());
    if (sums.defined()) {
        check(sums, "sums", at::kFloat, 1, &ids);
        check_shape(sums, "sums", {ids.size(0)});
    }
    const On on(ids);
    Tensor dp = at::empty({ids.size(0), experts}, w.options());
    check_ok(lapsum_expert_topk_vjp(ptr<int32_t>(ids), ptr<float>(w), ptr<float>(dw), ptr<float>(sums), ids.size(0),
                                    experts, ids.size(1), sums.defined(), ptr<float>(dp), on.stream),
             "lapsum_expert_topk_vjp");
    return dp;
}

std::tuple<Tensor, Tensor, Tensor> sort(const Tensor& ids, int64_t experts) {
    check(ids, "ids", at::kInt, 2);
    TORCH_CHECK_VALUE(experts >= 1 && experts <= LAPSUM_MAX_EXPERTS, "experts must be between 1 and ",
                      LAPSUM_MAX_EXPERTS, " (got ", experts, ")");
    TORCH_CHECK_VALUE(ids.size(1) >= 1 && ids.size(1) <= LAPSUM_MAX_SLOTS, "ids must have between 1 and ",
                      LAPSUM_MAX_SLOTS, " slots (got ", ids.size(1), ")");
    const On on(ids);
    const int64_t pairs = ids.numel();
    Tensor offsets = at::empty({experts + 1}, ids.options()), order = at::empty({pairs}, ids.options()),
           place = at::empty(ids.sizes(), ids.options()), scratch;
    if (const size_t n = lapsum_expert_sort_scratch_bytes(pairs, experts))
        scratch = at::empty({(int64_t)n}, ids.options().dtype(at::kByte));
    check_ok(lapsum_expert_sort(ptr<int32_t>(ids), pairs, experts, ptr<int32_t>(offsets), ptr<int32_t>(order),
                                ptr<int32_t>(place), ptr<void>(scratch), on.stream),
             "lapsum_expert_sort");
    return {offsets, order, place};
}

Tensor dispatch_call(const Tensor& x, const Plan& plan) {
    check_rows(x, "x");
    check_shape(x, "x", {plan.tokens(), x.size(1)});
    const On on(x);
    Tensor xs = at::empty({plan.pairs(), x.size(1)}, x.options());
    check_ok(lapsum_expert_dispatch(ptr<void>(x), type_of(x), plan.tokens(), plan.slots(), x.size(1), plan.experts,
                                    plan.off(), plan.at(), ptr<void>(xs), on.stream),
             "lapsum_expert_dispatch");
    return xs;
}

Tensor dispatch_vjp_call(const Tensor& dxs, const Plan& plan) {
    check_rows(dxs, "dxs");
    check_shape(dxs, "dxs", {plan.pairs(), dxs.size(1)});
    const On on(dxs);
    Tensor dx = at::empty({plan.tokens(), dxs.size(1)}, dxs.options());
    check_ok(lapsum_expert_dispatch_vjp(ptr<void>(dxs), type_of(dxs), plan.tokens(), plan.slots(), dxs.size(1),
                                        plan.at(), ptr<void>(dx), on.stream),
             "lapsum_expert_dispatch_vjp");
    return dx;
}

void check_linear(const Tensor& xs, const Tensor& weight, const Plan& plan, const Tensor& bias) {
    check_rows(xs, "xs");
    check(weight, "weight", xs.scalar_type(), 3, &xs);
    check_shape(xs, "xs", {plan.pairs(), weight.size(2)});
    check_shape(weight, "weight", {plan.experts, weight.size(1), weight.size(2)});
    TORCH_CHECK_VALUE(std::max(weight.size(1), weight.size(2)) <= LAPSUM_MAX_PAIRS, "weight must have at most ",
                      LAPSUM_MAX_PAIRS, " rows and columns an expert (got ", weight.size(1), " x ", weight.size(2), ")");
    if (bias.defined()) {
        check(bias, "bias", xs.scalar_type(), 2, &xs);
        check_shape(bias, "bias", {plan.experts, weight.size(1)});
    }
}

// ys and, with `keep` and an activation, z
std::tuple<Tensor, Tensor> linear_call(const Tensor& xs, const Tensor& weight, const Tensor& bias, const Plan& plan,
                                       int act, bool keep) {
    check_linear(xs, weight, plan, bias);
    const On on(xs);
    const int64_t rows = xs.size(0), out = weight.size(1);
    Tensor ys = at::empty({rows, out}, xs.options()), z;
    if (keep && act != LAPSUM_ACT_NONE) z = at::empty({rows, out}, xs.options().dtype(z_type(xs)));
    check_ok(lapsum_expert_linear(ptr<void>(xs), ptr<void>(weight), ptr<void>(bias), type_of(xs), rows, xs.size(1),
                                  out, plan.experts, plan.off(), (lapsum_act_t)act, ptr<void>(ys), ptr<void>(z),
                                  on.stream),
             "lapsum_expert_linear");
    return {ys, z};
}

// xs is read for dweight only, weight for dxs only: where those are not wanted
// either may be missing.
std::tuple<Tensor, Tensor, Tensor> linear_vjp_call(const Tensor& xs, const Tensor& weight, const Plan& plan,
                                                   const Tensor& z, const Tensor& dys, int act,
                                                   std::array<bool, 3> want) {
    const int64_t rows = dys.size(0), out = dys.size(1),
                  in = xs.defined() ? xs.size(1) : weight.defined() ? weight.size(2) : 0;
    if (act != LAPSUM_ACT_NONE) {
        TORCH_CHECK_VALUE(z.defined(), "z is needed with an activation");
        check(z, "z", z_type(dys), 2, &dys);
        check_shape(z, "z", {rows, out});
    }
    const On on(dys);
    Tensor dxs, dweight, dbias, scratch;
    if (want[0]) dxs = at::empty({rows, in}, dys.options());
    if (want[1]) dweight = at::empty({plan.experts, out, in}, dys.options());
    if (want[2]) dbias = at::empty({plan.experts, out}, dys.options());
    int64_t elements = 0;
    for (const Tensor* t : {&dxs, &dweight, &dbias}) elements += t->defined() ? t->numel() : 0;
    if (elements == 0) return {dxs, dweight, dbias};
    const auto dt = type_of(dys);
    if (const size_t n = lapsum_expert_linear_vjp_scratch_bytes(dt, rows, in, out, plan.experts, (lapsum_act_t)act,
                                                                want[2]))
        scratch = at::empty({(int64_t)n}, dys.options().dtype(at::kByte));
    check_ok(lapsum_expert_linear_vjp(ptr<void>(xs), ptr<void>(weight), ptr<void>(z), ptr<void>(dys), dt, rows, in, out,
                                      plan.experts, plan.off(), (lapsum_act_t)act, ptr<void>(dxs), ptr<void>(dweight),
                                      ptr<void>(dbias), ptr<void>(scratch), on.stream),
             "lapsum_expert_linear_vjp");
    return {dxs, dweight, dbias};
}

void check_combine(const Tensor& ys, const Tensor& w, const Plan& plan) {
    check_rows(ys, "ys");
    check_shape(ys, "ys", {plan.pairs(), ys.size(1)});
    check(w, "w", at::kFloat, 2, &ys);
    check_shape(w, "w", {plan.tokens(), plan.slots()});
}

Tensor combine_call(const Tensor& ys, const Tensor& w, const Tensor& residual, const Plan& plan) {
    check_combine(ys, w, plan);
    if (residual.defined()) {
        check(residual, "residual", ys.scalar_type(), 2, &ys);
        check_shape(residual, "residual", {plan.tokens(), ys.size(1)});
    }
    const On on(ys);
    Tensor out = at::empty({plan.tokens(), ys.size(1)}, ys.options());
    check_ok(lapsum_expert_combine(ptr<void>(ys), ptr<float>(w), ptr<void>(residual), type_of(ys), plan.tokens(),
                                   plan.slots(), ys.size(1), plan.at(), ptr<void>(out), on.stream),
             "lapsum_expert_combine");
    return out;
}

// ys is read for dw only: where that is not wanted it may be missing.
std::tuple<Tensor, Tensor> combine_vjp_call(const Tensor& ys, const Tensor& w, const Plan& plan, const Tensor& dout,
                                            std::array<bool, 2> want) {
    const On on(dout);
    const int64_t width = dout.size(1);
    Tensor dys, dw;
    if (want[0]) dys = at::empty({plan.pairs(), width}, dout.options());
    if (want[1]) dw = at::empty(w.sizes(), w.options());
    if ((dys.defined() ? dys.numel() : 0) + (dw.defined() ? dw.numel() : 0) == 0) return {dys, dw};
    check_ok(lapsum_expert_combine_vjp(ptr<void>(ys), ptr<float>(w), ptr<void>(dout), type_of(dout), plan.tokens(),
                                       plan.slots(), width, plan.experts, plan.off(), plan.at(), ptr<void>(dys),
                                       ptr<float>(dw), on.stream),
             "lapsum_expert_combine_vjp");
    return {dys, dw};
}

// ---- autograd nodes --------------------------------------------------------------
// needs_input_grad counts the tensors that were given: where an optional one
// is missing, the next is a plan's array, which needs none.

Plan saved_plan(AutogradContext* ctx, const Tensor& offsets, const Tensor& place) {
    return {ctx->saved_data["experts"].toInt(), offsets, place};
}

struct TopK : torch::autograd::Function<TopK> {
    static variable_list forward(AutogradContext* ctx, const Tensor& p, int64_t m, double floor, bool normalize) {
        at::AutoDispatchBelowADInplaceOrView below;
        auto [ids, w, sums] = topk_call(p.contiguous(), m, floor, normalize);
        ctx->save_for_backward({ids, w, sums});
        ctx->saved_data["experts"] = p.size(1);
        ctx->mark_non_differentiable({ids});
        ctx->set_materialize_grads(false);
        return {ids, w};
    }
    static variable_list backward(AutogradContext* ctx, variable_list g) {
        if (!g[1].defined()) return {Tensor(), Tensor(), Tensor(), Tensor()};
        check_once("expert_topk");
        const auto s = ctx->get_saved_variables();
        return {topk_vjp(s[0], s[1], g[1].contiguous(), ctx->saved_data["experts"].toInt(),
                         s[2].defined() ? std::optional<Tensor>(s[2]) : std::nullopt),
                Tensor(), Tensor(), Tensor()};
    }
};

struct Dispatch : torch::autograd::Function<Dispatch> {
    static Tensor forward(AutogradContext* ctx, const Tensor& x, int64_t experts, const Tensor& offsets,
                          const Tensor& place) {
        at::AutoDispatchBelowADInplaceOrView below;
        ctx->save_for_backward({offsets, place});
        ctx->saved_data["experts"] = experts;
        return dispatch_call(x.contiguous(), {experts, offsets, place});
    }
    static variable_list backward(AutogradContext* ctx, variable_list g) {
        check_once("expert_dispatch");
        const auto s = ctx->get_saved_variables();
        return {dispatch_vjp_call(g[0].contiguous(), saved_plan(ctx, s[0], s[1])), Tensor(), Tensor(), Tensor()};
    }
};

struct Linear : torch::autograd::Function<Linear> {
    static Tensor forward(AutogradContext* ctx, const Tensor& xs_, const Tensor& weight_,
                          const std::optional<Tensor>& bias_, int64_t experts, const Tensor& offsets,
                          const Tensor& place, int64_t act) {
        at::AutoDispatchBelowADInplaceOrView below;
        const Tensor xs = xs_.contiguous(), weight = weight_.contiguous(), bias = bias_.value_or(Tensor());
        auto [ys, z] = linear_call(xs, weight, bias.defined() ? bias.contiguous() : bias, {experts, offsets, place},
                                   (int)act, true);
        // what the gradients that are wanted read, and no more
        ctx->save_for_backward({recorded(weight_) ? xs : Tensor(), recorded(xs_) ? weight : Tensor(), z, offsets, place});
        ctx->saved_data["experts"] = experts;
        ctx->saved_data["act"] = act;
        return ys;
    }
    static variable_list backward(AutogradContext* ctx, variable_list g) {
        check_once("expert_linear");
        const auto s = ctx->get_saved_variables();
        auto [dxs, dweight, dbias] = linear_vjp_call(
            s[0], s[1], saved_plan(ctx, s[3], s[4]), s[2], g[0].contiguous(), (int)ctx->saved_data["act"].toInt(),
            {ctx->needs_input_grad(0), ctx->needs_input_grad(1), ctx->needs_input_grad(2)});
        return {dxs, dweight, dbias, Tensor(), Tensor(), Tensor(), Tensor()};
    }
};

struct Combine : torch::autograd::Function<Combine> {
    static Tensor forward(AutogradContext* ctx, const Tensor& ys_, const Tensor& w_,
                          const std::optional<Tensor>& residual_, int64_t experts, const Tensor& offsets,
                          const Tensor& place) {
        at::AutoDispatchBelowADInplaceOrView below;
        const Tensor ys = ys_.contiguous(), w = w_.contiguous(), residual = residual_.value_or(Tensor());
        ctx->save_for_backward({recorded(w_) ? ys : Tensor(), w, offsets, place});
        ctx->saved_data["experts"] = experts;
        return combine_call(ys, w, residual.defined() ? residual.contiguous() : residual, {experts, offsets, place});
    }
    static variable_list backward(AutogradContext* ctx, variable_list g) {
        check_once("expert_combine");
        const auto s = ctx->get_saved_variables();
        auto [dys, dw] = combine_vjp_call(s[0], s[1], saved_plan(ctx, s[2], s[3]), g[0].contiguous(),
                                          {ctx->needs_input_grad(0), ctx->needs_input_grad(1)});
        return {dys, dw, ctx->needs_input_grad(2) ? g[0] : Tensor(), Tensor(), Tensor(), Tensor()};
    }
};

// ---- what Python calls -------------------------------------------------------------

std::tuple<Tensor, Tensor> topk(const Tensor& p, int64_t m, double floor, bool normalize) {
    check_tangents("expert_topk", p);
    if (at::GradMode::is_enabled() && recorded(p)) {
        auto r = TopK::apply(p, m, floor, normalize);
        return {r[0], r[1]};
    }
    auto r = topk_call(p.contiguous(), m, floor, normalize);
    return {std::get<0>(r), std::get<1>(r)};
}

Tensor dispatch(const Tensor& x, int64_t experts, const Tensor& offsets, const Tensor& order, const Tensor& place) {
    const Plan plan = make_plan(experts, offsets, order, place, x);
    check_tangents("expert_dispatch", x);
    if (at::GradMode::is_enabled() && recorded(x)) return Dispatch::apply(x, experts, offsets, place);
    return dispatch_call(x.contiguous(), plan);
}
Tensor dispatch_vjp(const Tensor& dxs, int64_t experts, const Tensor& offsets, const Tensor& order,
                    const Tensor& place) {
    return dispatch_vjp_call(dxs, make_plan(experts, offsets, order, place, dxs));
}

Tensor linear(const Tensor& xs, const Tensor& weight, const std::optional<Tensor>& bias_, const std::string& activation,
              int64_t experts, const Tensor& offsets, const Tensor& order, const Tensor& place) {
    const Tensor bias = bias_.value_or(Tensor());
    const int act = act_of(activation);
    const Plan plan = make_plan(experts, offsets, order, place, xs);
    check_tangents("expert_linear", xs, weight, bias);
    if (at::GradMode::is_enabled() && (recorded(xs) || recorded(weight) || recorded(bias)))
        return Linear::apply(xs, weight, bias_, experts, offsets, place, (int64_t)act);
    return std::get<0>(linear_call(xs.contiguous(), weight.contiguous(), bias.defined() ? bias.contiguous() : bias,
                                   plan, act, false));
}
std::tuple<Tensor, std::optional<Tensor>> linear_forward(const Tensor& xs, const Tensor& weight,
                                                         const std::optional<Tensor>& bias,
                                                         const std::string& activation, int64_t experts,
                                                         const Tensor& offsets, const Tensor& order,
                                                         const Tensor& place) {
    auto [ys, z] = linear_call(xs, weight, bias.value_or(Tensor()), make_plan(experts, offsets, order, place, xs),
                               act_of(activation), true);
    return {ys, z.defined() ? std::optional<Tensor>(z) : std::nullopt};
}

std::tuple<std::optional<Tensor>, std::optional<Tensor>, std::optional<Tensor>> linear_vjp(
    const Tensor& xs, const Tensor& weight, const std::optional<Tensor>& z, const Tensor& dys,
    const std::string& activation, std::array<bool, 3> want, int64_t experts, const Tensor& offsets,
    const Tensor& order, const Tensor& place) {
    const Plan plan = make_plan(experts, offsets, order, place, xs);
    check_linear(xs, weight, plan, Tensor());
    check(dys, "dys", xs.scalar_type(), 2, &xs);
    check_shape(dys, "dys", {xs.size(0), weight.size(1)});
    auto [a, b, c] = linear_vjp_call(xs, weight, plan, z.value_or(Tensor()), dys, act_of(activation), want);
    return {maybe(a), maybe(b), maybe(c)};
}

Tensor combine(const Tensor& ys, const Tensor& w, const std::optional<Tensor>& residual_, int64_t experts,
               const Tensor& offsets, const Tensor& order, const Tensor& place) {
    const Tensor residual = residual_.value_or(Tensor());
    const Plan plan = make_plan(experts, offsets, order, place, ys);
    check_tangents("expert_combine", ys, w, residual);
    if (at::GradMode::is_enabled() && (recorded(ys) || recorded(w) || recorded(residual)))
        return Combine::apply(ys, w, residual_, experts, offsets, place);
    return combine_call(ys.contiguous(), w.contiguous(), residual.defined() ? residual.contiguous() : residual, plan);
}
std::tuple<std::optional<Tensor>, std::optional<Tensor>> combine_vjp(const Tensor& ys, const Tensor& w,
                                                                     const Tensor& dout, std::array<bool, 2> want,
                                                                     int64_t experts, const Tensor& offsets,
                                                                     const Tensor& order, const Tensor& place) {
    const Plan plan = make_plan(experts, offsets, order, place, ys);
    check_combine(ys, w, plan);
    check(dout, "dout", ys.scalar_type(), 2, &ys);
    check_shape(dout, "dout", {plan.tokens(), ys.size(1)});
    auto [a, b] = combine_vjp_call(ys, w, plan, dout, want);
    return {maybe(a), maybe(b)};
}

}  // namespace

// layers_torch.cpp
void define_layers(py::module_& m);

PYBIND11_MODULE(_experts_torch, m) {
    define_layers(m);
    py::register_exception_translator([](std::exception_ptr p) {
        try {
            if (p) std::rethrow_exception(p);
        } catch (const StatusError& e) {
            const py::object cls = py::module_::import("differentiable_exact_budget_amd._binding").attr("LapsumError");
            PyErr_SetObject(cls.ptr(), cls(e.code, e.where).ptr());
        } catch (const c10::Error&) {
            torch::translate_exception_to_python(p);
        }
    });
    m.def("topk", &topk);
    m.def("topk_vjp", &topk_vjp);
    m.def("sort", &sort);
    m.def("dispatch", &dispatch);
    m.def("dispatch_vjp", &dispatch_vjp);
    m.def("linear", &linear);
    m.def("linear_forward", &linear_forward);
    m.def("linear_vjp", &linear_vjp);
    m.def("combine", &combine);
    m.def("combine_vjp", &combine_vjp);
}

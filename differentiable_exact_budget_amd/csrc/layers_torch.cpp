// The norm, the loss and the experts' products in 8 bits for torch: argument
// checks, outputs and autograd nodes over the C ABIs of lapsum_layers.h and
// lapsum_experts8.h.
#include "lapsum_layers.h"

#include "lapsum_experts8.h"
#include "lapsum_torch.h"

using namespace lapsum_torch;

namespace {

Tensor scratch_of(size_t bytes, const Tensor& like) {
    return bytes ? at::empty({(int64_t)bytes}, like.options().dtype(at::kByte)) : Tensor();
}
// whether a call has anything to write (what has no elements has no address)
template <class... Tensors>
bool written(const Tensors&... out) {
    return ((out.defined() && out.numel() > 0) || ...);
}
Tensor laid_out(const Tensor& x) { return x.defined() ? x.contiguous() : x; }

// rows of one of the three types, of any number of dimensions, at least one
void check_any_rows(const Tensor& x, const char* name) {
    TORCH_CHECK_VALUE(x.is_cuda(), name, " must be on a GPU device (got ", x.device(), ")");
    TORCH_CHECK_VALUE(x.dim() >= 1, name, " must have at least 1 dimension");
    TORCH_CHECK_VALUE(row_type(x.scalar_type()), name, " must be float32, bfloat16 or float16 (got ", x.scalar_type(),
                      ")");
}
void check_like(const Tensor& x, const char* name, at::ScalarType t, at::IntArrayRef shape, const Tensor& like) {
    TORCH_CHECK_VALUE(x.device() == like.device(), name, " must be on ", like.device(), " (got ", x.device(), ")");
    TORCH_CHECK_VALUE(x.scalar_type() == t, name, " must be ", t, " (got ", x.scalar_type(), ")");
    check_shape(x, name, shape);
}

// ---- layer norm -------------------------------------------------------------------

// the type of weight and bias
at::ScalarType norm_wtype(const Tensor& x, const Tensor& weight, const Tensor& bias) {
    return weight.defined() ? weight.scalar_type() : bias.defined() ? bias.scalar_type() : x.scalar_type();
}
void check_norm(const Tensor& x, const Tensor& weight, const Tensor& bias) {
    check_any_rows(x, "x");
    TORCH_CHECK_VALUE(x.size(-1) >= 1, "x must have a last dimension of at least 1");
    const auto w = norm_wtype(x, weight, bias);
    TORCH_CHECK_VALUE(w == x.scalar_type() || w == at::kFloat, weight.defined() ? "weight" : "bias", " must be ",
                      x.scalar_type(), " or float32 (got ", w, ")");
    if (weight.defined()) check_like(weight, "weight", w, {x.size(-1)}, x);
    if (bias.defined()) check_like(bias, "bias", w, {x.size(-1)}, x);
}

std::tuple<Tensor, Tensor, Tensor> norm_call(const Tensor& x, const Tensor& weight, const Tensor& bias, double eps,
                                             bool keep) {
    TORCH_CHECK_VALUE(eps >= 0, "eps must be at least 0 (got ", eps, ")");
    const On on(x);
    const int64_t width = x.size(-1), rows = x.numel() / width;
    Tensor y = at::empty(x.sizes(), x.options()), mean, rstd;
    if (keep) {
        const auto shape = x.sizes().slice(0, x.dim() - 1);
        mean = at::empty(shape, x.options().dtype(at::kFloat));
        rstd = at::empty(shape, x.options().dtype(at::kFloat));
    }
    check_ok(lapsum_layer_norm(ptr<void>(x), ptr<void>(weight), ptr<void>(bias), type_of(x),
                               *row_type(norm_wtype(x, weight, bias)), rows, width, (float)eps, ptr<void>(y),
                               ptr<float>(mean), ptr<float>(rstd), on.stream),
             "lapsum_layer_norm");
    return {y, mean, rstd};
}

// x is read for dx and dweight, weight for dx only.
std::tuple<Tensor, Tensor, Tensor> norm_vjp_call(const Tensor& x, const Tensor& weight, const Tensor& mean,
                                                 const Tensor& rstd, const Tensor& dy, at::ScalarType wtype,
                                                 std::array<bool, 3> want) {
    const On on(dy);
    const int64_t width = dy.size(-1), rows = dy.numel() / width;
    Tensor dx, dw, db, scratch;
    if (want[0]) dx = at::empty(dy.sizes(), dy.options());
    if (want[1]) dw = at::empty({width}, dy.options().dtype(wtype));
    if (want[2]) db = at::empty({width}, dy.options().dtype(wtype));
    if (!written(dx, dw, db)) return {dx, dw, db};
    if (want[1] || want[2]) scratch = scratch_of(lapsum_layer_norm_vjp_scratch_bytes(type_of(dy), rows, width), dy);
    check_ok(lapsum_layer_norm_vjp(ptr<void>(x), ptr<void>(weight), ptr<float>(mean), ptr<float>(rstd), ptr<void>(dy),
                                   type_of(dy), *row_type(wtype), rows, width, ptr<void>(dx), ptr<void>(dw),
                                   ptr<void>(db), ptr<void>(scratch), on.stream),
             "lapsum_layer_norm_vjp");
    return {dx, dw, db};
}

struct Norm : torch::autograd::Function<Norm> {
    static Tensor forward(AutogradContext* ctx, const Tensor& x_, const std::optional<Tensor>& weight_,
                          const std::optional<Tensor>& bias_, double eps) {
        at::AutoDispatchBelowADInplaceOrView below;
        const Tensor x = x_.contiguous(), weight = laid_out(weight_.value_or(Tensor())),
                     bias = laid_out(bias_.value_or(Tensor()));
        auto [y, mean, rstd] = norm_call(x, weight, bias, eps, true);
        ctx->save_for_backward({x, recorded(x_) ? weight : Tensor(), mean, rstd});
        ctx->saved_data["wtype"] = (int64_t)norm_wtype(x, weight, bias);
        // needs_input_grad counts the tensors that were given
        ctx->saved_data["weight"] = weight.defined();
        ctx->saved_data["bias"] = bias.defined();
        return y;
    }
    static variable_list backward(AutogradContext* ctx, variable_list g) {
        check_once("layer_norm");
        const auto s = ctx->get_saved_variables();
        const bool weight = ctx->saved_data["weight"].toBool(), bias = ctx->saved_data["bias"].toBool();
        auto [dx, dw, db] = norm_vjp_call(s[0], s[1], s[2], s[3], g[0].contiguous(),
                                          (at::ScalarType)ctx->saved_data["wtype"].toInt(),
                                          {ctx->needs_input_grad(0), weight && ctx->needs_input_grad(1),
                                           bias && ctx->needs_input_grad(weight ? 2 : 1)});
        return {dx, dw, db, Tensor()};
    }
};

Tensor layer_norm(const Tensor& x, const std::optional<Tensor>& weight_, const std::optional<Tensor>& bias_, double eps) {
    const Tensor weight = weight_.value_or(Tensor()), bias = bias_.value_or(Tensor());
    check_norm(x, weight, bias);
    check_tangents("layer_norm", x, weight, bias);
    if (at::GradMode::is_enabled() && (recorded(x) || recorded(weight) || recorded(bias)))
        return Norm::apply(x, weight_, bias_, eps);
    return std::get<0>(norm_call(x.contiguous(), laid_out(weight), laid_out(bias), eps, false));
}
std::tuple<Tensor, Tensor, Tensor> layer_norm_forward(const Tensor& x, const std::optional<Tensor>& weight_,
                                                      const std::optional<Tensor>& bias_, double eps) {
    const Tensor weight = weight_.value_or(Tensor()), bias = bias_.value_or(Tensor());
    check_norm(x, weight, bias);
    return norm_call(x.contiguous(), laid_out(weight), laid_out(bias), eps, true);
}
std::tuple<std::optional<Tensor>, std::optional<Tensor>, std::optional<Tensor>> layer_norm_vjp(
    const Tensor& x, const std::optional<Tensor>& weight_, const Tensor& mean, const Tensor& rstd, const Tensor& dy,
    std::array<bool, 3> want) {
    const Tensor weight = weight_.value_or(Tensor());
    check_norm(x, weight, Tensor());
    const auto shape = x.sizes().slice(0, x.dim() - 1);
    check_like(mean, "mean", at::kFloat, shape, x);
    check_like(rstd, "rstd", at::kFloat, shape, x);
    check_like(dy, "dy", x.scalar_type(), x.sizes(), x);
    auto [dx, dw, db] = norm_vjp_call(x.contiguous(), laid_out(weight), mean.contiguous(), rstd.contiguous(),
                                      dy.contiguous(), norm_wtype(x, weight, Tensor()), want);
    return {maybe(dx), maybe(dw), maybe(db)};
}

// ---- the loss ---------------------------------------------------------------------

lapsum_reduction_t reduction_of(const std::string& r) {
    if (r == "none") return LAPSUM_REDUCE_NONE;
    if (r == "sum") return LAPSUM_REDUCE_SUM;
    if (r == "mean") return LAPSUM_REDUCE_MEAN;
    TORCH_CHECK_VALUE(false, "reduction must be one of none, sum, mean (got '", r, "')");
}

void check_loss(const Tensor& x, const Tensor& weight, const Tensor& target, const Tensor& bias) {
    check_any_rows(x, "x");
    TORCH_CHECK_VALUE(weight.dim() == 2, "weight must have 2 dimensions (got ", weight.dim(), ")");
    check_like(weight, "weight", x.scalar_type(), {weight.size(0), x.size(-1)}, x);
    const int64_t vocab = weight.size(0), width = x.size(-1), rows = target.numel();
    TORCH_CHECK_VALUE(vocab >= 1, "weight must have at least 1 row");
    TORCH_CHECK_VALUE(std::max({vocab, width, rows}) <= LAPSUM_MAX_LOSS_SIDE, "rows, vocabulary and width must be at most ",
                      LAPSUM_MAX_LOSS_SIDE, " (got ", rows, ", ", vocab, ", ", width, ")");
    check_like(target, "target", at::kLong, x.sizes().slice(0, x.dim() - 1), x);
    if (bias.defined()) check_like(bias, "bias", x.scalar_type(), {vocab}, x);
}

// the loss and, with `keep`, lse
std::tuple<Tensor, Tensor> loss_call(const Tensor& x, const Tensor& weight, const Tensor& target, const Tensor& bias,
                                     lapsum_reduction_t reduction, bool keep) {
    const On on(x);
    const int64_t rows = target.numel(), vocab = weight.size(0), width = x.size(-1);
    const auto f32 = x.options().dtype(at::kFloat);
    Tensor loss = reduction == LAPSUM_REDUCE_NONE ? at::empty(target.sizes(), f32) : at::empty({}, f32), lse;
    if (keep) lse = at::empty(target.sizes(), f32);
    const Tensor scratch = scratch_of(lapsum_linear_cross_entropy_scratch_bytes(type_of(x), rows, vocab, width), x);
    check_ok(lapsum_linear_cross_entropy(ptr<void>(x), ptr<void>(weight), ptr<void>(bias), ptr<int64_t>(target),
                                         type_of(x), rows, vocab, width, reduction, ptr<float>(loss), ptr<float>(lse),
                                         ptr<void>(scratch), on.stream),
             "lapsum_linear_cross_entropy");
    return {loss, lse};
}

std::tuple<Tensor, Tensor, Tensor> loss_vjp_call(const Tensor& x, const Tensor& weight, const Tensor& target,
                                                 const Tensor& bias, const Tensor& lse, const Tensor& dloss,
                                                 lapsum_reduction_t reduction, std::array<bool, 3> want) {
    const On on(x);
    const int64_t rows = target.numel(), vocab = weight.size(0), width = x.size(-1);
    Tensor dx, dw, db;
    if (want[0]) dx = at::empty(x.sizes(), x.options());
    if (want[1]) dw = at::empty(weight.sizes(), weight.options());
    if (want[2]) db = at::empty({vocab}, weight.options());
    if (!written(dx, dw, db)) return {dx, dw, db};
    const Tensor scratch =
        scratch_of(lapsum_linear_cross_entropy_vjp_scratch_bytes(type_of(x), rows, vocab, width), x);
    check_ok(lapsum_linear_cross_entropy_vjp(ptr<void>(x), ptr<void>(weight), ptr<void>(bias), ptr<int64_t>(target),
                                             ptr<float>(lse), ptr<float>(dloss), type_of(x), rows, vocab, width,
                                             reduction, ptr<void>(dx), ptr<void>(dw), ptr<void>(db), ptr<void>(scratch),
                                             on.stream),
             "lapsum_linear_cross_entropy_vjp");
    return {dx, dw, db};
}

struct Loss : torch::autograd::Function<Loss> {
    static Tensor forward(AutogradContext* ctx, const Tensor& x_, const Tensor& weight_, const Tensor& target_,
                          const std::optional<Tensor>& bias_, int64_t reduction) {
        at::AutoDispatchBelowADInplaceOrView below;
        const Tensor x = x_.contiguous(), weight = weight_.contiguous(), target = target_.contiguous(),
                     bias = laid_out(bias_.value_or(Tensor()));
        auto [loss, lse] = loss_call(x, weight, target, bias, (lapsum_reduction_t)reduction, true);
        ctx->save_for_backward({x, weight, target, bias, lse});
        ctx->saved_data["reduction"] = reduction;
        return loss;
    }
    static variable_list backward(AutogradContext* ctx, variable_list g) {
        check_once("linear_cross_entropy");
        const auto s = ctx->get_saved_variables();
        auto [dx, dw, db] = loss_vjp_call(s[0], s[1], s[2], s[3], s[4], g[0].contiguous(),
                                          (lapsum_reduction_t)ctx->saved_data["reduction"].toInt(),
                                          {ctx->needs_input_grad(0), ctx->needs_input_grad(1),
                                           s[3].defined() && ctx->needs_input_grad(3)});
        return {dx, dw, Tensor(), db, Tensor()};
    }
};

Tensor linear_cross_entropy(const Tensor& x, const Tensor& weight, const Tensor& target,
                            const std::optional<Tensor>& bias_, const std::string& reduction) {
    const Tensor bias = bias_.value_or(Tensor());
    const auto r = reduction_of(reduction);
    check_loss(x, weight, target, bias);
    check_tangents("linear_cross_entropy", x, weight, bias);
    if (at::GradMode::is_enabled() && (recorded(x) || recorded(weight) || recorded(bias)))
        return Loss::apply(x, weight, target, bias_, (int64_t)r);
    return std::get<0>(loss_call(x.contiguous(), weight.contiguous(), target.contiguous(), laid_out(bias), r, false));
}
std::tuple<Tensor, Tensor> linear_cross_entropy_forward(const Tensor& x, const Tensor& weight, const Tensor& target,
                                                        const std::optional<Tensor>& bias_, const std::string& reduction) {
    const Tensor bias = bias_.value_or(Tensor());
    check_loss(x, weight, target, bias);
    return loss_call(x.contiguous(), weight.contiguous(), target.contiguous(), laid_out(bias), reduction_of(reduction),
                     true);
}
std::tuple<std::optional<Tensor>, std::optional<Tensor>, std::optional<Tensor>> linear_cross_entropy_vjp(
    const Tensor& x, const Tensor& weight, const Tensor& target, const Tensor& lse, const Tensor& dloss,
    const std::optional<Tensor>& bias_, const std::string& reduction, std::array<bool, 3> want) {
    const Tensor bias = bias_.value_or(Tensor());
    const auto r = reduction_of(reduction);
    check_loss(x, weight, target, bias);
    check_like(lse, "lse", at::kFloat, target.sizes(), x);
    check_like(dloss, "dloss", at::kFloat, r == LAPSUM_REDUCE_NONE ? target.sizes() : at::IntArrayRef(), x);
    auto [dx, dw, db] = loss_vjp_call(x.contiguous(), weight.contiguous(), target.contiguous(), laid_out(bias),
                                      lse.contiguous(), dloss.contiguous(), r, want);
    return {maybe(dx), maybe(dw), maybe(db)};
}

// ---- rows in 8 bits ------------------------------------------------------------------

int64_t blocks_of(int64_t width) { return (width + LAPSUM_BLOCK8 - 1) / LAPSUM_BLOCK8; }

void check_rows8(const Tensor& values, const Tensor& scales, int64_t width, const char* name) {
    TORCH_CHECK_VALUE(values.is_cuda(), name, ".values must be on a GPU device (got ", values.device(), ")");
    TORCH_CHECK_VALUE(scales.device() == values.device(), name, ".scales must be on ", values.device(), " (got ",
                      scales.device(), ")");
    TORCH_CHECK_VALUE(values.scalar_type() == at::kFloat8_e4m3fn, name, ".values must be float8_e4m3fn (got ",
                      values.scalar_type(), ")");
    TORCH_CHECK_VALUE(scales.scalar_type() == at::kFloat8_e8m0fnu, name, ".scales must be float8_e8m0fnu (got ",
                      scales.scalar_type(), ")");
    TORCH_CHECK_VALUE(values.dim() >= 1 && width >= 0, name, " must have at least 1 dimension and no negative width");
    auto shape = values.sizes().vec();
    shape.back() = blocks_of(width) * LAPSUM_BLOCK8;
    TORCH_CHECK_VALUE(values.sizes() == at::IntArrayRef(shape), name, ".values must have a last dimension of ",
                      shape.back(), ", whole blocks of ", LAPSUM_BLOCK8, " for its width (got ", values.sizes(), ")");
    shape.back() = blocks_of(width);
    TORCH_CHECK_VALUE(scales.sizes() == at::IntArrayRef(shape), name, ".scales must have the shape ",
                      at::IntArrayRef(shape), " (got ", scales.sizes(), ")");
    TORCH_CHECK_VALUE(values.is_contiguous() && scales.is_contiguous(), name, " must be contiguous");
    TORCH_CHECK_VALUE((reinterpret_cast<uintptr_t>(values.data_ptr()) & 15) == 0, name, ".values must start on 16 bytes");
    TORCH_CHECK(!(at::GradMode::is_enabled() && (recorded(values) || recorded(scales))), name,
                " in 8 bits have no gradient: detach them");
}

std::tuple<Tensor, Tensor> quantize(const Tensor& x_) {
    check_any_rows(x_, "x");
    TORCH_CHECK(!(at::GradMode::is_enabled() && recorded(x_)), "expert_quantize has no gradient: detach x");
    check_tangents("expert_quantize", x_);
    const On on(x_);
    const Tensor x = x_.contiguous();
    const int64_t width = x.size(-1), rows = width ? x.numel() / width : 0;
    auto shape = x.sizes().vec();
    shape.back() = blocks_of(width) * LAPSUM_BLOCK8;
    Tensor values = at::empty(shape, x.options().dtype(at::kFloat8_e4m3fn));
    shape.back() = blocks_of(width);
    Tensor scales = at::empty(shape, x.options().dtype(at::kFloat8_e8m0fnu));
    check_ok(lapsum_expert_quantize(ptr<void>(x), type_of(x), rows, width, ptr<void>(values), ptr<void>(scales), on.stream),
             "lapsum_expert_quantize");
    return {values, scales};
}

at::ScalarType out_type(const py::object& dtype) {
    TORCH_CHECK_TYPE(THPDtype_Check(dtype.ptr()), "dtype must be a torch.dtype");
    const auto t = reinterpret_cast<THPDtype*>(dtype.ptr())->scalar_type;
    TORCH_CHECK_VALUE(row_type(t), "dtype must be float32, bfloat16 or float16 (got ", t, ")");
    return t;
}

Tensor dequantize(const Tensor& values, const Tensor& scales, int64_t width, const py::object& dtype) {
    check_rows8(values, scales, width, "rows");
    const auto t = out_type(dtype);
    const On on(values);
    auto shape = values.sizes().vec();
    shape.back() = width;
    Tensor x = at::empty(shape, values.options().dtype(t));
    check_ok(lapsum_expert_dequantize(ptr<void>(values), ptr<void>(scales), type_of(x), width ? x.numel() / width : 0,
                                      width, ptr<void>(x), on.stream),
             "lapsum_expert_dequantize");
    return x;
}

Tensor linear_fp8(const Tensor& xs, const Tensor& xs_scales, int64_t xs_width, const Tensor& weight,
                  const Tensor& weight_scales, int64_t width, const std::optional<Tensor>& bias_,
                  const std::string& activation, const py::object& dtype, int64_t experts, const Tensor& offsets,
                  const Tensor& order, const Tensor& place) {
    const Tensor bias = laid_out(bias_.value_or(Tensor()));
    const int act = act_of(activation);
    check_rows8(xs, xs_scales, xs_width, "xs");
    check_rows8(weight, weight_scales, width, "weight");
    const auto t = out_type(dtype);
    const Plan plan = make_plan(experts, offsets, order, place, xs);
    TORCH_CHECK_VALUE(weight.device() == xs.device(), "weight must be on ", xs.device(), " (got ", weight.device(), ")");
    TORCH_CHECK_VALUE(xs_width == width, "xs and weight must have the same width (got ", xs_width, " and ", width, ")");
    TORCH_CHECK_VALUE(width <= LAPSUM_MAX_WIDTH8, "xs must have a width of at most ", LAPSUM_MAX_WIDTH8, " (got ", width,
                      ")");
    TORCH_CHECK_VALUE(xs.dim() == 2 && xs.size(0) == plan.pairs(), "xs must have the rows [", plan.pairs(),
                      "] (got ", xs.sizes(), ")");
    TORCH_CHECK_VALUE(weight.dim() == 3 && weight.size(0) == experts, "weight must have the rows [", experts,
                      ", out] (got ", weight.sizes(), ")");
    const int64_t out = weight.size(1);
    if (bias.defined()) check_like(bias, "bias", t, {experts, out}, xs);
    TORCH_CHECK(!(at::GradMode::is_enabled() && recorded(bias)), "expert_linear_fp8 has no gradient: detach bias");
    check_tangents("expert_linear_fp8", bias);
    const On on(xs);
    Tensor ys = at::empty({xs.size(0), out}, xs.options().dtype(t));
    check_ok(lapsum_expert_linear_fp8(ptr<void>(xs), ptr<void>(xs_scales), ptr<void>(weight), ptr<void>(weight_scales),
                                      ptr<void>(bias), type_of(ys), xs.size(0), width, out, experts, plan.off(),
                                      (lapsum_act_t)act, ptr<void>(ys), on.stream),
             "lapsum_expert_linear_fp8");
    return ys;
}

}  // namespace

void define_layers(py::module_& m) {
    m.def("layer_norm", &layer_norm);
    m.def("layer_norm_forward", &layer_norm_forward);
    m.def("layer_norm_vjp", &layer_norm_vjp);
    m.def("linear_cross_entropy", &linear_cross_entropy);
    m.def("linear_cross_entropy_forward", &linear_cross_entropy_forward);
    m.def("linear_cross_entropy_vjp", &linear_cross_entropy_vjp);
    m.def("quantize", &quantize);
    m.def("dequantize", &dequantize);
    m.def("linear_fp8", &linear_fp8);
}

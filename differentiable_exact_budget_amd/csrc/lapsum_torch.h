// What the torch modules over the C ABIs share: argument checks, statuses, and
// the device and stream of a call.
#pragma once
#include <ATen/TracerMode.h>
#include <c10/core/AutogradState.h>
#include <c10/core/DeviceGuard.h>
#include <c10/hip/HIPStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/extension.h>

#include <optional>
#include <tuple>

#include "lapsum_experts.h"

namespace lapsum_torch {

using at::Tensor;
using torch::autograd::AutogradContext;
using torch::autograd::variable_list;

// ---- checks -------------------------------------------------------------------

inline const char* const kActs[] = {"none", "relu", "silu", "gelu"};

inline int act_of(const std::string& a) {
    for (int i = 0; i < 4; ++i)
        if (a == kActs[i]) return i;
    TORCH_CHECK_VALUE(false, "activation must be one of none, relu, silu, gelu (got '", a, "')");
}

inline std::optional<lapsum_dtype_t> row_type(at::ScalarType t) {
    if (t == at::kFloat) return LAPSUM_F32;
    if (t == at::kBFloat16) return LAPSUM_BF16;
    if (t == at::kHalf) return LAPSUM_F16;
    return std::nullopt;
}
inline lapsum_dtype_t type_of(const Tensor& x) { return *row_type(x.scalar_type()); }
// the type z is kept in
inline at::ScalarType z_type(const Tensor& xs) { return xs.scalar_type() == at::kFloat ? at::kFloat : at::kHalf; }

inline void check_place(const Tensor& x, const char* name, int64_t dims, const Tensor* like) {
    TORCH_CHECK_VALUE(x.is_cuda(), name, " must be on a GPU device (got ", x.device(), ")");
    TORCH_CHECK_VALUE(!like || x.device() == like->device(), name, " must be on ", like->device(), " (got ", x.device(),
                      ")");
    TORCH_CHECK_VALUE(x.dim() == dims, name, " must have ", dims, " dimensions (got ", x.dim(), ")");
    TORCH_CHECK_VALUE(x.is_contiguous(), name, " must be contiguous");
}
inline void check(const Tensor& x, const char* name, at::ScalarType t, int64_t dims, const Tensor* like = nullptr) {
    check_place(x, name, dims, like);
    TORCH_CHECK_VALUE(x.scalar_type() == t, name, " must be ", t, " (got ", x.scalar_type(), ")");
}
inline void check_rows(const Tensor& x, const char* name) {
    check_place(x, name, 2, nullptr);
    TORCH_CHECK_VALUE(row_type(x.scalar_type()), name, " must be float32, bfloat16 or float16 (got ", x.scalar_type(),
                      ")");
}
inline void check_shape(const Tensor& x, const char* name, at::IntArrayRef shape) {
    TORCH_CHECK_VALUE(x.sizes() == shape, name, " must have the shape ", shape, " (got ", x.sizes(), ")");
}
// A status of the C ABI, the package's LapsumError in Python.
struct StatusError : std::runtime_error {
    int code;
    const char* where;
    StatusError(int rc, const char* name)
        : std::runtime_error(std::string(name) + ": " + lapsum_status_string((lapsum_status_t)rc)),
          code(rc),
          where(name) {}
};
inline void check_ok(int rc, const char* name) {
    if (rc != LAPSUM_OK) throw StatusError(rc, name);
}
// There are gradients in reverse mode only: a forward-mode tangent would be
// dropped where nothing requires a gradient.
template <class... Tensors>
void check_tangents(const char* name, const Tensors&... inputs) {
    if (!c10::AutogradState::get_tls_state().get_fw_grad_mode()) return;
    const bool any = ((inputs.defined() && inputs._fw_grad(/*level=*/0).defined()) || ...);
    TORCH_CHECK(!any, name, " has no forward-mode derivative");
}
// The gradients are kernels of their own, not recorded in turn.
inline void check_once(const char* name) {
    TORCH_CHECK(!at::GradMode::is_enabled(), name, " is not differentiable twice (create_graph)");
}

inline bool recorded(const Tensor& x) { return x.defined() && x.requires_grad(); }

template <class T>
T* ptr(const Tensor& x) {
    return x.defined() ? static_cast<T*>(x.data_ptr()) : nullptr;
}

// The device of x made current, and its current stream.
struct On {
    c10::DeviceGuard guard;
    lapsum_stream_t stream;
    explicit On(const Tensor& x)
        : guard(x.device()),
          stream(reinterpret_cast<lapsum_stream_t>(c10::hip::getCurrentHIPStream(x.device().index()).stream())) {
        // a trace would keep the outputs' allocation and none of the work
        TORCH_CHECK(!at::tracer::impl::is_dispatch_enabled(), "these operators cannot be traced (torch.jit.trace)");
    }
};

// A plan's arrays as they travel through autograd.
struct Plan {
    int64_t experts;
    Tensor offsets, place;
    int64_t tokens() const { return place.size(0); }
    int64_t slots() const { return place.size(1); }
    int64_t pairs() const { return place.numel(); }
    const int32_t* off() const { return ptr<const int32_t>(offsets); }
    const int32_t* at() const { return ptr<const int32_t>(place); }
};
inline Plan make_plan(int64_t experts, const Tensor& offsets, const Tensor& order, const Tensor& place, const Tensor& like) {
    check(offsets, "plan.offsets", at::kInt, 1, &like);
    check(order, "plan.order", at::kInt, 1, &like);
    check(place, "plan.place", at::kInt, 2, &like);
    check_shape(offsets, "plan.offsets", {experts + 1});
    check_shape(order, "plan.order", {place.numel()});
    return {experts, offsets, place};
}
inline std::optional<Tensor> maybe(const Tensor& t) { return t.defined() ? std::optional<Tensor>(t) : std::nullopt; }

}  // namespace lapsum_torch

// C ABI of the expert operators: argument checks and launches.  No call
// allocates, waits or keeps state.
#include <cmath>

#include "lapsum_expert_ops.h"
#include "lapsum_experts.h"

using namespace lapsum;

namespace {

// rows, and a product's widths: the ends of tiles and of a sum's steps stay
// below 2^31
constexpr int64_t kRowsMax = LAPSUM_MAX_PAIRS;
constexpr int64_t kWidthMax = 0x7FFFFFFFll;

hipStream_t stream_of(lapsum_stream_t s) { return reinterpret_cast<hipStream_t>(s); }
lapsum_status_t launched() { return hipGetLastError() == hipSuccess ? LAPSUM_OK : LAPSUM_ERR_HIP; }

bool good_dtype(int d) { return d == LAPSUM_F32 || d == LAPSUM_BF16 || d == LAPSUM_F16; }
bool good_act(int a) { return a >= LAPSUM_ACT_NONE && a <= LAPSUM_ACT_GELU; }
bool good_experts(int64_t e) { return e >= 1 && e <= LAPSUM_MAX_EXPERTS; }
bool good_tokens(int64_t tokens, int64_t slots) {
    return tokens >= 0 && slots >= 1 && slots <= LAPSUM_MAX_SLOTS && tokens <= kRowsMax / slots;
}
bool good_width(int64_t width) { return width >= 0 && width <= kWidthMax; }
bool good_product(int64_t rows, int64_t in, int64_t out) {
    for (const int64_t n : {rows, in, out})
        if (n < 0 || n > kRowsMax) return false;
    return true;
}

// dz of the 16-byte aligned scratch, then the bias gradient's partial sums
struct VjpScratch {
    size_t dz = 0, part = 0;
    size_t bytes() const { return dz + part; }
};
VjpScratch vjp_scratch(int dtype, int64_t rows, int64_t out, int64_t experts, int act, bool want_dbias) {
    VjpScratch s;
    if (act != LAPSUM_ACT_NONE) s.dz = ((size_t)rows * (size_t)out * dtype_size(dtype) + 255) & ~(size_t)255;
    if (want_dbias) s.part = sizeof(float) * (size_t)max_row_tiles<kDzRows>(rows, (int)experts) * (size_t)out;
    return s;
}

}  // namespace

extern "C" {

lapsum_status_t lapsum_expert_topk(const float* gates, int64_t tokens, int64_t experts, int64_t slots, float floor,
                                   int32_t normalize, int32_t* ids, float* weights, float* sums,
                                   lapsum_stream_t stream) {
    if (!good_experts(experts) || !good_tokens(tokens, slots) || slots > experts || std::isnan(floor))
        return LAPSUM_ERR_INVALID_ARGUMENT;
    if (tokens > 0 && (!gates || !ids || !weights || (normalize && !sums))) return LAPSUM_ERR_INVALID_ARGUMENT;
    if (tokens == 0) return LAPSUM_OK;
    launch_expert_topk(gates, tokens, (int)experts, (int)slots, floor, ids, weights, normalize ? sums : nullptr,
                       stream_of(stream));
    return launched();
}

lapsum_status_t lapsum_expert_topk_vjp(const int32_t* ids, const float* weights, const float* dweights,
                                       const float* sums, int64_t tokens, int64_t experts, int64_t slots,
                                       int32_t normalize, float* dgates, lapsum_stream_t stream) {
    if (!good_experts(experts) || !good_tokens(tokens, slots) || slots > experts) return LAPSUM_ERR_INVALID_ARGUMENT;
    if (tokens > 0 && (!ids || !dweights || !dgates || (normalize && (!weights || !sums))))
        return LAPSUM_ERR_INVALID_ARGUMENT;
    if (tokens == 0) return LAPSUM_OK;
    launch_expert_topk_vjp(ids, weights, dweights, normalize ? sums : nullptr, tokens, (int)experts, (int)slots,
                           dgates, stream_of(stream));
    return launched();
}

size_t lapsum_expert_sort_scratch_bytes(int64_t pairs, int64_t experts) {
    if (pairs < 0 || pairs > kRowsMax || !good_experts(experts)) return 0;
    return expert_sort_scratch(pairs, (int)experts);
}

lapsum_status_t lapsum_expert_sort(const int32_t* ids, int64_t pairs, int64_t experts, int32_t* offsets,
                                   int32_t* order, int32_t* place, void* scratch, lapsum_stream_t stream) {
    if (pairs < 0 || pairs > kRowsMax || !good_experts(experts) || !offsets) return LAPSUM_ERR_INVALID_ARGUMENT;
    if (pairs > 0 && (!ids || !order || !place)) return LAPSUM_ERR_INVALID_ARGUMENT;
    if (expert_sort_scratch(pairs, (int)experts) && (!scratch || !aligned16(scratch)))
        return LAPSUM_ERR_INVALID_ARGUMENT;
    launch_expert_sort(ids, pairs, (int)experts, offsets, order, place, (uint32_t*)scratch, stream_of(stream));
    return launched();
}

lapsum_status_t lapsum_expert_dispatch(const void* x, lapsum_dtype_t dtype, int64_t tokens, int64_t slots,
                                       int64_t width, int64_t experts, const int32_t* offsets, const int32_t* place,
                                       void* xs, lapsum_stream_t stream) {
    if (!good_dtype(dtype) || !good_tokens(tokens, slots) || !good_width(width) || !good_experts(experts))
        return LAPSUM_ERR_INVALID_ARGUMENT;
    if (tokens == 0 || width == 0) return LAPSUM_OK;
    if (!x || !offsets || !place || !xs) return LAPSUM_ERR_INVALID_ARGUMENT;
    launch_dispatch(x, dtype, tokens, (int)slots, width, (int)experts, offsets, place, xs, stream_of(stream));
    return launched();
}

lapsum_status_t lapsum_expert_dispatch_vjp(const void* dxs, lapsum_dtype_t dtype, int64_t tokens, int64_t slots,
                                           int64_t width, const int32_t* place, void* dx, lapsum_stream_t stream) {
    if (!good_dtype(dtype) || !good_tokens(tokens, slots) || !good_width(width)) return LAPSUM_ERR_INVALID_ARGUMENT;
    if (tokens == 0 || width == 0) return LAPSUM_OK;
    if (!dxs || !place || !dx) return LAPSUM_ERR_INVALID_ARGUMENT;
    launch_dispatch_vjp(dxs, dtype, tokens, (int)slots, width, place, dx, stream_of(stream));
    return launched();
}

lapsum_status_t lapsum_expert_combine(const void* ys, const float* weights, const void* residual, lapsum_dtype_t dtype,
                                      int64_t tokens, int64_t slots, int64_t width, const int32_t* place, void* out,
                                      lapsum_stream_t stream) {
    if (!good_dtype(dtype) || !good_tokens(tokens, slots) || !good_width(width)) return LAPSUM_ERR_INVALID_ARGUMENT;
    if (tokens == 0 || width == 0) return LAPSUM_OK;
    if (!ys || !weights || !place || !out) return LAPSUM_ERR_INVALID_ARGUMENT;
    launch_combine(ys, weights, residual, dtype, tokens, (int)slots, width, place, out, stream_of(stream));
    return launched();
}

lapsum_status_t lapsum_expert_combine_vjp(const void* ys, const float* weights, const void* dout, lapsum_dtype_t dtype,
                                          int64_t tokens, int64_t slots, int64_t width, int64_t experts,
                                          const int32_t* offsets, const int32_t* place, void* dys, float* dweights,
                                          lapsum_stream_t stream) {
    if (!good_dtype(dtype) || !good_tokens(tokens, slots) || !good_width(width) || !good_experts(experts) ||
        (!dys && !dweights))
        return LAPSUM_ERR_INVALID_ARGUMENT;
    if (tokens == 0) return LAPSUM_OK;
    if (!weights || !place || !offsets || (width > 0 && (!dout || (dweights && !ys))))
        return LAPSUM_ERR_INVALID_ARGUMENT;
    launch_combine_vjp(ys, weights, dout, dtype, tokens, (int)slots, width, (int)experts, offsets, place, dys,
                       dweights, stream_of(stream));
    return launched();
}

lapsum_status_t lapsum_expert_linear(const void* xs, const void* weight, const void* bias, lapsum_dtype_t dtype,
                                     int64_t rows, int64_t in, int64_t out, int64_t experts, const int32_t* offsets,
                                     lapsum_act_t act, void* ys, void* z_out, lapsum_stream_t stream) {
    if (!good_dtype(dtype) || !good_act(act) || !good_product(rows, in, out) ||
        !good_experts(experts))
        return LAPSUM_ERR_INVALID_ARGUMENT;
    if (rows == 0 || out == 0) return LAPSUM_OK;
    if (!offsets || !ys || (in > 0 && (!xs || !weight))) return LAPSUM_ERR_INVALID_ARGUMENT;
    LinearArgs g{xs, weight, bias, ys, act == LAPSUM_ACT_NONE ? nullptr : z_out, offsets, (int)rows, (int)experts,
                 (int)in, (int)out, act};
    launch_expert_product(kFormY, dtype, g, stream_of(stream));
    return launched();
}

size_t lapsum_expert_linear_vjp_scratch_bytes(lapsum_dtype_t dtype, int64_t rows, int64_t in, int64_t out,
                                              int64_t experts, lapsum_act_t act, int32_t want_dbias) {
    if (!good_dtype(dtype) || !good_act(act) || !good_product(rows, in, out) ||
        !good_experts(experts))
        return 0;
    return vjp_scratch(dtype, rows, out, experts, act, want_dbias != 0).bytes();
}

lapsum_status_t lapsum_expert_linear_vjp(const void* xs, const void* weight, const void* z, const void* dys,
                                         lapsum_dtype_t dtype, int64_t rows, int64_t in, int64_t out, int64_t experts,
                                         const int32_t* offsets, lapsum_act_t act, void* dxs, void* dweight,
                                         void* dbias, void* scratch, lapsum_stream_t stream) {
    if (!good_dtype(dtype) || !good_act(act) || !good_product(rows, in, out) ||
        !good_experts(experts) || (!dxs && !dweight && !dbias) || !offsets)
        return LAPSUM_ERR_INVALID_ARGUMENT;
    const bool work = rows > 0 && out > 0;
    if (work && (!dys || (act != LAPSUM_ACT_NONE && !z) || (dxs && in > 0 && !weight) || (dweight && in > 0 && !xs)))
        return LAPSUM_ERR_INVALID_ARGUMENT;
    const VjpScratch s = vjp_scratch(dtype, rows, out, experts, act, dbias != nullptr);
    if (s.bytes() && (!scratch || !aligned16(scratch))) return LAPSUM_ERR_INVALID_ARGUMENT;
    hipStream_t st = stream_of(stream);
    const int P = (int)rows, E = (int)experts, N = (int)out;
    void* dz = act == LAPSUM_ACT_NONE ? nullptr : scratch;
    float* part = dbias ? reinterpret_cast<float*>(static_cast<char*>(scratch) + s.dz) : nullptr;
    launch_expert_dz(z, dys, dtype, act, offsets, P, E, N, dz, part, st);
    if (dbias) launch_expert_dbias(part, dtype, offsets, P, E, N, dbias, st);
    LinearArgs g{dz ? dz : dys, weight, nullptr, dxs, nullptr, offsets, P, E, (int)in, N, LAPSUM_ACT_NONE};
    if (dxs) launch_expert_product(kFormDx, dtype, g, st);
    g.b = xs;
    g.c = dweight;
    if (dweight) launch_expert_product(kFormDw, dtype, g, st);
    return launched();
}

}  // extern "C"

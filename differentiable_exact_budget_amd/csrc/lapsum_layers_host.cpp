// C ABI of the norm, the loss and the experts' products in 8 bits: argument
// checks and launches.  No call allocates, waits or keeps state.
#include "lapsum_layers.h"

#include "lapsum_experts8.h"
#include "lapsum_layer_ops.h"

using namespace lapsum;

namespace {

hipStream_t stream_of(lapsum_stream_t s) { return reinterpret_cast<hipStream_t>(s); }
lapsum_status_t launched() { return hipGetLastError() == hipSuccess ? LAPSUM_OK : LAPSUM_ERR_HIP; }

bool good_dtype(int d) { return d == LAPSUM_F32 || d == LAPSUM_BF16 || d == LAPSUM_F16; }
bool good_count(int64_t n) { return n >= 0 && n <= LAPSUM_MAX_PAIRS; }

bool good_norm(int dtype, int wtype, int64_t rows, int64_t width) {
    return good_dtype(dtype) && (wtype == dtype || wtype == LAPSUM_F32) && good_count(rows) && width >= 1 &&
           width <= 0x7FFFFFFFll;
}

bool good_loss(int dtype, int64_t rows, int64_t vocab, int64_t width) {
    for (const int64_t n : {rows, vocab, width})
        if (n < 0 || n > LAPSUM_MAX_LOSS_SIDE) return false;
    return good_dtype(dtype) && vocab >= 1;
}
bool good_reduction(int r) { return r >= LAPSUM_REDUCE_NONE && r <= LAPSUM_REDUCE_MEAN; }

LossArgs loss_args(const void* x, const void* w, const void* bias, const int64_t* target, int64_t rows, int64_t vocab,
                   int64_t width) {
    return {x, w, bias, target, (int)rows, (int)vocab, (int)width};
}

}  // namespace

extern "C" {

lapsum_status_t lapsum_layer_norm(const void* x, const void* weight, const void* bias, lapsum_dtype_t dtype,
                                  lapsum_dtype_t wtype, int64_t rows, int64_t width, float eps, void* y, float* mean,
                                  float* rstd, lapsum_stream_t stream) {
    if (!good_norm(dtype, wtype, rows, width) || !(eps >= 0.0f)) return LAPSUM_ERR_INVALID_ARGUMENT;
    if (rows == 0) return LAPSUM_OK;
    if (!x || !y) return LAPSUM_ERR_INVALID_ARGUMENT;
    launch_norm(x, weight, bias, dtype, wtype, rows, width, eps, y, mean, rstd, stream_of(stream));
    return launched();
}

size_t lapsum_layer_norm_vjp_scratch_bytes(lapsum_dtype_t dtype, int64_t rows, int64_t width) {
    return good_norm(dtype, dtype, rows, width) ? norm_vjp_scratch(dtype, rows, width) : 0;
}

lapsum_status_t lapsum_layer_norm_vjp(const void* x, const void* weight, const float* mean, const float* rstd,
                                      const void* dy, lapsum_dtype_t dtype, lapsum_dtype_t wtype, int64_t rows,
                                      int64_t width, void* dx, void* dweight, void* dbias, void* scratch,
                                      lapsum_stream_t stream) {
    if (!good_norm(dtype, wtype, rows, width) || (!dx && !dweight && !dbias)) return LAPSUM_ERR_INVALID_ARGUMENT;
    if (rows > 0 && (!x || !mean || !rstd || !dy)) return LAPSUM_ERR_INVALID_ARGUMENT;
    if ((dweight || dbias) && (!scratch || !aligned16(scratch))) return LAPSUM_ERR_INVALID_ARGUMENT;
    if (rows == 0 && !dweight && !dbias) return LAPSUM_OK;
    launch_norm_vjp(x, weight, mean, rstd, dy, dtype, wtype, rows, width, dx, dweight, dbias, (float*)scratch,
                    stream_of(stream));
    return launched();
}

size_t lapsum_linear_cross_entropy_scratch_bytes(lapsum_dtype_t dtype, int64_t rows, int64_t vocab, int64_t width) {
    if (!good_loss(dtype, rows, vocab, width)) return 0;
    const LossArgs g = loss_args(nullptr, nullptr, nullptr, nullptr, rows, vocab, width);
    // whatever the addresses' alignment
    const size_t any = loss_any_parts(dtype, g).bytes;
    return loss_tile_takes(dtype, g) ? std::max(any, loss_tile_parts(g).bytes) : any;
}

lapsum_status_t lapsum_linear_cross_entropy(const void* x, const void* weight, const void* bias,
                                            const int64_t* target, lapsum_dtype_t dtype, int64_t rows, int64_t vocab,
                                            int64_t width, lapsum_reduction_t reduction, float* loss, float* lse,
                                            void* scratch, lapsum_stream_t stream) {
    if (!good_loss(dtype, rows, vocab, width) || !good_reduction(reduction)) return LAPSUM_ERR_INVALID_ARGUMENT;
    if (rows == 0 && reduction == LAPSUM_REDUCE_NONE) return LAPSUM_OK;
    if (!loss) return LAPSUM_ERR_INVALID_ARGUMENT;
    if (rows > 0 && (!target || (width > 0 && (!x || !weight)) || !scratch || !aligned16(scratch)))
        return LAPSUM_ERR_INVALID_ARGUMENT;
    const LossArgs g = loss_args(x, weight, bias, target, rows, vocab, width);
    hipStream_t st = stream_of(stream);
    char* s = static_cast<char*>(scratch);
    float* each = loss;
    if (rows > 0) {
        const bool tile = loss_tile_takes(dtype, g);
        const LossParts p = tile ? loss_tile_parts(g) : loss_any_parts(dtype, g);
        if (tile) launch_loss_tile(dtype, g, p, s, st);
        else launch_loss_any(dtype, g, p, s, st);
        if (reduction != LAPSUM_REDUCE_NONE) each = reinterpret_cast<float*>(s + p.loss);
        launch_loss_rows(g, p, s, each, lse, st);
    }
    if (reduction != LAPSUM_REDUCE_NONE) launch_loss_reduce(g, each, reduction, loss, st);
    return launched();
}

size_t lapsum_linear_cross_entropy_vjp_scratch_bytes(lapsum_dtype_t dtype, int64_t rows, int64_t vocab,
                                                     int64_t width) {
    if (!good_loss(dtype, rows, vocab, width)) return 0;
    const LossArgs g = loss_args(nullptr, nullptr, nullptr, nullptr, rows, vocab, width);
    const size_t any = loss_any_plan(dtype, g).bytes;
    return loss_tile_takes(dtype, g) ? std::max(any, loss_tile_plan(g).bytes) : any;
}

lapsum_status_t lapsum_linear_cross_entropy_vjp(const void* x, const void* weight, const void* bias,
                                                const int64_t* target, const float* lse, const float* dloss,
                                                lapsum_dtype_t dtype, int64_t rows, int64_t vocab, int64_t width,
                                                lapsum_reduction_t reduction, void* dx, void* dweight, void* dbias,
                                                void* scratch, lapsum_stream_t stream) {
    if (!good_loss(dtype, rows, vocab, width) || !good_reduction(reduction) || (!dx && !dweight && !dbias))
        return LAPSUM_ERR_INVALID_ARGUMENT;
    if (!scratch || !aligned16(scratch)) return LAPSUM_ERR_INVALID_ARGUMENT;
    if (rows > 0 && (!target || !lse || !dloss || (width > 0 && (!x || !weight)))) return LAPSUM_ERR_INVALID_ARGUMENT;
    const LossArgs g = loss_args(x, weight, bias, target, rows, vocab, width);
    hipStream_t st = stream_of(stream);
    char* s = static_cast<char*>(scratch);
    const bool tile = loss_tile_takes(dtype, g) && aligned16(dx) && aligned16(dweight);
    const LossVjpPlan p = tile ? loss_tile_plan(g) : loss_any_plan(dtype, g);
    launch_loss_grad_rows(dtype, g, dloss, reduction, reinterpret_cast<float*>(s + p.g), dweight ? s + p.x : nullptr, st);
    if (tile) launch_loss_tile_vjp(dtype, g, p, lse, s, dx, dweight, dbias, st);
    else launch_loss_any_vjp(dtype, g, p, lse, s, dx, dweight, dbias, st);
    return launched();
}

lapsum_status_t lapsum_expert_quantize(const void* x, lapsum_dtype_t dtype, int64_t rows, int64_t width, void* values,
                                       void* scales, lapsum_stream_t stream) {
    if (!good_dtype(dtype) || !good_count(rows) || !good_count(width)) return LAPSUM_ERR_INVALID_ARGUMENT;
    if (rows == 0 || width == 0) return LAPSUM_OK;
    if (!x || !values || !scales || !aligned16(values)) return LAPSUM_ERR_INVALID_ARGUMENT;
    launch_quantize(x, dtype, rows, width, (uint8_t*)values, (uint8_t*)scales, stream_of(stream));
    return launched();
}

lapsum_status_t lapsum_expert_dequantize(const void* values, const void* scales, lapsum_dtype_t dtype, int64_t rows,
                                         int64_t width, void* x, lapsum_stream_t stream) {
    if (!good_dtype(dtype) || !good_count(rows) || !good_count(width)) return LAPSUM_ERR_INVALID_ARGUMENT;
    if (rows == 0 || width == 0) return LAPSUM_OK;
    if (!x || !values || !scales || !aligned16(values)) return LAPSUM_ERR_INVALID_ARGUMENT;
    launch_dequantize((const uint8_t*)values, (const uint8_t*)scales, dtype, rows, width, x, stream_of(stream));
    return launched();
}

lapsum_status_t lapsum_expert_linear_fp8(const void* xs, const void* xs_scales, const void* weight,
                                         const void* weight_scales, const void* bias, lapsum_dtype_t dtype,
                                         int64_t rows, int64_t width, int64_t out, int64_t experts,
                                         const int32_t* offsets, lapsum_act_t act, void* ys, lapsum_stream_t stream) {
    if (!good_dtype(dtype) || act < LAPSUM_ACT_NONE || act > LAPSUM_ACT_GELU || !good_count(rows) ||
        !good_count(out) || width < 0 || width > LAPSUM_MAX_WIDTH8 || experts < 1 || experts > LAPSUM_MAX_EXPERTS)
        return LAPSUM_ERR_INVALID_ARGUMENT;
    if (rows == 0 || out == 0) return LAPSUM_OK;
    if (expert_linear8_tiles(rows, experts, out) > LAPSUM_MAX_TILES8) return LAPSUM_ERR_INVALID_ARGUMENT;
    if (!offsets || !ys) return LAPSUM_ERR_INVALID_ARGUMENT;
    if (width > 0 && (!xs || !xs_scales || !weight || !weight_scales || !aligned16(xs) || !aligned16(weight)))
        return LAPSUM_ERR_INVALID_ARGUMENT;
    const Linear8Args g{(const uint8_t*)xs, (const uint8_t*)xs_scales, (const uint8_t*)weight,
                        (const uint8_t*)weight_scales, bias, ys, offsets, (int)rows, (int)experts,
                        (int)ceil_div(width, kBlock8), (int)out, act};
    launch_expert_linear8(dtype, g, stream_of(stream));
    return launched();
}

}  // extern "C"

// Launchers of the operators around a routed layer (each defined next to its
// kernels): layer norm, the loss over a vocabulary, 8-bit rows.
#pragma once
#include <algorithm>

#include "lapsum_expert_ops.h"

namespace lapsum {

// lapsum_norm.hip.  mean, rstd may be null in the forward pass; dx, and both
// dweight and dbias, in the backward pass, whose part has norm_vjp_scratch bytes.
void launch_norm(const void* x, const void* weight, const void* bias, int dtype, int wtype, long long rows, long long D,
                 float eps, void* y, float* mean, float* rstd, hipStream_t st);
size_t norm_vjp_scratch(int dtype, long long rows, long long D);
void launch_norm_vjp(const void* x, const void* weight, const float* mean, const float* rstd, const void* dy, int dtype,
                     int wtype, long long rows, long long D, void* dx, void* dweight, void* dbias, float* part,
                     hipStream_t st);

// The loss: rows x[T, D], a vocabulary's weights w[V, D] and bias (may be
// null), targets (a row whose target is outside [0, V) is ignored).
struct LossArgs {
    const void* x;
    const void* w;
    const void* bias;
    const int64_t* target;
    int T, V, D;
};
enum Reduction : int { kReduceNone = 0, kReduceSum = 1, kReduceMean = 2 };

// The gradient's pieces of the vocabulary, and its scratch (all offsets in
// bytes, each on 256): g[T] and its factor, x[T, D] of the rows that have a
// gradient, d[T, ld] of one piece, fp32 rows [, ld] whose sum is db's piece (d
// before its rounding), dx's partial sums [shares, T, D] (where there is more than
// one).
struct LossVjpPlan {
    int width;   // columns of a piece
    int ld;      // elements between rows of d: the width on a multiple of 8
    int pieces;
    int shares;  // of dx's sum over a piece
    size_t g, x, d, db, dx, bytes;
};

// lapsum_entropy.hip: every type, width and alignment, and the steps around the
// products
struct LossParts {
    int parts;           // partial (maximum, sum) pairs of a row
    size_t pairs, zt, loss, bytes;  // scratch, as above; pairs[parts][T]
    size_t logits;       // [T, width] of one piece, where they are formed by themselves (else 0)
    int width;
};
LossParts loss_any_parts(int dtype, const LossArgs& g);
LossVjpPlan loss_any_plan(int dtype, const LossArgs& g);
void launch_loss_any(int dtype, const LossArgs& g, const LossParts& p, char* scratch, hipStream_t st);
void launch_loss_any_vjp(int dtype, const LossArgs& g, const LossVjpPlan& p, const float* lse, char* scratch, void* dx,
                         void* dw, void* db, hipStream_t st);
// lse and, with loss (may be null), the rows' losses; then their sum or mean
void launch_loss_rows(const LossArgs& g, const LossParts& p, char* scratch, float* loss, float* lse, hipStream_t st);
void launch_loss_reduce(const LossArgs& g, const float* loss, int reduction, float* out, hipStream_t st);
// g[t] over the largest, and what results are multiplied by behind it; x's rows,
// zeros for those without a gradient, to `live` (may be null)
void launch_loss_grad_rows(int dtype, const LossArgs& g, const float* dloss, int reduction, float* rows, void* live,
                           hipStream_t st);
// db of n columns from their partial rows
void launch_loss_db(int dtype, const float* part, int ld, int rows, int n, const float* unscale, void* db,
                    hipStream_t st);
void launch_loss_dx(int dtype, const float* part, int shares, long long n, const float* unscale, void* dx,
                    hipStream_t st);

// lapsum_entropy_tile.hip: 16-bit rows whose width and addresses are on 16 bytes
bool loss_tile_takes(int dtype, const LossArgs& g);
LossParts loss_tile_parts(const LossArgs& g);
LossVjpPlan loss_tile_plan(const LossArgs& g);
void launch_loss_tile(int dtype, const LossArgs& g, const LossParts& p, char* scratch, hipStream_t st);
void launch_loss_tile_vjp(int dtype, const LossArgs& g, const LossVjpPlan& p, const float* lse, char* scratch,
                          void* dx, void* dw, void* db, hipStream_t st);

// lapsum_rows8.hip: rows in blocks of kBlock8 e4m3 values with an e8m0 scale
constexpr int kBlock8 = 128;
void launch_quantize(const void* x, int dtype, long long rows, long long D, uint8_t* q, uint8_t* scale, hipStream_t st);
void launch_dequantize(const uint8_t* q, const uint8_t* scale, int dtype, long long rows, long long D, void* x,
                       hipStream_t st);
// lapsum_expert_fp8.hip
struct Linear8Args {
    const uint8_t *a, *as;  // rows [P, blocks * 128], scales [P, blocks]
    const uint8_t *b, *bs;  // weights [E, out, blocks * 128], scales [E, out, blocks]
    const void* bias;       // [E, out], may be null
    void* c;                // [P, out]
    const int32_t* off;
    int P, E, blocks, out, act;
};
// the widest tiles of a launch, at most
inline long long expert_linear8_tiles(long long P, long long E, long long out) {
    return max_row_tiles<256>(P, (int)E) * ceil_div(out, 256);
}
void launch_expert_linear8(int dtype, const Linear8Args& g, hipStream_t st);

}  // namespace lapsum

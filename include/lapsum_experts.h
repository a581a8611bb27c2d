/*
 * lapsum_experts.h -- C ABI of the expert operators: from exact-budget gates
 * to routed tokens, through the experts' products, and back.
 *
 * The solver gives every token a row of gates p[E] with sum(p) equal to its
 * budget (lapsum_forward_batched).  These operators are the rest of a routed
 * layer:
 *
 *   topk      ids[t, j], w[t, j]: the m largest gates of row t
 *   sort      the T m (token, slot) pairs in expert order
 *   dispatch  xs[pos] = x[token of the pair at pos]
 *   linear    ys[pos] = act(xs[pos] W_e^T + b_e), e the expert of pos
 *   combine   out[t] = residual[t] + sum_j w[t, j] ys[place[t, j]]
 *
 * and their vector-Jacobian products.
 *
 * A plan is three int32 arrays that lapsum_expert_sort fills: offsets[E + 1]
 * (the pairs of expert e are the positions offsets[e] .. offsets[e + 1] - 1,
 * and offsets[E] is the number of pairs in use), order[T m] (the pair
 * t * m + j at a position, -1 past offsets[E]) and place[T * m] (the position
 * of a pair, -1 for an empty slot).  Every array that goes by positions has
 * T m rows whatever the ids are, so no call waits for a count; its rows past
 * offsets[E] are written as zeros.
 *
 * Conventions for every entry point:
 *  - Pointers are DEVICE pointers (gfx950) owned by the caller, rows
 *    contiguous; outputs alias nothing else.
 *  - All work is ordered on `stream`; nothing is allocated, nothing waits for
 *    the device, and no state is kept between calls.  Scratch memory, where a
 *    call needs some, is the caller's (its size is asked for first) and free
 *    again when the call's work on the stream is done.  Calls may be captured
 *    into a graph.
 *  - Argument errors are returned before anything is launched and nothing is
 *    written.  A call over no tokens or no columns writes what is left to
 *    write (an empty plan's offsets, an empty product's zeros) and returns
 *    LAPSUM_OK.
 *  - Results are the same every run: no sum's order depends on timing.
 *  - Sums are held in fp32; a result in a 16-bit type is rounded once.
 *  - Plans are only bounds-checked on the device: positions outside
 *    [0, T m) count as empty slots, offsets are clamped to [0, T m].  A plan
 *    that lapsum_expert_sort did not make gives wrong rows, not faults.
 *  - No exception crosses this ABI; calls may come from several host threads.
 */
#ifndef LAPSUM_EXPERTS_H_
#define LAPSUM_EXPERTS_H_

#include "lapsum.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Element types of rows and weights. */
typedef enum { LAPSUM_F32 = 0, LAPSUM_BF16 = 1, LAPSUM_F16 = 2 } lapsum_dtype_t;

/* Activations: z, max(z, 0), z / (1 + e^-z), z (1 + erf(z / sqrt 2)) / 2. */
typedef enum { LAPSUM_ACT_NONE = 0, LAPSUM_ACT_RELU = 1, LAPSUM_ACT_SILU = 2, LAPSUM_ACT_GELU = 3 } lapsum_act_t;

#define LAPSUM_MAX_EXPERTS 1024 /* experts of a row, at most */
#define LAPSUM_MAX_SLOTS 64     /* slots of a token, at most */
#define LAPSUM_MAX_PAIRS 0x7FFF0000 /* tokens * slots, and each side of a product, at most */

/*
 * The m largest gates of every row.
 *   gates   : fp32[tokens, experts].
 *   floor   : gates must be greater than this to be chosen (-inf: every gate
 *             but NaN and -inf; NaN is an argument error).
 *   ids     : int32[tokens, slots], in descending order of the gates, ties to
 *             the lowest expert; -1 where no gate above the floor is left.
 *   weights : fp32[tokens, slots], the chosen gates, 0 in empty slots; with
 *             normalize != 0 divided by their sum over the row (all 0 when
 *             that sum is not above 0).
 *   sums    : fp32[tokens], those sums, for the VJP; written when
 *             normalize != 0, and then required.
 * 1 <= experts <= LAPSUM_MAX_EXPERTS, 1 <= slots <= min(experts,
 * LAPSUM_MAX_SLOTS), tokens >= 0, tokens * slots <= LAPSUM_MAX_PAIRS.
 */
lapsum_status_t lapsum_expert_topk(const float* gates, int64_t tokens, int64_t experts, int64_t slots, float floor,
                                   int32_t normalize, int32_t* ids, float* weights, float* sums,
                                   lapsum_stream_t stream);

/* dgates[tokens, experts] (every element is written): dweights scattered to
 * the chosen experts, through the division when normalize != 0
 * (dgate_j = (dw_j - sum_i dw_i w_i) / sum; 0 where the weights were set to
 * 0).  The choice itself has no gradient.  ids, weights and sums are the
 * forward's; weights and sums are not read when normalize is 0. */
lapsum_status_t lapsum_expert_topk_vjp(const int32_t* ids, const float* weights, const float* dweights,
                                       const float* sums, int64_t tokens, int64_t experts, int64_t slots,
                                       int32_t normalize, float* dgates, lapsum_stream_t stream);

/*
 * The pairs in expert order: a stable counting sort, so the pairs of one
 * expert keep their order.
 *   ids     : int32[pairs]; an id outside [0, experts) is an empty slot.
 *   offsets : int32[experts + 1].
 *   order   : int32[pairs].    place: int32[pairs].
 *   scratch : lapsum_expert_sort_scratch_bytes(pairs, experts) bytes, 16-byte
 *             aligned; may be NULL when that is 0.
 * 0 <= pairs <= LAPSUM_MAX_PAIRS, 1 <= experts <= LAPSUM_MAX_EXPERTS.
 */
size_t lapsum_expert_sort_scratch_bytes(int64_t pairs, int64_t experts);
lapsum_status_t lapsum_expert_sort(const int32_t* ids, int64_t pairs, int64_t experts, int32_t* offsets,
                                   int32_t* order, int32_t* place, void* scratch, lapsum_stream_t stream);

/*
 * Token rows to their pairs' places.  x: dtype[tokens, width], xs:
 * dtype[tokens * slots, width].  tokens * slots <= LAPSUM_MAX_PAIRS, width <
 * 2^31.  The VJP sums a token's rows of dxs in the order of its slots.
 */
lapsum_status_t lapsum_expert_dispatch(const void* x, lapsum_dtype_t dtype, int64_t tokens, int64_t slots,
                                       int64_t width, int64_t experts, const int32_t* offsets, const int32_t* place,
                                       void* xs, lapsum_stream_t stream);
lapsum_status_t lapsum_expert_dispatch_vjp(const void* dxs, lapsum_dtype_t dtype, int64_t tokens, int64_t slots,
                                           int64_t width, const int32_t* place, void* dx, lapsum_stream_t stream);

/*
 * Weighted rows back to their tokens, summed in the order of the slots.
 *   ys       : dtype[tokens * slots, width].  weights: fp32[tokens, slots]
 *              (those of empty slots are not read into the sum, NaN or not).
 *   residual : dtype[tokens, width] or NULL.  out: dtype[tokens, width].
 * The VJP writes dys (dtype[tokens * slots, width]: w dout) and dweights
 * (fp32[tokens, slots]: <dout, ys>, 0 for empty slots); either may be NULL,
 * and ys may be NULL when dweights is.  The residual's gradient is dout.
 */
lapsum_status_t lapsum_expert_combine(const void* ys, const float* weights, const void* residual, lapsum_dtype_t dtype,
                                      int64_t tokens, int64_t slots, int64_t width, const int32_t* place, void* out,
                                      lapsum_stream_t stream);
lapsum_status_t lapsum_expert_combine_vjp(const void* ys, const float* weights, const void* dout, lapsum_dtype_t dtype,
                                          int64_t tokens, int64_t slots, int64_t width, int64_t experts,
                                          const int32_t* offsets, const int32_t* place, void* dys, float* dweights,
                                          lapsum_stream_t stream);

/*
 * Every expert's product over its rows: ys = act(z), z = xs W_e^T + b_e.
 *   xs     : dtype[rows, in].        weight: dtype[experts, out, in].
 *   bias   : dtype[experts, out] or NULL.
 *   ys     : dtype[rows, out].
 *   z_out  : NULL, or fp16 (fp32 for LAPSUM_F32)[rows, out]: z as the VJP
 *            wants it (not written past offsets[experts]).  z is kept in
 *            fp16 whatever the 16-bit type, infinite beyond its range: only
 *            the activation's slope is taken from it, which is 0 or 1 there.
 * rows, in and out <= LAPSUM_MAX_PAIRS.
 */
lapsum_status_t lapsum_expert_linear(const void* xs, const void* weight, const void* bias, lapsum_dtype_t dtype,
                                     int64_t rows, int64_t in, int64_t out, int64_t experts, const int32_t* offsets,
                                     lapsum_act_t act, void* ys, void* z_out, lapsum_stream_t stream);

/*
 * With dz = dys act'(z), rounded to dtype once: dxs = dz W_e, dweight_e =
 * dz^T xs over the rows of e, dbias_e = sum of dz over them (summed before
 * the rounding).  Experts without rows get zeros.
 *   z       : the forward's z_out; NULL when act is LAPSUM_ACT_NONE.
 *   dxs, dweight, dbias: dtype, shaped as xs, weight, bias; each may be NULL.
 *   scratch : lapsum_expert_linear_vjp_scratch_bytes(...) bytes, 16-byte
 *             aligned; may be NULL when that is 0.
 */
size_t lapsum_expert_linear_vjp_scratch_bytes(lapsum_dtype_t dtype, int64_t rows, int64_t in, int64_t out,
                                              int64_t experts, lapsum_act_t act, int32_t want_dbias);
lapsum_status_t lapsum_expert_linear_vjp(const void* xs, const void* weight, const void* z, const void* dys,
                                         lapsum_dtype_t dtype, int64_t rows, int64_t in, int64_t out, int64_t experts,
                                         const int32_t* offsets, lapsum_act_t act, void* dxs, void* dweight,
                                         void* dbias, void* scratch, lapsum_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* LAPSUM_EXPERTS_H_ */

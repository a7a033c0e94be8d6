/*
 * mp_block.h — C ABI of libmpadamw.so, third part: what a transformer block
 * computes between its matrix products, in training: RMS norm with the
 * residual's addition, rotary positions, the gated activation, each with its
 * backward pass; and activations kept in 8 bits, which the norm's and the
 * activation's forward passes write and their backward passes read.
 *
 * The conventions of mp_adamw.h and mp_train.h hold: device pointers owned by
 * the caller, every call only enqueues work on `stream`, arguments are checked
 * on the host before any launch, nothing is allocated; matrices are row-major
 * with contiguous rows, `*_stride` elements apart; elements are an mp_dtype_t,
 * widened to fp32, every sum is held in fp32, a result is rounded to nearest
 * even once; any row count, length, stride and element-aligned address is
 * accepted, and rows on 16-B boundaries of a multiple of 16 bytes run fastest.
 * Results are bit-identical on every run with the same arguments, sizes and
 * alignments on the same GPU model (no float atomics).
 *
 * An output may be the same matrix (address and stride) as an input of the same
 * element size where said; otherwise outputs overlap neither inputs nor one another.
 * Rows are read in whole aligned pieces of up to 16 bytes, which may hold bytes
 * beside them; those are not used.
 * Waits inside a kernel (RMS norm's) end after a second at most. Should one run out
 * (a fault of the GPU), every element that it touches is NaN.
 *
 * Rows in 8 bits: e4m3 values (1 sign, 4 exponent, 3 mantissa bits, bias 7, no
 * infinities, 448 the largest) and their scales, value = e4m3 * scale, as mp_scale8_t says:
 *  MP_SCALE_ROW    float[rows]: scale = max(amax / 448, 2^-126), amax the row's
 *                  largest magnitude; it and the quotients by it to a few fp32
 *                  roundings, so that a quotient next to the middle of two
 *                  e4m3 values may become either. A row that holds NaN or an
 *                  infinity has scale NaN and reads back as NaN throughout.
 *  MP_SCALE_BLOCK  uint8[rows, ceil(d / 32)], contiguous: for every 32 columns
 *                  (the last block may be shorter) a power of two, held as its
 *                  exponent + 127: the least one with amax <= 448 * scale, or
 *                  2^-127. 255 is NaN, as for a row. (In blocks whose largest
 *                  magnitude is above 1.75 times the largest power of two of
 *                  the element type, magnitudes are limited to 240 * scale, so that nothing
 *                  reads back above the type's range. For y8, made from fp32 values, that
 *                  type is fp32.)
 */
#ifndef MP_BLOCK_H
#define MP_BLOCK_H

#include "mp_train.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef enum mp_scale8 {
    MP_SCALE_ROW = 1,
    MP_SCALE_BLOCK = 2
} mp_scale8_t;

/* ---------------------------------------------------------------------------
 * RMS norm with the residual's addition, forward. Per row of d values:
 *
 *   h    = x + residual, rounded to `type` (h = x without a residual)
 *   rstd = 1 / sqrt(sum(h^2) / d + eps)
 *   y[j] = h[j] * rstd * weight[j]
 *
 * The norm is that of the rounded sum, so the backward pass, which reads the
 * stored h, differentiates what was computed.
 *
 *   y           [rows, d] of `type`, written; may be x or residual itself; NULL
 *               when y8 is given and no other form is wanted.
 *   h           [rows, d] of `type`, written when residual is given (the next
 *               residual); may be x or residual itself; NULL: not wanted.
 *   rstd        float[rows], written for the backward pass; may be NULL.
 *   y8          [rows, d], y in 8 bits (from its fp32 value) with y8_scale of
 *               kind y8_kind; NULL: not wanted.
 *   h8          [rows, d], h in 8 bits with h8_scale of kind MP_SCALE_BLOCK, for
 *               the backward pass; NULL: not wanted.
 *   x, residual [rows, d] of `type`; residual NULL: none.
 *   weight      [d] of `weight_type`; NULL: ones.
 *   rows >= 0 (0 is a no-op), d in [1, 2^24], eps finite and >= 0.
 * The sum of squares is fp32: a row whose sum is above 3.4e38 has rstd 0, and
 * squares below 2^-150 add nothing (with eps = 0 a row of such values, zeros among
 * them, has rstd infinity). For MP_SCALE_ROW the largest |h * weight| is taken
 * before it is multiplied by rstd: above 3.4e38 it makes the row NaN.
 * Errors: MP_ERR_NULL (also when no output is given), MP_ERR_ALIGN,
 *         MP_ERR_RANGE, MP_ERR_CUDA.
 * ------------------------------------------------------------------------- */
int mp_rmsnorm_forward(void* y, void* h, float* rstd, void* y8, void* y8_scale, void* h8, void* h8_scale,
                       const void* x, const void* residual, const void* weight, int64_t rows, int64_t d,
                       int64_t y_stride, int64_t h_stride, int64_t y8_stride, int64_t h8_stride, int64_t x_stride,
                       int64_t residual_stride, float eps, int32_t type, int32_t weight_type, int32_t y8_kind,
                       void* stream);

/* ---------------------------------------------------------------------------
 * RMS norm, backward. With xh = h * rstd and g = dy * weight:
 *
 *   dx[j]      = dh[j] + rstd * (g[j] - xh[j] * sum(g * xh) / d)     per row
 *   dweight[j] = sum over rows of dy[j] * xh[j]
 *
 *   dx          [rows, d] of `type`, written: the gradient of x and of the
 *               residual; may be dy, dh or (in `type`) h itself; NULL: not wanted.
 *   dweight     [d] of `weight_type` (for instance a range of the flat bf16
 *               gradient buffer), written, not added to; NULL: not wanted. The
 *               sums over rows are fp32, added in a fixed order and rounded
 *               once. With rows = 0 they are zero.
 *   dy          [rows, d] of `type`.
 *   dh          [rows, d] of `type`: the gradient that reaches h by its other
 *               uses; NULL: zero.
 *   h           [rows, d] of `type`; or, with h_scale, in 8 bits with scales of
 *               kind MP_SCALE_BLOCK.
 *   weight      [d] of `weight_type`; NULL: ones.
 *   rstd        float[rows], the forward pass's.
 *   workspace   device scratch of at least mp_rmsnorm_workspace_bytes(rows, d)
 *               bytes, 16-B aligned, not shared with another call in flight;
 *               may be NULL when dweight is.
 *   rows, d     as the forward pass.
 * Errors: MP_ERR_NULL, MP_ERR_ALIGN, MP_ERR_RANGE, MP_ERR_WORKSPACE,
 *         MP_ERR_CUDA.
 * ------------------------------------------------------------------------- */
size_t mp_rmsnorm_workspace_bytes(int64_t rows, int64_t d);

int mp_rmsnorm_backward(void* dx, void* dweight, const void* dy, const void* dh, const void* h, const void* h_scale,
                        const void* weight, const float* rstd, int64_t rows, int64_t d, int64_t dx_stride,
                        int64_t dy_stride, int64_t dh_stride, int64_t h_stride, int32_t type, int32_t weight_type,
                        void* workspace, size_t workspace_bytes, void* stream);

/* ---------------------------------------------------------------------------
 * Rotary positions. A pair (a, b) of a head's values that has frequency f, at
 * position p, becomes
 *
 *   (a cos(p f) - b sin(p f),  a sin(p f) + b cos(p f)) * factor
 *
 * and with inverse != 0 the same with -p f: the gradient of the rotation is its
 * inverse (with the same factor). Pair i of rotary_dim / 2: columns i and
 * i + rotary_dim / 2, or with interleaved != 0 columns 2 i and 2 i + 1. A head's
 * columns from rotary_dim on are copied.
 *
 * Frequencies are given in turns a position, as 64-bit fractions: turns[i] =
 * f / (2 pi) * 2^64, so that the product with any position is exact modulo one
 * turn, and far positions lose nothing.
 *
 *   q_out, q    [tokens, q_heads, head_dim] of `type`: token and head distances
 *               given, a head's values contiguous. q_out may be q itself (same
 *               distances), not k.
 *   k_out, k    the same with k_heads; unused when k_heads is 0. k_out is not q.
 *   turns       uint64[rotary_dim / 2], 8-B aligned, on the device.
 *   positions   [tokens] of `index_type`, any value (negative ones turn
 *               backwards); NULL: first_position + t.
 *   tokens in [0, 2^31 - 1] (0 is a no-op), q_heads and k_heads in [0, 1024], not
 *   both 0, head_dim in [2, 1024], rotary_dim even, in [2, head_dim], factor
 *   finite. Distances at least head_dim, and the one of tokens at least (heads -
 *   1) * the one of heads + head_dim or the other way round (heads outermost).
 * Errors: MP_ERR_NULL, MP_ERR_ALIGN, MP_ERR_RANGE, MP_ERR_CUDA.
 * ------------------------------------------------------------------------- */
int mp_rope(void* q_out, const void* q, void* k_out, const void* k, const uint64_t* turns, const void* positions,
            int64_t first_position, int64_t tokens, int32_t q_heads, int32_t k_heads, int32_t head_dim,
            int32_t rotary_dim, int64_t q_out_token_stride, int64_t q_out_head_stride, int64_t q_token_stride,
            int64_t q_head_stride, int64_t k_out_token_stride, int64_t k_out_head_stride, int64_t k_token_stride,
            int64_t k_head_stride, float factor, int32_t interleaved, int32_t inverse, int32_t type,
            int32_t index_type, void* stream);

/* How the frequencies base^(-2 i / rotary_dim) are changed for contexts `factor`
 * times as long as the `context` positions trained with. */
typedef enum mp_rope_kind {
    MP_ROPE_NONE = 0,   /* not at all */
    MP_ROPE_LINEAR = 1, /* every frequency / factor */
    MP_ROPE_BASE = 2,   /* base * factor^(r / (r - 2)), r = rotary_dim: the slowest pair / factor, the fastest kept */
    MP_ROPE_BANDS = 3,  /* with u = context f / (2 pi), a pair's turns in the context: s = (u - low) / (high - low)
                         * limited to [0, 1]; f * ((1 - s) / factor + s) */
    MP_ROPE_RAMP = 4    /* by the pair's index i: i(u) = r ln(context / (2 pi u)) / (2 ln base), lo = floor(i(high)) >= 0,
                         * hi = ceil(i(low)) <= r - 1, s = (i - lo) / max(hi - lo, 0.001) limited to [0, 1];
                         * f * (s / factor + 1 - s), and results times 0.1 ln(factor) + 1 */
} mp_rope_kind_t;

typedef struct mp_rope_scaling {
    int32_t kind;     /* mp_rope_kind_t */
    int32_t reserved; /* 0 */
    double factor;    /* >= 1 */
    double context;   /* > 0 (BANDS and RAMP) */
    double low, high; /* 0 < low < high (BANDS and RAMP) */
} mp_rope_scaling_t;

/* Host only: turns[rotary_dim / 2] (host memory, to be copied to the device) for
 * base > 1 and a scaling (NULL: none), and in *factor (may be NULL) what mp_rope
 * takes as its factor. Errors: MP_ERR_NULL, MP_ERR_RANGE. */
int mp_rope_frequencies(uint64_t* turns, float* factor, int32_t rotary_dim, double base,
                        const mp_rope_scaling_t* scaling);

/* ---------------------------------------------------------------------------
 * The gated activation, forward: y = act(gate) * up, or act(gate) without up.
 *
 *   MP_ACT_SILU   act(a) = a / (1 + exp(-a))
 *   MP_ACT_GELU   act(a) = a / 2 * (1 + tanh(sqrt(2 / pi) (a + 0.044715 a^3)))
 *
 *   y           [rows, d] of `type`, written; may be gate or up itself.
 *   gate, up    [rows, d] of `type` (for instance the halves of one product's
 *               output); up NULL: none.
 *   gate8, up8  [rows, d], gate and up in 8 bits with gate8_scale and up8_scale
 *               of kind MP_SCALE_BLOCK, for the backward pass; NULL: not wanted.
 *   rows in [0, 2^31 - 1] (0 is a no-op), d in [1, 2^24].
 * (GELU in its form with tanh, which is up to 5e-4 from the one with erf.) A gate
 * of -inf gives NaN. The factor of a in act, in both passes, is 0 where it would be below 2^-126.
 * Errors: MP_ERR_NULL, MP_ERR_ALIGN, MP_ERR_RANGE, MP_ERR_CUDA.
 * ------------------------------------------------------------------------- */
typedef enum mp_activation {
    MP_ACT_SILU = 0,
    MP_ACT_GELU = 1
} mp_activation_t;

int mp_gated_forward(void* y, void* gate8, void* gate8_scale, void* up8, void* up8_scale, const void* gate,
                     const void* up, int64_t rows, int64_t d, int64_t y_stride, int64_t gate8_stride,
                     int64_t up8_stride, int64_t gate_stride, int64_t up_stride, int32_t activation, int32_t type,
                     void* stream);

/* ---------------------------------------------------------------------------
 * Its backward pass:
 *
 *   dgate = dy * up * act'(gate),   dup = dy * act(gate)
 *
 *   dgate       [rows, d] of `type`, written; may be dy or (in `type`) gate or up itself.
 *   dup         the same for up; NULL exactly when up is NULL.
 *   y           [rows, d] of `type`, act(gate) * up computed again (for the
 *               weight gradient of the product behind it); NULL: not wanted;
 *               may be dy itself where neither of the others is.
 *   dy          [rows, d] of `type`.
 *   gate, up    [rows, d] of `type`; or, with gate_scale and up_scale, both in 8
 *               bits with scales of kind MP_SCALE_BLOCK.
 *   rows, d     as the forward pass.
 * Errors: as the forward pass.
 * ------------------------------------------------------------------------- */
int mp_gated_backward(void* dgate, void* dup, void* y, const void* dy, const void* gate, const void* gate_scale,
                      const void* up, const void* up_scale, int64_t rows, int64_t d, int64_t dgate_stride,
                      int64_t dup_stride, int64_t y_stride, int64_t dy_stride, int64_t gate_stride,
                      int64_t up_stride, int32_t activation, int32_t type, void* stream);

/* ---------------------------------------------------------------------------
 * Activations in 8 bits, by themselves: q and scale (of `kind`) from x; and x
 * from them, a value above `type`'s range as infinity.
 *
 *   x           [rows, d] of `type`.
 *   q           [rows, d] e4m3.
 *   rows in [0, 2^31 - 1] (0 is a no-op), d in [1, 2^24].
 * Errors: MP_ERR_NULL, MP_ERR_ALIGN, MP_ERR_RANGE, MP_ERR_CUDA.
 * ------------------------------------------------------------------------- */
int mp_pack8(void* q, void* scale, const void* x, int64_t rows, int64_t d, int64_t q_stride, int64_t x_stride,
             int32_t type, int32_t kind, void* stream);
int mp_unpack8(void* x, const void* q, const void* scale, int64_t rows, int64_t d, int64_t x_stride,
               int64_t q_stride, int32_t type, int32_t kind, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* MP_BLOCK_H */

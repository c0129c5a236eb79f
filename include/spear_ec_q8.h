/*
 * spear_ec_q8.h -- C ABI of libspear_ec, the 8-bit path for AMD Instinct
 * MI355X (gfx950): matrix products of int8 activations and weights, plain and
 * gated, and the operators that make their operands: the root-mean-square norm
 * with the residual's addition, and the quantization of rows.  It serves the
 * layers that 4 bits hurt too much beside the 4-bit layers of spear_ec.h, whose
 * status codes and conventions it shares.
 *
 * The format.  A row (a token's activations, an output channel's weights) is
 * `width` int8 codes c and one fp32 scale s; an element stands for c * s.
 * Quantizing a row of values v:
 *   s = RN_fp32(max|v| / 127), 1 where that is 0
 *   c = clamp(rint(v / s), -127, 127), ties to even
 * with ratios as 64-bit arithmetic gives them.  A row that holds an infinity or
 * NaN gets the scale NaN and codes 0, so that every product with it is NaN.
 * Products take any int8 code, -128 too, and any scale.
 *
 * Conventions shared by every entry point: those of spear_ec.h (caller-owned
 * device pointers, none kept, nothing allocated; asynchronous on `stream`;
 * every argument validated before any HIP call, with the status codes of
 * spear_ec.h and spear_ec_last_error(); matrices 16-byte aligned, vectors of
 * scales 4-byte aligned).  Rows are contiguous, one after the other, but where
 * a stride is given.  width and d_in are multiples of 16 up to 65536, so that
 * rows begin on 16 bytes; rows are at most 2^30.
 */
#ifndef SPEAR_EC_Q8_H
#define SPEAR_EC_Q8_H

#include "spear_ec.h"

#ifdef __cplusplus
extern "C" {
#endif

/* desc.flags, besides SPEAR_EC_OUT_F32 */
#define SPEAR_EC_Q8_GATED 8 /* y = act(a) * b over two projections */
#define SPEAR_EC_Q8_GELU 16 /* act is GELU's tanh form instead of SiLU (with SPEAR_EC_Q8_GATED) */

/*
 * Shape of one product.  Supported set:
 *   d_in   a multiple of 16, 16 .. 65536
 *   d_out  a multiple of 16, 16 .. 262144 (columns of y; the weights have
 *          2 * d_out rows with SPEAR_EC_Q8_GATED)
 *   flags  SPEAR_EC_OUT_F32, SPEAR_EC_Q8_GATED, SPEAR_EC_Q8_GATED | SPEAR_EC_Q8_GELU
 *          in any combination
 * Passed by pointer and read during the call only.
 */
typedef struct spear_ec_q8_desc {
  int32_t d_in;
  int32_t d_out;
  int32_t flags;
} spear_ec_q8_desc;

/*
 * Quantize rows: x bf16, or fp32 with x_f32 != 0, row r at r * x_stride
 * elements (a multiple of 8, at least width), to codes int8 [rows][width] and
 * scales fp32 [rows].  For activations, and for weights (the rows of
 * [d_out][d_in]) when a model is loaded.  rows 0 launches nothing.  No output
 * may overlap x or the other.
 */
int spear_ec_q8_quantize(int32_t rows, int32_t width, const void* x, int32_t x_f32,
                         int64_t x_stride, int8_t* codes, float* scales, hipStream_t stream);

/* Read rows back: fp32 out [rows][width] = c * s, rounded once. */
int spear_ec_q8_dequant_f32(int32_t rows, int32_t width, const int8_t* codes, const float* scales,
                            float* out, hipStream_t stream);

/*
 * Root-mean-square norm of rows, with the residual's addition before it and
 * the quantization of its result:
 *   h = x, or with a residual h = RN_bf16(x + residual), written to sum
 *   u = h * weight / sqrt(mean(h^2) + eps)
 *   y = RN_bf16(u), and/or codes and scales = u quantized as above, from the
 *   unrounded u
 *   x        bf16, row r at r * x_stride elements (a multiple of 8, at least width)
 *   residual, sum  bf16 [rows][width], both or neither
 *   weight   bf16 [width]
 *   eps      positive, at most 1e300
 *   y        bf16 [rows][width], or NULL (what a 4-bit layer of spear_ec.h reads)
 *   codes, scales  as in spear_ec_q8_quantize, both or neither; at least one
 *            of y and codes is given
 * sum may be x (with x_stride == width) or residual itself; no other output
 * may overlap an input or another output.  The mean is held in 64 bits, its sum in
 * an order that goes with rows and width: a scale or code that lies within a few
 * 64-bit steps of a border between two may be either.  y is off by at most
 * (1 + 2^-12) half steps of bf16, or by 2^-149 / sqrt(mean(h^2) + eps) if that is
 * more (products h * weight below fp32's normal range).  A row with an infinity or
 * NaN in h, or any row if weight holds one, gets NaN throughout y, the scale NaN
 * and codes 0; so does one whose scale leaves fp32.
 */
int spear_ec_q8_rmsnorm(int32_t rows, int32_t width, const void* x, int64_t x_stride,
                        const void* residual, void* sum, const void* weight, double eps, void* y,
                        int8_t* codes, float* scales, hipStream_t stream);

/*
 * Bytes of scratch device memory spear_ec_q8_linear needs for up to max_tokens
 * tokens.  As with the layer's workspace its first use requires it to be
 * zero-filled, every call leaves its counters at zero again, and calls that
 * overlap on one workspace race.  0 for an invalid desc or count.
 */
size_t spear_ec_q8_workspace_bytes(const spear_ec_q8_desc* desc, int32_t max_tokens);

/*
 * Matrix product, 0 .. 2^20 tokens (0: nothing is launched), tokens * d_out at
 * most 2^37:
 *   p[t][n] = xs[t] * ws[n] * sum_k xq[t][k] * wq[n][k]
 *   y[t][n] = p[t][n], or with SPEAR_EC_Q8_GATED act(p[t][n]) * p[t][n + d_out]
 *   act(a)  = a * sigmoid(a), or with SPEAR_EC_Q8_GELU
 *             a * (1 + tanh(sqrt(2 / pi) (a + 0.044715 a^3))) / 2
 *   xq int8 [tokens][d_in], xs fp32 [tokens]
 *   wq int8 [d_out or 2 d_out][d_in], ws fp32 [d_out or 2 d_out]
 *   y  bf16 [tokens][d_out] (fp32 with SPEAR_EC_OUT_F32), no input's memory
 * Sums are exact 32-bit integers, whatever way the work is split: a row of y
 * depends on its own token and weight rows alone, bit for bit.  p takes three
 * fp32 roundings (the sum's conversion, times xs, times ws); where the sum times
 * xs leaves fp32's normal range so may p.  A bf16 y below 2^-126 may be zero.
 * act is computed in fp32, its sigmoid within 2^-15 of itself where that is
 * above 2^-126.
 */
int spear_ec_q8_linear(const spear_ec_q8_desc* desc, int32_t tokens, const int8_t* xq,
                       const float* xs, const int8_t* wq, const float* ws, void* y,
                       void* workspace, size_t workspace_bytes, hipStream_t stream);

#ifdef __cplusplus
}
#endif
#endif /* SPEAR_EC_Q8_H */

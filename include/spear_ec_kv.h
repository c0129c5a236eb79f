/*
 * spear_ec_kv.h -- C ABI of libspear_ec, the 4-bit paged key/value cache for
 * AMD Instinct MI355X (gfx950): appending keys and values (with the rotary
 * position embedding on the way), attention over the cache, and reading rows
 * of it back.  It is the serving loop's other memory-bound half next to the
 * 4-bit linear layer of spear_ec.h, whose status codes, conventions and
 * quantization rules it shares.
 *
 * The cache.  For every (token, kv head) one key and one value vector of
 * head_dim 4-bit codes c, each vector with one positive fp16 scale s and one zero-point
 * z (0 .. 15, or 8 throughout without SPEAR_EC_ZEROS); an element stands for
 * (c - z) * s.  Tokens lie in pages of page_tokens; a page holds every kv
 * head's vectors of its tokens.  Three caller-owned device arrays:
 *   codes  uint8 [pages][kv_heads][page_tokens/16][16 * head_dim]
 *          16-token blocks: first the keys, [16 tokens][head_dim/2] bytes,
 *          then the values, [head_dim/2][16 tokens] bytes; byte i of a vector
 *          holds dimension 2i in bits 0-3 and 2i + 1 in bits 4-7
 *   scales fp16  [pages][kv_heads][page_tokens/16][2][16]
 *          per block the keys' 16 scales, then the values'
 *   zeros  uint8 [pages][kv_heads][page_tokens/16][16]
 *          the key's zero-point in bits 0-3, the value's in bits 4-7; NULL
 *          without SPEAR_EC_ZEROS
 * Values lie byte-transposed so that a matrix-core operand (one dimension,
 * consecutive tokens) is loaded as it is; a single token still writes whole
 * bytes.  Slots that no token was appended to may hold anything.
 *
 * Conventions shared by every entry point: those of spear_ec.h (caller-owned
 * device pointers, none kept, nothing allocated; asynchronous on `stream`;
 * every host-side argument validated before any HIP call, with the status
 * codes of spear_ec.h and spear_ec_last_error()).  The arrays named in a
 * batch are device memory that the host cannot check; what the kernels do
 * with entries out of range is stated at each call, and none of them reads or
 * writes outside the cache for it.
 */
#ifndef SPEAR_EC_KV_H
#define SPEAR_EC_KV_H

#include "spear_ec.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Error bit of a workspace (spear_ec_workspace_status): an attention call met
 * a page number outside [0, pages) or a sequence longer than its page-table
 * row; the affected output rows hold NaN. */
#define SPEAR_EC_WS_BAD_PAGE 2

/*
 * Shape of one layer's cache.  Supported set:
 *   q_heads     a multiple of kv_heads, at most 128 per kv head; query head h
 *               reads kv head h / (q_heads / kv_heads)
 *   kv_heads    1 .. 256
 *   head_dim    64 or 128
 *   page_tokens a power of two, 16 .. 4096
 *   pages       >= 1; pages * kv_heads * page_tokens/16 at most 2^31 - 1
 *   max_pages   >= 1: entries of a page-table row; max_pages * page_tokens,
 *               the longest sequence, is at most 2^30
 *   flags       0 or SPEAR_EC_ZEROS
 * Passed by pointer and read during the call only.
 */
typedef struct spear_ec_kv_desc {
  int32_t q_heads;
  int32_t kv_heads;
  int32_t head_dim;
  int32_t page_tokens;
  int32_t pages;
  int32_t max_pages;
  int32_t flags;
} spear_ec_kv_desc;

/*
 * The sequences of one call.  Rows q_offsets[b] .. q_offsets[b + 1] of the
 * token arrays (q, k, v, out ...) are the newest tokens of sequence b, in
 * order; seq_lens[b] counts its tokens including them, so row i of its n is
 * the token at position seq_lens[b] - n + i.  Token j of the sequence lies in
 * page page_table[b][j / page_tokens].  q_offsets must ascend from 0; NULL
 * means one row per sequence (tokens == n_seqs); with other offsets rows may
 * be left out or hold anything.  Rows behind
 * q_offsets[n_seqs] belong to no sequence: no call reads or writes them.  A
 * row at a negative position (seq_lens[b] < n) is padding.
 *   n_seqs 0 .. 65536, tokens 0 .. 2^20, tokens * q_heads at most 2^27
 *   (0 of either count: nothing is launched)
 * Passed by pointer and read during the call only; the three arrays are int32
 * device memory, read by the kernels, so a captured call follows their
 * contents at each replay.
 */
typedef struct spear_ec_kv_batch {
  int32_t n_seqs;
  int32_t tokens;
  const int32_t* q_offsets;  /* [n_seqs + 1], or NULL */
  const int32_t* seq_lens;   /* [n_seqs] */
  const int32_t* page_table; /* [n_seqs][max_pages] */
} spear_ec_kv_batch;

/*
 * Rotary position embedding: row p of cos_sin (fp32 [rows][dim], device, 16-byte aligned)
 * holds dim/2 cosines, then dim/2 sines, for position p.  The first dim
 * elements (a multiple of 16, at most head_dim) of a head are rotated in
 * pairs (a, b) -> (a cos_i - b sin_i, b cos_i + a sin_i): elements i and
 * i + dim/2, or 2i and 2i + 1 with interleaved != 0.
 */
typedef struct spear_ec_kv_rope {
  const float* cos_sin;
  int32_t rows;
  int32_t dim;
  int32_t interleaved;
} spear_ec_kv_rope;

/*
 * Append the batch's rows to the cache: k (rotated) and v are quantized and
 * stored at their positions, and q, rotated, is written to q_out in bf16.
 *   q, k, v   bf16, row t at t * stride elements, [heads][head_dim] in a row
 *             (strides multiples of 8, e.g. slices of one projection's output)
 *   rope      NULL: no rotation
 *   q_out     bf16 rows of q_out_stride elements; may be q itself with the
 *             same stride, and must not overlap any input otherwise.  q and
 *             q_out may both be NULL: nothing but keys and values
 * What is stored is what 64-bit arithmetic gives, without rounding to bf16
 * between rotation and quantization; q_out is off by at most (1 + 2^-14) half
 * steps of bf16.  Quantization is spear_ec_quantize_rtn's over one vector:
 *   symmetric   s = RN_fp16(max|x| / 7), c = clamp(rint(x / s), -8, 7) + 8
 *   asymmetric  lo = min(0, x), hi = max(0, x), s = RN_fp16((hi - lo) / 15),
 *               z = clamp(rint(-lo / s), 0, 15), c = clamp(rint(x / s) + z, 0, 15)
 * (a scale that rounds to 0 becomes 1, one beyond 65504 is 65504; a NaN
 * element is skipped by the maxima and stored as code 0).
 * Padding rows store nothing and get zeros in q_out.  A row whose page is
 * outside [0, pages), whose position is past the page-table row, or past
 * rope->rows, stores nothing and gets NaN in q_out.  Rows of one call must
 * have different slots: where two share one, either's bytes may remain.
 */
int spear_ec_kv_append(const spear_ec_kv_desc* desc, const spear_ec_kv_batch* batch, const void* q,
                       int64_t q_stride, const void* k, int64_t k_stride, const void* v,
                       int64_t v_stride, const spear_ec_kv_rope* rope, uint8_t* codes, void* scales,
                       uint8_t* zeros, void* q_out, int64_t q_out_stride, hipStream_t stream);

/*
 * Bytes of scratch device memory spear_ec_kv_attention needs for up to n_seqs
 * sequences and up to `tokens` rows.  As with the layer's workspace its first
 * use requires it to be zero-filled, every call leaves its counters at zero
 * again, calls that overlap on one workspace race, and
 * spear_ec_workspace_status reads its error word.  0 for an invalid desc or
 * count.
 */
size_t spear_ec_kv_workspace_bytes(const spear_ec_kv_desc* desc, int32_t n_seqs, int32_t tokens);

/*
 * Attention of the batch's rows over their sequences' cached tokens.  The row
 * at position p attends to positions p - window + 1 .. p (window 0: 0 .. p):
 *   S_j = softmax_scale * q . K~_j,  m = max S_j,  l = sum exp(S_j - m)
 *   out = sum exp(S_j - m) V~_j / l,  lse = m + ln l
 *   q    bf16, row t at t * q_stride elements, [q_heads][head_dim] in a row
 *   out  bf16 [tokens][q_heads][head_dim], must not overlap q
 *   lse  fp32 [tokens][q_heads], or NULL
 * Keys meet q exactly, but for elements below 2^-19 of their row's largest in
 * calls of many rows, which are off by at most 2^-27 of it; products and sums are
 * held in fp32 (those of a value's codes and of its zero-point apart in calls of
 * few rows).  A probability and a value are rounded to fp16 on their way
 * (2^-11 relative each), whatever the scales of other tokens: a probability times
 * its value's scale is off by no more than 2^-11 of itself or, in calls of many
 * rows, 2^-24 of the row's largest such product, in calls of few 2^-38 of its
 * largest probability times its largest scale, if that is more.  Whatever a row of
 * q holds, the others keep these bounds.
 * Scores past 2^23 (in powers of two), whose digits below 1 fp32 does not hold,
 * decide by the digits that it does; a row whose scores leave fp32 itself may hold
 * anything.
 * A call of few rows is one with tokens * (q_heads / kv_heads) / n_seqs at most 64,
 * or 128 in small calls.  That is an average, which single tokens and a long chunk
 * in one call fit badly: two calls are faster there.
 * A padding row attends to nothing: zeros, lse = -inf.  softmax_scale is
 * positive and at most 2^64.  A q row holding an infinity or NaN gives NaN in that
 * row alone.  Bad pages: see SPEAR_EC_WS_BAD_PAGE.
 */
int spear_ec_kv_attention(const spear_ec_kv_desc* desc, const spear_ec_kv_batch* batch,
                          const void* q, int64_t q_stride, const uint8_t* codes,
                          const void* scales, const uint8_t* zeros, float softmax_scale,
                          int32_t window, void* out, float* lse, void* workspace,
                          size_t workspace_bytes, hipStream_t stream);

/*
 * Read the batch's rows back: fp32 (c - z) * s, exact, to k_out and v_out
 * [tokens][kv_heads][head_dim].  q_offsets that span seq_lens read whole
 * sequences.  Padding rows give zeros, rows on bad pages NaN.
 */
int spear_ec_kv_dequant_f32(const spear_ec_kv_desc* desc, const spear_ec_kv_batch* batch,
                            const uint8_t* codes, const void* scales, const uint8_t* zeros,
                            float* k_out, float* v_out, hipStream_t stream);

#ifdef __cplusplus
}
#endif
#endif /* SPEAR_EC_KV_H */

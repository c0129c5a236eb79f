// C ABI of the 4-bit paged key/value cache (spear_ec_kv.h): argument
// validation and planning.  Every check runs before any HIP call; no C++
// exception leaves this file.
#include "internal.hpp"
#include "kv.hpp"
#include "spear_ec_kv.h"

namespace spear {
namespace {

bool aligned(const void* p, uintptr_t n) { return ((uintptr_t)p & (n - 1)) == 0; }

int check_kv_desc(const spear_ec_kv_desc* d) {
  if (!d) return fail(SPEAR_EC_ERR_INVALID_ARGUMENT, "desc is NULL");
  if (d->q_heads <= 0 || d->kv_heads <= 0 || d->head_dim <= 0 || d->page_tokens <= 0 ||
      d->pages <= 0 || d->max_pages <= 0)
    return fail(SPEAR_EC_ERR_INVALID_ARGUMENT, "desc has a non-positive size");
  if (d->flags & ~SPEAR_EC_ZEROS)
    return fail(SPEAR_EC_ERR_INVALID_ARGUMENT, "unknown desc.flags bits");
  if (d->kv_heads > 256 || d->q_heads % d->kv_heads != 0 || d->q_heads / d->kv_heads > 128)
    return fail(SPEAR_EC_ERR_UNSUPPORTED,
                "q_heads must be 1 .. 128 times kv_heads, kv_heads at most 256");
  if (d->head_dim != 64 && d->head_dim != 128)
    return fail(SPEAR_EC_ERR_UNSUPPORTED, "head_dim must be 64 or 128");
  if (d->page_tokens < 16 || d->page_tokens > 4096 || (d->page_tokens & (d->page_tokens - 1)))
    return fail(SPEAR_EC_ERR_UNSUPPORTED, "page_tokens must be a power of two, 16 .. 4096");
  if ((int64_t)d->max_pages * d->page_tokens > (int64_t)1 << 30)
    return fail(SPEAR_EC_ERR_UNSUPPORTED, "max_pages * page_tokens must be at most 2^30");
  if ((int64_t)d->pages * d->kv_heads * (d->page_tokens / 16) > 0x7FFFFFFF)
    return fail(SPEAR_EC_ERR_UNSUPPORTED, "a cache has at most 2^31 - 1 blocks of 16 tokens and one head");
  return SPEAR_EC_OK;
}

int check_kv_batch(const spear_ec_kv_desc* d, const spear_ec_kv_batch* b) {
  if (!b) return fail(SPEAR_EC_ERR_INVALID_ARGUMENT, "batch is NULL");
  if (b->n_seqs < 0 || b->tokens < 0)
    return fail(SPEAR_EC_ERR_INVALID_ARGUMENT, "batch has a negative count");
  if (b->n_seqs > kKvMaxSeqs || b->tokens > kKvMaxTokens)
    return fail(SPEAR_EC_ERR_UNSUPPORTED, "at most 65536 sequences and 2^20 rows");
  if ((int64_t)b->tokens * d->q_heads > (int64_t)1 << 27)
    return fail(SPEAR_EC_ERR_UNSUPPORTED, "tokens * q_heads must be at most 2^27");
  if (b->n_seqs == 0 || b->tokens == 0) return SPEAR_EC_OK;
  if (!b->seq_lens || !b->page_table)
    return fail(SPEAR_EC_ERR_INVALID_ARGUMENT, "seq_lens and page_table are required");
  if (!b->q_offsets && b->tokens != b->n_seqs)
    return fail(SPEAR_EC_ERR_INVALID_ARGUMENT, "without q_offsets tokens must equal n_seqs");
  if (!aligned(b->q_offsets, 4) || !aligned(b->seq_lens, 4) || !aligned(b->page_table, 4))
    return fail(SPEAR_EC_ERR_MISALIGNED, "a batch array is not 4-byte aligned");
  return SPEAR_EC_OK;
}

int check_kv_cache(const spear_ec_kv_desc* d, const uint8_t* codes, const void* scales,
                   const uint8_t* zeros) {
  if (!codes || !scales) return fail(SPEAR_EC_ERR_INVALID_ARGUMENT, "codes and scales are required");
  if ((d->flags & SPEAR_EC_ZEROS) && !zeros)
    return fail(SPEAR_EC_ERR_INVALID_ARGUMENT, "zeros is required with SPEAR_EC_ZEROS");
  if (!aligned(codes, 16) || !aligned(scales, 16) ||
      ((d->flags & SPEAR_EC_ZEROS) && !aligned(zeros, 16)))
    return fail(SPEAR_EC_ERR_MISALIGNED, "a cache array is not 16-byte aligned");
  return SPEAR_EC_OK;
}

// A token array of `heads` heads a row: present, aligned, rows that do not overlap.
int check_rows(const spear_ec_kv_desc* d, const void* p, int64_t stride, int heads) {
  if (!p) return fail(SPEAR_EC_ERR_INVALID_ARGUMENT, "a token array is NULL");
  if (!aligned(p, 16)) return fail(SPEAR_EC_ERR_MISALIGNED, "a pointer is not 16-byte aligned");
  if (stride < (int64_t)heads * d->head_dim || stride > ((int64_t)1 << 32))
    return fail(SPEAR_EC_ERR_INVALID_ARGUMENT, "a row stride is shorter than its row or over 2^32");
  if (stride % 8 != 0)
    return fail(SPEAR_EC_ERR_MISALIGNED, "a row stride is not a multiple of 8 elements");
  return SPEAR_EC_OK;
}

KvShape make_kv_shape(const spear_ec_kv_desc* d) {
  KvShape s;
  s.q_heads = d->q_heads;
  s.kv_heads = d->kv_heads;
  s.D = d->head_dim;
  s.page_shift = 0;
  while ((1 << s.page_shift) < d->page_tokens) ++s.page_shift;
  s.pages = d->pages;
  s.max_pages = d->max_pages;
  s.zeros = (d->flags & SPEAR_EC_ZEROS) != 0;
  return s;
}

KvBatch make_kv_batch(const spear_ec_kv_batch* b) {
  return KvBatch{b->n_seqs, b->tokens, b->q_offsets, b->seq_lens, b->page_table};
}

KvCache make_kv_cache(const KvShape& s, const uint8_t* codes, const void* scales,
                      const uint8_t* zeros) {
  return KvCache{const_cast<uint8_t*>(codes),
                 static_cast<uint16_t*>(const_cast<void*>(scales)),
                 s.zeros ? const_cast<uint8_t*>(zeros) : nullptr};
}

// Which calls take the kernel for many rows.  The one for few rows reads and
// unpacks a cached token again for every 16 rows (token, query head of one kv
// head) of its sequence, the one for many for every 128 or 256, but it starts
// and joins slower: it pays past 64 rows a sequence, or past 128 where 16 at a
// time make no more items than there are compute units.  Few / many rows'
// kernel, heads of 128 behind 4096 tokens: 8 chats of 64 rows 25 / 35 us, of 72
// 36 / 36, of 128 45 / 39; 9 chats of 64 33 / 61, 16 of 64 47 / 55, 32 of 48
// 78 / 92, 32 of 64 101 / 93; one chat of 128 13 / 27; one of 72 behind 65536
// 57 / 69, of 128 76 / 77, of 192 114 / 106; 40 of 64, heads of 64 behind 1024,
// 37 / 47.  The lengths of the rows are device data: the rule goes by their
// average, and these calls are even.
constexpr int kFewRows = 64, kFewItems = 256;

bool many_rows(const KvShape& s, int n_seqs, int tokens) {
  const int64_t rows = ((int64_t)tokens * s.group() + n_seqs - 1) / n_seqs;
  return rows > kFewRows &&
         (rows > 2 * kFewRows || (rows + 15) / 16 * n_seqs * s.kv_heads > kFewItems);
}

// Covers every call of at most `tokens` tokens: one of several sequences that
// takes the second kernel has more than 128 rows, as one sequence does then too.
size_t attention_workspace(const KvShape& s, int tokens) {
  const size_t d = kv_decode_workspace(s), p = kv_prefill_workspace(s);
  return many_rows(s, 1, tokens) && p > d ? p : d;
}

}  // namespace
}  // namespace spear

using namespace spear;

extern "C" {

int spear_ec_kv_append(const spear_ec_kv_desc* desc, const spear_ec_kv_batch* batch, const void* q,
                       int64_t q_stride, const void* k, int64_t k_stride, const void* v,
                       int64_t v_stride, const spear_ec_kv_rope* rope, uint8_t* codes, void* scales,
                       uint8_t* zeros, void* q_out, int64_t q_out_stride, hipStream_t stream) {
  clear_error();
  int rc = check_kv_desc(desc);
  if (!rc) rc = check_kv_batch(desc, batch);
  if (rc) return rc;
  if (rope) {
    if (rope->rows <= 0 || rope->dim <= 0 || !rope->cos_sin)
      return fail(SPEAR_EC_ERR_INVALID_ARGUMENT, "rope needs cos_sin, rows and dim");
    if (rope->dim % 16 != 0 || rope->dim > desc->head_dim)
      return fail(SPEAR_EC_ERR_UNSUPPORTED, "rope dim must be a multiple of 16 up to head_dim");
    if (!aligned(rope->cos_sin, 16))
      return fail(SPEAR_EC_ERR_MISALIGNED, "cos_sin is not 16-byte aligned");
  }
  if (batch->n_seqs == 0 || batch->tokens == 0) return SPEAR_EC_OK;
  rc = check_kv_cache(desc, codes, scales, zeros);
  if (!rc) rc = check_rows(desc, k, k_stride, desc->kv_heads);
  if (!rc) rc = check_rows(desc, v, v_stride, desc->kv_heads);
  if (!rc && (q || q_out)) {
    if (!q || !q_out)
      rc = fail(SPEAR_EC_ERR_INVALID_ARGUMENT, "q and q_out are given together or not at all");
    if (!rc) rc = check_rows(desc, q, q_stride, desc->q_heads);
    if (!rc) rc = check_rows(desc, q_out, q_out_stride, desc->q_heads);
    if (!rc && q == q_out && q_stride != q_out_stride)
      rc = fail(SPEAR_EC_ERR_INVALID_ARGUMENT, "q_out in place of q needs q's stride");
  }
  if (rc) return rc;
  const KvShape s = make_kv_shape(desc);
  KvAppendArgs a;
  a.q = static_cast<const uint16_t*>(q);
  a.k = static_cast<const uint16_t*>(k);
  a.v = static_cast<const uint16_t*>(v);
  a.q_stride = q_stride;
  a.k_stride = k_stride;
  a.v_stride = v_stride;
  a.rope = rope ? KvRope{rope->cos_sin, rope->rows, rope->dim, rope->interleaved}
                : KvRope{nullptr, 0, 0, 0};
  a.cache = make_kv_cache(s, codes, scales, zeros);
  a.q_out = static_cast<uint16_t*>(q_out);
  a.q_out_stride = q_out_stride;
  return hip_status(launch_kv_append(s, make_kv_batch(batch), a, stream),
                    "cache append kernel launch");
}

size_t spear_ec_kv_workspace_bytes(const spear_ec_kv_desc* desc, int32_t n_seqs, int32_t tokens) {
  if (check_kv_desc(desc) != SPEAR_EC_OK || n_seqs < 0 || tokens < 0 || n_seqs > kKvMaxSeqs ||
      tokens > kKvMaxTokens)
    return 0;
  return attention_workspace(make_kv_shape(desc), tokens);
}

int spear_ec_kv_attention(const spear_ec_kv_desc* desc, const spear_ec_kv_batch* batch,
                          const void* q, int64_t q_stride, const uint8_t* codes,
                          const void* scales, const uint8_t* zeros, float softmax_scale,
                          int32_t window, void* out, float* lse, void* workspace,
                          size_t workspace_bytes, hipStream_t stream) {
  clear_error();
  int rc = check_kv_desc(desc);
  if (!rc) rc = check_kv_batch(desc, batch);
  if (rc) return rc;
  if (!(softmax_scale > 0.f) || softmax_scale > 0x1p64f)  // past that scores leave fp32
    return fail(SPEAR_EC_ERR_INVALID_ARGUMENT, "softmax_scale must be positive and at most 2^64");
  if (window < 0) return fail(SPEAR_EC_ERR_INVALID_ARGUMENT, "window is negative");
  if (batch->n_seqs == 0 || batch->tokens == 0) return SPEAR_EC_OK;
  rc = check_kv_cache(desc, codes, scales, zeros);
  if (!rc) rc = check_rows(desc, q, q_stride, desc->q_heads);
  if (rc) return rc;
  if (!out) return fail(SPEAR_EC_ERR_INVALID_ARGUMENT, "out is required");
  if (out == q) return fail(SPEAR_EC_ERR_INVALID_ARGUMENT, "out must not alias q");
  if (!workspace) return fail(SPEAR_EC_ERR_WORKSPACE, "workspace is NULL");
  if (!aligned(out, 16) || !aligned(workspace, 16))
    return fail(SPEAR_EC_ERR_MISALIGNED, "a pointer is not 16-byte aligned");
  if (!aligned(lse, 4)) return fail(SPEAR_EC_ERR_MISALIGNED, "lse is not 4-byte aligned");
  const KvShape s = make_kv_shape(desc);
  if (workspace_bytes < attention_workspace(s, batch->tokens))
    return fail(SPEAR_EC_ERR_WORKSPACE, "workspace is smaller than spear_ec_kv_workspace_bytes()");
  KvAttentionArgs a;
  a.q = static_cast<const uint16_t*>(q);
  a.q_stride = q_stride;
  a.cache = make_kv_cache(s, codes, scales, zeros);
  a.scale = softmax_scale;
  // no row sees more tokens than a page-table row holds
  a.window = window < s.max_pages << s.page_shift ? window : 0;
  a.out = static_cast<uint16_t*>(out);
  a.lse = lse;
  const auto launch = many_rows(s, batch->n_seqs, batch->tokens) ? launch_kv_prefill : launch_kv_decode;
  return hip_status(launch(s, make_kv_batch(batch), a, workspace, stream),
                    "cache attention kernel launch");
}

int spear_ec_kv_dequant_f32(const spear_ec_kv_desc* desc, const spear_ec_kv_batch* batch,
                            const uint8_t* codes, const void* scales, const uint8_t* zeros,
                            float* k_out, float* v_out, hipStream_t stream) {
  clear_error();
  int rc = check_kv_desc(desc);
  if (!rc) rc = check_kv_batch(desc, batch);
  if (rc) return rc;
  if (batch->n_seqs == 0 || batch->tokens == 0) return SPEAR_EC_OK;
  rc = check_kv_cache(desc, codes, scales, zeros);
  if (rc) return rc;
  if (!k_out || !v_out) return fail(SPEAR_EC_ERR_INVALID_ARGUMENT, "k_out and v_out are required");
  if (!aligned(k_out, 16) || !aligned(v_out, 16))
    return fail(SPEAR_EC_ERR_MISALIGNED, "a pointer is not 16-byte aligned");
  const KvShape s = make_kv_shape(desc);
  return hip_status(launch_kv_dequant(s, make_kv_batch(batch), make_kv_cache(s, codes, scales, zeros),
                                      k_out, v_out, stream),
                    "cache dequant kernel launch");
}

}  // extern "C"

// The 4-bit paged key/value cache: shapes handed to the kernels and the
// launchers' declarations (kv_api.hip, k_kv_*.hip).
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace spear {

constexpr int kKvBlock = 16;          // tokens of a cache block
constexpr int kKvMaxTokens = 1 << 20;  // rows of one call
constexpr int kKvMaxSeqs = 65536;

struct KvShape {
  int q_heads, kv_heads, D;
  int page_shift;  // log2(page_tokens)
  int pages, max_pages;
  bool zeros;
  __host__ __device__ int group() const { return q_heads / kv_heads; }
};

struct KvBatch {
  int n_seqs, tokens;
  const int* q_offsets;  // NULL: row b is sequence b's
  const int* seq_lens;
  const int* page_table;
};

struct KvCache {
  uint8_t* codes;
  uint16_t* scales;
  uint8_t* zeros;
};

struct KvRope {
  const float* cos_sin;  // NULL: no rotation
  int rows, dim, interleaved;
};

struct KvAppendArgs {
  const uint16_t *q, *k, *v;
  int64_t q_stride, k_stride, v_stride;
  KvRope rope;
  KvCache cache;
  uint16_t* q_out;
  int64_t q_out_stride;
};

struct KvAttentionArgs {
  const uint16_t* q;
  int64_t q_stride;
  KvCache cache;
  float scale;
  int window;  // 0: every earlier token
  uint16_t* out;
  float* lse;
};

hipError_t launch_kv_append(const KvShape& s, const KvBatch& b, const KvAppendArgs& a,
                            hipStream_t st);
hipError_t launch_kv_dequant(const KvShape& s, const KvBatch& b, const KvCache& c, float* k_out,
                             float* v_out, hipStream_t st);
// Bytes of workspace (counter words, then partial results) and launch of the
// attention kernels.
size_t kv_decode_workspace(const KvShape& s);
hipError_t launch_kv_decode(const KvShape& s, const KvBatch& b, const KvAttentionArgs& a,
                            void* workspace, hipStream_t st);
size_t kv_prefill_workspace(const KvShape& s);
hipError_t launch_kv_prefill(const KvShape& s, const KvBatch& b, const KvAttentionArgs& a,
                             void* workspace, hipStream_t st);

}  // namespace spear

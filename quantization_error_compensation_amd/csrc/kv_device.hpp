// Device helpers of the key/value cache kernels: the batch's rows and the
// cache's addresses.
#pragma once

#include "common.hpp"
#include "kv.hpp"

namespace spear {

// Sequence and position of a row of the batch.
struct KvRow {
  int seq;  // -1: the row belongs to no sequence
  int pos;  // negative: padding
};

// Row t's sequence: the number of offsets at or below t, counted by the whole
// wave (64 offsets a step), so the search costs one memory round trip for up
// to 64 sequences.  Offsets that do not ascend can only yield "none" or a
// row inside the sequence it names.  Wave-uniform t; every lane takes part.
__device__ __forceinline__ KvRow kv_row(const KvBatch& b, int t) {
  KvRow r{-1, -1};
  if (!b.q_offsets) {
    r.seq = t;  // tokens == n_seqs
    r.pos = max(__builtin_amdgcn_readfirstlane(b.seq_lens[t]), 0) - 1;
    return r;
  }
  const int lane = threadIdx.x & 63;
  int below = 0;  // offsets <= t
  for (int i = 0; i <= b.n_seqs; i += 64) {
    const bool le = i + lane <= b.n_seqs && b.q_offsets[i + lane] <= t;
    const int c = __popcll(__ballot(le));
    below += c;
    if (c < 64) break;
  }
  const int s = below - 1;
  if (s < 0 || s >= b.n_seqs) return r;
  const int first = __builtin_amdgcn_readfirstlane(b.q_offsets[s]);
  const int end = __builtin_amdgcn_readfirstlane(b.q_offsets[s + 1]);
  if (t < first || t >= end) return r;
  r.seq = s;
  r.pos = max(__builtin_amdgcn_readfirstlane(b.seq_lens[s]), 0) - (end - t);
  return r;
}

// Index of a (page, head)'s 16-token block in the cache, -1 for a position
// past the page-table row or a page that is not in the cache.
__device__ __forceinline__ int64_t kv_block(const KvShape& s, const KvBatch& b, int seq, int pos,
                                            int head) {
  const int p = pos >> s.page_shift;
  if (p >= s.max_pages) return -1;
  const int page = b.page_table[(int64_t)seq * s.max_pages + p];
  if ((unsigned)page >= (unsigned)s.pages) return -1;
  const int per = 1 << (s.page_shift - 4);  // blocks of a (page, head)
  return ((int64_t)page * s.kv_heads + head) * per + ((pos >> 4) & (per - 1));
}

}  // namespace spear

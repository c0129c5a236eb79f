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
// wave (64 offsets a step), so that the search costs one memory round trip for
// up to 63 sequences; their lengths come along with it.  Offsets that do not
// ascend can only yield "none" or a row inside the sequence it names.
// Wave-uniform t; every lane takes part.
__device__ __forceinline__ KvRow kv_row(const KvBatch& b, int t) {
  const int lane = threadIdx.x & 63;
  if (!b.q_offsets)  // tokens == n_seqs
    return KvRow{t, max(__builtin_amdgcn_readfirstlane(b.seq_lens[t]), 0) - 1};
  const int off = b.q_offsets[min(lane, b.n_seqs)];
  const int len = b.seq_lens[min(lane, b.n_seqs - 1)];
  int below = __popcll(__ballot(lane <= b.n_seqs && off <= t));
  for (int c = 64; c <= b.n_seqs && below == c; c += 64) {
    const int o = b.q_offsets[min(c + lane, b.n_seqs)];
    below += __popcll(__ballot(c + lane <= b.n_seqs && o <= t));
  }
  const int s = below - 1;
  if (s < 0 || s >= b.n_seqs) return KvRow{-1, -1};
  int first, end, n;
  if (s < 63) {
    first = __builtin_amdgcn_readlane(off, s);
    end = __builtin_amdgcn_readlane(off, s + 1);
    n = __builtin_amdgcn_readlane(len, s);
  } else {
    first = __builtin_amdgcn_readfirstlane(b.q_offsets[s]);
    end = __builtin_amdgcn_readfirstlane(b.q_offsets[s + 1]);
    n = __builtin_amdgcn_readfirstlane(b.seq_lens[s]);
  }
  if (t < first || t >= min(end, b.tokens)) return KvRow{-1, -1};
  return KvRow{s, max(n, 0) - (end - t)};
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

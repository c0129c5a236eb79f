// Code, operand and softmax helpers shared by the cache's attention kernels.
#pragma once

#include "kv_device.hpp"

namespace spear {

// Codes of a word's low and high half bytes, one a byte.  A byte c below 16 is
// the 8-bit float (e4m3) of value c 2^-9, normal or not, so that the
// conversions with a scale of 2^9 give the bf16 or fp16 pair of two codes
// exactly, and with the sign bit set of their negatives.
__device__ __forceinline__ uint32_t low_codes(uint32_t w) { return w & 0x0F0F0F0Fu; }
__device__ __forceinline__ uint32_t high_codes(uint32_t w) { return (w >> 4) & 0x0F0F0F0Fu; }
__device__ __forceinline__ uint32_t bf16_01(uint32_t b) {
  return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(b, 512.f, false));
}
__device__ __forceinline__ uint32_t bf16_23(uint32_t b) {
  return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(b, 512.f, true));
}
__device__ __forceinline__ uint32_t f16_01(uint32_t b) {
  return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(b, 512.f, false));
}
__device__ __forceinline__ uint32_t f16_23(uint32_t b) {
  return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(b, 512.f, true));
}
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
__device__ __forceinline__ f16x2 as_f16x2(uint32_t w) { return __builtin_bit_cast(f16x2, w); }
__device__ __forceinline__ uint32_t as_u32(f16x2 v) { return __builtin_bit_cast(uint32_t, v); }

__device__ __forceinline__ f32x4 mfma16x16x32_f16(u32x4 a, u32x4 b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a),
                                                __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
}
__device__ __forceinline__ f32x16 mfma32x32x16_f16(u32x4 a, u32x4 b, f32x16 c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8, a),
                                                __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
}

// Two fp32 -> fp16 pair and bf16 pair, nearest even.
__device__ __forceinline__ uint32_t pack_f16(float a, float b) {
  f16x2 r;
  r.x = (_Float16)a;
  r.y = (_Float16)b;
  return as_u32(r);
}
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
  bf16x2 r;
  r.x = (__bf16)a;
  r.y = (__bf16)b;
  return __builtin_bit_cast(uint32_t, r);
}

// Larger and smaller halves of two pairs of non-negative fp16 values.
__device__ __forceinline__ uint32_t max_pairs(uint32_t a, uint32_t b) {
  typedef unsigned short u16x2 __attribute__((ext_vector_type(2)));
  const u16x2 x = __builtin_bit_cast(u16x2, a), y = __builtin_bit_cast(u16x2, b);
  return __builtin_bit_cast(uint32_t, __builtin_elementwise_max(x, y));
}
__device__ __forceinline__ uint32_t min_pairs(uint32_t a, uint32_t b) {
  typedef unsigned short u16x2 __attribute__((ext_vector_type(2)));
  const u16x2 x = __builtin_bit_cast(u16x2, a), y = __builtin_bit_cast(u16x2, b);
  return __builtin_bit_cast(uint32_t, __builtin_elementwise_min(x, y));
}

__device__ __forceinline__ float fast_exp2(float x) { return __builtin_amdgcn_exp2f(x); }
constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kLn2 = 0.69314718055994530942f;

__device__ __forceinline__ uint64_t div_u64(uint64_t a, uint64_t b) {
  return ((a | b) >> 32) == 0 ? (uint64_t)((uint32_t)a / (uint32_t)b) : a / b;
}

// Inclusive prefix sum and maximum over the wave's lanes of non-negative
// 32-bit values: data-parallel-primitive moves within rows of 16 lanes (shifts
// by 1, 2, 4, 8), then across rows (lane 15 of a row to the next, lane 31 to
// the upper half).  Lane 63 holds the whole wave's.
template <int CTRL, int ROWS>
__device__ __forceinline__ int dpp_move(int v) {
  return __builtin_amdgcn_update_dpp(0, v, CTRL, ROWS, 0xF, false);
}
__device__ __forceinline__ int wave_prefix(int v) {
  v += dpp_move<0x111, 0xF>(v);
  v += dpp_move<0x112, 0xF>(v);
  v += dpp_move<0x114, 0xF>(v);
  v += dpp_move<0x118, 0xF>(v);
  v += dpp_move<0x142, 0xA>(v);
  v += dpp_move<0x143, 0xC>(v);
  return v;
}
__device__ __forceinline__ int wave_max(int v) {
  v = max(v, dpp_move<0x111, 0xF>(v));
  v = max(v, dpp_move<0x112, 0xF>(v));
  v = max(v, dpp_move<0x114, 0xF>(v));
  v = max(v, dpp_move<0x118, 0xF>(v));
  v = max(v, dpp_move<0x142, 0xA>(v));
  v = max(v, dpp_move<0x143, 0xC>(v));
  return __builtin_amdgcn_readlane(v, 63);
}

// v of the lane and of its partner 16 (32) lanes away, joined by op: the swap
// of rows leaves both in the two results.
template <typename F>
__device__ __forceinline__ float join16(float v, F op) {
  const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return op(__uint_as_float(r[0]), __uint_as_float(r[1]));
}
template <typename F>
__device__ __forceinline__ float join32(float v, F op) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return op(__uint_as_float(r[0]), __uint_as_float(r[1]));
}
__device__ __forceinline__ float larger(float a, float b) { return fmaxf(a, b); }
__device__ __forceinline__ float sum2(float a, float b) { return a + b; }

template <typename T>
__device__ __forceinline__ T wave_sum(T v) {
  #pragma unroll
  for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o, 64);
  return v;
}

// What the attention kernels' splits need of a sequence: its rows, and the
// range of its tokens that they see, in units of UNIT tokens.
struct Seq {
  int first, n;  // its rows of the batch
  int len;       // tokens with them
  int tiles;     // row tiles of a kv head
  int u0, nb;    // first unit and number of units (at least 1: an empty
                 // sequence's rows are still written)
};

template <int ROWS, int UNIT>
__device__ __forceinline__ Seq load_seq(const KvShape& s, const KvBatch& b, int window, int i) {
  Seq q;
  int first = i, end = i + 1;
  if (b.q_offsets) {
    first = min(max(b.q_offsets[i], 0), b.tokens);
    end = min(max(b.q_offsets[i + 1], first), b.tokens);
  }
  q.first = first;
  q.n = end - first;
  q.len = max(b.seq_lens[i], 0);
  q.tiles = (q.n * s.group() + ROWS - 1) / ROWS;
  const int last = min(q.len, s.max_pages << s.page_shift) - 1;
  const int lo = window ? max(0, min(q.len - q.n - window + 1, last)) : 0;
  q.u0 = lo / UNIT;
  q.nb = last < 0 ? 1 : last / UNIT - q.u0 + 1;
  return q;
}

// For up to 64 sequences, one a lane with its work w (32-bit sums): the lane
// whose work holds x, -1 past the end, and the work before it.
__device__ __forceinline__ int lane_of(int w, int x, int& base) {
  const int upto = wave_prefix(w);
  const uint64_t above = __ballot(upto > x);
  if (!above) return -1;
  const int who = __builtin_amdgcn_readfirstlane(__ffsll((unsigned long long)above) - 1);
  base = __builtin_amdgcn_readlane(upto, who) - __builtin_amdgcn_readlane(w, who);
  return who;
}
__device__ __forceinline__ Seq seq_of_lane(const Seq& own, int who) {
  Seq q;
  q.first = __builtin_amdgcn_readlane(own.first, who);
  q.n = __builtin_amdgcn_readlane(own.n, who);
  q.len = __builtin_amdgcn_readlane(own.len, who);
  q.tiles = __builtin_amdgcn_readlane(own.tiles, who);
  q.u0 = __builtin_amdgcn_readlane(own.u0, who);
  q.nb = __builtin_amdgcn_readlane(own.nb, who);
  return q;
}

// Work of the sequences before each 64 of them, and where a piece of work
// lies: every workgroup adds the lengths up itself, since they are device
// data.
constexpr int kMaxChunks = kKvMaxSeqs / 64;

// before[c + 1]: work of chunks 0 .. c.  Only needed with more than 64
// sequences; contains barriers.  weight(i): work of sequence i.
template <int WAVES, typename F>
__device__ __forceinline__ void sum_chunks(int64_t* before, int n_seqs, F weight) {
  const int lane = threadIdx.x & 63, chunks = (n_seqs + 63) / 64;
  for (int c = wave_id(); c < chunks; c += WAVES) {
    const int i = 64 * c + lane;
    const int64_t w = wave_sum(i < n_seqs ? weight(i) : (int64_t)0);
    if (lane == 0) before[c + 1] = w;
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    before[0] = 0;
    for (int c = 0; c < chunks; ++c) before[c + 1] += before[c];
  }
  __syncthreads();
}

// The sequence that holds work x (which is below the total) and the work
// before it.
template <typename F>
__device__ __forceinline__ int find_seq(const int64_t* before, int n_seqs, int64_t x, F weight,
                                        int64_t& seq_base) {
  const int lane = threadIdx.x & 63, chunks = (n_seqs + 63) / 64;
  int chunk = 0;
  int64_t base = 0;
  if (chunks > 1) {
    int lo = 0, hi = chunks;  // before[lo] <= x < before[hi]
    while (hi - lo > 1) {
      const int mid = (lo + hi) / 2;
      if (before[mid] <= x) lo = mid; else hi = mid;
    }
    chunk = lo;
    base = before[lo];
  }
  const int i = 64 * chunk + lane;
  const int64_t w = i < n_seqs ? weight(i) : (int64_t)0;
  int64_t upto = w;  // inclusive prefix
  #pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const int64_t y = __shfl_up(upto, o, 64);
    if (lane >= o) upto += y;
  }
  const int who = __builtin_amdgcn_readfirstlane(
      __ffsll((unsigned long long)__ballot(base + upto > x)) - 1);
  const int64_t mine = base + upto - w;
  const uint32_t low = __builtin_amdgcn_readlane((uint32_t)mine, who);
  const uint32_t high = __builtin_amdgcn_readlane((uint32_t)(mine >> 32), who);
  seq_base = (int64_t)(((uint64_t)high << 32) | low);
  return 64 * chunk + who;
}

}  // namespace spear

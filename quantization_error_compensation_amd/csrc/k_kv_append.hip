// Appending to and reading the 4-bit paged key/value cache (spear_ec_kv.h).
//
// Append.  One vector of head_dim elements (a query, key or value head of one
// token) takes head_dim / 8 lanes, 8 elements each, so a 16-byte load and a
// 4-byte store of codes a lane.  The stored codes are those of the rotation
// and the quotients in exact arithmetic.  They are evaluated in fp32 first (the
// rotation a cos - b sin with the product's error added back, 2^-23 of itself),
// together with a test whether any scale or code lies so near a border between
// two fp16 values or two codes that fp32 could choose the other one.  A wave
// that has one (about one in 30) evaluates its vectors again in fp64: there
// bf16 x fp32 products are exact, their difference is rounded once, and a
// quotient is checked against its exact residual.  Measured on the keys and
// values of 6803 tokens of 8 heads of 128: all in fp64 31 us, so 18 us.  Queries
// are only rounded to bf16 and take the fp32 rotation.  Calls with many rows a
// sequence go by blocks of 16 positions: a token's value bytes lie 16 bytes
// apart, and written one by one they cost as much as all the arithmetic (24 us
// by rows).  With 64 query heads the call moves 250 MB in 56 us.
//
// Reading back.  A wave takes one head of a 16-token block.  Values lie with
// the tokens of a byte column side by side, keys with the bytes of a token:
// keys go through LDS, and then a lane holds one byte column of 16 tokens
// either way and each token's row is written by consecutive lanes.
#include <algorithm>

#include "kv_math.hpp"

namespace spear {
namespace {

// Rows a sequence has on average from which a call goes by blocks of
// positions instead of rows.  By rows / by blocks, 64 and 8 heads of 128: 64
// sequences of 4 rows 6.3 / 7.4 us, of 12 10.9 / 11.2, of 16 13.4 / 12.3, of 32
// 21 / 18; one of 8 to 64 rows the same within 4%.  All of them even calls.
constexpr int kChunkRows = 16;

// Joins over the LANES (8 or 16) lanes of a vector by lane exchanges within
// rows of 16: neighbours, pairs, halves of 8, halves of 16.
template <int CTRL>
__device__ __forceinline__ double dpp_f64(double v) {
  const uint64_t b = (uint64_t)__double_as_longlong(v);
  const uint32_t lo = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)b, CTRL, 0xF, 0xF, false);
  const uint32_t hi = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(b >> 32), CTRL, 0xF, 0xF, false);
  return __longlong_as_double((long long)(((uint64_t)hi << 32) | lo));
}
template <int CTRL>
__device__ __forceinline__ float dpp_f32(float v) {
  return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), CTRL, 0xF, 0xF, false));
}
template <int LANES>
__device__ __forceinline__ float vector_max(float v) {
  v = fmaxf(v, dpp_f32<0xB1>(v));
  v = fmaxf(v, dpp_f32<0x4E>(v));
  v = fmaxf(v, dpp_f32<0x141>(v));
  if constexpr (LANES == 16) v = fmaxf(v, dpp_f32<0x140>(v));
  return v;
}
template <int LANES>
__device__ __forceinline__ double vector_max(double v) {
  v = fmax(v, dpp_f64<0xB1>(v));
  v = fmax(v, dpp_f64<0x4E>(v));
  v = fmax(v, dpp_f64<0x141>(v));
  if constexpr (LANES == 16) v = fmax(v, dpp_f64<0x140>(v));
  return v;
}

// rint(x / s) for s > 0 and r = 1 / s: the estimate rint(x r) is off by one at
// most, next to a border, where the residual x - q s (exact) tells.
__device__ __forceinline__ double rint_quotient(double x, double s, double r) {
  double q = rint(x * r);
  const double e = 2.0 * __builtin_fma(-q, s, x);
  if (fabs(e) >= s) {
    const bool odd = q - 2.0 * floor(q * 0.5) != 0.0;
    if (fabs(e) > s || odd) q += e > 0.0 ? 1.0 : -1.0;  // a tie goes to the even one
  }
  return q;
}

// What a vector is stored as: the codes of the lane's 8 elements (nibble i =
// element i), the vector's scale bits and zero-point.  LANES lanes hold it.
struct Stored {
  uint32_t codes;
  uint16_t scale;
  int zero;
};

// rint(x / s) from the estimate q of x / s, off by one at most: x is a bf16, s
// an fp16 value, so that the residual is exact in fp32 for quotients up to 15.
__device__ __forceinline__ float rint_quotient(float x, float s, float q) {
  float n = rintf(q);
  const float e = 2.f * __builtin_fmaf(-n, s, x);
  const bool odd = n - 2.f * floorf(n * 0.5f) != 0.f;
  if (fabsf(e) > s || (fabsf(e) == s && odd)) n += e > 0.f ? 1.f : -1.f;  // a tie goes to the even one
  return n;
}

// In fp32.  EXACT: the elements are bf16 values as they are; otherwise they are
// known to 2^-23 of themselves.  `sure` is false where the exact result may be
// another one.  Errors: the scale's quotient 2^-22 of itself (tested with
// 2^-21); x (1 / s), at most 15 where the code depends on it,
// 15 (2^-23 + 2^-23 + 2^-24) < 2^-17 (tested with 2^-16).  Few-digit elements
// often meet a border exactly: EXACT decides those by the residual.
template <int LANES, bool EXACT>
__device__ __forceinline__ Stored quantize8(const float (&x)[8], bool asym, bool& sure) {
  constexpr float kNear = 0.5f - 0x1p-16f;
  float hi = 0.f, neg = 0.f;  // max(0, x), max(0, -x)
  #pragma unroll
  for (int i = 0; i < 8; ++i) {
    hi = fmaxf(hi, asym ? x[i] : fabsf(x[i]));
    if (asym) neg = fmaxf(neg, -x[i]);
  }
  hi = vector_max<LANES>(hi);
  if (asym) neg = vector_max<LANES>(neg);
  const float y = fminf(asym ? (hi + neg) * (1.f / 15.f) : hi * (1.f / 7.f), 65504.f);
  const _Float16 below = (_Float16)(y * (1.f - 0x1p-21f)), above = (_Float16)(y * (1.f + 0x1p-21f));
  sure = below == above;
  Stored o;
  o.scale = __builtin_bit_cast(uint16_t, (_Float16)y);
  if ((o.scale & 0x7FFFu) == 0) o.scale = 0x3C00u;
  const float s = half_bits_to_f32(o.scale), r = __builtin_amdgcn_rcpf(s);
  float z = 8.f;
  if (asym) {
    const float q = neg * r, n = EXACT ? rint_quotient(neg, s, q) : rintf(q);
    if (!EXACT) sure = sure && !(fabsf(q - n) >= kNear);
    z = fminf(15.f, n);
  }
  o.zero = (int)z;
  float n[8], far = 0.f;  // far: largest distance from the nearest code
  #pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float q = x[i] * r;
    n[i] = rintf(q);
    far = fmaxf(far, fabsf(q - n[i]));
  }
  if constexpr (EXACT) {
    if (far >= kNear)
      #pragma unroll
      for (int i = 0; i < 8; ++i) n[i] = rint_quotient(x[i], s, x[i] * r);
  } else {
    sure = sure && far < kNear;
  }
  const float lo = asym ? -z : -8.f, up = asym ? 15.f - z : 7.f;
  float half[2];  // four codes less z as the digits of an integer in fp32
  #pragma unroll
  for (int h = 0; h < 2; ++h) {
    float w = 0.f;
    #pragma unroll
    for (int i = 3; i >= 0; --i)
      w = __builtin_fmaf(w, 16.f, fminf(up, fmaxf(lo, n[4 * h + i])));  // a NaN becomes lo
    half[h] = __builtin_fmaf(z, 4369.f, w);  // z in all four digits
  }
  o.codes = (uint32_t)half[0] | ((uint32_t)half[1] << 16);
  return o;
}

// The same in fp64, exact.
template <int LANES>
__device__ __forceinline__ Stored quantize8(const double (&x)[8], bool asym) {
  double hi = 0.0, neg = 0.0;  // max(0, x), max(0, -x)
  #pragma unroll
  for (int i = 0; i < 8; ++i) {
    hi = fmax(hi, asym ? x[i] : fabs(x[i]));
    if (asym) neg = fmax(neg, -x[i]);
  }
  hi = vector_max<LANES>(hi);
  if (asym) neg = vector_max<LANES>(neg);
  Stored o;
  o.scale = f64_to_f16_rne_sat(asym ? (hi + neg) / 15.0 : hi / 7.0);
  if ((o.scale & 0x7FFFu) == 0) o.scale = 0x3C00u;
  const double s = (double)half_bits_to_f32(o.scale), r = 1.0 / s;
  const double z = asym ? fmin(15.0, fmax(0.0, rint_quotient(neg, s, r))) : 8.0;
  o.zero = (int)z;
  const double lo = asym ? -z : -8.0, up = asym ? 15.0 - z : 7.0;
  o.codes = 0;
  #pragma unroll
  for (int i = 0; i < 8; ++i) {
    const double q = fmin(up, fmax(lo, rint_quotient(x[i], s, r)));
    o.codes |= (uint32_t)(int)(q + z) << (4 * i);
  }
  return o;
}

// Eight elements without rotation.
__device__ __forceinline__ void widen8(double (&x)[8], u32x4 raw) {
  #pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = (double)bf16_lo(raw[i]);
    x[2 * i + 1] = (double)bf16_hi(raw[i]);
  }
}

// A lane's cosines and signed sines for its 8 elements of a vector at
// position pos (elements past the rotated ones: 1 and 0).
struct Turn {
  float c[8], s[8];
};
__device__ __forceinline__ void load_turn(Turn& t, const KvRope& rope, int pos, int sub) {
  const int half = rope.dim / 2, d0 = 8 * sub;
  const float* row = rope.cos_sin + (int64_t)pos * rope.dim;
  #pragma unroll
  for (int i = 0; i < 8; ++i) {
    t.c[i] = 1.f;
    t.s[i] = 0.f;
  }
  if (d0 >= rope.dim) return;
  if (rope.interleaved) {
    const float4 c = *reinterpret_cast<const float4*>(row + d0 / 2);
    const float4 s = *reinterpret_cast<const float4*>(row + half + d0 / 2);
    const float cf[4] = {c.x, c.y, c.z, c.w}, sf[4] = {s.x, s.y, s.z, s.w};
    #pragma unroll
    for (int i = 0; i < 8; ++i) {
      t.c[i] = cf[i / 2];
      t.s[i] = (i & 1) ? sf[i / 2] : -sf[i / 2];
    }
    return;
  }
  const bool first = d0 < half;
  const int at = first ? d0 : d0 - half;
  const float4* c = reinterpret_cast<const float4*>(row + at);
  const float4* s = reinterpret_cast<const float4*>(row + half + at);
  const float4 c0 = c[0], c1 = c[1], s0 = s[0], s1 = s[1];
  const float cf[8] = {c0.x, c0.y, c0.z, c0.w, c1.x, c1.y, c1.z, c1.w};
  const float sf[8] = {s0.x, s0.y, s0.z, s0.w, s1.x, s1.y, s1.z, s1.w};
  #pragma unroll
  for (int i = 0; i < 8; ++i) {
    t.c[i] = cf[i];
    t.s[i] = first ? -sf[i] : sf[i];
  }
}

// The other elements of the lane's pairs: neighbours, or dim/16 lanes away in
// the same vector.
__device__ __forceinline__ u32x4 partners(u32x4 raw, const KvRope& rope, int sub) {
  u32x4 other;
  if (rope.interleaved) {
    #pragma unroll
    for (int i = 0; i < 4; ++i) other[i] = __builtin_amdgcn_alignbit(raw[i], raw[i], 16);
  } else {
    const int away = rope.dim / 16, lane = threadIdx.x & 63;
    const int from = 16 * sub < rope.dim ? lane + away : lane - away;
    #pragma unroll
    for (int i = 0; i < 4; ++i) other[i] = __shfl(raw[i], from & 63, 64);
  }
  return other;
}

__device__ __forceinline__ float element(u32x4 raw, int i) {
  return (i & 1) ? bf16_hi(raw[i / 2]) : bf16_lo(raw[i / 2]);
}

// The lane's 8 elements rotated: x c + (its pair's other element) s, in fp64, and
// in fp32 with the error of the second product (exact) added back.  A product
// that is infinite has no such error: the result is not to be used then.
__device__ __forceinline__ void rotate8(double (&f)[8], u32x4 raw, u32x4 other, const Turn& t) {
  #pragma unroll
  for (int i = 0; i < 8; ++i)
    f[i] = __builtin_fma((double)element(raw, i), (double)t.c[i],
                         (double)element(other, i) * (double)t.s[i]);
}
__device__ __forceinline__ bool rotate8(float (&f)[8], u32x4 raw, u32x4 other, const Turn& t) {
  float most = 0.f;
  #pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float y = element(other, i), p = y * t.s[i];
    const float low = __builtin_fmaf(y, t.s[i], -p);
    f[i] = __builtin_fmaf(element(raw, i), t.c[i], p) + low;
    most = fmaxf(most, fabsf(p));
  }
  return most < INFINITY;
}
__device__ __forceinline__ void widen8(float (&x)[8], u32x4 raw) {
  #pragma unroll
  for (int i = 0; i < 8; ++i) x[i] = element(raw, i);
}

// Slot of a row: the cache block of kv head 0 that its position lies in.
// Negative: padding (pos < 0), a bad page or a position past the rotation's
// table, whose row is not stored.
__device__ __forceinline__ int64_t row_block(const KvShape& s, const KvBatch& b, const KvRope& rope,
                                             int seq, int pos) {
  if (pos < 0 || (rope.cos_sin && pos >= rope.rows)) return -1;
  return kv_block(s, b, seq, pos, 0);
}

// A row's query heads head0, head0 + step, ..., QUERIES of them.
template <int D, int QUERIES>
__device__ __forceinline__ void append_queries(const KvShape& s, const KvBatch& b,
                                               const KvAppendArgs& a, int t, int head0, int step,
                                               int sub) {
  // the elements are on their way while the row is looked up
  u32x4 raw[QUERIES];
  #pragma unroll
  for (int u = 0; u < QUERIES; ++u)
    raw[u] = load16(a.q + (int64_t)t * a.q_stride + min(head0 + u * step, s.q_heads - 1) * D + 8 * sub);
  const KvRow r = kv_row(b, t);
  if (r.seq < 0) return;
  const int64_t blk = row_block(s, b, a.rope, r.seq, r.pos);
  Turn turn;
  const bool turned = a.rope.cos_sin && blk >= 0;
  if (turned) load_turn(turn, a.rope, r.pos, sub);
  #pragma unroll
  for (int u = 0; u < QUERIES; ++u) {
    u32x4 o = raw[u];
    if (blk < 0) {
      const uint32_t fill = r.pos < 0 ? 0u : 0x7FC07FC0u;
      o = u32x4{fill, fill, fill, fill};
    } else if (turned) {
      float f[8];
      const u32x4 other = partners(raw[u], a.rope, sub);
      if (!rotate8(f, raw[u], other, turn)) {
        double d[8];
        rotate8(d, raw[u], other, turn);
        #pragma unroll
        for (int e = 0; e < 8; ++e) f[e] = (float)d[e];
      }
      if (8 * sub < a.rope.dim)
        #pragma unroll
        for (int e = 0; e < 4; ++e) o[e] = pack_bf16(f[2 * e], f[2 * e + 1]);
    }
    if (head0 + u * step < s.q_heads)
      *reinterpret_cast<u32x4*>(a.q_out + (int64_t)t * a.q_out_stride + (head0 + u * step) * D + 8 * sub) = o;
  }
}

// What the lane's part of a token's key and value is stored as.  Every lane of
// a vector takes part.
template <int D>
__device__ __forceinline__ void store_form(const KvShape& s, const KvRope& rope, u32x4 kraw,
                                           u32x4 vraw, const Turn& turn, int sub, Stored& sk,
                                           Stored& sv) {
  constexpr int LANES = D / 8;
  u32x4 other = {0, 0, 0, 0};
  const bool turned = rope.cos_sin && 8 * sub < rope.dim;
  if (rope.cos_sin) other = partners(kraw, rope, sub);
  bool k_sure, v_sure, finite = true;
  {
    float x[8];
    widen8(x, kraw);
    if (rope.cos_sin) {
      if (turned) finite = rotate8(x, kraw, other, turn);
      sk = quantize8<LANES, false>(x, s.zeros, k_sure);
    } else {
      sk = quantize8<LANES, true>(x, s.zeros, k_sure);
    }
    widen8(x, vraw);
    sv = quantize8<LANES, true>(x, s.zeros, v_sure);
  }
  if (__any(!k_sure || !v_sure || !finite)) {
    double x[8];
    widen8(x, kraw);
    if (turned) rotate8(x, kraw, other, turn);
    sk = quantize8<LANES>(x, s.zeros);
    widen8(x, vraw);
    sv = quantize8<LANES>(x, s.zeros);
  }
}

// Few rows a sequence: a workgroup per row and 256 / LANES heads, first the
// row's kv heads (key and value together: they share a zero-point byte), then
// its query heads.
template <int D>
__global__ __launch_bounds__(256) void append_rows_kernel(KvShape s, KvBatch b, KvAppendArgs a) {
  constexpr int LANES = D / 8, kGroup = 256 / LANES;
  const int sub = threadIdx.x % LANES, which = threadIdx.x / LANES;
  const int kv_groups = (s.kv_heads + kGroup - 1) / kGroup;
  const int t = blockIdx.x;
  if ((int)blockIdx.y >= kv_groups) {
    append_queries<D, 1>(s, b, a, t, ((int)blockIdx.y - kv_groups) * kGroup + which, 0, sub);
    return;
  }
  const int head = blockIdx.y * kGroup + which;
  const int at = min(head, s.kv_heads - 1) * D + 8 * sub;
  const u32x4 kraw = load16(a.k + (int64_t)t * a.k_stride + at);
  const u32x4 vraw = load16(a.v + (int64_t)t * a.v_stride + at);
  const KvRow r = kv_row(b, t);
  if (r.seq < 0) return;
  const int64_t blk = row_block(s, b, a.rope, r.seq, r.pos);
  if (blk < 0) return;
  Turn turn;
  if (a.rope.cos_sin) load_turn(turn, a.rope, r.pos, sub);
  Stored sk, sv;
  store_form<D>(s, a.rope, kraw, vraw, turn, sub, sk, sv);
  if (head >= s.kv_heads) return;
  const int j = r.pos & 15;
  const int64_t hb = blk + ((int64_t)head << (s.page_shift - 4));
  uint8_t* codes = a.cache.codes + hb * (16 * D);
  *reinterpret_cast<uint32_t*>(codes + j * (D / 2) + 4 * sub) = sk.codes;
  uint8_t* col = codes + 8 * D + 64 * sub + j;
  #pragma unroll
  for (int c = 0; c < 4; ++c) col[16 * c] = (uint8_t)(sv.codes >> (8 * c));
  if (sub == 0) {
    a.cache.scales[hb * 32 + j] = sk.scale;
    a.cache.scales[hb * 32 + 16 + j] = sv.scale;
    if (s.zeros) a.cache.zeros[hb * 16 + j] = (uint8_t)(sk.zero | (sv.zero << 4));
  }
}

// Blocks of 16 positions that a sequence's rows lie in (padding rows in
// blocks of negative positions).
__device__ __forceinline__ int row_blocks(const Seq& q) {
  return q.n > 0 ? ((q.len - 1) >> 4) - ((q.len - q.n) >> 4) + 1 : 0;
}

// The sequence and first position of the batch's x-th such block; false past
// the last.  SMALL: at most 64 sequences.  Contains barriers otherwise.
template <bool SMALL>
__device__ __forceinline__ bool find_block(const KvShape& s, const KvBatch& b, int64_t* before, int x,
                                           Seq& q, int& seq, int& p0) {
  const int lane = threadIdx.x & 63;
  const auto seq_at = [&](int i) { return load_seq<16, 16>(s, b, 0, i); };
  int base;
  if constexpr (SMALL) {
    Seq own{0, 0, 0, 0, 0, 1};
    if (lane < b.n_seqs) own = seq_at(lane);
    seq = lane_of(row_blocks(own), x, base);
    if (seq < 0) return false;
    q = seq_of_lane(own, seq);
  } else {
    const auto weight = [&](int i) { return (int64_t)row_blocks(seq_at(i)); };
    sum_chunks<4>(before, b.n_seqs, weight);
    if (x >= before[(b.n_seqs + 63) / 64]) return false;
    int64_t base64;
    seq = find_seq(before, b.n_seqs, x, weight, base64);
    base = (int)base64;
    q = seq_at(seq);
  }
  p0 = (((q.len - q.n) >> 4) + x - base) << 4;
  return true;
}

// Many rows a sequence: the first `blocks` workgroups along x take a block of 16
// positions, 16 / LANES kv heads for each y, so that the byte-transposed values
// leave as whole 16-byte pieces; the others a row and 4 * 256 / LANES query
// heads each.
template <int D, bool SMALL>
__global__ __launch_bounds__(256) void append_chunk_kernel(KvShape s, KvBatch b, KvAppendArgs a,
                                                           int blocks, int query_groups) {
  constexpr int LANES = D / 8, kHeads = 16 / LANES;
  __shared__ int64_t before[SMALL ? 1 : kMaxChunks + 1];
  __shared__ __attribute__((aligned(16))) uint8_t cols[kHeads][D / 2][16];
  const int sub = threadIdx.x % LANES, which = threadIdx.x / LANES;
  if ((int)blockIdx.x >= blocks) {
    const int i = ((int)blockIdx.x - blocks) * gridDim.y + blockIdx.y;
    if (i >= b.tokens * query_groups) return;
    append_queries<D, 4>(s, b, a, i / query_groups, (i % query_groups) * (4 * 256 / LANES) + which,
                         256 / LANES, sub);
    return;
  }
  Seq q;
  int seq, p0;
  if (!find_block<SMALL>(s, b, before, blockIdx.x, q, seq, p0)) return;
  const int j = which & 15, hh = which >> 4;
  const int first = q.len - q.n, pos = p0 + j;
  if (p0 < 0) return;  // padding only
  const bool row = pos >= first && pos < q.len;
  const int64_t t = q.first + (row ? pos - first : 0);
  const int step = gridDim.y * kHeads;
  u32x4 kraw, vraw;
  const auto load = [&](int head) {
    const int at = min(head, s.kv_heads - 1) * D + 8 * sub;
    kraw = row ? load16(a.k + t * a.k_stride + at) : u32x4{0, 0, 0, 0};
    vraw = row ? load16(a.v + t * a.v_stride + at) : u32x4{0, 0, 0, 0};
  };
  load(blockIdx.y * kHeads + hh);
  const int64_t page = kv_block(s, b, seq, p0, 0);
  if (page < 0) return;
  const int limit = a.rope.cos_sin ? min(q.len, a.rope.rows) : q.len;  // rows past the table stay out
  const bool kept = row && pos < limit;
  const bool whole = p0 >= first && p0 + 15 < limit;  // every position of the block is a row
  Turn turn;
  if (a.rope.cos_sin) load_turn(turn, a.rope, min(pos, a.rope.rows - 1), sub);
  for (int head0 = blockIdx.y * kHeads; head0 < s.kv_heads; head0 += step) {
    const int head = head0 + hh;
    const u32x4 kcur = kraw, vcur = vraw;
    if (head0 + step < s.kv_heads) load(head + step);
    Stored sk, sv;
    store_form<D>(s, a.rope, kcur, vcur, turn, sub, sk, sv);
    const int64_t hb = page + ((int64_t)min(head, s.kv_heads - 1) << (s.page_shift - 4));
    uint8_t* codes = a.cache.codes + hb * (16 * D);
    if (kept && head < s.kv_heads) {
      *reinterpret_cast<uint32_t*>(codes + j * (D / 2) + 4 * sub) = sk.codes;
      if (sub == 0) {
        a.cache.scales[hb * 32 + j] = sk.scale;
        a.cache.scales[hb * 32 + 16 + j] = sv.scale;
        if (s.zeros) a.cache.zeros[hb * 16 + j] = (uint8_t)(sk.zero | (sv.zero << 4));
      }
      if (!whole) {  // other tokens' bytes are not this call's to write
        uint8_t* col = codes + 8 * D + 64 * sub + j;
        #pragma unroll
        for (int c = 0; c < 4; ++c) col[16 * c] = (uint8_t)(sv.codes >> (8 * c));
      }
    }
    if (!whole) continue;
    #pragma unroll
    for (int c = 0; c < 4; ++c) cols[hh][4 * sub + c][j] = (uint8_t)(sv.codes >> (8 * c));
    __syncthreads();
    // 64 columns of 16 bytes: one head of 128 or two of 64
    if (threadIdx.x < 64) {
      const int h2 = threadIdx.x / (D / 2), c = threadIdx.x % (D / 2);
      if (head0 + h2 < s.kv_heads) {
        uint8_t* to = a.cache.codes + (page + ((int64_t)(head0 + h2) << (s.page_shift - 4))) * (16 * D) + 8 * D;
        *reinterpret_cast<u32x4*>(to + 16 * c) = *reinterpret_cast<const u32x4*>(&cols[h2][c][0]);
      }
    }
    __syncthreads();  // the columns are free for the next heads
  }
}

typedef float f32x2 __attribute__((ext_vector_type(2)));

// A workgroup per block and four kv heads.
template <int D, bool SMALL>
__global__ __launch_bounds__(256) void kv_dequant_kernel(KvShape s, KvBatch b, KvCache c,
                                                         float* __restrict__ k_out,
                                                         float* __restrict__ v_out) {
  __shared__ int64_t before[SMALL ? 1 : kMaxChunks + 1];
  __shared__ __attribute__((aligned(16))) uint8_t keys[4][8 * D];
  const int lane = threadIdx.x & 63, wave = wave_id();
  const int head = blockIdx.y * 4 + wave;
  Seq q;
  int seq, p0;
  if (!find_block<SMALL>(s, b, before, blockIdx.x, q, seq, p0) || head >= s.kv_heads) return;
  const int first = q.len - q.n;  // position of the first row
  const int64_t blk = p0 < 0 ? -1 : kv_block(s, b, seq, p0, head);
  const int64_t bl = max(blk, (int64_t)0);
  constexpr int kCols = D / 2;
  const int col = lane % kCols;
  // tokens of the block: lane's byte column of all 16 (head_dim 64: lanes 32
  // and up take tokens 8 to 15)
  constexpr int kTokens = 16 * kCols / 64;
  const int j0 = (lane / kCols) * kTokens;
  const uint8_t* codes = c.codes + bl * (16 * D);
  uint8_t kb[kTokens], vb[kTokens];
  {
    // keys: the block's bytes as they lie, then every 64th (32nd) of them
    if constexpr (D == 128) {
      *reinterpret_cast<u32x4*>(&keys[wave][16 * lane]) = load16(codes + 16 * lane);
    } else {
      *reinterpret_cast<u32x2*>(&keys[wave][8 * lane]) = *reinterpret_cast<const u32x2*>(codes + 8 * lane);
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    #pragma unroll
    for (int j = 0; j < kTokens; ++j) kb[j] = keys[wave][(j0 + j) * kCols + col];
    uint32_t w[kTokens / 4];
    const uint8_t* vp = codes + 8 * D + 16 * col + j0;
    if constexpr (D == 128) {
      const u32x4 r = load16(vp);
      #pragma unroll
      for (int i = 0; i < 4; ++i) w[i] = r[i];
    } else {
      const u32x2 r = *reinterpret_cast<const u32x2*>(vp);
      #pragma unroll
      for (int i = 0; i < 2; ++i) w[i] = r[i];
    }
    #pragma unroll
    for (int j = 0; j < kTokens; ++j) vb[j] = (uint8_t)(w[j / 4] >> (8 * (j % 4)));
  }
  // scales and zero-points of the lane's tokens
  u32x4 ks4[kTokens / 8], vs4[kTokens / 8];
  uint32_t z4[kTokens / 4];
  const uint8_t* sp = reinterpret_cast<const uint8_t*>(c.scales) + bl * 64 + 2 * j0;
  #pragma unroll
  for (int i = 0; i < kTokens / 8; ++i) {
    ks4[i] = load16(sp + 16 * i);
    vs4[i] = load16(sp + 32 + 16 * i);
  }
  #pragma unroll
  for (int i = 0; i < kTokens / 4; ++i)
    z4[i] = s.zeros ? *reinterpret_cast<const uint32_t*>(c.zeros + bl * 16 + j0 + 4 * i) : 0x88888888u;
  #pragma unroll
  for (int j = 0; j < kTokens; ++j) {
    const int pos = p0 + j0 + j;
    const uint32_t kw = ks4[j >> 3][(j >> 1) & 3], vw = vs4[j >> 3][(j >> 1) & 3];
    const float ks = half_bits_to_f32((uint16_t)((j & 1) ? kw >> 16 : kw));
    const float vs = half_bits_to_f32((uint16_t)((j & 1) ? vw >> 16 : vw));
    const uint32_t z = z4[j >> 2] >> (8 * (j & 3));
    const float kz = (float)(z & 15u), vz = (float)((z >> 4) & 15u);
    if (pos < first || pos >= q.len) continue;
    f32x2 k = {((float)(kb[j] & 15) - kz) * ks, ((float)(kb[j] >> 4) - kz) * ks};
    f32x2 v = {((float)(vb[j] & 15) - vz) * vs, ((float)(vb[j] >> 4) - vz) * vs};
    if (blk < 0) {
      const float fill = pos < 0 ? 0.f : __uint_as_float(0x7FC00000u);
      k = v = f32x2{fill, fill};
    }
    const int64_t at = ((int64_t)(q.first + pos - first) * s.kv_heads + head) * D + 2 * col;
    // written once, not read back by this kernel: past the caches (84 -> 70 us
    // for 42597 tokens of 8 heads of 128, 5.6 TB/s)
    __builtin_nontemporal_store(k, reinterpret_cast<f32x2*>(k_out + at));
    __builtin_nontemporal_store(v, reinterpret_cast<f32x2*>(v_out + at));
  }
}

int ceil_div(int a, int b) { return (a + b - 1) / b; }

}  // namespace

// n rows of a sequence lie in at most n / 16 + 2 blocks
int block_bound(const KvBatch& b) { return b.tokens / 16 + 2 * std::min(b.n_seqs, b.tokens); }

hipError_t launch_kv_append(const KvShape& s, const KvBatch& b, const KvAppendArgs& a,
                            hipStream_t st) {
  const int lanes = s.D / 8, group = 256 / lanes;
  if (b.tokens < kChunkRows * b.n_seqs) {
    const dim3 grid(b.tokens, ceil_div(s.kv_heads, group) + (a.q ? ceil_div(s.q_heads, group) : 0));
    if (s.D == 64)
      hipLaunchKernelGGL(append_rows_kernel<64>, grid, dim3(256), 0, st, s, b, a);
    else
      hipLaunchKernelGGL(append_rows_kernel<128>, grid, dim3(256), 0, st, s, b, a);
    return hipGetLastError();
  }
  // several heads a workgroup once there are enough workgroups to fill the chip
  const int blocks = block_bound(b), all = ceil_div(s.kv_heads, 16 / lanes);
  const int groups = ceil_div(all, std::max(1, std::min(4, blocks * all / 1024)));
  const int query_groups = a.q ? ceil_div(s.q_heads, 4 * group) : 0;
  const dim3 grid(blocks + ceil_div(b.tokens * query_groups, groups), groups);
  const auto go = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, grid, dim3(256), 0, st, s, b, a, blocks, query_groups);
  };
  if (s.D == 64) {
    if (b.n_seqs <= 64) go(append_chunk_kernel<64, true>); else go(append_chunk_kernel<64, false>);
  } else {
    if (b.n_seqs <= 64) go(append_chunk_kernel<128, true>); else go(append_chunk_kernel<128, false>);
  }
  return hipGetLastError();
}

hipError_t launch_kv_dequant(const KvShape& s, const KvBatch& b, const KvCache& c, float* k_out,
                             float* v_out, hipStream_t st) {
  const dim3 grid(block_bound(b), ceil_div(s.kv_heads, 4));
  const auto go = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, grid, dim3(256), 0, st, s, b, c, k_out, v_out);
  };
  if (s.D == 64) {
    if (b.n_seqs <= 64) go(kv_dequant_kernel<64, true>); else go(kv_dequant_kernel<64, false>);
  } else {
    if (b.n_seqs <= 64) go(kv_dequant_kernel<128, true>); else go(kv_dequant_kernel<128, false>);
  }
  return hipGetLastError();
}

}  // namespace spear

// Attention of few rows per sequence over the 4-bit paged key/value cache:
// one pass over the cache with a running maximum and sum, work split evenly
// over the cached tokens of all sequences.
//
// Work.  The rows (token, query head) of a sequence that read one kv head are
// taken 16 at a time; an item is one such row tile and one kv head, a unit 128
// tokens of an item.  Workgroups take equal runs of units (the lengths are
// device data, so every workgroup adds them up itself), the four waves of a
// workgroup every fourth unit of a run.  Runs cut items: each workgroup that
// holds a piece of a cut item leaves (O, m, l) in its slot of the workspace
// and the last one to arrive joins them in workgroup order, so results do not
// depend on the order of arrival.
//
// Matrix cores.  Scores come as S^T = K q^T (16x16x32, bf16): a lane then
// holds one query row and 32 of the unit's 128 tokens, so the softmax's
// maximum and sum need two exchanges per unit, and the probabilities are
// already the operand of O^T = V^T P^T: lane and token order agree because
// key tile t, row m is token 32 (m / 4) + 4 t + m % 4.  A key's code c becomes
// the bf16 value 16 + c, a value's the fp16 value 64 + c (its nibble under the
// top of the mantissa, one byte permute a pair); the offset 16 + z comes out
// with the row's sum of q for keys, and for values with one matrix step of
// -(64 + z) against the same probabilities, added once a unit, so that it
// never grows with the sequence.  Keys and q meet exactly.  A probability
// times its value's scale is rounded to fp16 (2^-11 relative, an eighth of the
// output's bf16 rounding): the running reference M is the rows' maximum score
// plus the exponent of the largest value scale so far, less 14, so that
// w = 2^(score - M) s stays below 2^14 and is exact to its 11 bits down to
// 2^-28 of that.  Every sum is fp32.
#include "internal.hpp"
#include "kv_math.hpp"
#include "spear_ec_kv.h"

namespace spear {
namespace {

constexpr int kUnit = 128;       // tokens of a unit
constexpr int kRows = 16;        // rows of an item
constexpr int kGroups = 512;     // workgroups: two per compute unit of gfx950
constexpr int kWaves = 4;

template <int D>
constexpr int slot_floats() { return kRows * D + 2 * kRows; }

// Codes, scales and zero-points of one unit in a lane's registers.
template <int D, bool ZEROS>
struct Unit {
  uint32_t k[8][D / 32];  // key tile t: D / 8 bytes of its token
  u32x4 v[D / 32][2];     // byte column 16 tau + lane % 16, tokens 32 kb + 16 half ..
  u32x4 ks[2][2], vs[2][2];
  u32x4 z[2];
};

template <int D, bool ZEROS>
__device__ __forceinline__ void load_keys(Unit<D, ZEROS>& u, const KvCache& c, const int (&blk)[2],
                                          int n, int kb) {
  #pragma unroll
  for (int t = 0; t < 8; ++t) {
    const uint8_t* p = c.codes + (int64_t)blk[t >> 2] * (16 * D) +
                       ((4 * (t & 3) + (n & 3)) * (D / 2) + kb * (D / 8));
    if constexpr (D == 128) {
      const u32x4 w = load16(p);
      #pragma unroll
      for (int i = 0; i < 4; ++i) u.k[t][i] = w[i];
    } else {
      const u32x2 w = *reinterpret_cast<const u32x2*>(p);
      #pragma unroll
      for (int i = 0; i < 2; ++i) u.k[t][i] = w[i];
    }
  }
}

template <int D, bool ZEROS>
__device__ __forceinline__ void load_values(Unit<D, ZEROS>& u, const KvCache& c,
                                            const int (&blk)[2], int n) {
  #pragma unroll
  for (int h = 0; h < 2; ++h) {
    const uint8_t* sp = reinterpret_cast<const uint8_t*>(c.scales) + (int64_t)blk[h] * 64;
    #pragma unroll
    for (int i = 0; i < 2; ++i) u.ks[h][i] = load16(sp + 16 * i);
    #pragma unroll
    for (int i = 0; i < 2; ++i) u.vs[h][i] = load16(sp + 32 + 16 * i);
    if constexpr (ZEROS) u.z[h] = load16(c.zeros + (int64_t)blk[h] * 16);
  }
  #pragma unroll
  for (int t = 0; t < D / 32; ++t)
    #pragma unroll
    for (int h = 0; h < 2; ++h)
      u.v[t][h] = load16(c.codes + (int64_t)blk[h] * (16 * D) + 8 * D + (16 * t + n) * 16);
}

// fp16 scale of the lane's token i (0 .. 31) of the unit.
__device__ __forceinline__ float scale_of(const u32x4 (&s)[2][2], int i) {
  const uint32_t w = s[i >> 4][(i >> 3) & 1][(i >> 1) & 3];
  return half_bits_to_f32((uint16_t)((i & 1) ? w >> 16 : w));
}

template <int D, bool ZEROS>
__global__ __launch_bounds__(256, 2) void decode_attention_kernel(KvShape s, KvBatch b,
                                                                  KvAttentionArgs a, int* counters,
                                                                  float* slots, uint32_t slot_bytes) {
  __shared__ int64_t before[kMaxChunks + 1];  // work before each 64 sequences
  __shared__ float osh[kWaves][kRows][D + 4];
  __shared__ float msh[kWaves][kRows], lsh[kWaves][kRows];
  __shared__ int flag;
  const int lane = threadIdx.x & 63, wave = wave_id();
  const int n = lane & 15, kb = lane >> 4;
  const int capacity = s.max_pages << s.page_shift;

  // ---- the split: equal runs of units
  const auto seq_at = [&](int i) { return load_seq<kRows, kUnit>(s, b, a.window, i); };
  int64_t units = 0, items = 0;
  int longest = 0;
  for (int i = lane; i < b.n_seqs; i += 64) {
    const Seq q = seq_at(i);
    const int64_t it = (int64_t)q.tiles * s.kv_heads;
    items += it;
    units += it * q.nb;
    if (it) longest = max(longest, q.nb);
  }
  units = wave_sum(units);
  items = wave_sum(items);
  #pragma unroll
  for (int o = 32; o > 0; o >>= 1) longest = max(longest, __shfl_xor(longest, o, 64));
  int64_t run = max((units + kGroups - 1) / kGroups, (int64_t)kWaves);
  // A workgroup per item where that takes at most two more steps of its four
  // waves than the even split: nothing is cut and nothing joined.
  const bool whole = items <= gridDim.x && longest <= 4 * ((run + 3) / 4 + 2);
  if (whole) run = 1;  // counted in items
  const int64_t total = whole ? items : units;
  int64_t x0 = (int64_t)blockIdx.x * run;
  const int64_t x1 = min(x0 + run, total);
  if (x0 >= x1) return;
  const auto weight = [&](int i) {
    const Seq q = seq_at(i);
    return (int64_t)q.tiles * s.kv_heads * (whole ? 1 : q.nb);
  };
  if (b.n_seqs > 64) sum_chunks<kWaves>(before, b.n_seqs, weight);

  while (x0 < x1) {
    // ---- the item that holds work x0
    int64_t seq_base;
    const int seq = find_seq(before, b.n_seqs, x0, weight, seq_base);
    const Seq q = seq_at(seq);
    const int first = q.first, rows_n = q.n, len = q.len, tiles = q.tiles, u0 = q.u0, nb = q.nb;
    const int64_t local = x0 - seq_base;
    const int64_t item = whole ? local : (int64_t)div_u64(local, nb);
    const int ub = whole ? 0 : (int)(local - item * nb);
    const int take = whole ? nb : (int)min((int64_t)(nb - ub), x1 - x0);
    const int head = (int)div_u64(item, tiles);
    const int tile = (int)(item - (int64_t)head * tiles);

    // ---- the lane's query row
    const int group = s.group();
    const int row = tile * kRows + n;
    const bool live = row < rows_n * group;
    const int tok = live ? row / group : 0;
    const int qh = head * group + (live ? row - tok * group : 0);
    const int pos = live ? len - rows_n + tok : -1;
    const int hi = min(pos, capacity - 1);
    const int lo = a.window && pos >= a.window ? pos - a.window + 1 : 0;
    const uint16_t* qp = a.q + (int64_t)(first + tok) * a.q_stride + qh * D + kb * (D / 4);
    u32x4 qf[D / 32];
    float qs = 0.f;
    #pragma unroll
    for (int i = 0; i < D / 32; ++i) {
      const u32x4 r = live ? load16(qp + 8 * i) : u32x4{0, 0, 0, 0};
      #pragma unroll
      for (int j = 0; j < 4; ++j) qs += bf16_lo(r[j]) + bf16_hi(r[j]);
      qf[i] = x_permute8(r);
    }
    qs += __shfl_xor(qs, 16, 64);
    qs += __shfl_xor(qs, 32, 64);
    const float f = a.scale * kLog2e;  // scores in powers of two
    // tokens that some row of the tile sees: a unit inside is unmasked
    int all_lo = live ? lo : 0, all_hi = live ? hi : 0x7FFFFFFF;
    int any_lo = live && hi >= lo ? lo : 0x7FFFFFFF, any_hi = live ? hi : -1;
    #pragma unroll
    for (int o = 1; o < 16; o <<= 1) {
      all_lo = max(all_lo, __shfl_xor(all_lo, o, 64));
      all_hi = min(all_hi, __shfl_xor(all_hi, o, 64));
      any_lo = min(any_lo, __shfl_xor(any_lo, o, 64));
      any_hi = max(any_hi, __shfl_xor(any_hi, o, 64));
    }

    // mx, ev: the row's largest score and value-scale exponent; m: their reference M
    float mx = -INFINITY, m = -INFINITY, l = 0.f;  // l: the lane's own tokens
    int ev = 0;
    f32x4 o[D / 32][2];
    #pragma unroll
    for (int t = 0; t < D / 32; ++t) o[t][0] = o[t][1] = f32x4{0.f, 0.f, 0.f, 0.f};

    for (int ui = wave; ui < take; ui += kWaves) {
      const int j0 = (u0 + ub + ui) * kUnit;
      // the unit's 8 blocks, one lane each; positions nobody sees stand for
      // the nearest one that somebody does
      int my = 0;
      bool bad = false;
      if (any_hi >= any_lo) {
        const int at = min(max(j0 + 16 * (lane & 7), any_lo & ~15), any_hi);
        const int page = b.page_table[(int64_t)seq * s.max_pages + (at >> s.page_shift)];
        bad = (unsigned)page >= (unsigned)s.pages;
        const int per = 1 << (s.page_shift - 4);
        my = bad ? 0 : (page * s.kv_heads + head) * per + ((at >> 4) & (per - 1));
      }
      const uint64_t bads = __ballot(bad);
      const int kblk[2] = {__shfl(my, 2 * (n >> 2), 64), __shfl(my, 2 * (n >> 2) + 1, 64)};
      const int vblk[2] = {__shfl(my, 2 * kb, 64), __shfl(my, 2 * kb + 1, 64)};
      Unit<D, ZEROS> u;
      load_keys(u, a.cache, kblk, n, kb);
      load_values(u, a.cache, vblk, n);

      // scores: x = (sum (16 + c) q - (16 + z) sum q) s
      float x[32];
      const float init = (ZEROS ? -16.f : -24.f) * qs;
      #pragma unroll
      for (int t = 0; t < 8; ++t) {
        f32x4 acc = {init, init, init, init};
        #pragma unroll
        for (int i = 0; i < D / 32; ++i) {
          const uint32_t e = even16(u.k[t][i]), d = odd16(u.k[t][i]), top = 0x41414141u;
          const u32x4 kf = {pair01(e, top), pair23(e, top), pair01(d, top), pair23(d, top)};
          acc = mfma16x16x32(kf, qf[i], acc);
        }
        #pragma unroll
        for (int i = 0; i < 4; ++i) {
          float v = acc[i];
          if constexpr (ZEROS)
            v -= (float)((u.z[t >> 2][t & 3] >> (8 * i)) & 15u) * qs;
          x[4 * t + i] = v * scale_of(u.ks, 4 * t + i);
        }
      }
      if (bads & 0xFF) {  // tokens on a page outside the cache: NaN where they are seen
        #pragma unroll
        for (int h = 0; h < 2; ++h)
          if ((bads >> (2 * kb + h)) & 1)
            #pragma unroll
            for (int i = 0; i < 16; ++i) x[16 * h + i] = __uint_as_float(0x7FC00000u);
      }
      const bool masked = j0 < all_lo || j0 + kUnit - 1 > all_hi;
      if (masked) {
        #pragma unroll
        for (int i = 0; i < 32; ++i) {
          const int j = j0 + 32 * kb + i;
          if (j < lo || j > hi) x[i] = -INFINITY;
        }
      }
      float top = x[0];
      #pragma unroll
      for (int i = 1; i < 32; ++i) top = fmaxf(top, x[i]);
      uint32_t big_s = 0;  // largest value scale (fp16 bits) of the lane's tokens
      if (!masked) {
        uint32_t p = u.vs[0][0][0];
        #pragma unroll
        for (int i = 1; i < 16; ++i) p = max_pairs(p, u.vs[i >> 3][(i >> 2) & 1][i & 3]);
        big_s = max(p & 0xFFFFu, p >> 16);
      } else {  // an unwritten slot's scale may be anything
        #pragma unroll
        for (int i = 0; i < 32; ++i) {
          const uint32_t w = u.vs[i >> 4][(i >> 3) & 1][(i >> 1) & 3];
          if (x[i] != -INFINITY) big_s = max(big_s, (i & 1) ? w >> 16 : w & 0xFFFFu);
        }
      }
      top = fmaxf(top, __shfl_xor(top, 16, 64));
      top = fmaxf(top, __shfl_xor(top, 32, 64));
      big_s = max(big_s, (uint32_t)__shfl_xor((int)big_s, 16, 64));
      big_s = max(big_s, (uint32_t)__shfl_xor((int)big_s, 32, 64));
      mx = fmaxf(mx, top * f);
      ev = max(ev, (int)((big_s & 0x7FFFu) >> 10));
      const float mn = mx + (float)(ev - 28);  // scale < 2^(ev - 14)
      if (__any(mn != m)) {
        const float alpha = mn == m ? 1.f : fast_exp2(m - mn);
        l *= alpha;
        #pragma unroll
        for (int t = 0; t < D / 32; ++t)
          #pragma unroll
          for (int h = 0; h < 2; ++h) o[t][h] *= alpha;
        m = mn;
      }
      const float ref = m == -INFINITY ? 0.f : m;
      u32x4 pf[4];  // probabilities times value scales, 8 tokens a step
      #pragma unroll
      for (int i = 0; i < 32; i += 2) {
        const float p0 = fast_exp2(__builtin_fmaf(x[i], f, -ref));
        const float p1 = fast_exp2(__builtin_fmaf(x[i + 1], f, -ref));
        l += p0 + p1;
        float w0 = p0 * scale_of(u.vs, i), w1 = p1 * scale_of(u.vs, i + 1);
        if (masked) {
          w0 = p0 == 0.f ? 0.f : w0;
          w1 = p1 == 0.f ? 0.f : w1;
        }
        pf[i >> 3][(i >> 1) & 3] = pack_f16(w0, w1);
      }
      f32x4 off = {0.f, 0.f, 0.f, 0.f};
      #pragma unroll
      for (int st = 0; st < 4; ++st) {
        const int h = st >> 1, d0 = 2 * (st & 1);
        u32x4 zf = {0xD480D480u, 0xD480D480u, 0xD480D480u, 0xD480D480u};  // -72
        if constexpr (ZEROS) {
          const uint32_t a0 = odd64(u.z[h][d0]), a1 = odd64(u.z[h][d0 + 1]), neg = 0xD4D4D4D4u;
          zf = u32x4{pair01(a0, neg), pair23(a0, neg), pair01(a1, neg), pair23(a1, neg)};
        }
        off = mfma16x16x32_f16(zf, pf[st], off);
        #pragma unroll
        for (int t = 0; t < D / 32; ++t) {
          const uint32_t w0 = u.v[t][h][d0], w1 = u.v[t][h][d0 + 1], top64 = 0x54545454u;
          const uint32_t e0 = even64(w0), e1 = even64(w1), o0 = odd64(w0), o1 = odd64(w1);
          const u32x4 evn = {pair01(e0, top64), pair23(e0, top64), pair01(e1, top64), pair23(e1, top64)};
          const u32x4 odd = {pair01(o0, top64), pair23(o0, top64), pair01(o1, top64), pair23(o1, top64)};
          o[t][0] = mfma16x16x32_f16(evn, pf[st], o[t][0]);
          o[t][1] = mfma16x16x32_f16(odd, pf[st], o[t][1]);
        }
      }
      #pragma unroll
      for (int t = 0; t < D / 32; ++t)
        #pragma unroll
        for (int h = 0; h < 2; ++h) o[t][h] += off;
      if ((bads & 0xFF) && lane == 0) {
        // only a token that some row sees makes an output NaN
        bool seen = false;
        #pragma unroll
        for (int i = 0; i < 8; ++i)
          if ((bads >> i) & 1) seen |= j0 + 16 * i <= any_hi && j0 + 16 * i + 15 >= any_lo;
        if (seen) atomicOr(counters + kCtrError, SPEAR_EC_WS_BAD_PAGE);
      }
    }
    l += __shfl_xor(l, 16, 64);
    l += __shfl_xor(l, 32, 64);

    // ---- the four waves' results joined
    if (kb == 0) {
      msh[wave][n] = m;
      lsh[wave][n] = l;
    }
    __syncthreads();
    {
      const float big = fmaxf(fmaxf(msh[0][n], msh[1][n]), fmaxf(msh[2][n], msh[3][n]));
      const float k = m == -INFINITY ? 0.f : fast_exp2(m - big);
      #pragma unroll
      for (int t = 0; t < D / 32; ++t) {
        // byte columns 16 t + 4 kb + i: eight dimensions in a row
        float* dst = &osh[wave][n][32 * t + 8 * kb];
        #pragma unroll
        for (int i = 0; i < 4; ++i) {
          dst[2 * i] = o[t][0][i] * k;
          dst[2 * i + 1] = o[t][1][i] * k;
        }
      }
    }
    __syncthreads();
    constexpr int kPer = D / 16;  // elements a thread finishes
    const int r = threadIdx.x >> 4, d0 = (threadIdx.x & 15) * kPer;
    float acc[kPer];
    float big = -INFINITY, sum = 0.f;
    for (int w2 = 0; w2 < kWaves; ++w2) big = fmaxf(big, msh[w2][r]);
    #pragma unroll
    for (int i = 0; i < kPer; ++i) acc[i] = 0.f;
    for (int w2 = 0; w2 < kWaves; ++w2) {
      const float mw = msh[w2][r], lw = lsh[w2][r];
      sum += mw == -INFINITY ? lw : lw * fast_exp2(mw - big);
      #pragma unroll
      for (int i = 0; i < kPer; ++i) acc[i] += osh[w2][r][d0 + i];
    }

    // ---- a piece of a cut item: leave it, and join the pieces if it is the last
    const int my_row = tile * kRows + r;
    const bool mine = my_row < rows_n * group;
    bool last = true;
    if (take < nb) {
      const int64_t i0 = seq_base + item * nb;              // the item's units
      const int wa = (int)div_u64(i0, run);
      const int wb = (int)div_u64(i0 + nb - 1, run);
      const rsrc_t rs = make_rsrc(slots, slot_bytes);
      const uint32_t stride = slot_floats<D>() * 4;
      const uint32_t to = (2 * blockIdx.x + (x0 == (int64_t)blockIdx.x * run ? 0 : 1)) * stride;
      if (mine) {
        #pragma unroll
        for (int i = 0; i < kPer; i += 4)
          bstore16_dev(rs, to + (r * D + d0 + i) * 4, 0,
                       f32x4{acc[i], acc[i + 1], acc[i + 2], acc[i + 3]});
        if ((threadIdx.x & 15) == 0) {
          bstore_dev(rs, to + (kRows * D + r) * 4, 0, big);
          bstore_dev(rs, to + (kRows * D + kRows + r) * 4, 0, sum);
        }
      }
      wait_vmem();
      __syncthreads();
      if (threadIdx.x == 0) {
        int* ctr = counters + kCtrBand + wa;
        const int arrived = __hip_atomic_fetch_add(ctr, 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        flag = arrived == wb - wa;
        if (arrived == wb - wa) store_dev(ctr, 0);
      }
      __syncthreads();
      last = flag != 0;
      if (last && mine) {
        // the first piece starts its item inside workgroup wa's run, or with it
        const uint32_t first_slot = 2 * wa + (i0 == (int64_t)wa * run ? 0 : 1);
        big = -INFINITY;
        for (int w2 = wa; w2 <= wb; ++w2) {
          const uint32_t from = (w2 == wa ? first_slot : 2 * w2) * stride;
          big = fmaxf(big, bload_dev(rs, from + (kRows * D + r) * 4, 0));
        }
        sum = 0.f;
        #pragma unroll
        for (int i = 0; i < kPer; ++i) acc[i] = 0.f;
        for (int w2 = wa; w2 <= wb; ++w2) {
          const uint32_t from = (w2 == wa ? first_slot : 2 * w2) * stride;
          const float mw = bload_dev(rs, from + (kRows * D + r) * 4, 0);
          const float lw = bload_dev(rs, from + (kRows * D + kRows + r) * 4, 0);
          const float k = mw == -INFINITY ? 1.f : fast_exp2(mw - big);  // an empty piece is zeros
          sum += lw * k;
          #pragma unroll
          for (int i = 0; i < kPer; i += 4) {
            const u32x4 v = bload16_dev(rs, from + (r * D + d0 + i) * 4, 0);
            #pragma unroll
            for (int j = 0; j < 4; ++j) acc[i + j] += __uint_as_float(v[j]) * k;
          }
        }
      }
    }
    if (last && mine) {
      const int t = my_row / group;
      const int h = head * group + my_row - t * group;
      const int64_t at = (int64_t)(first + t) * s.q_heads + h;
      const bool past = len - rows_n + t >= capacity;  // longer than its page-table row
      float inv = sum == 0.f ? 0.f : 1.f / sum;
      if (past) inv = sum = __uint_as_float(0x7FC00000u);
      uint32_t out[kPer / 2];
      #pragma unroll
      for (int i = 0; i < kPer / 2; ++i) out[i] = pack_bf16(acc[2 * i] * inv, acc[2 * i + 1] * inv);
      uint32_t* dst = reinterpret_cast<uint32_t*>(a.out + at * D + d0);
      #pragma unroll
      for (int i = 0; i < kPer / 2; ++i) dst[i] = out[i];
      if ((threadIdx.x & 15) == 0) {
        if (a.lse) a.lse[at] = (big + log2f(sum)) * kLn2;
        if (past) atomicOr(counters + kCtrError, SPEAR_EC_WS_BAD_PAGE);
      }
    }
    __syncthreads();  // the shared arrays are free for the next item
    x0 += whole ? 1 : take;
  }
}

}  // namespace

size_t kv_decode_workspace(const KvShape& s) {
  return sizeof(int) * kCounterSlots +
         sizeof(float) * 2 * kGroups * (s.D == 64 ? slot_floats<64>() : slot_floats<128>());
}

hipError_t launch_kv_decode(const KvShape& s, const KvBatch& b, const KvAttentionArgs& a,
                            void* workspace, hipStream_t st) {
  int* counters = static_cast<int*>(workspace);
  float* slots = reinterpret_cast<float*>(counters + kCounterSlots);
  const uint32_t bytes = (uint32_t)(kv_decode_workspace(s) - sizeof(int) * kCounterSlots);
  const auto go = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, dim3(kGroups), dim3(256), 0, st, s, b, a, counters, slots, bytes);
  };
  if (s.D == 64) {
    if (s.zeros) go(decode_attention_kernel<64, true>); else go(decode_attention_kernel<64, false>);
  } else {
    if (s.zeros) go(decode_attention_kernel<128, true>); else go(decode_attention_kernel<128, false>);
  }
  return hipGetLastError();
}

}  // namespace spear

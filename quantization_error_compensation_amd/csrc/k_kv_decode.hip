// Attention of few rows per sequence over the 4-bit paged key/value cache:
// one pass over the cache with a running maximum and sum, work split evenly
// over the cached tokens of all sequences.
//
// Work.  The rows (token, query head) of a sequence that read one kv head are
// taken 16 at a time; an item is one such row tile and one kv head, a unit 128
// tokens of an item.  The lengths are device data, so every workgroup adds them
// up itself.  Either the items are cut into pieces of one size, one a workgroup,
// the row tiles of one piece next to each other on one XCD, whose L2 then reads
// the cache once for them (8 chats of 64 rows behind 4096 tokens 29 -> 25 us);
// or, where that would make the longest piece more than a step longer than an
// even share, the workgroups take equal runs of all items' units laid end to
// end.  The waves of a workgroup take every eighth unit.
// Each workgroup that holds a piece of a cut item leaves (O, M, l) in its slot
// of the workspace, and the last one to arrive joins them in order, so results
// do not depend on the order of arrival.
//
// Matrix cores.  Scores come as S^T = K q^T (16x16x32, bf16): a lane then
// holds one query row and 32 of the unit's 128 tokens, so the softmax's
// maximum and sum need two exchanges per unit, and the probabilities are
// already the operand of O^T = V^T P^T: lane and token order agree because
// key tile t, row m is token 32 (m / 4) + 4 t + m % 4.  Codes become bf16
// (keys) and fp16 (values) operands by the 8-bit float conversions: a code c
// alone in its byte is the 8-bit float c 2^-9.  The zero-point comes out with
// the row's sum of q for keys, and for values with one matrix step of z
// against the same probabilities, subtracted once a unit, so that it never
// grows with the sequence.  Keys and q meet exactly.  A probability
// times its value's scale is rounded to fp16 (2^-11 relative, an eighth of the
// output's bf16 rounding): the running reference M is the row's maximum score,
// down to a whole number, plus the exponent of the largest value scale so far,
// less 14, so that w = 2^(score - M) s stays below 2^15 and is exact to its 11 bits
// down to 2^-29 of that.  Every sum is fp32.  Scores past 2^23 count times a power
// of two that brings them below it.
#include <type_traits>

#include "internal.hpp"
#include "kv_math.hpp"
#include "spear_ec_kv.h"

namespace spear {
namespace {

constexpr int kUnit = 128;       // tokens of a unit
constexpr int kRows = 16;        // rows of an item
constexpr int kGroups = 256;     // workgroups: one per compute unit of gfx950
constexpr int kXcds = 8;         // consecutive workgroups go to them in turn
constexpr int kWaves = 8;
constexpr int kThreads = 64 * kWaves;
constexpr float kLarge = 0x1p23f;  // scores past it count times a power of two below it

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

// Product of an fp32 value and the lane's token i's fp16 scale (0 .. 31 of the
// unit), the half taken from its pair by the instruction.
__device__ __forceinline__ float times_scale(float v, const u32x4 (&s)[2][2], int i) {
  const uint32_t w = s[i >> 4][(i >> 3) & 1][(i >> 1) & 3];
  // with an addend of +0 this is one mixed-precision instruction
  return __builtin_fmaf(v, half_bits_to_f32((uint16_t)((i & 1) ? w >> 16 : w)), 0.f);
}

// N consecutive floats of a piece, to and from every XCD (device scope).
template <int N>
__device__ __forceinline__ void store_piece(rsrc_t rs, uint32_t at, const float (&v)[N]) {
  if constexpr (N == 4)
    bstore16_dev(rs, at, f32x4{v[0], v[1], v[2], v[3]});
  else
    __builtin_amdgcn_raw_buffer_store_b64(u32x2{__float_as_uint(v[0]), __float_as_uint(v[1])}, rs, at, 0,
                                          kDeviceScope);
}
template <int N>
__device__ __forceinline__ void load_piece(rsrc_t rs, uint32_t at, float (&v)[N]) {
  if constexpr (N == 4) {
    const u32x4 w = bload16_dev(rs, at, 0);
    #pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = __uint_as_float(w[i]);
  } else {
    const u32x2 w = __builtin_amdgcn_raw_buffer_load_b64(rs, at, 0, kDeviceScope);
    v[0] = __uint_as_float(w.x);
    v[1] = __uint_as_float(w.y);
  }
}

// a / b of non-negative counts.
__device__ __forceinline__ int quotient(int a, int b) { return (int)((uint32_t)a / (uint32_t)b); }
__device__ __forceinline__ int64_t quotient(int64_t a, int64_t b) { return (int64_t)div_u64(a, b); }

// Where a workgroup's next piece of work lies.
struct Piece {
  int seq, head, tile;
  int ub, take;           // its units of the item
  int parts, part;        // pieces of the item, this one's number
  int counter;            // arrival counter of the item (its first workgroup)
  int slot0, slot1, step; // slots of piece 0 and 1; the others follow by step
};

template <int D, bool ZEROS, bool SMALL>
__global__ __launch_bounds__(kThreads, 2) void decode_attention_kernel(KvShape s, KvBatch b,
                                                                  KvAttentionArgs a, int* counters,
                                                                  float* slots, uint32_t slot_bytes) {
  __shared__ int64_t before[SMALL ? 1 : kMaxChunks + 1];  // work before each 64 sequences
  __shared__ float osh[kWaves][kRows][D + 4];
  __shared__ float msh[kRows][kRows], lsh[kRows][kRows];
  __shared__ int flag;
  // what the loop over units does not use, out of the registers: the lanes'
  // sequences and work up to them (SMALL), the piece
  __shared__ Seq seqs[SMALL ? 64 : 1];
  __shared__ int uptos[SMALL ? 64 : 1];
  __shared__ Piece kept;
  const int lane = threadIdx.x & 63, wave = wave_id();
  const int n = lane & 15, kb = lane >> 4;
  const int capacity = s.max_pages << s.page_shift;
  const int group = s.group();

  // ---- the split
  const auto seq_at = [&](int i) { return load_seq<kRows, kUnit>(s, b, a.window, i); };
  using count_t = typename std::conditional<SMALL, int, int64_t>::type;
  count_t units = 0, items = 0;
  int longest = 0;
  Seq own{0, 0, 0, 0, 0, 1};  // SMALL: the lane's sequence
  count_t upto = 0;
  if constexpr (SMALL) {
    if (lane < b.n_seqs) own = seq_at(lane);
    const int it = own.tiles * s.kv_heads;
    upto = wave_prefix(it * own.nb);
    items = __builtin_amdgcn_readlane(wave_prefix(it), 63);
    units = __builtin_amdgcn_readlane(upto, 63);
    longest = wave_max(it ? own.nb : 0);
  } else {
    for (int i = lane; i < b.n_seqs; i += 64) {
      const Seq q = seq_at(i);
      const int64_t it = (int64_t)q.tiles * s.kv_heads;
      items += it;
      units += it * q.nb;
      if (it) longest = max(longest, q.nb);
    }
    units = wave_sum(units);
    items = wave_sum(items);
    longest = wave_max(longest);
  }
  if (items == 0) return;
  const count_t run = max((count_t)((units + kGroups - 1) / kGroups), (count_t)kWaves);
  // Pieces of at most c units, one a workgroup and no more of them than there
  // are: as many for each item as for the longest, or, an item's last piece being
  // short, units / c + items of them, or, uneven lengths filling fewer, what lies
  // between that and an even share; at least a step of the waves.  Pieces / runs:
  // one chat of 1000 tokens with 32 heads 7.7 / 23.9 us (runs are a step of all
  // waves at least), 16 chats up to 4096 16.5 / 19.6, 30 chats of 4096 28 / 32,
  // but 20 of 8192, whose 160 items leave a third of the workgroups without one,
  // 48 / 42.  With as many pieces for each item as for the longest alone: 12
  // chats up to 4096 tokens 20.0 us, so 17.5; one to 16 even ones 0.1 to 0.3 less.
  int c = 0;
  if (items <= kGroups) {
    const auto steps = [](int c) { return (c + kWaves - 1) / kWaves; };
    const int even = (int)((units + kGroups - 1) / kGroups);
    const int k = kGroups / (int)items;
    c = (longest + k - 1) / k;
    if (c > kWaves) {
      const int spare = kGroups - (int)items;
      if (spare) c = (int)min((count_t)c, (count_t)((units + spare - 1) / spare));
      if constexpr (SMALL) {
        int low = max(even, kWaves);
        while (low < c && (c - low > low / 16 || steps(low) < steps(c))) {
          const int mid = (low + c) / 2;
          const int n = own.tiles * s.kv_heads * ((own.nb + mid - 1) / mid);
          if (__builtin_amdgcn_readlane(wave_prefix(n), 63) <= kGroups) c = mid;
          else low = mid + 1;
        }
      }
    }
    c = max(c, kWaves);
    if (steps(c) > steps(even) + 1) c = 0;
  }
  count_t pieces = 0;
  const auto parts_of = [&](const Seq& q) { return (q.nb + c - 1) / c; };
  if constexpr (SMALL)
    if (c) {
      upto = wave_prefix(own.tiles * s.kv_heads * parts_of(own));
      pieces = __builtin_amdgcn_readlane(upto, 63);
    }
  if constexpr (SMALL) {  // every wave the same
    seqs[lane] = own;
    uptos[lane] = upto;
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  }
  const int me = (int)(blockIdx.x % kXcds) * (kGroups / kXcds) + (int)(blockIdx.x / kXcds);
  if constexpr (!SMALL)
    if (c) {
      int64_t n = 0;
      for (int i = lane; i < b.n_seqs; i += 64) {
        const Seq q = seq_at(i);
        n += (int64_t)q.tiles * s.kv_heads * parts_of(q);
      }
      pieces = wave_sum(n);
    }
  count_t x0 = c ? (count_t)me : (count_t)me * run;
  const count_t x1 = c ? min(x0 + 1, pieces) : min(x0 + run, units);
  if (x0 >= x1) return;
  const auto weight = [&](int i) {
    const Seq q = seq_at(i);
    return (int64_t)q.tiles * s.kv_heads * (c ? parts_of(q) : q.nb);
  };
  if constexpr (!SMALL)
    if (b.n_seqs > 64) sum_chunks<kWaves>(before, b.n_seqs, weight);

  while (x0 < x1) {
    // ---- the piece that starts with work x0
    Seq q;
    Piece pc;
    count_t seq_base;
    if constexpr (SMALL) {
      const int who = __builtin_amdgcn_readfirstlane(__ffsll((unsigned long long)__ballot(uptos[lane] > x0)) - 1);
      pc.seq = who;
      const Seq& at = seqs[who];
      q.first = __builtin_amdgcn_readfirstlane(at.first);
      q.n = __builtin_amdgcn_readfirstlane(at.n);
      q.len = __builtin_amdgcn_readfirstlane(at.len);
      q.tiles = __builtin_amdgcn_readfirstlane(at.tiles);
      q.u0 = __builtin_amdgcn_readfirstlane(at.u0);
      q.nb = __builtin_amdgcn_readfirstlane(at.nb);
      seq_base = __builtin_amdgcn_readfirstlane(uptos[who]) - q.tiles * s.kv_heads * (c ? parts_of(q) : q.nb);
    } else {
      int64_t base;
      pc.seq = find_seq(before, b.n_seqs, x0, weight, base);
      seq_base = base;
      q = seq_at(pc.seq);
    }
    const int nb = q.nb;
    const count_t local = x0 - seq_base;
    if (c) {
      // a head's pieces one after the other, each for all row tiles
      const int at = (int)local;
      pc.parts = parts_of(q);
      pc.head = at / (q.tiles * pc.parts);
      const int rest = at - pc.head * (q.tiles * pc.parts);
      pc.part = rest / q.tiles;
      pc.tile = rest - pc.part * q.tiles;
      const int per = (nb + pc.parts - 1) / pc.parts;
      pc.ub = pc.part * per;
      pc.take = min(per, nb - pc.ub);
      pc.counter = me - pc.part * q.tiles;
      pc.slot0 = 2 * pc.counter;
      pc.step = 2 * q.tiles;
      pc.slot1 = pc.slot0 + pc.step;
    } else {
      const count_t item = quotient(local, (count_t)nb);
      pc.ub = (int)(local - item * nb);
      pc.take = (int)min((count_t)(nb - pc.ub), x1 - x0);
      const count_t i0 = seq_base + item * nb;  // the item's units
      const int wa = (int)quotient(i0, run), wb = (int)quotient(i0 + nb - 1, run);
      pc.part = me - wa;
      pc.parts = wb - wa + 1;
      pc.counter = wa;
      // a workgroup's first piece takes its slot 0, an item it starts later slot 1
      pc.slot0 = 2 * wa + (i0 == (count_t)wa * run ? 0 : 1);
      pc.slot1 = 2 * (wa + 1);
      pc.step = 2;
      pc.head = (int)quotient(item, (count_t)q.tiles);
      pc.tile = (int)(item - (count_t)pc.head * q.tiles);
    }
    kept = pc;  // for the join; every wave the same
    const int rows_n = q.n * group, start = q.len - q.n;
    const int rows = min(kRows, rows_n - pc.tile * kRows);  // rows of the tile

    // ---- the lane's query row
    const bool live = n < rows;
    const int row = pc.tile * kRows + (live ? n : 0);
    const int tok = row / group;
    const int qh = pc.head * group + row - tok * group;
    const int pos = live ? start + tok : -1;
    const int hi = min(pos, capacity - 1);
    const int lo = a.window && pos >= a.window ? pos - a.window + 1 : 0;
    const uint16_t* qp = a.q + (int64_t)(q.first + tok) * a.q_stride + qh * D + kb * (D / 4);
    u32x4 qf[D / 32];
    #pragma unroll
    for (int i = 0; i < D / 32; ++i) qf[i] = live ? load16(qp + 8 * i) : u32x4{0, 0, 0, 0};
    // tokens that every row, and that some row of the tile sees (its rows are
    // consecutive tokens; padding rows see none)
    const int first_pos = start + pc.tile * kRows / group;
    const int last_pos = start + (pc.tile * kRows + rows - 1) / group;
    const int all_hi = min(first_pos, capacity - 1);
    const int all_lo = a.window && last_pos >= a.window ? last_pos - a.window + 1 : 0;
    const int any_hi = min(last_pos, capacity - 1);
    const int any_lo = a.window && first_pos >= a.window
                           ? min(first_pos - a.window + 1, max(any_hi, 0)) : 0;

    // the unit's 8 blocks, one lane each; positions nobody sees stand for the
    // nearest one that somebody does
    const int per = 1 << (s.page_shift - 4);
    const auto block_of = [&](int ui) {
      if (any_hi < 0) return 0;
      const int at = min(max((q.u0 + pc.ub + ui) * kUnit + 16 * (lane & 7), any_lo & ~15), any_hi);
      const int page = b.page_table[(int64_t)pc.seq * s.max_pages + (at >> s.page_shift)];
      return (unsigned)page < (unsigned)s.pages
                 ? (page * s.kv_heads + pc.head) * per + ((at >> 4) & (per - 1)) : -1;
    };
    const auto spread = [&](int my, int (&kblk)[2], int (&vblk)[2]) {
      my = max(my, 0);
      kblk[0] = __shfl(my, 2 * (n >> 2), 64);
      kblk[1] = __shfl(my, 2 * (n >> 2) + 1, 64);
      vblk[0] = __shfl(my, 2 * kb, 64);
      vblk[1] = __shfl(my, 2 * kb + 1, 64);
    };
    Unit<D, ZEROS> u;
    int kblk[2], vblk[2];
    uint64_t bads = 0;
    int next = 0;
    if (wave < pc.take) {
      const int my = block_of(wave);
      bads = __ballot(my < 0) & 0xFF;
      spread(my, kblk, vblk);
      load_keys(u, a.cache, kblk, n, kb);
      if (wave + kWaves < pc.take) next = block_of(wave + kWaves);
    }
    float qs = 0.f;
    #pragma unroll
    for (int i = 0; i < D / 32; ++i) {
      #pragma unroll
      for (int j = 0; j < 4; ++j) qs += bf16_lo(qf[i][j]) + bf16_hi(qf[i][j]);
      qf[i] = x_permute8(qf[i]);
    }
    qs = join32(join16(qs, sum2), sum2);
    float f = a.scale * kLog2e;  // scores in powers of two

    // mx, ev: the row's largest score, down to a whole number, and value-scale
    // exponent; M = mx + ev - 28
    float mx = -INFINITY, l = 0.f;  // l: the lane's own tokens
    int ev = 0;
    f32x4 o[D / 32][2];
    #pragma unroll
    for (int t = 0; t < D / 32; ++t) o[t][0] = o[t][1] = f32x4{0.f, 0.f, 0.f, 0.f};

    for (int ui = wave; ui < pc.take; ui += kWaves) {
      const int j0 = (q.u0 + pc.ub + ui) * kUnit;
      const bool more = ui + kWaves < pc.take;
      load_values(u, a.cache, vblk, n);
      // all of them before the scores: scheduled among the matrix steps they were
      // issued later and took registers the longer (131001 tokens: 40.5 us; so 37.5)
      __builtin_amdgcn_sched_barrier(0);
      float x[32];
      const float init = (ZEROS ? 0.f : -8.f) * qs;
      #pragma unroll
      for (int t = 0; t < 8; ++t) {
        f32x4 acc = {init, init, init, init};
        #pragma unroll
        for (int i = 0; i < D / 32; ++i) {
          const uint32_t e = low_codes(u.k[t][i]), d = high_codes(u.k[t][i]);
          const u32x4 kf = {bf16_01(e), bf16_23(e), bf16_01(d), bf16_23(d)};
          acc = mfma16x16x32(kf, qf[i], acc);
        }
        #pragma unroll
        for (int i = 0; i < 4; ++i) {
          float v = acc[i];
          if constexpr (ZEROS)
            v -= (float)((u.z[t >> 2][t & 3] >> (8 * i)) & 15u) * qs;
          x[4 * t + i] = times_scale(v, u.ks, 4 * t + i);
        }
      }
      const uint64_t bad = bads;
      if (more) {  // the next keys arrive during the softmax
        bads = __ballot(next < 0) & 0xFF;
        spread(next, kblk, vblk);
        load_keys(u, a.cache, kblk, n, kb);
      }
      if (bad) {  // tokens on a page outside the cache: NaN where they are seen
        #pragma unroll
        for (int h = 0; h < 2; ++h)
          if ((bad >> (2 * kb + h)) & 1)
            #pragma unroll
            for (int i = 0; i < 16; ++i) x[16 * h + i] = __uint_as_float(0x7FC00000u);
        bool seen = false;
        for (int i = 0; i < 8; ++i)
          if ((bad >> i) & 1) seen |= j0 + 16 * i <= any_hi && j0 + 16 * i + 15 >= any_lo;
        if (seen && lane == 0) atomicOr(counters + kCtrError, SPEAR_EC_WS_BAD_PAGE);
      }
      const bool masked = j0 < all_lo || j0 + kUnit - 1 > all_hi;
      uint32_t big_s = 0;  // largest value scale (fp16 bits) of the lane's tokens
      if (masked) {
        #pragma unroll
        for (int i = 0; i < 32; ++i) {
          const int j = j0 + 32 * kb + i;
          const uint32_t w = u.vs[i >> 4][(i >> 3) & 1][(i >> 1) & 3];
          if (j < lo || j > hi) x[i] = -INFINITY;
          else big_s = max(big_s, (i & 1) ? w >> 16 : w & 0xFFFFu);  // elsewhere it may be anything
        }
      } else {
        uint32_t p = u.vs[0][0][0];
        #pragma unroll
        for (int i = 1; i < 16; ++i) p = max_pairs(p, u.vs[i >> 3][(i >> 2) & 1][i & 3]);
        big_s = max(p & 0xFFFFu, p >> 16);
      }
      float top = x[0];
      #pragma unroll
      for (int i = 1; i < 32; ++i) top = fmaxf(top, x[i]);
      top = join32(join16(top, larger), larger);
      // half bits order like their values, and are denormal floats: joined as integers
      big_s = max(big_s, (uint32_t)__shfl_xor((int)big_s, 16, 64));
      big_s = max(big_s, (uint32_t)__shfl_xor((int)big_s, 32, 64));
      top *= f;
      // Past kLarge fp32 leaves a score no digits below 1, and M none for ev: such
      // a row's scores count times a power of two from here on, which tells two of
      // them apart where their last digits do.
      const bool far = fabsf(top) > kLarge && fabsf(top) < INFINITY;
      if (__any(far)) {
        const int k = far ? 23 - __builtin_amdgcn_frexp_expf(top) : 0;
        top = __builtin_amdgcn_ldexpf(top, k);
        mx = __builtin_amdgcn_ldexpf(mx, k);
        f = __builtin_amdgcn_ldexpf(f, k);
      }
      const float nmx = fmaxf(mx, floorf(top));
      const int nev = max(ev, (int)((big_s & 0x7FFFu) >> 10));  // scale < 2^(ev - 14)
      if (__any(nmx != mx || nev != ev)) {
        const float alpha = fast_exp2((nmx == mx ? 0.f : mx - nmx) + (float)(ev - nev));
        l *= alpha;
        #pragma unroll
        for (int t = 0; t < D / 32; ++t)
          #pragma unroll
          for (int h = 0; h < 2; ++h) o[t][h] *= alpha;
        mx = nmx;
        ev = nev;
      }
      const float ref = mx == -INFINITY ? 0.f : mx + (float)(ev - 28);
      u32x4 pf[4];  // probabilities times value scales, 8 tokens a step
      #pragma unroll
      for (int i = 0; i < 32; i += 2) {
        const float p0 = fast_exp2(__builtin_fmaf(x[i], f, -ref));
        const float p1 = fast_exp2(__builtin_fmaf(x[i + 1], f, -ref));
        l += p0 + p1;
        float w0 = times_scale(p0, u.vs, i), w1 = times_scale(p1, u.vs, i + 1);
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
        u32x4 zf = {0x48004800u, 0x48004800u, 0x48004800u, 0x48004800u};  // 8
        if constexpr (ZEROS) {
          const uint32_t a0 = high_codes(u.z[h][d0]);
          const uint32_t a1 = high_codes(u.z[h][d0 + 1]);
          zf = u32x4{f16_01(a0), f16_23(a0), f16_01(a1), f16_23(a1)};
        }
        off = mfma16x16x32_f16(zf, pf[st], off);
        #pragma unroll
        for (int t = 0; t < D / 32; ++t) {
          const uint32_t w0 = u.v[t][h][d0], w1 = u.v[t][h][d0 + 1];
          const uint32_t e0 = low_codes(w0), e1 = low_codes(w1), o0 = high_codes(w0), o1 = high_codes(w1);
          const u32x4 evn = {f16_01(e0), f16_23(e0), f16_01(e1), f16_23(e1)};
          const u32x4 odd = {f16_01(o0), f16_23(o0), f16_01(o1), f16_23(o1)};
          o[t][0] = mfma16x16x32_f16(evn, pf[st], o[t][0]);
          o[t][1] = mfma16x16x32_f16(odd, pf[st], o[t][1]);
        }
      }
      if (more) {
        if (ui + 2 * kWaves < pc.take) next = block_of(ui + 2 * kWaves);
      }
      #pragma unroll
      for (int t = 0; t < D / 32; ++t)
        #pragma unroll
        for (int h = 0; h < 2; ++h) o[t][h] -= off;
    }
    l = join32(join16(l, sum2), sum2);
    l *= fast_exp2((float)(ev - 28));  // relative to mx from here on
    mx = __builtin_amdgcn_ldexpf(mx, __builtin_amdgcn_frexp_expf(a.scale * kLog2e) - __builtin_amdgcn_frexp_expf(f));

    // ---- the waves' results joined
    pc.part = __builtin_amdgcn_readfirstlane(kept.part);
    pc.parts = __builtin_amdgcn_readfirstlane(kept.parts);
    pc.counter = __builtin_amdgcn_readfirstlane(kept.counter);
    pc.slot0 = __builtin_amdgcn_readfirstlane(kept.slot0);
    pc.slot1 = __builtin_amdgcn_readfirstlane(kept.slot1);
    pc.step = __builtin_amdgcn_readfirstlane(kept.step);
    if (kb == 0) {
      msh[wave][n] = mx;
      lsh[wave][n] = l;
    }
    __syncthreads();
    {
      float big = msh[0][n];
      #pragma unroll
      for (int w = 1; w < kWaves; ++w) big = fmaxf(big, msh[w][n]);
      const float kf = mx == -INFINITY ? 0.f : fast_exp2(mx - big + (float)(ev - 28));
      #pragma unroll
      for (int t = 0; t < D / 32; ++t) {
        // byte columns 16 t + 4 kb + i: eight dimensions in a row
        float* dst = &osh[wave][n][32 * t + 8 * kb];
        #pragma unroll
        for (int i = 0; i < 4; ++i) {
          dst[2 * i] = o[t][0][i] * kf;
          dst[2 * i + 1] = o[t][1][i] * kf;
        }
      }
    }
    __syncthreads();
    constexpr int kLanes = kThreads / kRows, kPer = D / kLanes;  // threads a row, elements a thread
    int r = threadIdx.x / kLanes;
    const int d0 = (threadIdx.x % kLanes) * kPer;
    float acc[kPer];
    float big = -INFINITY, sum = 0.f;
    #pragma unroll
    for (int w = 0; w < kWaves; ++w) big = fmaxf(big, msh[w][r]);
    #pragma unroll
    for (int i = 0; i < kPer; ++i) acc[i] = 0.f;
    #pragma unroll
    for (int w = 0; w < kWaves; ++w) {
      const float mw = msh[w][r], lw = lsh[w][r];
      sum += mw == -INFINITY ? lw : lw * fast_exp2(mw - big);
      #pragma unroll
      for (int i = 0; i < kPer; ++i) acc[i] += osh[w][r][d0 + i];
    }

    // ---- a piece of a cut item: leave it, and join the pieces if it is the last
    bool mine = r < rows;
    bool last = true;
    if (pc.parts > 1) {
      const rsrc_t rs = make_rsrc(slots, slot_bytes);
      const uint32_t stride = slot_floats<D>() * 4;
      const auto at_slot = [&](int i) {
        return (uint32_t)(i == 0 ? pc.slot0 : pc.slot1 + pc.step * (i - 1)) * stride;
      };
      if (mine) {
        const uint32_t to = at_slot(pc.part);
        store_piece<kPer>(rs, to + (r * D + d0) * 4, acc);
        if (threadIdx.x % kLanes == 0) {
          bstore_dev(rs, to + (kRows * D + r) * 4, 0, big);
          bstore_dev(rs, to + (kRows * D + kRows + r) * 4, 0, sum);
        }
      }
      wait_vmem();
      __syncthreads();
      if (threadIdx.x == 0) {
        int* ctr = counters + kCtrBand + pc.counter;
        const int arrived = __hip_atomic_fetch_add(ctr, 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        flag = arrived == pc.parts - 1;
        if (arrived == pc.parts - 1) store_dev(ctr, 0);
      }
      __syncthreads();
      last = flag != 0;
      if (last) {
        // kLanes threads a row; with few rows the pieces are dealt to `teams` of them
        int rp = kRows;
        while (rp > 1 && rows <= rp / 2) rp /= 2;
        const int teams = kRows / rp, team = r / rp;
        const int my = r;
        r &= rp - 1;
        const int rr = min(r, rows - 1);  // rows past the tile's load another's
        big = -INFINITY;
        sum = 0.f;
        #pragma unroll
        for (int i = 0; i < kPer; ++i) acc[i] = 0.f;
        constexpr int kBatch = 4;  // pieces in flight
        for (int p = team; p < pc.parts; p += kBatch * teams) {
          float ms[kBatch], ls[kBatch];
          float v[kBatch][kPer];
          #pragma unroll
          for (int i = 0; i < kBatch; ++i) {
            const uint32_t from = at_slot(min(p + i * teams, pc.parts - 1));
            ms[i] = bload_dev(rs, from + (kRows * D + rr) * 4, 0);
            ls[i] = bload_dev(rs, from + (kRows * D + kRows + rr) * 4, 0);
            load_piece<kPer>(rs, from + (rr * D + d0) * 4, v[i]);
          }
          float bn = big;
          #pragma unroll
          for (int i = 0; i < kBatch; ++i) bn = fmaxf(bn, ms[i]);
          if (bn != big) {
            const float kf = fast_exp2(big - bn);
            sum *= kf;
            #pragma unroll
            for (int i = 0; i < kPer; ++i) acc[i] *= kf;
            big = bn;
          }
          #pragma unroll
          for (int i = 0; i < kBatch; ++i) {
            // an empty piece is zeros (or NaN); one counted twice counts once
            float kf = ms[i] == -INFINITY ? 1.f : fast_exp2(ms[i] - big);
            if (p + i * teams < pc.parts) {
              sum += ls[i] * kf;
              #pragma unroll
              for (int j = 0; j < kPer; ++j) acc[j] += v[i][j] * kf;
            }
          }
        }
        if (teams > 1) {  // the teams' results, in order
          float* flat = &osh[0][0][0];
          #pragma unroll
          for (int i = 0; i < kPer; ++i) flat[my * D + d0 + i] = acc[i];
          if (threadIdx.x % kLanes == 0) {
            msh[team][r] = big;
            lsh[team][r] = sum;
          }
          __syncthreads();
          big = -INFINITY;
          sum = 0.f;
          for (int t = 0; t < teams; ++t) big = fmaxf(big, msh[t][r]);
          #pragma unroll
          for (int i = 0; i < kPer; ++i) acc[i] = 0.f;
          for (int t = 0; t < teams; ++t) {
            const float kf = msh[t][r] == -INFINITY ? 1.f : fast_exp2(msh[t][r] - big);
            sum += lsh[t][r] * kf;
            #pragma unroll
            for (int i = 0; i < kPer; ++i) acc[i] += flat[(t * rp + r) * D + d0 + i] * kf;
          }
          mine = team == 0 && r < rows;
        }
      }
    }
    if (last && mine) {
      const int out_row = pc.tile * kRows + r;
      const int t = out_row / group;
      const int64_t at = (int64_t)(q.first + t) * s.q_heads + pc.head * group + out_row - t * group;
      const bool past = start + t >= capacity;  // longer than its page-table row
      float inv = sum == 0.f ? 0.f : 1.f / sum;
      if (past) inv = sum = __uint_as_float(0x7FC00000u);
      uint32_t out[kPer / 2];
      #pragma unroll
      for (int i = 0; i < kPer / 2; ++i) out[i] = pack_bf16(acc[2 * i] * inv, acc[2 * i + 1] * inv);
      uint32_t* dst = reinterpret_cast<uint32_t*>(a.out + at * D + d0);
      #pragma unroll
      for (int i = 0; i < kPer / 2; ++i) dst[i] = out[i];
      if (threadIdx.x % kLanes == 0) {
        if (a.lse) a.lse[at] = (big + log2f(sum)) * kLn2;
        if (past) atomicOr(counters + kCtrError, SPEAR_EC_WS_BAD_PAGE);
      }
    }
    if (c) return;
    __syncthreads();  // the shared arrays are free for the next piece
    x0 += pc.take;
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
  // at most this many items (also where offsets do not ascend), of at most this
  // many units: 32-bit sums for the common calls, one sequence a lane
  const int64_t items = ((int64_t)b.tokens * s.group() / kRows + 1) * b.n_seqs * s.kv_heads;
  const int64_t longest = ((int64_t)s.max_pages << s.page_shift) / kUnit + 2;
  const bool small = b.n_seqs <= 64 && items * longest < (int64_t)1 << 30;
  const auto go = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, dim3(kGroups), dim3(kThreads), 0, st, s, b, a, counters, slots, bytes);
  };
  const auto pick = [&](auto d, auto z) {
    constexpr int D = decltype(d)::value;
    constexpr bool Z = decltype(z)::value;
    if (small) go(decode_attention_kernel<D, Z, true>); else go(decode_attention_kernel<D, Z, false>);
  };
  const std::integral_constant<int, 64> d64;
  const std::integral_constant<int, 128> d128;
  if (s.D == 64) {
    if (s.zeros) pick(d64, std::true_type{}); else pick(d64, std::false_type{});
  } else {
    if (s.zeros) pick(d128, std::true_type{}); else pick(d128, std::false_type{});
  }
  return hipGetLastError();
}

}  // namespace spear

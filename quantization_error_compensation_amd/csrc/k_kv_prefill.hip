// Attention of many rows per sequence over the 4-bit paged key/value cache:
// 256 rows a workgroup, 64 cached tokens a step, matrix cores fed from LDS.
//
// Work.  An item is 256 rows (token, query head) of a sequence that read one
// kv head; its eight waves hold 32 rows each, and walk the tokens that the
// item sees in tiles of 64.  Where the items alone leave compute units idle
// each is cut into runs of tiles, whose results (O, M, l) the last
// one to arrive joins in order.
//
// A tile.  Waves 0-3 load a block's codes each (keys and values) one tile
// ahead and write them to LDS as fp16 matrix operands, so that the codes are
// unpacked once per item and tile: keys as c - z, exact; values as
// (c - z) s 2^-e with e the exponent of the block's largest scale, rounded
// once (2^-11), or, where that scale is more than 128 times the block's smallest,
// as c - z, whose scale the probability takes.  Two waves share a SIMD, w and
// w + 4; the first stages the next tile before its own work on this one, so that
// its matrix steps meet the other's vector work (staging by all eight waves, half
// a block each, before their work: 817 us for prompts of 4096 tokens with 64
// heads of 128, by waves 4-7 after theirs: 812, so: 785 on the same card).
// Items of 128 rows leave the staging to waves 0-3 alone, two tiles ahead, and
// the rows to waves 4-7: such calls read the cache more often per row, and
// waited for it (8 chats of 72 rows behind 4096 tokens: two workgroups of four
// waves a compute unit 45 us, this one 42, with the cut by the items that there
// are and all waves joining 35, with scales and queries held over their whole
// range 36).
//
// Scores.  S^T = K q^T (32x32x16): a lane holds one row and, with key row
// bits 2 and 3 exchanged when the tile is written, runs of 8 consecutive
// tokens, which is the operand order that O^T = V^T P^T wants.  q enters as
// fp16 times a power of two, one for the item's rows (its largest element below
// 2^15) unless that leaves a row's largest below 4, which takes its own then and
// has its scores multiplied: bf16 has 8 significant bits and fp16 eleven, so an
// element is exact unless it is below 2^-19 of its row's largest, and then off by
// at most 2^-27 of it.  A row's probabilities are w = 2^(score + e - M), rounded to fp16
// (2^-11); the sum l takes w 2^-e in fp32.  The reference M is 2^7 below the
// largest score plus its block's e up to some tile and stays there until a lane's
// eight w add up to more than fp16 holds, so most tiles need no maximum: their w
// are taken at once, and again, against a new M, where the sum says so (a
// maximum per tile: 801 and 164 us for prompts of 4096 and a chunk of 512
// tokens, so, before scales and scores were held over their whole range: 789 and
// 159 us).  In a block of scales far apart a token counts with its own exponent
// and only for rows that see it, so that no row depends on the scales of tokens
// without weight in it: half of fp16's smallest step is at most
// 2^-25 kAlike 2 2^-kBelow = 2^-24 of the row's largest product of probability and
// scale, fp32's own rounding of that.
//
// Bound.  A tile of 64 tokens against 64 rows a SIMD is 2048 cycles of matrix
// steps and takes about 4500 (prompts of 4096 tokens 782-807 us, 843-870 TFLOP/s).
// Counters there: matrix cores busy 37% of the time, vector units 50%, LDS 34%:
// two waves a SIMD wait for each other's results rather than for one unit (32
// fewer vector instructions a tile in the staging waves gained 0.5%); more do not
// fit, since items of 256 rows with heads of 128 take all 256 registers (10 or 11
// more live in scratch memory, in the join alone).  Computing a tile's scores
// beside the previous tile's softmax in one wave, with eight or four waves a
// workgroup, took 1.09 to 1.2 times as long; staging by all waves and wave
// priorities gained nothing.
#include <algorithm>
#include <type_traits>
#include <utility>

#include "internal.hpp"
#include "kv_math.hpp"
#include "spear_ec_kv.h"

namespace spear {
namespace {

constexpr int kTileTokens = 64;
// Items fewer than the compute units are cut into runs, up to 32 (one chat of
// 128 rows behind 65536 tokens 77 us, up to 16 104 us) of at least 4 tiles (of
// 4096 tokens: 27 us, at least 2 38 us).  Cut for two workgroups a compute unit,
// 8 chats of 72 rows took 57 us instead of 44.
constexpr int kTileTarget = 256;
constexpr int kTileMaxSplits = 32;
constexpr int kMinTiles = 4;
constexpr int kWaves = 8, kThreads = 64 * kWaves;
constexpr float kNever = -3e38f;     // M before any score: below any, and finite
constexpr float kLarge = 0x1p23f;    // scores past it count times a power of two below it
constexpr float kBelow = 7.f;        // M stands this far below the largest score plus e
constexpr float kApart = 3e38f;      // an exponent that leaves no sum of weights below kMostSum
constexpr float kMostSum = 65504.f;  // of a lane's eight weights, fp16's largest: above it M is raised
// Ratio of a block's value scales that takes them apart: with kBelow it bounds
// what fp16's smallest step costs.  Prompts of 4096 tokens with normal logarithms
// of the scales, of deviation 0.3 / 0.6 / 1 / 2: 792 / 954 / 1522 / 1563 us with a
// ratio of 16, 792 / 791 / 891 / 1545 with 128.
constexpr float kAlike = 128.f;

// One tile as operands.  Rows are padded by 16 bytes, so that eight
// consecutive lanes' 16-byte reads meet different banks and every offset is a
// constant.
template <int D>
struct Staged {
  uint16_t k[kTileTokens][D + 8];  // row: token with bits 2 and 3 exchanged
  uint16_t v[D][kTileTokens + 8];
  float ks[kTileTokens];       // key scale times softmax scale and log2 e, over q's power of two
  float e[4];                  // exponents of the four blocks' value scales, or kApart
  float ea[4];                 // where it is that, their exponents, and their
  float vf[kTileTokens];       // scales over 2^ea, which are not in v
};

// A thread's part of a tile on its way from the cache.
template <int D>
struct Fetched {
  uint32_t k[D / 32], ks, kz;  // token lane / 4: codes, scale, zero-point byte
  uint32_t v[D / 32];          // codes of a value column, D / 8 tokens
  u32x4 vs[D / 64];            // value scales of those tokens
  uint32_t vz[D / 32];         // and zero-point bytes
  bool bad;                    // the block lies on a page outside the cache
  int page;                    // page of the wave's part of the tile fetched next
};

template <int D, bool ZEROS, bool NARROW, bool SMALL>
__global__ __launch_bounds__(kThreads, 2) void prefill_attention_kernel(KvShape s, KvBatch b,
                                                                   KvAttentionArgs a,
                                                                   int* counters, float* slots) {
  __shared__ int64_t before[SMALL ? 1 : kMaxChunks + 1];
  __shared__ __attribute__((aligned(16))) Staged<D> buf[2];
  __shared__ float red[kWaves];
  __shared__ float row_factor[kWaves][32];  // each wave its own, as is
  __shared__ int row_shrunk[kWaves][32];
  __shared__ int flag;
  constexpr int kTileRows = NARROW ? 128 : 256, kRowFloats = D + 2;
  const int lane = threadIdx.x & 63, wave = wave_id();
  const int n = lane & 31, half = lane >> 5;
  const int capacity = s.max_pages << s.page_shift;
  const int group = s.group();

  // ---- the item: heads fastest (one head's items on one XCD), a sequence's
  // last rows first (they see the most tokens)
  const int head = blockIdx.x % s.kv_heads;
  const int rest = blockIdx.x / s.kv_heads;
  const auto seq_at = [&](int i) { return load_seq<kTileRows, kTileTokens>(s, b, a.window, i); };
  const auto cuts = [&](int64_t tiles) {  // runs an item is cut into
    const int items = (int)min(tiles * s.kv_heads, (int64_t)kTileTarget);
    return items ? min(kTileMaxSplits, (kTileTarget + items - 1) / items) : 1;
  };
  int seq, seq_base, splits;
  Seq q;
  if constexpr (SMALL) {
    Seq own{0, 0, 0, 0, 0, 1};
    if (lane < b.n_seqs) own = seq_at(lane);
    splits = cuts(__builtin_amdgcn_readlane(wave_prefix(own.tiles), 63));
    seq = lane_of(own.tiles, rest / splits, seq_base);
    if (seq < 0) return;
    q = seq_of_lane(own, seq);
  } else {
    const auto weight = [&](int i) { return (int64_t)seq_at(i).tiles; };
    sum_chunks<kWaves>(before, b.n_seqs, weight);
    const int64_t tiles = before[(b.n_seqs + 63) / 64];
    splits = cuts(tiles);
    if (rest / splits >= tiles) return;
    int64_t base;
    seq = find_seq(before, b.n_seqs, rest / splits, weight, base);
    seq_base = (int)base;
    q = seq_at(seq);
  }
  const int x = rest / splits, split = rest - x * splits;
  const int tile = q.tiles - 1 - (x - seq_base);
  const int rows_n = q.n * group;

  // ---- tokens that the item's rows see
  const int row0 = tile * kTileRows, row1 = min(row0 + kTileRows, rows_n) - 1;
  const int start = q.len - q.n;  // position of the sequence's first row
  const int item_hi = min(start + row1 / group, capacity - 1);
  const int pos0 = start + row0 / group;
  const int item_lo = a.window ? max(0, min(pos0, capacity - 1) - a.window + 1) : 0;
  const int t0 = item_lo / kTileTokens;
  const int nt = item_hi < 0 ? 0 : item_hi / kTileTokens - t0 + 1;
  // runs of at least kMinTiles tiles: short items are cut less, or not at all
  const int per = max((nt + splits - 1) / splits, kMinTiles);
  const int parts = max(1, (nt + per - 1) / per);
  if (split >= parts) return;
  const int tb = min(nt, split * per), te = min(nt, tb + per);

  // ---- the lane's query row
  const int row = row0 + (NARROW ? wave - 4 : wave) * 32 + n;
  const bool live = row < rows_n && (!NARROW || wave >= 4);
  const int tok = live ? row / group : 0;
  const int qh = head * group + (live ? row - tok * group : 0);
  const int pos = live ? start + tok : -1;
  const int hi = live ? min(pos, capacity - 1) : 0x7FFFFFFF;  // no row: nothing to mask
  const int lo = a.window && pos >= a.window ? pos - a.window + 1 : 0;
  u32x4 qf[D / 16];
  float big = 0.f;  // the row's largest element
  {
    const uint16_t* qp = a.q + (int64_t)(q.first + tok) * a.q_stride + qh * D + 8 * half;
    #pragma unroll
    for (int i = 0; i < D / 16; ++i) {
      qf[i] = pos >= 0 ? load16(qp + 16 * i) : u32x4{0, 0, 0, 0};  // padding may hold anything
      #pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float f0 = fabsf(bf16_lo(qf[i][j])), f1 = fabsf(bf16_hi(qf[i][j]));
        if (f0 < INFINITY) big = fmaxf(big, f0);
        if (f1 < INFINITY) big = fmaxf(big, f1);
      }
    }
  }
  big = join32(big, larger);
  float most_q = big;
  #pragma unroll
  for (int o = 16; o > 0; o >>= 1) most_q = fmaxf(most_q, __shfl_xor(most_q, o, 64));
  if (lane == 0) red[wave] = most_q;
  __syncthreads();
  for (int i = 0; i < kWaves; ++i) most_q = fmaxf(most_q, red[i]);
  // The item's power of two, and the row's own where the item's does not leave
  // its largest element between 2^2 and 2^15.  The bounds keep every factor finite
  // for softmax scales up to 2^64.
  const int qe = min(60, max(-26, 15 - __builtin_amdgcn_frexp_expf(most_q)));
  const int at_qe = __builtin_amdgcn_frexp_expf(big) + qe;
  const int own_qe = big == 0.f || (at_qe >= 3 && at_qe <= 15)
                         ? qe : min(min(127, qe + 126), max(-113, 15 - __builtin_amdgcn_frexp_expf(big)));
  bool scaled = __any(own_qe != qe);
  row_factor[wave][n] = __builtin_amdgcn_ldexpf(1.f, qe - own_qe);
  row_shrunk[wave][n] = 0;
  const float qmul = __builtin_amdgcn_ldexpf(1.f, own_qe);
  #pragma unroll
  for (int i = 0; i < D / 16; ++i) {
    const u32x4 r = x_permute8(qf[i]);
    #pragma unroll
    for (int j = 0; j < 4; ++j) {
      float f0 = bf16_lo(r[j]), f1 = bf16_hi(r[j]);
      // an infinity becomes NaN: its row's scores are all NaN then
      f0 = fabsf(f0) < INFINITY ? f0 * qmul : __uint_as_float(0x7FC00000u);
      f1 = fabsf(f1) < INFINITY ? f1 * qmul : __uint_as_float(0x7FC00000u);
      qf[i][j] = pack_f16(f0, f1);
    }
  }
  const float kmul = a.scale * kLog2e * __builtin_amdgcn_ldexpf(1.f, -qe);
  int all_lo = lo, all_hi = hi;
  int any_lo = live && hi >= lo ? lo : 0x7FFFFFFF, any_hi = live ? hi : -1;
  #pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    all_lo = max(all_lo, __shfl_xor(all_lo, o, 64));
    all_hi = min(all_hi, __shfl_xor(all_hi, o, 64));
    any_lo = min(any_lo, __shfl_xor(any_lo, o, 64));
    any_hi = max(any_hi, __shfl_xor(any_hi, o, 64));
  }
  all_lo = __builtin_amdgcn_readfirstlane(all_lo);
  all_hi = __builtin_amdgcn_readfirstlane(all_hi);
  any_lo = __builtin_amdgcn_readfirstlane(any_lo);
  any_hi = __builtin_amdgcn_readfirstlane(any_hi);

  // ---- staging: waves 0-3 fetch block w of a tile
  const bool stages = wave < 4;
  const int part = wave & 3;
  bool any_bad = false;
  // The wave's part of tile t: positions outside the item's range stand for
  // the nearest one inside.  The page number is left as loaded until it is
  // used a tile later (taken for a scalar it would be waited for at once; the
  // lane's zero keeps the compiler from that).
  int zero = 0;
  asm("" : "+v"(zero));
  const auto place = [&](int t) {
    return min(max(t * kTileTokens + 16 * part, item_lo & ~15), item_hi);
  };
  const int* table = b.page_table + (int64_t)seq * s.max_pages;
  const auto page_of = [&](int t) { return table[(place(t) >> s.page_shift) + zero]; };
  const auto block_of = [&](int page, int t) {
    page = __builtin_amdgcn_readfirstlane(page);
    const int pb = 1 << (s.page_shift - 4);
    return (unsigned)page < (unsigned)s.pages
               ? (page * s.kv_heads + head) * pb + ((place(t) >> 4) & (pb - 1)) : -1;
  };
  // values, head_dim 64: two lanes a column, eight of its tokens each
  const int col = D == 128 ? lane : lane >> 1, half_col = D == 128 ? 0 : lane & 1;
  const auto fetch = [&](Fetched<D>& fe, int blk) {
    const bool bad = fe.bad = blk < 0;
    any_bad |= bad;
    const int64_t bl = bad ? 0 : blk;
    const uint8_t* c = a.cache.codes + bl * (16 * D);
    const uint8_t* sc = reinterpret_cast<const uint8_t*>(a.cache.scales) + bl * 64;
    const auto codes = [&](const uint8_t* p, uint32_t (&to)[D / 32]) {
      if constexpr (D == 128) {
        const u32x4 w = load16(p + 16 * lane);
        #pragma unroll
        for (int i = 0; i < 4; ++i) to[i] = w[i];
      } else {
        const u32x2 w = *reinterpret_cast<const u32x2*>(p + 8 * lane);
        #pragma unroll
        for (int i = 0; i < 2; ++i) to[i] = w[i];
      }
    };
    {
      codes(c, fe.k);
      fe.ks = *reinterpret_cast<const uint16_t*>(sc + 2 * (lane >> 2));
      if constexpr (ZEROS) fe.kz = a.cache.zeros[bl * 16 + (lane >> 2)];
    }
    {
      codes(c + 8 * D, fe.v);
      #pragma unroll
      for (int i = 0; i < D / 64; ++i) fe.vs[i] = load16(sc + 32 + 16 * (i + half_col) + zero);
      if constexpr (ZEROS) {
        const uint8_t* zp = a.cache.zeros + bl * 16 + 8 * half_col + zero;
        #pragma unroll
        for (int i = 0; i < D / 32; ++i) fe.vz[i] = *reinterpret_cast<const uint32_t*>(zp + 4 * i);
      }
    }
  };
  const auto store = [&](Staged<D>& to, const Fetched<D>& fe, int t) {
    const bool bad = fe.bad;
    const int j0 = t * kTileTokens + 16 * part;  // the block's first position
    {
      const int token = 16 * part + (lane >> 2);
      const int r = (token & ~12) | ((token & 4) << 1) | ((token & 8) >> 1);
      f16x2 z = as_f16x2(0xC800C800u);  // -8
      if constexpr (ZEROS) z = as_f16x2(f16_01((fe.kz & 15u) * 0x0101u | 0x8080u));
      #pragma unroll
      for (int i = 0; i < D / 32; ++i) {
        const uint32_t e = low_codes(fe.k[i]), o = high_codes(fe.k[i]);
        const u32x4 c = {as_u32(as_f16x2(f16_01(e)) + z), as_u32(as_f16x2(f16_23(e)) + z),
                         as_u32(as_f16x2(f16_01(o)) + z), as_u32(as_f16x2(f16_23(o)) + z)};
        *reinterpret_cast<u32x4*>(&to.k[r][8 * ((D / 32) * (lane & 3) + i)]) = c;
      }
      if ((lane & 3) == 0)
        to.ks[token] = bad ? __uint_as_float(0x7FC00000u) : half_bits_to_f32((uint16_t)fe.ks) * kmul;
    }
    {
      // the lane's value scales; slots that nobody sees count as 0
      constexpr int kPairs = D / 16;
      uint32_t vs[kPairs];
      #pragma unroll
      for (int i = 0; i < kPairs; ++i) vs[i] = fe.vs[i >> 2][i & 3];
      if (bad || j0 < item_lo || j0 + 15 > item_hi) {
        #pragma unroll
        for (int i = 0; i < kPairs; ++i) {
          const int j = j0 + 8 * half_col + 2 * i;
          if (bad || j < item_lo || j > item_hi) vs[i] &= 0xFFFF0000u;
          if (bad || j + 1 < item_lo || j + 1 > item_hi) vs[i] &= 0x0000FFFFu;
        }
      }
      // largest and smallest, in pairs
      uint32_t mx[kPairs], mn[kPairs];
      #pragma unroll
      for (int i = 0; i < kPairs; ++i) mx[i] = mn[i] = vs[i];
      #pragma unroll
      for (int w = kPairs / 2; w > 0; w /= 2)
        #pragma unroll
        for (int i = 0; i < w; ++i) {
          mx[i] = max_pairs(mx[i], mx[i + w]);
          mn[i] = min_pairs(mn[i], mn[i + w]);
        }
      if constexpr (D == 64) {
        mx[0] = max_pairs(mx[0], (uint32_t)__shfl_xor((int)mx[0], 1, 64));
        mn[0] = min_pairs(mn[0], (uint32_t)__shfl_xor((int)mn[0], 1, 64));
      }
      const uint32_t most = max(mx[0] & 0xFFFFu, mx[0] >> 16);
      const uint32_t least = min(mn[0] & 0xFFFFu, mn[0] >> 16);
      // every scale is below 2^e; at most 2^14, so that 2^-e is an fp16 value
      const int e = (int)((most & 0x7FFFu) >> 10) - 14;
      if (lane == 0) to.e[part] = (float)e;
      const bool far_apart = __any(half_bits_to_f32((uint16_t)most) > kAlike * half_bits_to_f32((uint16_t)least));
      const auto put = [&](uint32_t unit, auto apart) {
        #pragma unroll
        for (int i = 0; i < D / 64; ++i) {  // 8 tokens: one chunk of two dimensions
          f16x2 z[4], sg[4];  // less the zero-point: before the scale, or with it for 8
          const auto value = [](uint32_t c, f16x2 z, f16x2 sg) {
            if constexpr (ZEROS) return as_u32((as_f16x2(c) + z) * sg);
            else return as_u32(__builtin_elementwise_fma(as_f16x2(c), sg, z));
          };
          #pragma unroll
          for (int j = 0; j < 4; ++j) {
            sg[j] = decltype(apart)::value ? as_f16x2(unit) : as_f16x2(vs[4 * i + j]) * as_f16x2(unit);
            z[j] = sg[j] * as_f16x2(0xC800C800u);  // -8 of them, exact
          }
          if constexpr (ZEROS) {
            const uint32_t a0 = high_codes(fe.vz[2 * i]) | 0x80808080u;
            const uint32_t a1 = high_codes(fe.vz[2 * i + 1]) | 0x80808080u;
            z[0] = as_f16x2(f16_01(a0));
            z[1] = as_f16x2(f16_23(a0));
            z[2] = as_f16x2(f16_01(a1));
            z[3] = as_f16x2(f16_23(a1));
          }
          #pragma unroll
          for (int odd = 0; odd < 2; ++odd) {
            const uint32_t w0 = odd ? high_codes(fe.v[2 * i]) : low_codes(fe.v[2 * i]);
            const uint32_t w1 = odd ? high_codes(fe.v[2 * i + 1]) : low_codes(fe.v[2 * i + 1]);
            const u32x4 c = {value(f16_01(w0), z[0], sg[0]), value(f16_23(w0), z[1], sg[1]),
                             value(f16_01(w1), z[2], sg[2]), value(f16_23(w1), z[3], sg[3])};
            *reinterpret_cast<u32x4*>(&to.v[2 * col + odd][16 * part + 8 * (i + half_col)]) = c;
          }
        }
      };
      put(pack_f16(__builtin_amdgcn_ldexpf(1.f, -e), __builtin_amdgcn_ldexpf(1.f, -e)), std::false_type{});
      // Scales far apart (a slot that counts as 0 makes them so, at an edge): the
      // values again, without them, behind the stores that are all nearly every
      // block needs (prompts of 4096 tokens 803 us; with the branch before them
      // 808; without the test at all 790 then, 771 against 783 now).
      if (far_apart) {
        put(0x3C003C00u, std::true_type{});
        if (lane == 0) {
          to.e[part] = kApart;
          to.ea[part] = (float)e;
        }
        if (lane <= half_col)  // a lane for each of the block's tokens
          #pragma unroll
          for (int i = 0; i < kPairs; ++i) {
            float* f = &to.vf[16 * part + 8 * half_col + 2 * i];
            f[0] = __builtin_amdgcn_ldexpf(half_bits_to_f32((uint16_t)vs[i]), -e);
            f[1] = __builtin_amdgcn_ldexpf(half_bits_to_f32((uint16_t)(vs[i] >> 16)), -e);
          }
      }
    }
  };

  // M, the lane's own share of l, and O
  float m = kNever, l = 0.f;
  bool started = false;  // M stands
  f32x16 o[D / 32];
  #pragma unroll
  for (int i = 0; i < D / 32; ++i)
    #pragma unroll
    for (int r = 0; r < 16; ++r) o[i][r] = 0.f;
  f32x16 sc[2];  // scores of a tile
  u32x4 pf[4];   // and its probabilities, the operands of its values
  const auto seen = [&](int ti) {
    const int j0 = (t0 + ti) * kTileTokens;
    return j0 <= any_hi && j0 + kTileTokens - 1 >= any_lo;
  };
  // Order of D / 8 matrix steps and the reads of their operands: four ahead (none
  // set: prompts of 4096 tokens 793 us, for the scores 780, for both 773).
  const auto read_ahead = [] {
    __builtin_amdgcn_sched_group_barrier(0x100, 4, 0);
    #pragma unroll
    for (int i = 0; i < D / 8 - 4; ++i) {
      __builtin_amdgcn_sched_group_barrier(0x8, 1, 0);
      __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
    }
    __builtin_amdgcn_sched_group_barrier(0x8, 4, 0);
  };
  const auto scores = [&](const Staged<D>& st) {
    #pragma unroll
    for (int r = 0; r < 16; ++r) sc[0][r] = sc[1][r] = 0.f;
    #pragma unroll
    for (int i = 0; i < D / 16; ++i)
      #pragma unroll
      for (int t = 0; t < 2; ++t) {
        const u32x4 kf = *reinterpret_cast<const u32x4*>(&st.k[32 * t + n][16 * i + 8 * half]);
        sc[t] = mfma32x32x16_f16(kf, qf[i], sc[t]);
      }
    read_ahead();
  };
  // The lane's tokens of a tile: 16 g + 8 half + 0 .. 7 for g = 0 .. 3.
  const auto key_scale = [&](const Staged<D>& st, int g, f32x4 (&k)[2]) {
    k[0] = *reinterpret_cast<const f32x4*>(&st.ks[16 * g + 8 * half]);
    k[1] = *reinterpret_cast<const f32x4*>(&st.ks[16 * g + 8 * half + 4]);
  };
  const auto hidden = [&](int j0, int g, int r) {
    const int j = j0 + 16 * g + 8 * half + r;
    return j < lo || j > hi;
  };
  // Their value scales over 2^e where these are not in the values.
  const auto value_scale = [&](const Staged<D>& st, int g, f32x4 (&f)[2]) {
    f[0] = *reinterpret_cast<const f32x4*>(&st.vf[16 * g + 8 * half]);
    f[1] = *reinterpret_cast<const f32x4*>(&st.vf[16 * g + 8 * half + 4]);
  };
  // Probabilities against M as it is, and their sums by group.
  const auto weights = [&](const Staged<D>& st, f32x4 eb, f32x4& sums) {
    #pragma unroll
    for (int g = 0; g < 4; ++g) {
      const float ref = m - eb[g];
      f32x4 k[2];
      key_scale(st, g, k);
      float sum = 0.f;
      #pragma unroll
      for (int r = 0; r < 8; r += 2) {
        const int at = 8 * (g & 1) + r;
        const float w0 = fast_exp2(fmaf(sc[g >> 1][at], k[r >> 2][r & 3], -ref));
        const float w1 = fast_exp2(fmaf(sc[g >> 1][at + 1], k[r >> 2][(r & 3) + 1], -ref));
        sum += w0 + w1;
        pf[g][r >> 1] = pack_f16(w0, w1);
      }
      sums[g] = sum;
    }
  };
  // The same of group g with tokens that the row does not see, and, in a block
  // of scales far apart, times its token's.
  const auto weights_of = [&](auto apart, int g, const Staged<D>& st, float e, int j0) {
    const float ref = m - e;
    f32x4 k[2], f[2];
    key_scale(st, g, k);
    if constexpr (decltype(apart)::value) value_scale(st, g, f);
    float sum = 0.f;
    #pragma unroll
    for (int r = 0; r < 8; r += 2) {
      const int at = 8 * (g & 1) + r;
      float w0 = fast_exp2(fmaf(sc[g >> 1][at], k[r >> 2][r & 3], -ref));
      float w1 = fast_exp2(fmaf(sc[g >> 1][at + 1], k[r >> 2][(r & 3) + 1], -ref));
      if (hidden(j0, g, r)) w0 = 0.f;
      if (hidden(j0, g, r + 1)) w1 = 0.f;
      sum += w0 + w1;
      if constexpr (decltype(apart)::value) {
        w0 *= f[r >> 2][r & 3];
        w1 *= f[r >> 2][(r & 3) + 1];
      }
      pf[g][r >> 1] = pack_f16(w0, w1);
    }
    return sum;
  };
  // Largest score of group g plus e, there of the token's own scale.
  const auto largest_of = [&](auto apart, int g, const Staged<D>& st, float e, int j0) {
    f32x4 k[2], f[2];
    key_scale(st, g, k);
    if constexpr (decltype(apart)::value) value_scale(st, g, f);
    float top = kNever;
    #pragma unroll
    for (int r = 0; r < 8; ++r) {
      float own = e;
      if constexpr (decltype(apart)::value)
        own += (float)(__builtin_amdgcn_frexp_expf(f[r >> 2][r & 3]) - 1);
      const float x = fmaf(sc[g >> 1][8 * (g & 1) + r], k[r >> 2][r & 3], own);
      if (!hidden(j0, g, r)) top = fmaxf(top, x);
    }
    return top;
  };
  // M becomes the largest so far less kBelow, a whole number, so that M - e is
  // exact.
  const auto raise = [&](float top) {
    const float mn = fmaxf(m, floorf(top - kBelow));
    const float alpha = fast_exp2(m - mn);
    l *= alpha;
    #pragma unroll
    for (int i = 0; i < D / 32; ++i) o[i] *= alpha;
    m = mn;
  };
  const auto softmax = [&](const Staged<D>& st, int j0) {
    f32x4 eb = *reinterpret_cast<const f32x4*>(st.e);
    f32x4 sums;
    bool done = false;
    if (started && !scaled && j0 >= all_lo && j0 + kTileTokens - 1 <= all_hi) {
      weights(st, eb, sums);
      const float most = fmaxf(fmaxf(sums[0], sums[1]), fmaxf(sums[2], sums[3]));
      done = !__any(most > kMostSum);
    }
    if (!done) {
      if (scaled) {
        const float f = row_factor[wave][n];
        sc[0] *= f;
        sc[1] *= f;
      }
      const std::true_type apart;
      const std::false_type alike;
      bool is_apart[4];
      #pragma unroll
      for (int g = 0; g < 4; ++g) {
        is_apart[g] = __builtin_amdgcn_readfirstlane(__float_as_int(eb[g])) == __float_as_int(kApart);
        if (is_apart[g]) eb[g] = st.ea[g];
      }
      const auto largest = [&] {
        float top = kNever;
        #pragma unroll
        for (int g = 0; g < 4; ++g)
          top = fmaxf(top, is_apart[g] ? largest_of(apart, g, st, eb[g], j0) : largest_of(alike, g, st, eb[g], j0));
        return join32(top, larger);
      };
      float top = largest();
      const bool far = fabsf(top) > kLarge && fabsf(top) < -kNever;
      if (__any(far)) {
        asm volatile("" ::: "memory");  // scales are read again: kept, they took 32 registers
        const int k = far ? __builtin_amdgcn_frexp_expf(top) - 23 : 0;
        const float f = __builtin_amdgcn_ldexpf(1.f, -k);
        sc[0] *= f;
        sc[1] *= f;
        if (m != kNever) m *= f;
        row_factor[wave][n] *= f;
        row_shrunk[wave][n] += k;
        scaled = true;
        top = largest();
      }
      raise(top);
      started = true;
      #pragma unroll
      for (int g = 0; g < 4; ++g)
        sums[g] = is_apart[g] ? weights_of(apart, g, st, eb[g], j0) : weights_of(alike, g, st, eb[g], j0);
    }
    #pragma unroll
    for (int g = 0; g < 4; ++g) l += __builtin_amdgcn_ldexpf(sums[g], -(int)eb[g]);
  };
  const auto values = [&](const Staged<D>& st) {
    #pragma unroll
    for (int g = 0; g < 4; ++g)
      #pragma unroll
      for (int i = 0; i < D / 32; ++i) {
        const u32x4 vf = *reinterpret_cast<const u32x4*>(&st.v[32 * i + n][16 * g + 8 * half]);
        o[i] = mfma32x32x16_f16(vf, pf[g], o[i]);
      }
    read_ahead();
  };
  // What the waves hand each other lies in LDS: nothing else is waited for.
  const auto meet = [&] {
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
  };
  // Tiles reach LDS by way of registers: the one that lies in f, `ti`, is
  // stored a tile ahead of its use, then the one kAhead later fetched into f.
  constexpr int kAhead = NARROW ? 2 : 1;
  const auto fetch_tile = [&](Fetched<D>& f, int ti) {
    if (ti < te) fetch(f, block_of(f.page, t0 + ti));
    if (ti + kAhead < te) f.page = page_of(t0 + ti + kAhead);
  };
  const auto advance = [&](Fetched<D>& f, int ti) {
    if (ti >= te) return;
    store(buf[ti & 1], f, t0 + ti);
    fetch_tile(f, ti + kAhead);
  };
  const auto attend = [&](int ti) {
    if (!seen(ti)) return;
    scores(buf[ti & 1]);
    softmax(buf[ti & 1], (t0 + ti) * kTileTokens);
    values(buf[ti & 1]);
  };
  if (tb < te) {
    Fetched<D> f[kAhead];
    if (stages) {
      #pragma unroll
      for (int i = 0; i < kAhead; ++i) f[i].page = page_of(t0 + min(tb + i, te - 1));
      #pragma unroll
      for (int i = 0; i < kAhead; ++i) fetch_tile(f[i], tb + i);
      advance(f[0], tb);
    }
    if constexpr (NARROW) {
      if (stages) {
        for (int ti = tb; ti < te; ti += 2) {
          meet();
          advance(f[1], ti + 1);
          if (ti + 1 < te) {
            meet();
            advance(f[0], ti + 2);
          }
        }
      } else {
        for (int ti = tb; ti < te; ++ti) {
          meet();
          attend(ti);
        }
      }
    } else {
      for (int ti = tb; ti < te; ++ti) {
        meet();
        if (stages) advance(f[0], ti + 1);
        attend(ti);
      }
    }
  }
  l += __shfl_xor(l, 32, 64);
  if (scaled) {  // rows of large scores: O over l, M their log-sum
    const int k = row_shrunk[wave][n];
    const bool far = k > 0 && l > 0.f;
    const float inv = far ? 1.f / l : 1.f;
    if (far) {
      m = __builtin_amdgcn_ldexpf(m + log2f(l), k);
      l = 1.f;
    }
    #pragma unroll
    for (int i = 0; i < D / 32; ++i) o[i] *= inv;
  }

  if (any_bad && lane == 0) atomicOr(counters + kCtrError, SPEAR_EC_WS_BAD_PAGE);
  // Eight bytes of a row's output and its log-sum; the reciprocal of l.
  const auto finish = [&](int row, float m, float l, bool first) {
    const int tok = row / group;
    const int64_t at = (int64_t)(q.first + tok) * s.q_heads + head * group + row - tok * group;
    const bool past = start + tok >= capacity;  // longer than its page-table row
    float inv = l == 0.f ? 0.f : 1.f / l;
    if (past) inv = l = __uint_as_float(0x7FC00000u);
    if (first) {
      if (a.lse) a.lse[at] = (m + log2f(l)) * kLn2;
      if (past) atomicOr(counters + kCtrError, SPEAR_EC_WS_BAD_PAGE);
    }
    return std::make_pair(a.out + at * D, inv);
  };
  const auto put = [](uint16_t* out, float inv, const float (&v)[4]) {
    u32x2 w;
    w.x = pack_bf16(v[0] * inv, v[1] * inv);
    w.y = pack_bf16(v[2] * inv, v[3] * inv);
    *reinterpret_cast<u32x2*>(out) = w;
  };

  // ---- the lane's row: dimensions 32 i + 8 (r / 4) + 4 half + r % 4
  if (parts == 1) {
    if (!live) return;
    const auto [out, inv] = finish(row, m, l, half == 0);
    #pragma unroll
    for (int i = 0; i < D / 32; ++i)
      #pragma unroll
      for (int r = 0; r < 16; r += 4) {
        const float v[4] = {o[i][r], o[i][r + 1], o[i][r + 2], o[i][r + 3]};
        put(out + 32 * i + 2 * r + 4 * half, inv, v);
      }
    return;
  }

  // ---- a run's results: [D / 4][rows][4], then M and l, so that lanes next to
  // each other store next to each other; the last workgroup joins the runs
  const int item = x * s.kv_heads + head;
  const uint32_t bytes = kRowFloats * kTileRows * 4;
  const auto slot = [&](int sp) {
    return make_rsrc(slots + (int64_t)(item * splits + sp) * (kRowFloats * kTileRows), bytes);
  };
  constexpr uint32_t kAtM = D * kTileRows * 4, kAtL = kAtM + kTileRows * 4;
  if (live) {
    const rsrc_t rs = slot(split);
    const uint32_t me = row - row0;
    #pragma unroll
    for (int i = 0; i < D / 32; ++i)
      #pragma unroll
      for (int r = 0; r < 16; r += 4)
        bstore16_dev(rs, ((8 * i + (r >> 1) + half) * kTileRows + me) * 16, 0,
                     f32x4{o[i][r], o[i][r + 1], o[i][r + 2], o[i][r + 3]});
    if (half == 0) {
      bstore_dev(rs, kAtM + me * 4, 0, m);
      bstore_dev(rs, kAtL + me * 4, 0, l);
    }
  }
  wait_vmem();
  __syncthreads();
  if (threadIdx.x == 0) {
    int* ctr = counters + kCtrBand + item;
    const int arrived = __hip_atomic_fetch_add(ctr, 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    flag = arrived == parts - 1;
    if (arrived == parts - 1) store_dev(ctr, 0);
  }
  __syncthreads();
  if (!flag) return;
  // a thread: kChunk of the D / 4 chunks of a row,
  // kBatch runs in flight
  constexpr int kChunk = D / 4 * kTileRows / kThreads, kBatch = NARROW ? 4 : 1;
  const int r = threadIdx.x % kTileRows, c0 = threadIdx.x / kTileRows * kChunk;
  if (row0 + r > row1) return;
  float most = kNever, sum = 0.f;
  float acc[kChunk][4];
  #pragma unroll
  for (int c = 0; c < kChunk; ++c)
    #pragma unroll
    for (int i = 0; i < 4; ++i) acc[c][i] = 0.f;
  for (int p = 0; p < parts; p += kBatch) {
    float ms[kBatch], ls[kBatch];
    u32x4 v[kBatch][kChunk];
    #pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const rsrc_t rs = slot(min(p + i, parts - 1));
      ms[i] = bload_dev(rs, kAtM + r * 4, 0);
      ls[i] = bload_dev(rs, kAtL + r * 4, 0);
      #pragma unroll
      for (int c = 0; c < kChunk; ++c) v[i][c] = bload16_dev(rs, ((c0 + c) * kTileRows + r) * 16, 0);
    }
    float bn = most;
    #pragma unroll
    for (int i = 0; i < kBatch; ++i) bn = fmaxf(bn, ms[i]);
    const float kf = fast_exp2(most - bn);
    sum *= kf;
    #pragma unroll
    for (int c = 0; c < kChunk; ++c)
      #pragma unroll
      for (int j = 0; j < 4; ++j) acc[c][j] *= kf;
    most = bn;
    #pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      if (p + i >= parts) break;
      const float k = fast_exp2(ms[i] - most);
      sum += ls[i] * k;
      #pragma unroll
      for (int c = 0; c < kChunk; ++c)
        #pragma unroll
        for (int j = 0; j < 4; ++j) acc[c][j] += __uint_as_float(v[i][c][j]) * k;
    }
  }
  const auto [out, inv] = finish(row0 + r, most, sum, c0 == 0);
  #pragma unroll
  for (int c = 0; c < kChunk; ++c) put(out + 4 * (c0 + c), inv, acc[c]);
}

// A call's rows are taken 128 at a time where its sequences have no more on
// average, or where that leaves fewer items than half the compute units, so that
// 256 rows an item would leave long runs or a large join; 256 at a time
// elsewhere.  Calls of 64 heads of 128 behind 4096 tokens, 128 rows / 256 rows:
// one chat of 64 tokens 31 / 50 us, of 128 39 / 46, of 256 59 / 58, of 1024
// 172 / 146; 32 chats of 16 tokens 101 / 130, of 32 199 / 165; 8 chats of 17
// 56 / 51.
bool narrow(const KvShape& s, int n_seqs, int tokens) {
  const int64_t rows = ((int64_t)tokens * s.group() + n_seqs - 1) / n_seqs;
  return rows <= 128 || (rows + 127) / 128 * n_seqs * s.kv_heads < kTileTarget / 2;
}

// Items of a call are at most this many (their number is device data).
int64_t item_bound(const KvShape& s, int n_seqs, int tokens, int tile_rows) {
  const int64_t rows = (int64_t)tokens * s.group();
  return (rows / tile_rows + std::min(n_seqs, tokens)) * s.kv_heads;
}

}  // namespace

size_t kv_prefill_workspace(const KvShape& s) {
  // items are cut where there are fewer than the target: into fewer than twice
  // the target runs, of 256 rows or fewer
  return sizeof(int) * kCounterSlots + sizeof(float) * 2 * kTileTarget * 256 * (s.D + 2);
}

hipError_t launch_kv_prefill(const KvShape& s, const KvBatch& b, const KvAttentionArgs& a,
                             void* workspace, hipStream_t st) {
  int* counters = static_cast<int*>(workspace);
  float* slots = reinterpret_cast<float*>(counters + kCounterSlots);
  const auto go = [&](auto d, auto z, auto w) {
    constexpr int D = decltype(d)::value;
    constexpr bool N = decltype(w)::value;
    // enough for the kernel's rule whatever the offsets: items are cut below the
    // target, into fewer than twice the target runs
    const int64_t items = item_bound(s, b.n_seqs, b.tokens, N ? 128 : 256);
    const int64_t grid = std::max<int64_t>(items, 2 * kTileTarget);
    const auto launch = [&](auto kernel) {
      hipLaunchKernelGGL(kernel, dim3((unsigned)grid), dim3(kThreads), 0, st, s, b, a, counters, slots);
    };
    if (b.n_seqs <= 64) launch(prefill_attention_kernel<D, decltype(z)::value, N, true>);
    else launch(prefill_attention_kernel<D, decltype(z)::value, N, false>);
  };
  const auto pick = [&](auto d, auto z) {
    if (narrow(s, b.n_seqs, b.tokens)) go(d, z, std::true_type{});
    else go(d, z, std::false_type{});
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

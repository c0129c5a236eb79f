// Attention of many rows per sequence over the 4-bit paged key/value cache:
// 256 rows a workgroup, 64 cached tokens a step, matrix cores fed from LDS.
//
// Work.  An item is 256 rows (token, query head) of a sequence that read one
// kv head; its eight waves hold 32 rows each, and walk the tokens that the
// item sees in tiles of 64.  Where the items alone leave compute units idle
// each is cut into `splits` runs of tiles, whose results (O, M, l) the last
// one to arrive joins in order.
//
// A tile.  Every thread loads 16 (head_dim 64: 8) bytes of codes one tile
// ahead: waves 0-3 a block of keys each, waves 4-7 a block of values, and
// writes them to LDS as fp16 matrix operands, so that the codes are unpacked
// once per 256 rows: keys as c - z, exact; values as (c - z) s 2^-e with e
// the exponent of the block's largest scale, rounded once (2^-11).  Both are
// laid out in 16-byte chunks whose place is XORed with the row, so that eight
// consecutive lanes' reads meet different banks.
//
// Scores.  S^T = K q^T (32x32x16): a lane holds one row and, with key row
// bits 2 and 3 exchanged when the tile is written, runs of 8 consecutive
// tokens, which is the operand order that O^T = V^T P^T wants.  q enters as
// fp16 times one power of two for the item's rows (its largest element below
// 2^15): bf16 has 8 significant bits and fp16 eleven, so an element is exact
// unless it is below 2^-29 of the largest, and then off by at most 2^-39 of
// it.  The running reference M of a row is the largest score plus its block's
// e, so that w = 2^(score + e - M) is at most 1, rounded to fp16 (2^-11); the
// sum l takes w 2^-e in fp32.
#include <algorithm>

#include "internal.hpp"
#include "kv_math.hpp"
#include "spear_ec_kv.h"

namespace spear {
namespace {

constexpr int kTileTokens = 64;
constexpr int kTileRows = 256;
constexpr int kTileWaves = 8;
constexpr int kTileTarget = 256;  // workgroups below which items are cut (one per compute unit)
constexpr int kTileMaxSplits = 16;

template <int D>
struct Staged {  // one tile as operands
  uint16_t k[kTileTokens][D];  // row: token with bits 2 and 3 exchanged
  uint16_t v[D][kTileTokens];
  float ks[kTileTokens];       // key scale times softmax scale and log2 e, over q's power of two
  int e[4];                    // exponents of the four blocks' value scales
};

// Byte offsets of 16-byte chunk c of a row.
template <int D>
__device__ __forceinline__ int k_chunk(int row, int c) { return row * (2 * D) + ((c ^ (row & 7)) << 4); }
__device__ __forceinline__ int v_chunk(int d, int c) {
  return d * (2 * kTileTokens) + ((c ^ ((d ^ (d >> 3)) & 7)) << 4);
}

// A thread's part of a tile on its way from the cache.
template <int D>
struct Fetched {
  uint32_t w[D / 32];   // codes: of token lane / 4 (keys); of a value column, D / 8 tokens
  uint32_t ks, kz;      // key scale and zero-point byte of that token
  u32x4 vs[D / 64];     // value scales of those tokens
  uint32_t vz[D / 32];  // and zero-point bytes
};

template <int D, bool ZEROS>
__global__ __launch_bounds__(512, 2) void prefill_attention_kernel(KvShape s, KvBatch b,
                                                                   KvAttentionArgs a, int splits,
                                                                   int* counters, float* slots) {
  __shared__ int64_t before[kMaxChunks + 1];
  __shared__ __attribute__((aligned(16))) Staged<D> buf[2];
  __shared__ float red[kTileWaves];
  __shared__ int flag;
  constexpr int kRowFloats = D + 2;
  const int lane = threadIdx.x & 63, wave = wave_id();
  const int n = lane & 31, half = lane >> 5;
  const int capacity = s.max_pages << s.page_shift;
  const int group = s.group();

  // ---- the item: heads fastest (one head's items on one XCD), a sequence's
  // last rows first (they see the most tokens)
  const auto weight = [&](int i) {
    return (int64_t)load_seq<kTileRows, kTileTokens>(s, b, a.window, i).tiles;
  };
  if (b.n_seqs > 64) sum_chunks<kTileWaves>(before, b.n_seqs, weight);
  const int head = blockIdx.x % s.kv_heads;
  const int rest = blockIdx.x / s.kv_heads;
  const int split = rest % splits;
  const int64_t x = rest / splits;
  int64_t total;
  if (b.n_seqs > 64) {
    total = before[(b.n_seqs + 63) / 64];
  } else {
    total = wave_sum(lane < b.n_seqs ? weight(lane) : (int64_t)0);
  }
  if (x >= total) return;
  int64_t seq_base;
  const int seq = __builtin_amdgcn_readfirstlane(find_seq(before, b.n_seqs, x, weight, seq_base));
  const Seq q = load_seq<kTileRows, kTileTokens>(s, b, a.window, seq);
  const int tile = q.tiles - 1 - (int)(x - seq_base);
  const int rows_n = q.n * group;

  // ---- tokens that the item's rows see
  const int row0 = tile * kTileRows, row1 = min(row0 + kTileRows, rows_n) - 1;
  const int start = q.len - q.n;  // position of the sequence's first row
  const int item_hi = min(start + row1 / group, capacity - 1);
  const int pos0 = start + row0 / group;
  const int item_lo = a.window ? max(0, min(pos0, capacity - 1) - a.window + 1) : 0;
  const int t0 = item_lo / kTileTokens;
  const int nt = item_hi < 0 ? 0 : item_hi / kTileTokens - t0 + 1;
  const int per = (nt + splits - 1) / splits;
  const int tb = min(nt, split * per), te = min(nt, tb + per);

  // ---- the lane's query row
  const int row = row0 + wave * 32 + n;
  const bool live = row < rows_n;
  const int tok = live ? row / group : 0;
  const int qh = head * group + (live ? row - tok * group : 0);
  const int pos = live ? start + tok : -1;
  const int hi = min(pos, capacity - 1);
  const int lo = a.window && pos >= a.window ? pos - a.window + 1 : 0;
  u32x4 qf[D / 16];
  float big = 0.f;
  {
    const uint16_t* qp = a.q + (int64_t)(q.first + tok) * a.q_stride + qh * D + 8 * half;
    #pragma unroll
    for (int i = 0; i < D / 16; ++i) {
      qf[i] = live ? load16(qp + 16 * i) : u32x4{0, 0, 0, 0};
      #pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float f0 = fabsf(bf16_lo(qf[i][j])), f1 = fabsf(bf16_hi(qf[i][j]));
        if (f0 < INFINITY) big = fmaxf(big, f0);
        if (f1 < INFINITY) big = fmaxf(big, f1);
      }
    }
  }
  #pragma unroll
  for (int o = 32; o > 0; o >>= 1) big = fmaxf(big, __shfl_xor(big, o, 64));
  if (lane == 0) red[wave] = big;
  __syncthreads();
  for (int i = 0; i < kTileWaves; ++i) big = fmaxf(big, red[i]);
  const int qe = min(110, max(-110, 15 - __builtin_amdgcn_frexp_expf(big)));  // big 2^qe < 2^15
  const float qmul = __builtin_amdgcn_ldexpf(1.f, qe);
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
  int all_lo = live ? lo : 0, all_hi = live ? hi : 0x7FFFFFFF;
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

  // ---- staging: wave w fetches block w % 4 of a tile, keys or values
  const bool is_v = wave >= 4;
  bool bad = false, any_bad = false;
  // cache block of the wave's part of tile t; positions outside the item's
  // range stand for the nearest one inside
  const auto block_of = [&](int t) {
    const int at = min(max(t * kTileTokens + 16 * (wave & 3), item_lo & ~15), item_hi);
    const int page = b.page_table[(int64_t)seq * s.max_pages + (at >> s.page_shift)];
    const bool out = (unsigned)page >= (unsigned)s.pages;
    const int pb = 1 << (s.page_shift - 4);
    return out ? -1 : (page * s.kv_heads + head) * pb + ((at >> 4) & (pb - 1));
  };
  Fetched<D> fe;
  const auto fetch = [&](int blk) {
    bad = blk < 0;
    const int64_t bl = bad ? 0 : blk;
    const uint8_t* c = a.cache.codes + bl * (16 * D) + (is_v ? 8 * D : 0);
    const uint8_t* sc = reinterpret_cast<const uint8_t*>(a.cache.scales) + bl * 64;
    // values, head_dim 64: two lanes a column, eight of its tokens each
    const int g = D == 128 ? 0 : lane & 1;
    if constexpr (D == 128) {
      const u32x4 w = load16(c + 16 * lane);
      #pragma unroll
      for (int i = 0; i < 4; ++i) fe.w[i] = w[i];
    } else {
      const u32x2 w = *reinterpret_cast<const u32x2*>(c + 8 * lane);
      #pragma unroll
      for (int i = 0; i < 2; ++i) fe.w[i] = w[i];
    }
    if (!is_v) {
      fe.ks = *reinterpret_cast<const uint16_t*>(sc + 2 * (lane >> 2));
      if constexpr (ZEROS) fe.kz = a.cache.zeros[bl * 16 + (lane >> 2)];
    } else {
      #pragma unroll
      for (int i = 0; i < D / 64; ++i) fe.vs[i] = load16(sc + 32 + 16 * (i + g));
      if constexpr (ZEROS) {
        const uint8_t* zp = a.cache.zeros + bl * 16 + 8 * g;
        #pragma unroll
        for (int i = 0; i < D / 32; ++i) fe.vz[i] = *reinterpret_cast<const uint32_t*>(zp + 4 * i);
      }
    }
  };
  const auto store = [&](Staged<D>& to, int t) {
    const int j0 = t * kTileTokens + 16 * (wave & 3);  // the block's first position
    uint8_t* kp = reinterpret_cast<uint8_t*>(to.k);
    uint8_t* vp = reinterpret_cast<uint8_t*>(to.v);
    if (!is_v) {
      const int token = 16 * (wave & 3) + (lane >> 2), part = lane & 3;
      const int r = (token & ~12) | ((token & 4) << 1) | ((token & 8) >> 1);
      f16x2 z = as_f16x2(0xD480D480u);  // -(64 + 8)
      if constexpr (ZEROS) {
        const uint32_t zb = 0xD400u | ((fe.kz & 15u) << 4);
        z = as_f16x2(zb | (zb << 16));
      }
      #pragma unroll
      for (int i = 0; i < D / 32; ++i) {
        const uint32_t e = even64(fe.w[i]), o = odd64(fe.w[i]), top = 0x54545454u;
        const u32x4 c = {as_u32(as_f16x2(pair01(e, top)) + z), as_u32(as_f16x2(pair23(e, top)) + z),
                         as_u32(as_f16x2(pair01(o, top)) + z), as_u32(as_f16x2(pair23(o, top)) + z)};
        *reinterpret_cast<u32x4*>(kp + k_chunk<D>(r, (D / 32) * part + i)) = c;
      }
      if (part == 0)
        to.ks[token] = bad ? __uint_as_float(0x7FC00000u) : half_bits_to_f32((uint16_t)fe.ks) * kmul;
      return;
    }
    // the lane's value scales; slots that nobody sees count as 0
    constexpr int kPairs = D / 16;
    const int g0 = D == 128 ? 0 : lane & 1;
    uint32_t vs[kPairs];
    #pragma unroll
    for (int i = 0; i < kPairs; ++i) vs[i] = fe.vs[i >> 2][i & 3];
    if (bad || j0 < item_lo || j0 + 15 > item_hi) {
      #pragma unroll
      for (int i = 0; i < kPairs; ++i) {
        const int j = j0 + 8 * g0 + 2 * i;
        if (bad || j < item_lo || j > item_hi) vs[i] &= 0xFFFF0000u;
        if (bad || j + 1 < item_lo || j + 1 > item_hi) vs[i] &= 0x0000FFFFu;
      }
    }
    uint32_t mp = vs[0];
    #pragma unroll
    for (int i = 1; i < kPairs; ++i) mp = max_pairs(mp, vs[i]);
    if constexpr (D == 64) mp = max_pairs(mp, (uint32_t)__shfl_xor((int)mp, 1, 64));
    const float mx = half_bits_to_f32((uint16_t)max(mp & 0xFFFFu, mp >> 16));
    const int e = mx > 0.f ? __builtin_amdgcn_frexp_expf(mx) : 0;  // every scale < 2^e
    if (lane == 0) to.e[wave & 3] = e;
    const int col = D == 128 ? lane : lane >> 1;
    #pragma unroll
    for (int i = 0; i < D / 64; ++i) {  // 8 tokens: one chunk of two dimensions
      const uint32_t w0 = fe.w[2 * i], w1 = fe.w[2 * i + 1], top = 0x54545454u;
      f16x2 z[4], sg[4];
      #pragma unroll
      for (int j = 0; j < 4; ++j) {
        const f16x2 h = as_f16x2(vs[4 * i + j]);
        sg[j] = as_f16x2(pack_f16(__builtin_amdgcn_ldexpf((float)h.x, -e),
                                  __builtin_amdgcn_ldexpf((float)h.y, -e)));
        z[j] = as_f16x2(0xD480D480u);
      }
      if constexpr (ZEROS) {
        const uint32_t a0 = odd64(fe.vz[2 * i]), a1 = odd64(fe.vz[2 * i + 1]), neg = 0xD4D4D4D4u;
        z[0] = as_f16x2(pair01(a0, neg));
        z[1] = as_f16x2(pair23(a0, neg));
        z[2] = as_f16x2(pair01(a1, neg));
        z[3] = as_f16x2(pair23(a1, neg));
      }
      const uint32_t e0 = even64(w0), e1 = even64(w1), o0 = odd64(w0), o1 = odd64(w1);
      const u32x4 ev = {as_u32((as_f16x2(pair01(e0, top)) + z[0]) * sg[0]),
                        as_u32((as_f16x2(pair23(e0, top)) + z[1]) * sg[1]),
                        as_u32((as_f16x2(pair01(e1, top)) + z[2]) * sg[2]),
                        as_u32((as_f16x2(pair23(e1, top)) + z[3]) * sg[3])};
      const u32x4 od = {as_u32((as_f16x2(pair01(o0, top)) + z[0]) * sg[0]),
                        as_u32((as_f16x2(pair23(o0, top)) + z[1]) * sg[1]),
                        as_u32((as_f16x2(pair01(o1, top)) + z[2]) * sg[2]),
                        as_u32((as_f16x2(pair23(o1, top)) + z[3]) * sg[3])};
      const int chunk = 2 * (wave & 3) + i + g0;
      *reinterpret_cast<u32x4*>(vp + v_chunk(2 * col, chunk)) = ev;
      *reinterpret_cast<u32x4*>(vp + v_chunk(2 * col + 1, chunk)) = od;
    }
  };

  float m = -INFINITY, l = 0.f;  // M and the lane's own share of l
  f32x16 o[D / 32];
  #pragma unroll
  for (int i = 0; i < D / 32; ++i)
    #pragma unroll
    for (int r = 0; r < 16; ++r) o[i][r] = 0.f;
  if (tb < te) {
    fetch(block_of(t0 + tb));
    any_bad |= bad;
    store(buf[tb & 1], t0 + tb);
  }
  for (int ti = tb; ti < te; ++ti) {
    __syncthreads();
    const Staged<D>& st = buf[ti & 1];
    const bool more = ti + 1 < te;
    if (more) fetch(block_of(t0 + ti + 1));
    const int j0 = (t0 + ti) * kTileTokens;
    if (j0 <= any_hi && j0 + kTileTokens - 1 >= any_lo) {
      const uint8_t* kp = reinterpret_cast<const uint8_t*>(st.k);
      const uint8_t* vp = reinterpret_cast<const uint8_t*>(st.v);
      f32x16 sc[2];
      #pragma unroll
      for (int t = 0; t < 2; ++t) {
        #pragma unroll
        for (int r = 0; r < 16; ++r) sc[t][r] = 0.f;
        #pragma unroll
        for (int i = 0; i < D / 16; ++i) {
          const u32x4 kf = *reinterpret_cast<const u32x4*>(kp + k_chunk<D>(32 * t + n, 2 * i + half));
          sc[t] = mfma32x32x16_f16(kf, qf[i], sc[t]);
        }
      }
      // lane's tokens: 16 g + 8 half + 0 .. 7 for g = 0 .. 3
      float top[4];
      #pragma unroll
      for (int g = 0; g < 4; ++g) {
        const f32x4 k0 = *reinterpret_cast<const f32x4*>(&st.ks[16 * g + 8 * half]);
        const f32x4 k1 = *reinterpret_cast<const f32x4*>(&st.ks[16 * g + 8 * half + 4]);
        #pragma unroll
        for (int r = 0; r < 8; ++r)
          sc[g >> 1][8 * (g & 1) + r] *= r < 4 ? k0[r & 3] : k1[r & 3];
      }
      if (j0 < all_lo || j0 + kTileTokens - 1 > all_hi) {
        #pragma unroll
        for (int g = 0; g < 4; ++g)
          #pragma unroll
          for (int r = 0; r < 8; ++r) {
            const int j = j0 + 16 * g + 8 * half + r;
            if (j < lo || j > hi) sc[g >> 1][8 * (g & 1) + r] = -INFINITY;
          }
      }
      float mn = m;
      float eb[4];
      #pragma unroll
      for (int g = 0; g < 4; ++g) {
        eb[g] = (float)st.e[g];
        top[g] = sc[g >> 1][8 * (g & 1)];
        #pragma unroll
        for (int r = 1; r < 8; ++r) top[g] = fmaxf(top[g], sc[g >> 1][8 * (g & 1) + r]);
        mn = fmaxf(mn, top[g] + eb[g]);
      }
      mn = fmaxf(mn, __shfl_xor(mn, 32, 64));
      if (__any(mn > m)) {
        const float alpha = mn == m ? 1.f : fast_exp2(m - mn);
        l *= alpha;
        #pragma unroll
        for (int i = 0; i < D / 32; ++i) o[i] *= alpha;
        m = mn;
      }
      u32x4 pf[4];
      #pragma unroll
      for (int g = 0; g < 4; ++g) {
        const float ref = m == -INFINITY ? 0.f : m - eb[g];
        float sum = 0.f;
        #pragma unroll
        for (int r = 0; r < 8; r += 2) {
          const float w0 = fast_exp2(sc[g >> 1][8 * (g & 1) + r] - ref);
          const float w1 = fast_exp2(sc[g >> 1][8 * (g & 1) + r + 1] - ref);
          sum += w0 + w1;
          pf[g][r >> 1] = pack_f16(w0, w1);
        }
        l += __builtin_amdgcn_ldexpf(sum, -st.e[g]);
      }
      #pragma unroll
      for (int g = 0; g < 4; ++g)
        #pragma unroll
        for (int i = 0; i < D / 32; ++i) {
          const u32x4 vf = *reinterpret_cast<const u32x4*>(vp + v_chunk(32 * i + n, 2 * g + half));
          o[i] = mfma32x32x16_f16(vf, pf[g], o[i]);
        }
    }
    if (more) {
      any_bad |= bad;
      store(buf[(ti + 1) & 1], t0 + ti + 1);
    }
  }
  l += __shfl_xor(l, 32, 64);

  // ---- the lane's row: dimensions 32 i + 8 (r / 4) + 4 half + r % 4
  const bool past = pos >= capacity;  // longer than its page-table row
  bool last = true;
  if (splits > 1) {
    // a run's results: [D + 2][256 rows], so that a wave's lanes store next to each other
    const int64_t item = x * s.kv_heads + head;
    const uint32_t bytes = kRowFloats * kTileRows * 4;
    const auto slot = [&](int sp) {
      return make_rsrc(slots + (item * splits + sp) * (kRowFloats * kTileRows), bytes);
    };
    const uint32_t me = (wave * 32 + n) * 4;
    {
      const rsrc_t rs = slot(split);
      #pragma unroll
      for (int i = 0; i < D / 32; ++i)
        #pragma unroll
        for (int r = 0; r < 16; ++r)
          bstore_dev(rs, (32 * i + 8 * (r >> 2) + 4 * half + (r & 3)) * (kTileRows * 4) + me, 0, o[i][r]);
      if (half == 0) {
        bstore_dev(rs, D * (kTileRows * 4) + me, 0, m);
        bstore_dev(rs, (D + 1) * (kTileRows * 4) + me, 0, l);
      }
    }
    wait_vmem();
    __syncthreads();
    if (threadIdx.x == 0) {
      int* ctr = counters + kCtrBand + (int)item;
      const int arrived = __hip_atomic_fetch_add(ctr, 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      flag = arrived == splits - 1;
      if (arrived == splits - 1) store_dev(ctr, 0);
    }
    __syncthreads();
    last = flag != 0;
    if (last) {
      float big_m = -INFINITY;
      for (int sp = 0; sp < splits; ++sp) big_m = fmaxf(big_m, bload_dev(slot(sp), D * (kTileRows * 4) + me, 0));
      l = 0.f;
      #pragma unroll
      for (int i = 0; i < D / 32; ++i)
        #pragma unroll
        for (int r = 0; r < 16; ++r) o[i][r] = 0.f;
      for (int sp = 0; sp < splits; ++sp) {
        const rsrc_t rs = slot(sp);
        const float ms = bload_dev(rs, D * (kTileRows * 4) + me, 0);
        const float k = ms == -INFINITY ? 1.f : fast_exp2(ms - big_m);  // an empty run is zeros
        l += bload_dev(rs, (D + 1) * (kTileRows * 4) + me, 0) * k;
        #pragma unroll
        for (int i = 0; i < D / 32; ++i)
          #pragma unroll
          for (int r = 0; r < 16; ++r)
            o[i][r] += bload_dev(rs, (32 * i + 8 * (r >> 2) + 4 * half + (r & 3)) * (kTileRows * 4) + me, 0) * k;
      }
      m = big_m;
    }
  }
  if (any_bad && lane == 0) atomicOr(counters + kCtrError, SPEAR_EC_WS_BAD_PAGE);
  if (last && live) {
    const int64_t at = (int64_t)(q.first + tok) * s.q_heads + qh;
    float inv = l == 0.f ? 0.f : 1.f / l;
    if (past) inv = l = __uint_as_float(0x7FC00000u);
    #pragma unroll
    for (int i = 0; i < D / 32; ++i)
      #pragma unroll
      for (int r = 0; r < 16; r += 4) {
        u32x2 w;
        w.x = pack_bf16(o[i][r] * inv, o[i][r + 1] * inv);
        w.y = pack_bf16(o[i][r + 2] * inv, o[i][r + 3] * inv);
        *reinterpret_cast<u32x2*>(a.out + at * D + 32 * i + 2 * r + 4 * half) = w;
      }
    if (half == 0) {
      if (a.lse) a.lse[at] = (m + log2f(l)) * kLn2;
      if (past) atomicOr(counters + kCtrError, SPEAR_EC_WS_BAD_PAGE);
    }
  }
}

// Items of a call are at most this many (their number is device data).
int64_t item_bound(const KvShape& s, int n_seqs, int tokens) {
  const int64_t rows = (int64_t)tokens * s.group();
  return (rows / kTileRows + std::min(n_seqs, tokens)) * s.kv_heads;
}

int split_count(const KvShape& s, int n_seqs, int tokens) {
  const int64_t items = std::max<int64_t>(1, item_bound(s, n_seqs, tokens));
  return (int)std::max<int64_t>(1, std::min<int64_t>(kTileMaxSplits, (kTileTarget + items - 1) / items));
}

}  // namespace

size_t kv_prefill_workspace(const KvShape& s) {
  // split_count(items) * items < kTileTarget + items <= 2 * kTileTarget where items are cut
  return sizeof(int) * kCounterSlots + sizeof(float) * 2 * kTileTarget * kTileRows * (s.D + 2);
}

hipError_t launch_kv_prefill(const KvShape& s, const KvBatch& b, const KvAttentionArgs& a,
                             void* workspace, hipStream_t st) {
  int* counters = static_cast<int*>(workspace);
  float* slots = reinterpret_cast<float*>(counters + kCounterSlots);
  const int splits = split_count(s, b.n_seqs, b.tokens);
  const int64_t wgs = item_bound(s, b.n_seqs, b.tokens) * splits;
  const auto go = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, dim3((unsigned)wgs), dim3(512), 0, st, s, b, a, splits, counters, slots);
  };
  if (s.D == 64) {
    if (s.zeros) go(prefill_attention_kernel<64, true>); else go(prefill_attention_kernel<64, false>);
  } else {
    if (s.zeros) go(prefill_attention_kernel<128, true>); else go(prefill_attention_kernel<128, false>);
  }
  return hipGetLastError();
}

}  // namespace spear

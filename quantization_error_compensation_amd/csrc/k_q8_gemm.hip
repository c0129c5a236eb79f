// Products of the 8-bit path for many tokens: int8 codes on the matrix cores.
//
//     p[t][n] = xs[t] ws[n] sum_k cx[t][k] cw[n][k],   y = p or act(p_n) p_(n + N)
//
// A workgroup multiplies a tile of BM tokens with BN weight rows, K by 128
// codes (one cache line of a row) through a ring of S stages in LDS, which
// loads that write LDS directly fill.  The sums are 32-bit integers in
// registers, exact for any order and split; scales and gate follow in fp32.
// A gated tile holds 32 rows of one projection, the 32 of the other for the
// same columns, and so on, so that a wave finds both in its own registers.
//
// Waves hold MT x NT results of the 32x32x32 instruction.  Operand reads take
// LDS (MT + NT) / (MT NT) of the matrix time at 128 bytes a cycle, so the waves
// are as square as eight of them can be; four waves of 128 x 128 would read a
// third less, but one wave a SIMD shows every wait (2.0 against 2.45 POP/s).
// One half of the waves, one of each SIMD, issues all loads right after the
// barrier while the other half computes, and computes when the other half is
// done: a wave that issues loads does not issue matrix steps (gated, 3999
// tokens 8192->28672: 1466 us, with every wave's own loads 1520 to 1575).  Tiles
// whose sums fit four waves beside four that load alone (256 x 128) read a quarter
// less from LDS that way, which is power: 512 tokens 28672->8192 122 -> 118 us, on
// zeros 102 and 103; with one tile of tokens, where loads bind, it is 2 to 6%
// slower, and 128 x 256 gains nothing.
//
// What bounds it.  The largest products: the card's power.  4096 tokens of
// 8192x8192 take 215 to 224 us (2.45 to 2.56 POP/s; the library's int8 product
// 2.1 here and 2.5 at best), the same on zeros 149 us, since the clock then
// stays up.  Smaller tiles: loads into LDS, about 30 cycles a KB and unit when
// they hit L2 and 41 from memory: a 128 x 256 tile waits 1500 to 2000 cycles for
// 1024 of matrix steps.  Prefetching lines into L2 with loads of their own costs
// more of that same path than it saves (512 tokens 28672->8192, then: 121 -> 127 us).
#include "common.hpp"
#include "internal.hpp"
#include "q8_math.hpp"
#include "q8_plan.hpp"

namespace spear {
namespace {

struct TileParams {
  const int8_t *xq, *wq;
  const float *xs, *ws;
  void* y;
  float* part;  // [tile][split][wave][16-byte piece][lane] partial sums
  int* ctr;     // [tile][wave][32 tokens] arrivals
  int T, K, N, tiles_m, tiles_n, splits;
  int gelu, out_f32;
};

// Token tiles side by side in a run of tiles: 4096 tokens of 8192x8192 277 us with
// 1, 235 with 2, 232 with 4 and 8, 265 with 16 (before the results went through
// LDS).
constexpr int kDeep = 4;

// BM tokens x BN weight rows a workgroup, WM x WN waves, K by BK codes, S stages,
// D waves more that only load.
template <int BM_, int BN_, int WM_, int WN_, int BK_, int S_, int D_ = 0>
struct Tile {
  static constexpr int BM = BM_, BN = BN_, WM = WM_, WN = WN_, BK = BK_, S = S_, D = D_;
  static constexpr int kWaves = WM * WN, kAll = kWaves + D;
  static constexpr int MT = BM / WM / 32, NT = BN / WN / 32;  // 32 x 32 results of a wave
  // The first half of the waves, one on each SIMD, issues every load, or the last D do.
  static constexpr int kFirstLoader = D ? kWaves : 0;
  static constexpr int kLoaders = D ? D : kWaves > 4 ? kWaves / 2 : kWaves;
  static constexpr int kRowsPerLoad = 1024 / BK;
  static constexpr int kXLoads = BM / kRowsPerLoad / kLoaders, kWLoads = BN / kRowsPerLoad / kLoaders;
  static constexpr int kLoads = kXLoads + kWLoads;
  static constexpr int kStage = (BM + BN) * BK;
  static constexpr int kRing = S * kStage;
  static constexpr int kLds = kRing + (BM + BN) * 4;  // the scales behind the ring
  static_assert(MT >= 1 && NT >= 1 && kXLoads >= 1 && kWLoads >= 1, "tile shape");
  static_assert(kXLoads * kLoaders * kRowsPerLoad == BM && kWLoads * kLoaders * kRowsPerLoad == BN, "loads");
  static_assert(BM * BN * 2 <= kRing, "the results' staging fits the ring");
  static_assert(kLds <= 160 * 1024, "LDS exceeds 160 KB");
};

// 16-byte piece a of row r lies at a ^ swizzle(r) of the row: 16 lanes that
// read one piece of 16 rows meet 16 different places of the 256 bytes that LDS
// serves at once.
template <int BK>
__device__ __forceinline__ int swizzle(int row) {
  return BK == 128 ? (row >> 1) & 7 : (row >> 2) & 3;
}

template <typename L, bool GATED>
__global__ __launch_bounds__(64 * L::kAll, 1) void tile_kernel(TileParams p) {
  constexpr int BM = L::BM, BN = L::BN, BK = L::BK, S = L::S, MT = L::MT, NT = L::NT;
  constexpr int kSteps = BK / 32;
  constexpr int kParts = GATED ? 2 : 1, kCols = BN / kParts;  // columns of y
  static_assert(NT % kParts == 0, "a wave holds both projections of its columns");
  __shared__ __attribute__((aligned(128))) uint8_t smem[L::kLds];
  const int lane = threadIdx.x & 63, wave = wave_id();
  const int wm = wave / L::WN, wn = wave % L::WN;
  const int i32 = lane & 31, h = lane >> 5;

  // Workgroup -> (split, tile).  Workgroups are dealt to the 8 XCDs in turn;
  // each XCD gets a run of tiles that lie next to each other, kDeep token
  // tiles deep, so that the ones it works on share rows in its L2.
  const int tiles = p.tiles_m * p.tiles_n, total = tiles * p.splits;
  const int per = total >> 3, more = total & 7, xcd = blockIdx.x & 7;
  const int idx = xcd * per + min(xcd, more) + (blockIdx.x >> 3);
  const int split = idx / tiles, tile = idx - split * tiles;
  const int band = kDeep * p.tiles_n;
  const int g0 = tile / band, in = tile - g0 * band;
  const int deep = min(kDeep, p.tiles_m - g0 * kDeep);
  const int tn = in / deep, tm = g0 * kDeep + in - tn * deep;
  const int m0 = tm * BM, n0 = tn * kCols;
  const int rows_m = min(BM, p.T - m0), rows_n = min(kCols, p.N - n0);
  const int blocks = (p.K + BK - 1) / BK;
  const int kb0 = (int)((int64_t)blocks * split / p.splits);
  const int kb1 = (int)((int64_t)blocks * (split + 1) / p.splits);

  const u32x4 xr = sdesc(p.xq + (size_t)m0 * p.K, (uint32_t)rows_m * p.K);
  const u32x4 wr = sdesc(p.wq + (size_t)n0 * p.K, (uint32_t)rows_n * p.K);
  const u32x4 ur = GATED ? sdesc(p.wq + ((size_t)p.N + n0) * p.K, (uint32_t)rows_n * p.K) : wr;
  const uint32_t lds0 = lds_addr(smem);

  // The tile's scales: tokens, then weight rows, first those of y's columns,
  // then with GATED the other projection's.
  {
    const u32x4 sx = sdesc(p.xs + m0, (uint32_t)rows_m * 4);
    const u32x4 sw = sdesc(p.ws + n0, (uint32_t)rows_n * 4);
    const u32x4 su = GATED ? sdesc(p.ws + p.N + n0, (uint32_t)rows_n * 4) : sw;
    for (int c = wave; c < (BM + BN) / 32; c += L::kAll) {  // 32 at a time, by half a wave
      const int f = c * 32 - BM;
      const uint32_t to = lds0 + L::kRing + c * 128;
      if (lane < 32) {
        if (f < 0) dma4(sx, to, (uint32_t)(c * 32 + lane) * 4);
        else if (f < kCols) dma4(sw, to, (uint32_t)(f + lane) * 4);
        else dma4(su, to, (uint32_t)(f - kCols + lane) * 4);
      }
    }
  }

  // Loads: R rows of BK bytes each, whole lines of a row side by side.  Rows
  // of the weights' stage: 32 of y's columns, with GATED the other
  // projection's for the same columns behind them.
  constexpr int R = L::kRowsPerLoad, P = BK / 16;
  const int lr = lane / P, lp = lane % P, lw = wave - L::kFirstLoader;
  uint32_t xoff[L::kXLoads], woff[L::kWLoads];  // at k = 0
  int xpiece[L::kXLoads];
  #pragma unroll
  for (int j = 0; j < L::kXLoads; ++j) {
    const int r = (lw * L::kXLoads + j) * R + lr;
    xpiece[j] = (lp ^ swizzle<BK>(r)) * 16;
    xoff[j] = (uint32_t)r * p.K + xpiece[j];
  }
  #pragma unroll
  for (int j = 0; j < L::kWLoads; ++j) {
    const int r = (lw * L::kWLoads + j) * R + lr;
    woff[j] = (uint32_t)(GATED ? (r >> 6) * 32 + (r & 31) : r) * p.K + (lp ^ swizzle<BK>(r)) * 16;
  }
  // Past K the tokens' codes are zeros (an offset out of range), so whatever
  // the weights' loads bring there counts nothing.
  auto issue = [&](int kb, int stage) {
    const uint32_t to = lds0 + stage * L::kStage;
    const int k0 = kb * BK;
    #pragma unroll
    for (int j = 0; j < L::kXLoads; ++j)
      dma16(xr, to + (lw * L::kXLoads + j) * 1024, k0 + xpiece[j] < p.K ? xoff[j] + k0 : 0x80000000u);
    #pragma unroll
    for (int j = 0; j < L::kWLoads; ++j) {
      const int first = (lw * L::kWLoads + j) * R;
      const bool other = GATED && (first & 32);
      dma16(other ? ur : wr, to + BM * BK + first * BK, woff[j] + k0);
    }
  };

  i32x16 acc[NT][MT];
  for (int a = 0; a < NT; ++a)
    for (int b = 0; b < MT; ++b)
      for (int v = 0; v < 16; ++v) acc[a][b][v] = 0;

  const int sw = swizzle<BK>(i32);
  const uint8_t* xl = smem + (wm * MT * 32 + i32) * BK;
  const uint8_t* wl = smem + BM * BK + (wn * NT * 32 + i32) * BK;
  auto read = [&](int stage, int s, u32x4 (&w)[NT], u32x4 (&x)[MT]) {
    const int at = stage * L::kStage + (((2 * s + h) ^ sw) * 16);
    #pragma unroll
    for (int a = 0; a < NT; ++a) w[a] = *reinterpret_cast<const u32x4*>(wl + at + a * 32 * BK);
    #pragma unroll
    for (int b = 0; b < MT; ++b) x[b] = *reinterpret_cast<const u32x4*>(xl + at + b * 32 * BK);
  };
  auto step = [&](const u32x4 (&w)[NT], const u32x4 (&x)[MT]) {
    #pragma unroll
    for (int a = 0; a < NT; ++a)
      #pragma unroll
      for (int b = 0; b < MT; ++b) acc[a][b] = mfma32x32x32_i8(w[a], x[b], acc[a][b]);
  };

  // At the top of block kb the loads of kb .. kb + S - 2 are in flight; after
  // the wait and the barrier kb's stage is whole and kb - 1's read by every
  // wave, so that kb + S - 1's loads go into it.  Past the last block they
  // begin again, which keeps the count in flight the same.  A block's last step
  // runs after the next barrier, while the first reads behind it are under way.
  // The order of the blocks is free (sums of integers): with one tile of tokens
  // every tile begins at another one, so that the rows' equal columns, which
  // lie a power of two apart, are not asked of the same memory channels at once.
  const bool loader = lw >= 0 && lw < L::kLoaders;
  int next = kb0 + (p.tiles_m == 1 ? first_block(tn, kb1 - kb0) : 0);
  auto load_next = [&](int stage) {
    issue(next, stage);
    next = next + 1 == kb1 ? kb0 : next + 1;
  };
  if (loader) {
    #pragma unroll
    for (int s = 0; s < S - 1; ++s) load_next(s);
  }
  if (L::D > 0 && loader) {  // the same waits and barriers as below, and nothing else
    for (int kb = kb0, into = S - 1; kb < kb1; ++kb) {
      wait_vmcnt<(S - 2) * L::kLoads>();
      __builtin_amdgcn_s_barrier();
      asm volatile("" ::: "memory");
      load_next(into);
      into = into + 1 == S ? 0 : into + 1;
    }
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    __syncthreads();
    return;
  }
  if (L::D > 0) wait_vmcnt<0>();  // this wave's share of the scales
  u32x4 wc[NT], xc[MT];  // the last step's operands
  for (int a = 0; a < NT; ++a) wc[a] = u32x4{0, 0, 0, 0};
  for (int b = 0; b < MT; ++b) xc[b] = u32x4{0, 0, 0, 0};
  int stage = 0, into = S - 1;
  for (int kb = kb0; kb < kb1; ++kb) {
    if (L::D == 0) wait_vmcnt<(S - 2) * L::kLoads>();
    __builtin_amdgcn_s_waitcnt(0xC07F);  // lgkmcnt(0)
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    u32x4 w[2][NT], x[2][MT];
    read(stage, 0, w[0], x[0]);
    if (L::D == 0 && loader) load_next(into);
    if (kb > kb0) step(wc, xc);
    #pragma unroll
    for (int s = 0; s + 1 < kSteps; ++s) {
      read(stage, s + 1, w[(s + 1) & 1], x[(s + 1) & 1]);
      step(w[s & 1], x[s & 1]);
    }
    #pragma unroll
    for (int a = 0; a < NT; ++a) wc[a] = w[(kSteps - 1) & 1][a];
    #pragma unroll
    for (int b = 0; b < MT; ++b) xc[b] = x[(kSteps - 1) & 1][b];
    stage = stage + 1 == S ? 0 : stage + 1;
    into = into + 1 == S ? 0 : into + 1;
  }
  step(wc, xc);
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
  __syncthreads();  // every load has landed and every stage is read

  // Split K.  A wave's sums meet those of the same wave of the tile's other
  // splits, one part (32 tokens) after the other: it stores a part, waits until
  // it has arrived and counts it; whoever counts a part last adds the others' to
  // its own, which are still in registers, and finishes that part.  No one
  // waits for another.  The splits take the parts in turned order, so that each
  // is likely to come last to other parts than the rest.
  uint32_t finish = (1u << MT) - 1;  // the parts that this wave finishes
  if (p.splits > 1) {
    constexpr int kFloats = BM * BN, kPartBytes = NT * 4 * 1024;
    const rsrc_t pr = make_rsrc(p.part + (size_t)tile * p.splits * kFloats, (uint32_t)p.splits * kFloats * 4);
    const uint32_t mine = (uint32_t)wave * (NT * MT * 4096) + lane * 16;
    int* ctr = p.ctr + (tile * L::kWaves + wave) * MT;
    const int first = split * MT / p.splits;
    finish = 0;
    for (int j = 1; j <= MT; ++j) {
      const int part = first + j < MT ? first + j : first + j - MT;
      #pragma unroll
      for (int b = 0; b < MT; ++b) {
        if (b != part) continue;
        #pragma unroll
        for (int a = 0; a < NT; ++a)
          #pragma unroll
          for (int g = 0; g < 4; ++g) {
            const i32x4 v = {acc[a][b][4 * g], acc[a][b][4 * g + 1], acc[a][b][4 * g + 2], acc[a][b][4 * g + 3]};
            bstore16_dev(pr, mine + (uint32_t)split * kFloats * 4 + b * kPartBytes + (a * 4 + g) * 1024,
                         __builtin_bit_cast(f32x4, v));
          }
      }
      wait_vmem();
      int seen = 0;
      if (lane == 0) seen = atomicAdd(ctr + part, 1);
      if (__builtin_amdgcn_readfirstlane(seen) == p.splits - 1) finish |= 1u << part;
    }
    #pragma unroll
    for (int b = 0; b < MT; ++b) {
      if (!(finish >> b & 1)) continue;
      if (lane == 0) store_dev(ctr + b, 0);
      for (int o = 0; o < p.splits; ++o) {
        if (o == split) continue;
        #pragma unroll
        for (int a = 0; a < NT; ++a)
          #pragma unroll
          for (int g = 0; g < 4; ++g) {
            const i32x4 v = __builtin_bit_cast(
                i32x4, bload16_dev(pr, mine + b * kPartBytes + (a * 4 + g) * 1024, (uint32_t)o * kFloats * 4));
            #pragma unroll
            for (int k = 0; k < 4; ++k) acc[a][b][4 * g + k] += v[k];
          }
      }
    }
    if (!finish) return;
  }

  // A lane holds token i32 of a block and weight rows 8 g + 4 h + 0 .. 3.
  const float* tok = reinterpret_cast<const float*>(smem + L::kRing) + wm * MT * 32 + i32;
  const float* row = reinterpret_cast<const float*>(smem + L::kRing) + BM + wn * (NT / kParts) * 32 + 4 * h;
  auto result = [&](int a, int b, int g) {
    const float xs = tok[b * 32];
    const f32x4 sc = *reinterpret_cast<const f32x4*>(row + a * 32 + 8 * g);
    f32x4 o;
    #pragma unroll
    for (int j = 0; j < 4; ++j) o[j] = (float)acc[a * kParts][b][4 * g + j] * xs * sc[j];
    if constexpr (GATED) {
      const f32x4 su = *reinterpret_cast<const f32x4*>(row + kCols + a * 32 + 8 * g);
      #pragma unroll
      for (int j = 0; j < 4; ++j)
        o[j] = gate(p.gelu, o[j], (float)acc[a * kParts + 1][b][4 * g + j] * xs * su[j]);
    }
    return o;
  };
  constexpr int NC = NT / kParts;               // blocks of 32 columns of a wave
  const int c0 = n0 + wn * NC * 32, t0 = m0 + wm * MT * 32;
  if (p.out_f32) {
    #pragma unroll
    for (int b = 0; b < MT; ++b) {
      if (!(finish >> b & 1)) continue;
      #pragma unroll
      for (int a = 0; a < NC; ++a)
        #pragma unroll
        for (int g = 0; g < 4; ++g) {
          const int t = t0 + b * 32 + i32, n = c0 + a * 32 + 8 * g + 4 * h;
          const f32x4 o = result(a, b, g);
          if (t < p.T && n < p.N)
            *reinterpret_cast<f32x4*>(static_cast<float*>(p.y) + (size_t)t * p.N + n) = o;
        }
    }
    return;
  }
  // Through LDS, a part of the ring for each wave, so that rows of y are
  // written as whole 64- or 128-byte runs: stored as the lanes hold them (8
  // bytes of 32 rows at a time) they cost 4096 tokens of 8192x8192 235 us, not 211.
  constexpr int kPieces = NC * 4, kShare = 16 / kPieces;  // 16-byte pieces of a row, rows of 256 bytes
  uint16_t* y = static_cast<uint16_t*>(p.y) + (size_t)t0 * p.N + c0;
  const int live = p.T - t0, cols = p.N - c0;
  #pragma unroll
  for (int b = 0; b < MT; ++b) {
    if (!(finish >> b & 1)) continue;
    uint8_t* own = smem + (wave * MT + b) * (32 * kPieces * 16);
    #pragma unroll
    for (int a = 0; a < NC; ++a)
      #pragma unroll
      for (int g = 0; g < 4; ++g) {
        const f32x4 o = result(a, b, g);
        const int piece = (a * 4 + g) ^ ((i32 / kShare) & (kPieces - 1));
        *reinterpret_cast<u32x2*>(own + i32 * kPieces * 16 + piece * 16 + 8 * h) =
            u32x2{bf16_pair(o[0], o[1]), bf16_pair(o[2], o[3])};
      }
    #pragma unroll
    for (int j = 0; j < kPieces / 2; ++j) {
      const int r = j * (64 / kPieces) + lane / kPieces;
      const int col = ((lane % kPieces) ^ ((r / kShare) & (kPieces - 1))) * 8;
      const u32x4 d = *reinterpret_cast<const u32x4*>(own + j * 1024 + lane * 16);
      if (b * 32 + r < live && col < cols) *reinterpret_cast<u32x4*>(y + (size_t)(b * 32 + r) * p.N + col) = d;
    }
  }
}

template <typename L>
hipError_t launch_tile(const Q8Shape& s, const Q8Product& a, int splits, void* workspace, hipStream_t st) {
  TileParams p;
  p.xq = a.xq;
  p.wq = a.wq;
  p.xs = a.xs;
  p.ws = a.ws;
  p.y = a.y;
  p.ctr = static_cast<int*>(workspace);
  p.part = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + kQ8CounterBytes);
  p.T = s.T;
  p.K = s.K;
  p.N = s.N;
  p.tiles_m = (s.T + L::BM - 1) / L::BM;
  const int cols = s.gated ? L::BN / 2 : L::BN;
  p.tiles_n = (s.N + cols - 1) / cols;
  p.splits = splits;
  p.gelu = s.gelu;
  p.out_f32 = s.out_f32;
  const dim3 grid(p.tiles_m * p.tiles_n * splits), block(64 * L::kAll);
  if (!s.gated)
    hipLaunchKernelGGL((tile_kernel<L, false>), grid, block, 0, st, p);
  else if constexpr (L::NT % 2 == 0)
    hipLaunchKernelGGL((tile_kernel<L, true>), grid, block, 0, st, p);
  else
    return hipErrorInvalidValue;
  return hipGetLastError();
}

// The shapes of kQ8Tiles, in its order.
template <typename L, int I>
hipError_t launch_shape(const Q8Shape& s, const Q8Product& a, int splits, void* workspace, hipStream_t st) {
  static_assert(L::BM == kQ8Tiles[I].bm && L::BN == kQ8Tiles[I].bn, "the plan's shapes");
  static_assert(kQ8Tiles[I].gated == (L::NT % 2 == 0), "the plan's shapes");
  static_assert(kQ8Tiles[I].held == (160 * 1024 / L::kLds < 2 ? 1 : 2), "workgroups a compute unit holds");
  return launch_tile<L>(s, a, splits, workspace, st);
}

}  // namespace

size_t q8_product_workspace(const Q8Shape& s) { return q8_workspace_for(s); }

hipError_t launch_q8_product(const Q8Shape& s, const Q8Product& a, void* workspace, hipStream_t st) {
  const Q8Stream f = plan_q8_stream(s);
  if (f.x) return launch_q8_stream(s, a, f, st);
  const Q8TilePlan pl = plan_q8_tiles(s);
  switch (pl.tile) {
    case 0: return launch_shape<Tile<256, 256, 2, 4, 128, 2>, 0>(s, a, pl.splits, workspace, st);
    case 1: return launch_shape<Tile<192, 256, 2, 4, 128, 2>, 1>(s, a, pl.splits, workspace, st);
    case 2:
      if (s.T > 256) return launch_shape<Tile<256, 128, 2, 2, 128, 3, 4>, 2>(s, a, pl.splits, workspace, st);
      return launch_shape<Tile<256, 128, 4, 2, 128, 3>, 2>(s, a, pl.splits, workspace, st);
    case 3: return launch_shape<Tile<128, 256, 2, 4, 128, 3>, 3>(s, a, pl.splits, workspace, st);
    case 4: return launch_shape<Tile<128, 128, 2, 4, 128, 4>, 4>(s, a, pl.splits, workspace, st);
    case 5: return launch_shape<Tile<64, 128, 2, 2, 128, 3>, 5>(s, a, pl.splits, workspace, st);
    case 6: return launch_shape<Tile<64, 64, 2, 2, 128, 4>, 6>(s, a, pl.splits, workspace, st);
    default: return launch_shape<Tile<32, 128, 1, 4, 128, 3>, 7>(s, a, pl.splits, workspace, st);
  }
}

}  // namespace spear

// Products of the 8-bit path for few tokens: the weights stream once from HBM.
//
//     p[t][n] = xs[t] ws[n] sum_k cx[t][k] cw[n][k],   y = p or act(p_n) p_(n + N)
//
// A workgroup holds 16 RT weight rows (of each projection) over the whole of K;
// its waves take K's blocks of 128 codes, one cache line of a row, in turn and
// add their exact integer sums in LDS at the end.  No workgroup waits for
// another, and nothing but y is written.
//
// A wave fills a ring of its own with loads that write LDS directly and meets
// no barrier until its blocks are done: eight lanes read a row's line, where
// loads into registers in the matrix operands' layout would have neighbouring
// lanes read different rows.  Tokens come the same way, 8 rows a load; rows past
// the last token are out of range and cost no traffic.  They are read again by
// every workgroup, hence more rows a workgroup the more tokens there are
// (q8_plan.hpp).
//
// HBM-bound: 28672->8192 at one token 40.2 us (5.8 TB/s), gated 8192->28672 76 us
// (6.2), 8192->10240 at 16 tokens 17.8 us (4.7), 4096x4096 at one token 4.5 us,
// of which the weights at that rate are 3.  Three or four blocks in flight a wave
// are no faster than two (8192x8192 at 16 tokens 14.06 and 14.35 against 14.01):
// what a unit has in flight comes from several workgroups.
#include "common.hpp"
#include "q8_math.hpp"
#include "q8_plan.hpp"

namespace spear {
namespace {

struct StreamParams {
  const int8_t *xq, *wq;
  const float *xs, *ws;
  void* y;
  int T, K, N, gelu, out_f32;
};

constexpr int kBlock = 128;  // K codes of a block

// XL: x loads of 8 tokens a block, RT: tiles of 16 weight rows (of each
// projection), W waves.
template <int XL, int RT, bool GATED, int W>
__global__ __launch_bounds__(64 * W) void stream_kernel(StreamParams p) {
  constexpr int S = 2;  // blocks of a wave in flight
  constexpr int MT = (XL + 1) / 2, kParts = GATED ? 2 : 1, kTiles = RT * kParts;
  constexpr int kLoads = 2 * kTiles + XL;  // of a block
  constexpr int kSlot = (2 * kTiles + 2 * MT) * 1024;
  constexpr int kSums = W * kTiles * MT * 1024;
  constexpr int kLds = W * S * kSlot > kSums ? W * S * kSlot : kSums;
  static_assert(kLds <= 160 * 1024, "LDS exceeds 160 KB");
  __shared__ __attribute__((aligned(128))) uint8_t smem[kLds];
  const int lane = threadIdx.x & 63, wave = wave_id();
  const int i16 = lane & 15, q = lane >> 4;
  const int n0 = blockIdx.x * 16 * RT;
  const int rows_n = min(16 * RT, p.N - n0);

  const u32x4 xr = sdesc(p.xq, (uint32_t)p.T * p.K);
  const u32x4 wr = sdesc(p.wq + (size_t)n0 * p.K, (uint32_t)rows_n * p.K);
  const u32x4 ur = GATED ? sdesc(p.wq + ((size_t)p.N + n0) * p.K, (uint32_t)rows_n * p.K) : wr;
  const uint32_t ring = lds_addr(smem) + wave * S * kSlot;

  const int lr = lane >> 3, lp = lane & 7;
  // 16-byte piece a of row r lies at a ^ ((r >> 1) & 7): rows 8 j + lr
  const int even = (lp ^ (lr >> 1)) * 16, odd = (lp ^ ((lr + 8) >> 1)) * 16;
  const uint32_t row0 = (uint32_t)lr * p.K, rows8 = 8u * p.K;
  const int blocks = (p.K + kBlock - 1) / kBlock;
  const int turn = first_block(blockIdx.x, blocks);
  auto issue = [&](int kb, int slot) {
    const uint32_t to = ring + slot * kSlot;
    const int at = kb + turn < blocks ? kb + turn : kb + turn - blocks;
    const int k0 = kb < blocks ? at * kBlock : p.K;  // past the last block nothing is read
    const int ke = k0 + even, ko = k0 + odd;
    const uint32_t e = ke < p.K ? row0 + ke : 0x80000000u, o = ko < p.K ? row0 + ko : 0x80000000u;
    #pragma unroll
    for (int j = 0; j < 2 * RT; ++j) {
      const uint32_t from = j & 1 ? o : e;
      dma16(wr, to + j * 1024, from + j * rows8);
      if (GATED) dma16(ur, to + (2 * RT + j) * 1024, from + j * rows8);
    }
    #pragma unroll
    for (int j = 0; j < XL; ++j)
      dma16(xr, to + (2 * kTiles + j) * 1024, (j & 1 ? o : e) + j * rows8);
  };

  i32x4 acc[kTiles][MT];
  for (int a = 0; a < kTiles; ++a)
    for (int b = 0; b < MT; ++b) acc[a][b] = i32x4{0, 0, 0, 0};
  #pragma unroll
  for (int s = 0; s < S; ++s) issue(wave + s * W, s);
  const int sw = (i16 >> 1) & 7;
  int slot = 0;
  for (int kb = wave; kb < blocks; kb += W) {
    wait_vmcnt<(S - 1) * kLoads>();
    const uint8_t* at = smem + (wave * S + slot) * kSlot + i16 * 128;
    u32x4 w[kTiles][2], x[MT][2];
    #pragma unroll
    for (int s = 0; s < 2; ++s) {
      const int o = ((4 * s + q) ^ sw) * 16;
      #pragma unroll
      for (int a = 0; a < kTiles; ++a) w[a][s] = *reinterpret_cast<const u32x4*>(at + a * 2048 + o);
      #pragma unroll
      for (int b = 0; b < MT; ++b)
        x[b][s] = *reinterpret_cast<const u32x4*>(at + (kTiles + b) * 2048 + o);
    }
    __builtin_amdgcn_s_waitcnt(0xC07F);  // lgkmcnt(0): the slot is read
    asm volatile("" ::: "memory");
    issue(kb + S * W, slot);
    #pragma unroll
    for (int s = 0; s < 2; ++s)
      #pragma unroll
      for (int a = 0; a < kTiles; ++a)
        #pragma unroll
        for (int b = 0; b < MT; ++b) acc[a][b] = mfma16x16x64_i8(w[a][s], x[b][s], acc[a][b]);
    slot = slot + 1 == S ? 0 : slot + 1;
  }
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
  __syncthreads();  // every wave's loads have landed: the ring becomes the sums

  u32x4* sums = reinterpret_cast<u32x4*>(smem);
  #pragma unroll
  for (int a = 0; a < kTiles; ++a)
    #pragma unroll
    for (int b = 0; b < MT; ++b)
      sums[(wave * kTiles * MT + a * MT + b) * 64 + lane] = __builtin_bit_cast(u32x4, acc[a][b]);
  __syncthreads();
  for (int i = wave; i < RT * MT; i += W) {
    const int a = i / MT, b = i - a * MT;
    i32x4 v[kParts];
    #pragma unroll
    for (int k = 0; k < kParts; ++k) {
      v[k] = i32x4{0, 0, 0, 0};
      #pragma unroll
      for (int w = 0; w < W; ++w)
        v[k] += __builtin_bit_cast(i32x4, sums[(w * kTiles * MT + (a + k * RT) * MT + b) * 64 + lane]);
    }
    const int t = b * 16 + i16, n = n0 + a * 16 + 4 * q;
    if (t >= p.T || n >= p.N) continue;
    const float xs = p.xs[t];
    const f32x4 sc = {p.ws[n], p.ws[n + 1], p.ws[n + 2], p.ws[n + 3]};
    f32x4 o;
    #pragma unroll
    for (int j = 0; j < 4; ++j) o[j] = (float)v[0][j] * xs * sc[j];
    if constexpr (GATED) {
      const float* us = p.ws + p.N + n;
      #pragma unroll
      for (int j = 0; j < 4; ++j) o[j] = gate(p.gelu, o[j], (float)v[1][j] * xs * us[j]);
    }
    const size_t to = (size_t)t * p.N + n;
    if (p.out_f32) *reinterpret_cast<f32x4*>(static_cast<float*>(p.y) + to) = o;
    else
      *reinterpret_cast<u32x2*>(static_cast<uint16_t*>(p.y) + to) =
          u32x2{bf16_pair(o[0], o[1]), bf16_pair(o[2], o[3])};
  }
}

template <int XL, int RT, int W>
hipError_t launch_stream(const Q8Shape& s, const Q8Product& a, hipStream_t st) {
  const StreamParams p{a.xq, a.wq, a.xs, a.ws, a.y, s.T, s.K, s.N, s.gelu, s.out_f32};
  const dim3 grid((s.N + 16 * RT - 1) / (16 * RT)), block(64 * W);
  if (s.gated)
    hipLaunchKernelGGL((stream_kernel<XL, RT, true, W>), grid, block, 0, st, p);
  else
    hipLaunchKernelGGL((stream_kernel<XL, RT, false, W>), grid, block, 0, st, p);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_q8_stream(const Q8Shape& s, const Q8Product& a, const Q8Stream& f, hipStream_t st) {
  switch (f.x * 100 + f.tiles * 10 + f.waves) {
    case 114: return launch_stream<1, 1, 4>(s, a, st);
    case 118: return launch_stream<1, 1, 8>(s, a, st);
    case 214: return launch_stream<2, 1, 4>(s, a, st);
    case 218: return launch_stream<2, 1, 8>(s, a, st);
    case 224: return launch_stream<2, 2, 4>(s, a, st);
    case 244: return launch_stream<2, 4, 4>(s, a, st);
    case 414: return launch_stream<4, 1, 4>(s, a, st);
    case 424: return launch_stream<4, 2, 4>(s, a, st);
    case 444: return launch_stream<4, 4, 4>(s, a, st);
    case 614: return launch_stream<6, 1, 4>(s, a, st);
    case 624: return launch_stream<6, 2, 4>(s, a, st);
    case 814: return launch_stream<8, 1, 4>(s, a, st);
    case 824: return launch_stream<8, 2, 4>(s, a, st);
  }
  return hipErrorInvalidValue;
}

}  // namespace spear

// Attention over the 4-bit paged key/value cache (spear_ec_kv.h): one wave
// per (row, query head), 64 tokens a step, a running maximum and sum.
#include "internal.hpp"
#include "kv_device.hpp"
#include "spear_ec_kv.h"

namespace spear {
namespace {

template <int D>
__global__ __launch_bounds__(64) void attention_kernel(KvShape s, KvBatch b, KvAttentionArgs a,
                                                       int* __restrict__ counters) {
  __shared__ float qs[D];
  __shared__ float ps[64];
  __shared__ int64_t blks[4];
  const int t = blockIdx.x, h = blockIdx.y, lane = threadIdx.x;
  KvRow r = kv_row(b, t);
  if (r.seq < 0) return;
  const int capacity = s.max_pages << s.page_shift;
  const bool past = r.pos >= capacity;  // its sequence is longer than its page-table row
  r.pos = min(r.pos, capacity - 1);
  const int head = h / (s.q_heads / s.kv_heads);
  for (int d = lane; d < D; d += 64)
    qs[d] = bf16_lo(a.q[(int64_t)t * a.q_stride + h * D + d]) * a.scale;
  __syncthreads();
  float m = -INFINITY, l = 0.f, o0 = 0.f, o1 = 0.f;  // lane's dimensions 2 lane, 2 lane + 1
  bool bad = past;
  const int first = a.window && r.pos >= a.window ? r.pos - a.window + 1 : 0;
  for (int j0 = first & ~63; j0 <= r.pos; j0 += 64) {
    if (lane < 4) blks[lane] = j0 + 16 * lane <= r.pos ? kv_block(s, b, r.seq, j0 + 16 * lane, head) : 0;
    __syncthreads();
    const int j = j0 + lane;
    const int64_t blk = blks[lane >> 4];
    const bool seen = j >= first && j <= r.pos;
    if (seen && blk < 0) bad = true;
    float x = -INFINITY, vs = 0.f;
    int vz = 8;
    if (seen && blk >= 0) {
      int kz = 8;
      if (s.zeros) {
        const int z = a.cache.zeros[blk * 16 + (j & 15)];
        kz = z & 15;
        vz = z >> 4;
      }
      const uint32_t* kr = reinterpret_cast<const uint32_t*>(a.cache.codes + blk * (16 * D) +
                                                             (j & 15) * (D / 2));
      float acc = 0.f;
      for (int w = 0; w < D / 8; ++w) {
        const uint32_t c = kr[w];
        for (int i = 0; i < 8; ++i)
          acc += (float)((int)((c >> (4 * i)) & 15u) - kz) * qs[8 * w + i];
      }
      x = acc * half_bits_to_f32(a.cache.scales[blk * 32 + (j & 15)]);
      vs = half_bits_to_f32(a.cache.scales[blk * 32 + 16 + (j & 15)]);
    }
    float top = x;
    for (int o = 32; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor(top, o, 64));
    const float mn = fmaxf(m, top);
    const float base = mn == -INFINITY ? 0.f : mn;
    const float alpha = expf(m - base);
    const float p = expf(x - base);
    m = mn;
    l = l * alpha + p;
    o0 *= alpha;
    o1 *= alpha;
    __syncthreads();
    ps[lane] = seen ? p * vs : 0.f;
    __syncthreads();
    for (int i = 0; i < 64; ++i) {
      const int64_t bi = blks[i >> 4];
      if (j0 + i < first || j0 + i > r.pos || bi < 0) continue;
      const int z = __shfl(vz, i, 64);
      if (lane < D / 2) {
        const int c = a.cache.codes[bi * (16 * D) + 8 * D + 16 * lane + (i & 15)];
        o0 += ps[i] * (float)((c & 15) - z);
        o1 += ps[i] * (float)((c >> 4) - z);
      }
    }
    __syncthreads();
  }
  for (int o = 32; o > 0; o >>= 1) l += __shfl_xor(l, o, 64);
  const bool any_bad = __any(bad);
  const float nan = __uint_as_float(0x7FC00000u);
  float inv = l > 0.f ? 1.f / l : 0.f;
  if (!(l >= 0.f) || any_bad) inv = nan;
  if (lane < D / 2) {
    const uint32_t w = f32_to_bf16_rne(o0 * inv) | (f32_to_bf16_rne(o1 * inv) << 16);
    reinterpret_cast<uint32_t*>(a.out + ((int64_t)t * s.q_heads + h) * D)[lane] = w;
  }
  if (lane == 0 && a.lse) a.lse[(int64_t)t * s.q_heads + h] = any_bad ? nan : m + logf(l);
  if (lane == 0 && any_bad) atomicOr(counters + kCtrError, SPEAR_EC_WS_BAD_PAGE);
}

}  // namespace

size_t kv_attention_workspace(const KvShape&, int, int) { return sizeof(int) * kCounterSlots; }

hipError_t launch_kv_attention(const KvShape& s, const KvBatch& b, const KvAttentionArgs& a,
                               void* workspace, hipStream_t st) {
  int* counters = static_cast<int*>(workspace);
  const dim3 grid(b.tokens, s.q_heads);
  if (s.D == 64)
    hipLaunchKernelGGL(attention_kernel<64>, grid, dim3(64), 0, st, s, b, a, counters);
  else
    hipLaunchKernelGGL(attention_kernel<128>, grid, dim3(64), 0, st, s, b, a, counters);
  return hipGetLastError();
}

}  // namespace spear

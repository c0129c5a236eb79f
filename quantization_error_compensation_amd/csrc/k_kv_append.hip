// Appending to and reading the 4-bit paged key/value cache (spear_ec_kv.h).
//
// Append.  One vector of head_dim elements (a query, key or value head of one
// token) takes head_dim / 8 lanes, 8 elements each, so a 16-byte load and a
// 4-byte store of codes a lane.  The rotation a' = a cos - b sin is evaluated
// in double: bf16 x fp32 products are exact there and their difference is
// rounded once, so a code near a border between two steps falls on the side
// the definition says.  The scale's maximum runs over the vector's lanes.
#include "kv_device.hpp"

namespace spear {
namespace {

__device__ __forceinline__ double shfl_xor_f64(double v, int o) {
  return __longlong_as_double(__shfl_xor(__double_as_longlong(v), o, 64));
}

// Codes of the lane's 8 elements (nibble i = element i), the vector's scale
// bits and zero-point.  LANES lanes hold the vector.
template <int LANES>
__device__ __forceinline__ uint32_t quantize8(const double (&x)[8], bool asym, uint16_t& sb,
                                              int& zp) {
  double lo = 0.0, hi = 0.0;
  for (int i = 0; i < 8; ++i) {
    lo = fmin(lo, x[i]);
    hi = fmax(hi, x[i]);
  }
  for (int o = LANES / 2; o > 0; o >>= 1) {
    lo = fmin(lo, shfl_xor_f64(lo, o));
    hi = fmax(hi, shfl_xor_f64(hi, o));
  }
  sb = f64_to_f16_rne_sat(asym ? (hi - lo) / 15.0 : fmax(hi, -lo) / 7.0);
  if ((sb & 0x7FFFu) == 0) sb = 0x3C00u;
  const double s = (double)half_bits_to_f32(sb);
  const double z = asym ? fmin(15.0, fmax(0.0, rint(-lo / s))) : 8.0;
  zp = (int)z;
  uint32_t word = 0;
  for (int i = 0; i < 8; ++i) {
    const double q = rint(x[i] / s);
    const double c = asym ? fmin(15.0, fmax(0.0, q + z)) : fmin(7.0, fmax(-8.0, q)) + 8.0;
    word |= (uint32_t)c << (4 * i);
  }
  return word;
}

// Eight elements without rotation.
__device__ __forceinline__ void widen8(double (&x)[8], u32x4 raw) {
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = (double)bf16_lo(raw[i]);
    x[2 * i + 1] = (double)bf16_hi(raw[i]);
  }
}

// The lane's 8 elements rotated for position pos.  Pairs (i, i + dim/2) lie
// dim/16 lanes apart, in the same vector.
__device__ __forceinline__ void rotate8(double (&x)[8], u32x4 raw, const KvRope& rope, int pos,
                                        int sub) {
  widen8(x, raw);
  if (!rope.cos_sin) return;
  const int half = rope.dim / 2;
  const float* row = rope.cos_sin + (int64_t)pos * rope.dim;
  const int d0 = 8 * sub;
  if (rope.interleaved) {
    if (d0 >= rope.dim) return;
    for (int i = 0; i < 4; ++i) {
      const double c = (double)row[d0 / 2 + i], s = (double)row[half + d0 / 2 + i];
      const double a = x[2 * i], b = x[2 * i + 1];
      x[2 * i] = a * c - b * s;
      x[2 * i + 1] = b * c + a * s;
    }
    return;
  }
  const int lane = threadIdx.x & 63;
  const bool first = d0 < half;
  const int away = half / 8;  // lanes between the two of a pair
  const int from = first ? lane + away : lane - away;
  u32x4 other;
  for (int i = 0; i < 4; ++i) other[i] = __shfl(raw[i], from & 63, 64);
  if (d0 >= rope.dim) return;
  const int at = first ? d0 : d0 - half;
  for (int i = 0; i < 8; ++i) {
    const double c = (double)row[at + i], s = (double)row[half + at + i];
    const double o = (double)((i & 1) ? bf16_hi(other[i / 2]) : bf16_lo(other[i / 2]));
    x[i] = first ? x[i] * c - o * s : x[i] * c + o * s;
  }
}

// One workgroup per (token, 256 / LANES units): the token's units are its kv
// heads (key and value together: they share a zero-point byte), then its
// query heads.
template <int D>
__global__ __launch_bounds__(256) void append_kernel(KvShape s, KvBatch b, KvAppendArgs a) {
  constexpr int LANES = D / 8;
  const int t = blockIdx.x;
  const KvRow r = kv_row(b, t);
  if (r.seq < 0) return;
  const int unit = blockIdx.y * (256 / LANES) + threadIdx.x / LANES;
  const int sub = threadIdx.x % LANES;
  if (unit >= s.kv_heads + (a.q ? s.q_heads : 0)) return;  // whole vectors leave
  const bool is_q = unit >= s.kv_heads;
  const int head = is_q ? unit - s.kv_heads : unit;
  // -1 for padding, a bad page or a position past the rotation's table
  int64_t blk = r.pos < 0 ? -1 : kv_block(s, b, r.seq, r.pos, is_q ? 0 : head);
  if (a.rope.cos_sin && r.pos >= a.rope.rows) blk = -1;

  const uint16_t* src = is_q ? a.q + (int64_t)t * a.q_stride : a.k + (int64_t)t * a.k_stride;
  const u32x4 raw = load16(src + head * D + 8 * sub);
  if (blk < 0) {
    if (!is_q) return;
    const uint32_t fill = r.pos < 0 ? 0u : 0x7FC07FC0u;
    *reinterpret_cast<u32x4*>(a.q_out + (int64_t)t * a.q_out_stride + head * D + 8 * sub) =
        u32x4{fill, fill, fill, fill};
    return;
  }
  double x[8];
  rotate8(x, raw, a.rope, r.pos, sub);
  if (is_q) {
    u32x4 o;
    for (int i = 0; i < 4; ++i)
      o[i] = f32_to_bf16_rne((float)x[2 * i]) | (f32_to_bf16_rne((float)x[2 * i + 1]) << 16);
    *reinterpret_cast<u32x4*>(a.q_out + (int64_t)t * a.q_out_stride + head * D + 8 * sub) = o;
    return;
  }
  const u32x4 vraw = load16(a.v + (int64_t)t * a.v_stride + head * D + 8 * sub);
  uint16_t ks, vs;
  int kz, vz;
  const uint32_t kw = quantize8<LANES>(x, s.zeros, ks, kz);
  widen8(x, vraw);
  const uint32_t vw = quantize8<LANES>(x, s.zeros, vs, vz);
  const int j = r.pos & 15;
  uint8_t* codes = a.cache.codes + blk * (16 * D);
  *reinterpret_cast<uint32_t*>(codes + j * (D / 2) + 4 * sub) = kw;
  uint8_t* col = codes + 8 * D + 64 * sub + j;
  for (int i = 0; i < 4; ++i) col[16 * i] = (uint8_t)(vw >> (8 * i));
  if (sub == 0) {
    a.cache.scales[blk * 32 + j] = ks;
    a.cache.scales[blk * 32 + 16 + j] = vs;
    if (s.zeros) a.cache.zeros[blk * 16 + j] = (uint8_t)(kz | (vz << 4));
  }
}

// One workgroup per (token, 256 / LANES kv heads), 8 elements a lane.
template <int D>
__global__ __launch_bounds__(256) void kv_dequant_kernel(KvShape s, KvBatch b, KvCache c,
                                                         float* __restrict__ k_out,
                                                         float* __restrict__ v_out) {
  constexpr int LANES = D / 8;
  const int t = blockIdx.x;
  const KvRow r = kv_row(b, t);
  if (r.seq < 0) return;
  const int head = blockIdx.y * (256 / LANES) + threadIdx.x / LANES;
  const int sub = threadIdx.x % LANES;
  if (head >= s.kv_heads) return;
  const int64_t at = ((int64_t)t * s.kv_heads + head) * D + 8 * sub;
  float k[8], v[8];
  const int64_t blk = r.pos < 0 ? -1 : kv_block(s, b, r.seq, r.pos, head);
  if (blk < 0) {
    const float fill = r.pos < 0 ? 0.f : __uint_as_float(0x7FC00000u);
    for (int i = 0; i < 8; ++i) k[i] = v[i] = fill;
  } else {
    const int j = r.pos & 15;
    const uint8_t* codes = c.codes + blk * (16 * D);
    const uint32_t kw = *reinterpret_cast<const uint32_t*>(codes + j * (D / 2) + 4 * sub);
    const uint8_t* col = codes + 8 * D + 64 * sub + j;
    uint32_t vw = 0;
    for (int i = 0; i < 4; ++i) vw |= (uint32_t)col[16 * i] << (8 * i);
    const float ks = half_bits_to_f32(c.scales[blk * 32 + j]);
    const float vs = half_bits_to_f32(c.scales[blk * 32 + 16 + j]);
    int kz = 8, vz = 8;
    if (s.zeros) {
      const int z = c.zeros[blk * 16 + j];
      kz = z & 15;
      vz = z >> 4;
    }
    for (int i = 0; i < 8; ++i) {
      k[i] = (float)((int)((kw >> (4 * i)) & 15u) - kz) * ks;
      v[i] = (float)((int)((vw >> (4 * i)) & 15u) - vz) * vs;
    }
  }
  float4* kd = reinterpret_cast<float4*>(k_out + at);
  float4* vd = reinterpret_cast<float4*>(v_out + at);
  kd[0] = make_float4(k[0], k[1], k[2], k[3]);
  kd[1] = make_float4(k[4], k[5], k[6], k[7]);
  vd[0] = make_float4(v[0], v[1], v[2], v[3]);
  vd[1] = make_float4(v[4], v[5], v[6], v[7]);
}

int ceil_div(int a, int b) { return (a + b - 1) / b; }

}  // namespace

hipError_t launch_kv_append(const KvShape& s, const KvBatch& b, const KvAppendArgs& a,
                            hipStream_t st) {
  const int units = s.kv_heads + (a.q ? s.q_heads : 0);
  const dim3 grid(b.tokens, ceil_div(units, 256 / (s.D / 8)));
  if (s.D == 64)
    hipLaunchKernelGGL(append_kernel<64>, grid, dim3(256), 0, st, s, b, a);
  else
    hipLaunchKernelGGL(append_kernel<128>, grid, dim3(256), 0, st, s, b, a);
  return hipGetLastError();
}

hipError_t launch_kv_dequant(const KvShape& s, const KvBatch& b, const KvCache& c, float* k_out,
                             float* v_out, hipStream_t st) {
  const dim3 grid(b.tokens, ceil_div(s.kv_heads, 256 / (s.D / 8)));
  if (s.D == 64)
    hipLaunchKernelGGL(kv_dequant_kernel<64>, grid, dim3(256), 0, st, s, b, c, k_out, v_out);
  else
    hipLaunchKernelGGL(kv_dequant_kernel<128>, grid, dim3(256), 0, st, s, b, c, k_out, v_out);
  return hipGetLastError();
}

}  // namespace spear

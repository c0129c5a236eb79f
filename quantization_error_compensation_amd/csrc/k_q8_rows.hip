// Row operators of the 8-bit path: quantization of rows, the root-mean-square
// norm with the residual's addition and its quantized result, and rows read
// back as values.  HBM-bound, one pass: a row's elements stay in registers
// between its sums and its result.
//
// A workgroup takes a row; a thread holds C pieces of 8 elements.  What a row
// needs as a whole is one maximum and, for the norm, one sum of squares:
//     u_j = p_j r,  p_j = h_j w_j,  r = 1 / sqrt(mean(h^2) + eps)
//     s = RN_fp32(max|p| r / 127),  c_j = rint(p_j r / s),
// so both are reduced at once.  p_j is exact in fp32 (8 x 8 significant bits).
// The sum of squares and the ratio r / s are held in fp64, as codes next to a
// border between two steps would otherwise fall on the wrong side; one fp64
// fma with 1.5 * 2^52 as its addend multiplies, rounds half to even and leaves
// the integer in its low word.  Rows whose maximum or scale is near fp32's
// small end (where p_j is no longer exact, or s so coarse that codes exceed
// 127) take the definition as it stands: fp64 products, a division and a clamp.
#include "common.hpp"
#include "q8.hpp"

namespace spear {
namespace {

constexpr uint32_t kInfBits = 0x7F800000u;
constexpr float kSmallMax = 0x1p-100f, kSmallScale = 0x1p-120f;
constexpr double kRoundMagic = 6755399441055744.0;  // 1.5 * 2^52

// Maximum of v and sum of d over the workgroup, in every thread.  red: 2
// doubles per wave.  Contains barriers, the first of which also separates the
// reads of the call before.
template <bool SUM>
__device__ __forceinline__ void join_row(uint64_t& v, double& d, double* red) {
  for (int o = 32; o > 0; o >>= 1) {
    const uint64_t w = __shfl_xor((unsigned long long)v, o, 64);
    v = w > v ? w : v;
    if constexpr (SUM) d += __shfl_xor(d, o, 64);
  }
  const int waves = blockDim.x >> 6;
  if (waves == 1) return;
  __syncthreads();
  if ((threadIdx.x & 63) == 0) {
    red[2 * wave_id()] = __longlong_as_double((long long)v);
    red[2 * wave_id() + 1] = d;
  }
  __syncthreads();
  v = 0;
  d = 0;
  for (int w = 0; w < waves; ++w) {
    const uint64_t m = (uint64_t)__double_as_longlong(red[2 * w]);
    v = m > v ? m : v;
    if constexpr (SUM) d += red[2 * w + 1];
  }
}

// c = r / s: the code of p, for rows away from fp32's small end.
__device__ __forceinline__ uint32_t code_of(float p, double c) {
  return (uint32_t)__double2loint(fma((double)p, c, kRoundMagic)) & 0xFFu;
}
// The code of a value u as defined.
__device__ __forceinline__ uint32_t code_as_defined(double u, double s) {
  return (uint32_t)(int)fmin(fmax(rint(u / s), -127.0), 127.0) & 0xFFu;
}

// The scale of a row whose largest value is `top` (bits of a non-negative
// fp64): NaN where that or the scale is not finite.
__device__ __forceinline__ float scale_of(double top) {
  const float s = (float)(top / 127.0);
  if (!(s <= 3.4028234663852886e38f)) return __uint_as_float(0x7FC00000u);
  return s == 0.f ? 1.f : s;
}

template <int C, bool F32>
__global__ __launch_bounds__(1024) void quantize_kernel(const void* __restrict__ x, int64_t stride,
                                                        int8_t* __restrict__ codes,
                                                        float* __restrict__ scales, int rows,
                                                        int width) {
  __shared__ double red[32];
  const int pieces = width / 8;
  for (int row = blockIdx.x; row < rows; row += gridDim.x) {
    float v[C][8];
    uint32_t top = 0;
    #pragma unroll
    for (int c = 0; c < C; ++c) {
      const int i = threadIdx.x + c * blockDim.x;
      u32x4 a{0, 0, 0, 0}, b{0, 0, 0, 0};
      if (i < pieces) {
        if constexpr (F32) {
          const u32x4* at = reinterpret_cast<const u32x4*>(static_cast<const float*>(x) + row * stride) + 2 * i;
          a = at[0];
          b = at[1];
        } else {
          a = reinterpret_cast<const u32x4*>(static_cast<const uint16_t*>(x) + row * stride)[i];
        }
      }
      #pragma unroll
      for (int j = 0; j < 4; ++j) {
        if constexpr (F32) {
          v[c][j] = __uint_as_float(a[j]);
          v[c][4 + j] = __uint_as_float(b[j]);
        } else {
          v[c][2 * j] = bf16_lo(a[j]);
          v[c][2 * j + 1] = bf16_hi(a[j]);
        }
      }
      #pragma unroll
      for (int j = 0; j < 8; ++j) top = max(top, __float_as_uint(v[c][j]) & 0x7FFFFFFFu);
    }
    uint64_t most = top;
    double none = 0;
    join_row<false>(most, none, red);
    const double m = (double)__uint_as_float((uint32_t)most);
    const float s = (uint32_t)most >= kInfBits ? __uint_as_float(0x7FC00000u) : scale_of(m);
    const bool good = s == s, small = s < kSmallScale;
    const double inv = good ? 1.0 / (double)s : 0.0;
    if (threadIdx.x == 0) scales[row] = s;
    #pragma unroll
    for (int c = 0; c < C; ++c) {
      const int i = threadIdx.x + c * blockDim.x;
      if (i >= pieces) continue;
      u32x2 out{0, 0};
      #pragma unroll
      for (int j = 0; j < 8; ++j) {
        uint32_t code;
        if (F32 || small) code = code_as_defined((double)v[c][j], (double)s);
        else code = code_of(v[c][j], inv);
        out[j >> 2] |= code << (8 * (j & 3));
      }
      if (!good) out = u32x2{0, 0};
      *reinterpret_cast<u32x2*>(codes + (int64_t)row * width + 8 * i) = out;
    }
  }
}

template <int C>
__global__ __launch_bounds__(1024) void norm_kernel(Q8Norm a, int rows, int width) {
  __shared__ double red[32];
  const int pieces = width / 8;
  for (int row = blockIdx.x; row < rows; row += gridDim.x) {
    u32x4 h[C], w[C];
    double squares = 0;
    uint32_t top = 0;
    #pragma unroll
    for (int c = 0; c < C; ++c) {
      const int i = threadIdx.x + c * blockDim.x;
      h[c] = w[c] = u32x4{0, 0, 0, 0};
      if (i < pieces) {
        h[c] = reinterpret_cast<const u32x4*>(a.x + row * a.x_stride)[i];
        w[c] = reinterpret_cast<const u32x4*>(a.weight)[i];
        if (a.residual) {
          const u32x4 r = reinterpret_cast<const u32x4*>(a.residual + (int64_t)row * width)[i];
          #pragma unroll
          for (int j = 0; j < 4; ++j)
            h[c][j] = f32_to_bf16_rne(bf16_lo(h[c][j]) + bf16_lo(r[j])) |
                      f32_to_bf16_rne(bf16_hi(h[c][j]) + bf16_hi(r[j])) << 16;
        }
      }
    }
    #pragma unroll
    for (int c = 0; c < C; ++c) {
      const int i = threadIdx.x + c * blockDim.x;
      if (a.residual && i < pieces)
        reinterpret_cast<u32x4*>(a.sum + (int64_t)row * width)[i] = h[c];
      #pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float e = j & 1 ? bf16_hi(h[c][j >> 1]) : bf16_lo(h[c][j >> 1]);
        const float f = j & 1 ? bf16_hi(w[c][j >> 1]) : bf16_lo(w[c][j >> 1]);
        squares = fma((double)e, (double)e, squares);
        top = max(top, __float_as_uint(e * f) & 0x7FFFFFFFu);
      }
    }
    uint64_t most = top;
    join_row<true>(most, squares, red);
    const double r = 1.0 / sqrt(squares / width + a.eps);
    bool good = (uint32_t)most < kInfBits && squares < 1e300;
    double m = (double)__uint_as_float((uint32_t)most);
    bool small = m < kSmallMax;
    float s = scale_of(m * r);
    if (good && (small || s < kSmallScale)) {  // as defined, in fp64
      small = true;
      uint64_t exact_top = 0;
      for (int c = 0; c < C; ++c)
        for (int j = 0; j < 8; ++j) {
          const double e = j & 1 ? bf16_hi(h[c][j >> 1]) : bf16_lo(h[c][j >> 1]);
          const double f = j & 1 ? bf16_hi(w[c][j >> 1]) : bf16_lo(w[c][j >> 1]);
          const uint64_t bits = (uint64_t)__double_as_longlong(fabs(e * f));
          exact_top = bits > exact_top ? bits : exact_top;
        }
      double none = 0;
      join_row<false>(exact_top, none, red);
      m = __longlong_as_double((long long)exact_top);
      s = scale_of(m * r);
    }
    good = good && s == s;
    if (!good) s = __uint_as_float(0x7FC00000u);
    if (a.codes && threadIdx.x == 0) a.scales[row] = s;
    const double ratio = r / (double)s;
    const float r32 = (float)r;
    #pragma unroll
    for (int c = 0; c < C; ++c) {
      const int i = threadIdx.x + c * blockDim.x;
      if (i >= pieces) continue;
      u32x2 out{0, 0};
      u32x4 y{0, 0, 0, 0};
      #pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float e = j & 1 ? bf16_hi(h[c][j >> 1]) : bf16_lo(h[c][j >> 1]);
        const float f = j & 1 ? bf16_hi(w[c][j >> 1]) : bf16_lo(w[c][j >> 1]);
        const float p = e * f;
        if (a.codes) {
          const uint32_t code = small ? code_as_defined((double)e * (double)f * r, (double)s)
                                      : code_of(p, ratio);
          out[j >> 2] |= code << (8 * (j & 3));
        }
        if (a.y)
          y[j >> 1] |= f32_to_bf16_rne(small ? (float)((double)e * (double)f * r) : p * r32)
                       << (16 * (j & 1));
      }
      if (!good) {
        out = u32x2{0, 0};
        y = u32x4{0x7FC07FC0u, 0x7FC07FC0u, 0x7FC07FC0u, 0x7FC07FC0u};
      }
      if (a.codes) *reinterpret_cast<u32x2*>(a.codes + (int64_t)row * width + 8 * i) = out;
      if (a.y) reinterpret_cast<u32x4*>(a.y + (int64_t)row * width)[i] = y;
    }
  }
}

// Four codes a thread and step: consecutive lanes write consecutive 16 bytes.
__global__ __launch_bounds__(256) void dequant_kernel(const int8_t* __restrict__ codes,
                                                      const float* __restrict__ scales,
                                                      float* __restrict__ out, int rows, int width) {
  const int words = width / 4;
  for (int row = blockIdx.y; row < rows; row += gridDim.y) {
    const float s = scales[row];
    const uint32_t* from = reinterpret_cast<const uint32_t*>(codes + (int64_t)row * width);
    f32x4* to = reinterpret_cast<f32x4*>(out + (int64_t)row * width);
    for (int i = blockIdx.x * 256 + threadIdx.x; i < words; i += gridDim.x * 256) {
      const uint32_t c = from[i];
      f32x4 v;
      #pragma unroll
      for (int j = 0; j < 4; ++j) v[j] = (float)(int8_t)(c >> (8 * j)) * s;
      to[i] = v;
    }
  }
}

// Pieces a thread and threads a workgroup for rows of `pieces` pieces.
struct RowPlan {
  int c, threads;
};
RowPlan plan_rows(int pieces) {
  int c = 1;
  while (c < 8 && (pieces + c - 1) / c > 256) c *= 2;
  const int threads = ((pieces + c - 1) / c + 63) / 64 * 64;
  return RowPlan{c, threads};
}
constexpr int kMaxGrid = 65536;

}  // namespace

hipError_t launch_q8_quantize(int rows, int width, const void* x, bool x_f32, int64_t x_stride,
                              int8_t* codes, float* scales, hipStream_t st) {
  const RowPlan pl = plan_rows(width / 8);
  const dim3 grid(rows < kMaxGrid ? rows : kMaxGrid), block(pl.threads);
#define SPEAR_Q8_ROWS(C)                                                                       \
  case C:                                                                                      \
    if (x_f32)                                                                                 \
      hipLaunchKernelGGL((quantize_kernel<C, true>), grid, block, 0, st, x, x_stride, codes,   \
                         scales, rows, width);                                                 \
    else                                                                                       \
      hipLaunchKernelGGL((quantize_kernel<C, false>), grid, block, 0, st, x, x_stride, codes,  \
                         scales, rows, width);                                                 \
    break;
  switch (pl.c) { SPEAR_Q8_ROWS(1) SPEAR_Q8_ROWS(2) SPEAR_Q8_ROWS(4) SPEAR_Q8_ROWS(8) }
#undef SPEAR_Q8_ROWS
  return hipGetLastError();
}

hipError_t launch_q8_norm(int rows, int width, const Q8Norm& a, hipStream_t st) {
  const RowPlan pl = plan_rows(width / 8);
  const dim3 grid(rows < kMaxGrid ? rows : kMaxGrid), block(pl.threads);
  switch (pl.c) {
    case 1: hipLaunchKernelGGL(norm_kernel<1>, grid, block, 0, st, a, rows, width); break;
    case 2: hipLaunchKernelGGL(norm_kernel<2>, grid, block, 0, st, a, rows, width); break;
    case 4: hipLaunchKernelGGL(norm_kernel<4>, grid, block, 0, st, a, rows, width); break;
    case 8: hipLaunchKernelGGL(norm_kernel<8>, grid, block, 0, st, a, rows, width); break;
  }
  return hipGetLastError();
}

hipError_t launch_q8_dequant(int rows, int width, const int8_t* codes, const float* scales,
                             float* out, hipStream_t st) {
  const dim3 grid((width / 4 + 255) / 256, rows < 32768 ? rows : 32768);
  hipLaunchKernelGGL(dequant_kernel, grid, dim3(256), 0, st, codes, scales, out, rows, width);
  return hipGetLastError();
}

}  // namespace spear

// Row operators of the 8-bit path: quantization of rows, the root-mean-square
// norm with the residual's addition and its quantized result, and rows read
// back as values.  HBM-bound, one pass: a row's elements stay in registers
// between its sums and its result.
//
// What a row needs as a whole is one maximum and, for the norm, one sum of
// squares:
//     u_j = p_j r,  p_j = h_j w_j,  r = 1 / sqrt(mean(h^2) + eps)
//     s = RN_fp32(max|p| r / 127),  c_j = rint(p_j r / s),
// so both are reduced at once.  p_j is exact in fp32 (8 x 8 significant bits);
// as non-negative floats order like their bits, the maximum is one of integers,
// in which infinity and NaN come out on top.  The sum of squares and the ratio
// r / s are held in fp64, as codes next to a border between two steps would
// otherwise fall on the wrong side; one fp64 fma with 1.5 * 2^52 as its addend
// multiplies, rounds half to even and leaves the integer in its low word.  Rows
// whose maximum or scale is near fp32's small end (where p_j is no longer
// exact, or s so coarse that codes exceed 127), or whose products or r leave
// fp32, take the definition as it stands: fp64 products, a division and a clamp.
//
// Rows of up to 2048 elements belong to one wave or, of up to 256, to a part
// of one, and meet no barrier; wider ones to a workgroup.
//
// Norm with residual, 4096 x 8192: 43 to 46 us (5.5 to 5.1 TB/s; a copy reaches
// 4.9) over inputs and outputs that the last-level cache does not hold, 37 when the
// same ones come again; without residual 23.5 and 20 us, where the fp64 steps of the
// sum and the codes show.  Quantization of bf16 4096 x 8192 20 and 16 us (5.0 TB/s
// from memory), of fp32 11008 x 4096 38 to 41 and 32.5 (5.9 to 5.5).  One row of
// 4096: 3.4 to 3.6 us, most of it launch, one load's latency and the chain from the
// sums to the ratio.
#include "common.hpp"
#include "q8_math.hpp"

namespace spear {
namespace {

constexpr uint32_t kInfBits = 0x7F800000u, kNanBits = 0x7FC00000u;
constexpr float kSmallMax = 0x1p-100f, kSmallScale = 0x1p-120f;
constexpr double kRoundMagic = 6755399441055744.0;  // 1.5 * 2^52

template <int CTRL, int ROWS>
__device__ __forceinline__ uint32_t moved(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, ROWS, 0xF, false);
}
// v's value in the lane that data-parallel-primitive control CTRL names (0
// where there is none), added to or compared with the lane's own; lane 63 ends
// with the wave's after shifts by 1, 2, 4, 8 within rows of 16 lanes and two
// moves across rows.
template <int CTRL, int ROWS, typename T>
__device__ __forceinline__ T joined(T v) {
  if constexpr (sizeof(T) == 4) {
    return max(v, (T)moved<CTRL, ROWS>(v));
  } else {
    const uint64_t b = __builtin_bit_cast(uint64_t, v);
    const uint64_t o = (uint64_t)moved<CTRL, ROWS>((uint32_t)(b >> 32)) << 32 | moved<CTRL, ROWS>((uint32_t)b);
    if constexpr (__is_same(T, double)) return v + __builtin_bit_cast(double, o);
    else return max(v, (T)o);
  }
}
// Maximum (integers) or sum (double) of v over LANES neighbouring lanes, in all
// of them.
template <int LANES, typename T>
__device__ __forceinline__ T join_lanes(T v) {
  if constexpr (LANES == 64) {
    v = joined<0x111, 0xF>(v);
    v = joined<0x112, 0xF>(v);
    v = joined<0x114, 0xF>(v);
    v = joined<0x118, 0xF>(v);
    v = joined<0x142, 0xA>(v);
    v = joined<0x143, 0xC>(v);
    if constexpr (sizeof(T) == 4) {
      return (T)__builtin_amdgcn_readlane((uint32_t)v, 63);
    } else {
      const uint64_t b = __builtin_bit_cast(uint64_t, v);
      const uint64_t o = (uint64_t)__builtin_amdgcn_readlane((uint32_t)(b >> 32), 63) << 32 |
                         (uint32_t)__builtin_amdgcn_readlane((uint32_t)b, 63);
      return __builtin_bit_cast(T, o);
    }
  } else {
    #pragma unroll
    for (int o = LANES / 2; o > 0; o >>= 1) {
      if constexpr (__is_same(T, double)) v += __shfl_xor(v, o, 64);
      else if constexpr (sizeof(T) == 4) v = max(v, (T)__shfl_xor((int)v, o, 64));
      else v = max(v, (T)__shfl_xor((unsigned long long)v, o, 64));
    }
    return v;
  }
}

// A row's share of a workgroup: LANES lanes of a wave, or with LANES 0 all of
// its waves.
template <int LANES>
struct RowTeam {
  uint64_t* red;  // with LANES 0: 2 words a wave in LDS
  template <typename T>
  __device__ __forceinline__ T join(T v) const {
    if constexpr (LANES > 0) return join_lanes<LANES>(v);
    v = join_lanes<64>(v);
    const int waves = blockDim.x >> 6;
    if (waves == 1) return v;
    __syncthreads();  // the words of the join before are read
    if ((threadIdx.x & 63) == 0) reinterpret_cast<T*>(red)[wave_id()] = v;
    __syncthreads();
    T all = reinterpret_cast<T*>(red)[0];
    for (int w = 1; w < waves; ++w) {
      const T o = reinterpret_cast<T*>(red)[w];
      if constexpr (__is_same(T, double)) all += o;
      else all = max(all, o);
    }
    return all;
  }
  // A maximum and a sum at once.
  __device__ __forceinline__ void join2(uint32_t& m, double& d) const {
    if constexpr (LANES > 0) {
      m = join_lanes<LANES>(m);
      d = join_lanes<LANES>(d);
    } else {
      m = join_lanes<64>(m);
      d = join_lanes<64>(d);
      const int waves = blockDim.x >> 6;
      if (waves == 1) return;
      __syncthreads();
      if ((threadIdx.x & 63) == 0) {
        red[2 * wave_id()] = m;
        red[2 * wave_id() + 1] = __builtin_bit_cast(uint64_t, d);
      }
      __syncthreads();
      m = 0;
      d = 0;
      for (int w = 0; w < waves; ++w) {
        m = max(m, (uint32_t)red[2 * w]);
        d += __builtin_bit_cast(double, red[2 * w + 1]);
      }
    }
  }
};

// c = r / s: the code of p, in the low byte, for rows away from fp32's small end.
__device__ __forceinline__ uint32_t code_of(float p, double c) {
  return (uint32_t)__double2loint(fma((double)p, c, kRoundMagic));
}
// The low bytes of four words.
__device__ __forceinline__ uint32_t four(const uint32_t* w) {
  const uint32_t low = __builtin_amdgcn_perm(w[1], w[0], 0x0C0C0400u);
  const uint32_t high = __builtin_amdgcn_perm(w[3], w[2], 0x0C0C0400u);
  return low | high << 16;
}
// The same for a p of 24 significant bits, whose ratio to s may be a tie that
// the product with the reciprocal misses: border is set where the product, off
// by 2^-45 at most, is that near to one.  (11008 x 4096 32.5 us, 41 from memory;
// dividing every element instead 39 and 42; 28672 x 8192 203 and 220.)
__device__ __forceinline__ uint32_t code_or_border(float p, double inv, bool& border) {
  const double ratio = (double)p * inv, rounded = ratio + kRoundMagic;
  border |= fabs(fabs(ratio - (rounded - kRoundMagic)) - 0.5) < 0x1p-40;
  return (uint32_t)__double2loint(rounded);
}
// The code of a value u as defined.
__device__ __forceinline__ uint32_t code_as_defined(double u, double s) {
  return (uint32_t)(int)fmin(fmax(rint(u / s), -127.0), 127.0);
}
// The scale of a row whose largest value is `top`: NaN where that or the scale
// is not finite.
__device__ __forceinline__ float scale_of(double top) {
  const float s = (float)(top / 127.0);
  if (!(s <= 3.4028234663852886e38f)) return __uint_as_float(kNanBits);
  return s == 0.f ? 1.f : s;
}
// Two fp32 -> bf16 pair, subnormal ones too (the conversion instruction makes
// them zeros).
__device__ __forceinline__ uint32_t rounded_pair(float a, float b) {
  return f32_to_bf16_rne(a) | f32_to_bf16_rne(b) << 16;
}
__device__ __forceinline__ float element(const u32x4& v, int j) {  // j of 8 bf16
  return j & 1 ? bf16_hi(v[j >> 1]) : bf16_lo(v[j >> 1]);
}

// A thread's place among the rows of its workgroup and the lanes of its row.
template <int LANES>
struct RowPlace {
  int rows, sub, lane, lanes;  // rows of a workgroup, which of them
  __device__ RowPlace() {
    rows = LANES > 0 ? (int)blockDim.x / (LANES > 0 ? LANES : 1) : 1;
    sub = LANES > 0 ? threadIdx.x / (LANES > 0 ? LANES : 1) : 0;
    lane = LANES > 0 ? threadIdx.x % (LANES > 0 ? LANES : 1) : threadIdx.x;
    lanes = LANES > 0 ? LANES : blockDim.x;
  }
};

// C: pieces of 8 elements a thread.  Lanes of a row past the last one (rows
// that share a wave) go along with the last row's data and write nothing.
template <int C, int LANES, bool F32>
__global__ __launch_bounds__(LANES ? 256 : 1024) void quantize_kernel(const void* __restrict__ x,
                                                                      int64_t stride, int8_t* __restrict__ codes,
                                                                      float* __restrict__ scales, int rows,
                                                                      int width) {
  __shared__ uint64_t red[32];
  const RowTeam<LANES> team{red};
  const int pieces = width / 8;
  const RowPlace<LANES> at;
  for (int first = blockIdx.x * at.rows; first < rows; first += gridDim.x * at.rows) {
    const bool live = first + at.sub < rows;
    const int row = live ? first + at.sub : rows - 1;
    u32x4 v[C][F32 ? 2 : 1];
    uint32_t top = 0;
    #pragma unroll
    for (int c = 0; c < C; ++c) {
      const int i = at.lane + c * at.lanes;
      #pragma unroll
      for (int k = 0; k < (F32 ? 2 : 1); ++k) v[c][k] = u32x4{0, 0, 0, 0};
      if (i < pieces) {
        if constexpr (F32) {
          const u32x4* from = reinterpret_cast<const u32x4*>(static_cast<const float*>(x) + row * stride) + 2 * i;
          v[c][0] = from[0];
          v[c][1] = from[1];
        } else {
          v[c][0] = reinterpret_cast<const u32x4*>(static_cast<const uint16_t*>(x) + row * stride)[i];
        }
      }
    }
    auto value = [&](int c, int j) {
      if constexpr (F32) return __uint_as_float(v[c][j >> 2][j & 3]);
      else return element(v[c][0], j);
    };
    #pragma unroll
    for (int c = 0; c < C; ++c)
      #pragma unroll
      for (int j = 0; j < 8; ++j) top = max(top, __float_as_uint(value(c, j)) & 0x7FFFFFFFu);
    top = team.join(top);
    const float s = top >= kInfBits ? __uint_as_float(kNanBits) : scale_of((double)__uint_as_float(top));
    const bool good = s == s, small = s < kSmallScale;
    const double inv = good ? 1.0 / (double)s : 0.0;
    if (!live) continue;
    if (at.lane == 0) scales[row] = s;
    #pragma unroll
    for (int c = 0; c < C; ++c) {
      const int i = at.lane + c * at.lanes;
      if (i >= pieces) continue;
      uint32_t code[8];
      bool again = small;
      #pragma unroll
      for (int j = 0; j < 8; ++j) {
        if constexpr (F32) code[j] = code_or_border(value(c, j), inv, again);
        else code[j] = code_of(value(c, j), inv);
      }
      if (again) {
        #pragma unroll
        for (int j = 0; j < 8; ++j) code[j] = code_as_defined((double)value(c, j), (double)s);
      }
      u32x2 out = {four(code), four(code + 4)};
      if (!good) out = u32x2{0, 0};
      *reinterpret_cast<u32x2*>(codes + (int64_t)row * width + 8 * i) = out;
    }
  }
}

// Stores 16 bytes; EARLY: marked to leave the caches first.
template <bool EARLY>
__device__ __forceinline__ void put(u32x4 v, u32x4* p) {
  if constexpr (EARLY) __builtin_nontemporal_store(v, p);
  else *p = v;
}

template <int C, int LANES, bool EARLY>
__global__ __launch_bounds__(LANES ? 256 : 1024) void norm_kernel(Q8Norm a, int rows, int width) {
  __shared__ uint64_t red[32];
  const RowTeam<LANES> team{red};
  const int pieces = width / 8;
  const RowPlace<LANES> at;
  for (int first = blockIdx.x * at.rows; first < rows; first += gridDim.x * at.rows) {
    const bool live = first + at.sub < rows;
    const int row = live ? first + at.sub : rows - 1;
    const u32x4* xr = reinterpret_cast<const u32x4*>(a.x + row * a.x_stride);
    const u32x4* wr = reinterpret_cast<const u32x4*>(a.weight);
    u32x4* sr = reinterpret_cast<u32x4*>(a.sum + (int64_t)row * width);
    u32x4 h[C], w[C];
    #pragma unroll
    for (int c = 0; c < C; ++c) {
      const int i = at.lane + c * at.lanes;
      h[c] = w[c] = u32x4{0, 0, 0, 0};
      if (i < pieces) {
        h[c] = xr[i];
        w[c] = wr[i];
      }
    }
    if (a.residual) {
      const u32x4* rr = reinterpret_cast<const u32x4*>(a.residual + (int64_t)row * width);
      u32x4 d[C];
      #pragma unroll
      for (int c = 0; c < C; ++c) {
        const int i = at.lane + c * at.lanes;
        d[c] = u32x4{0, 0, 0, 0};
        if (i < pieces) d[c] = rr[i];
      }
      #pragma unroll
      for (int c = 0; c < C; ++c) {
        const int i = at.lane + c * at.lanes;
        #pragma unroll
        for (int j = 0; j < 4; ++j)  // as one rounding: fp32's 24 bits are at least 2 * 8 + 2
          h[c][j] = rounded_pair(bf16_lo(h[c][j]) + bf16_lo(d[c][j]), bf16_hi(h[c][j]) + bf16_hi(d[c][j]));
        if (live && i < pieces) put<EARLY>(h[c], sr + i);
      }
    }
    float p[C][8];
    double squares = 0;
    uint32_t top = 0;
    #pragma unroll
    for (int c = 0; c < C; ++c)
      #pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float e = element(h[c], j);
        squares = fma((double)e, (double)e, squares);
        p[c][j] = e * element(w[c], j);
        top = max(top, __float_as_uint(p[c][j]) & 0x7FFFFFFFu);
      }
    team.join2(top, squares);
    const double r = 1.0 / sqrt(squares / width + a.eps);
    const float r32 = (float)r;
    bool good = squares < 1e300;  // h is finite
    const double m = (double)__uint_as_float(top);
    float s = scale_of(m * r);
    // near fp32's small end, where a product leaves fp32 (or a weight is not finite)
    // and where r does (mean + eps past 2^-256 or 2^252: no fp32 of 24 bits holds
    // y's factor) the products are taken again, in fp64; not for a row of zeros
    // (padding: 4096 x 8192 of them 102 us, so 32), whose products are exact
    const bool again = good && (top >= kInfBits || !__builtin_isnormal(r32) ||
                                (squares > 0 && (m < kSmallMax || s < kSmallScale)));
    auto product = [&](int c, int j) {
      const int i = at.lane + c * at.lanes;
      if (i >= pieces) return 0.0;
      const uint16_t* hr = a.residual ? a.sum + (int64_t)row * width : a.x + row * a.x_stride;
      return (double)__uint_as_float((uint32_t)hr[8 * i + j] << 16) *
             (double)__uint_as_float((uint32_t)a.weight[8 * i + j] << 16);
    };
    if (again) {
      uint64_t most = 0;
      if (live)  // others' rows are being written
        for (int c = 0; c < C; ++c)
          for (int j = 0; j < 8; ++j) most = max(most, __builtin_bit_cast(uint64_t, fabs(product(c, j))));
      most = team.join(most);
      s = scale_of(__builtin_bit_cast(double, most) * r);
    }
    good = good && s == s;
    if (!good) s = __uint_as_float(kNanBits);
    if (!live) continue;
    if (a.codes && at.lane == 0) a.scales[row] = s;
    const double ratio = r / (double)s;
    #pragma unroll
    for (int c = 0; c < C; ++c) {
      const int i = at.lane + c * at.lanes;
      if (i >= pieces) continue;
      if (a.codes) {
        uint32_t code[8];
        #pragma unroll
        for (int j = 0; j < 8; ++j) code[j] = code_of(p[c][j], ratio);
        if (again)
          for (int j = 0; j < 8; ++j) code[j] = code_as_defined(product(c, j) * r, (double)s);
        u32x2 out = {four(code), four(code + 4)};
        if (!good) out = u32x2{0, 0};
        *reinterpret_cast<u32x2*>(a.codes + (int64_t)row * width + 8 * i) = out;
      }
      if (a.y) {
        float y[8];
        #pragma unroll
        for (int j = 0; j < 8; ++j) y[j] = p[c][j] * r32;
        if (again)
          for (int j = 0; j < 8; ++j) y[j] = (float)(product(c, j) * r);
        u32x4 out;
        #pragma unroll
        for (int j = 0; j < 4; ++j) out[j] = good ? rounded_pair(y[2 * j], y[2 * j + 1]) : 0x7FC07FC0u;
        put<EARLY>(out, reinterpret_cast<u32x4*>(a.y + (int64_t)row * width) + i);
      }
    }
  }
}

// Four codes a thread and step: consecutive lanes write consecutive 16 bytes.
// 2^share lanes of a workgroup take a row, so that narrow rows fill it too
// (100000 rows of 128: 22 us with a workgroup for each, 11.5 so).  The values, four
// times as many bytes as the codes, are marked to leave the caches first: from
// memory 4096 x 8192 33 -> 27 us, from the last-level cache the same.  A read of the
// values right behind takes back what was gained, more or less: with a conversion
// of them to bf16 1333 x 4096 14.1 -> 13.6 us, 4096 x 4096 32.9 -> 34.8, 4096 x 8192
// 63.5 -> 62.8, up to 512 x 4096 the same.  Codes are read next: so marked,
// quantizing 11008 x 4096 and reading it back takes 83 us instead of 73.
__global__ __launch_bounds__(256) void dequant_kernel(const int8_t* __restrict__ codes,
                                                      const float* __restrict__ scales,
                                                      float* __restrict__ out, int rows, int width, int share) {
  const int words = width / 4, lanes = 1 << share, per = 256 >> share;
  const int lane = threadIdx.x & (lanes - 1), sub = threadIdx.x >> share;
  for (int64_t row = (int64_t)blockIdx.y * per + sub; row < rows; row += (int64_t)gridDim.y * per) {
    const float s = scales[row];
    const uint32_t* from = reinterpret_cast<const uint32_t*>(codes + row * width);
    f32x4* to = reinterpret_cast<f32x4*>(out + row * width);
    for (int i = blockIdx.x * lanes + lane; i < words; i += gridDim.x * lanes) {
      const uint32_t c = from[i];
      f32x4 v;
      #pragma unroll
      for (int j = 0; j < 4; ++j) v[j] = (float)(int8_t)(c >> (8 * j)) * s;
      __builtin_nontemporal_store(v, to + i);
    }
  }
}

// How rows of `pieces` pieces are shared out.
struct RowPlan {
  int c, lanes, threads, rows;  // pieces a thread; lanes of a row (0: a workgroup); rows a workgroup
};
// A wave or part of it up to 256 pieces (2048 elements): 30000 rows of 1040 take
// 39 us with 3 pieces a lane of a wave, 46 with two waves a row.  Wider rows
// take the fewest waves of 2, 4, 8, 12, 16 that leave a thread at most 4 pieces,
// or 2 for fp32 (8192 x 4096 28 us, with 4 pieces 30) and in calls of fewer than
// 2048 rows, where a row's own time counts: waves
// that are no such number load the SIMDs unevenly, more pieces take registers
// from a second workgroup, fewer leave lanes idle.  Norm with residual, us, the same
// inputs again and again:
//   8192 x 4096  2 waves of 4 pieces 37, 8 of 1 46     512 x 4096  4 waves of 2 5.5, 2 of 4 6.6
//   4096 x 8192  4 of 4 37, 8 of 2 39, 6 of 3 48, 5 of 4 52
//   3000 x 11008 8 of 3 38, 6 of 4 45, 4 of 6 45, 12 of 2 51
//   2000 x 28672 12 of 5 93, 16 of 4 95, 8 of 7 103, 10 of 6 111
RowPlan plan_rows(int rows, int pieces, bool f32) {
  if (pieces <= 256) {
    const int lanes = pieces <= 16 ? 16 : pieces <= 32 ? 32 : 64;
    return RowPlan{(pieces + lanes - 1) / lanes, lanes, 256, 256 / lanes};
  }
  const int most = rows >= 2048 && !f32 ? 4 : 2;
  int threads = 1024;
  for (int t : {128, 256, 512, 768}) {
    if ((pieces + t - 1) / t > most) continue;
    threads = t;
    break;
  }
  return RowPlan{(pieces + threads - 1) / threads, 0, threads, 1};
}
constexpr int kMaxGrid = 65536;

template <typename F>
hipError_t with_plan(int rows, int width, bool f32, F launch) {
  const RowPlan pl = plan_rows(rows, width / 8, f32);
  const int groups = (int)(((int64_t)rows + pl.rows - 1) / pl.rows);
  const dim3 grid(groups < kMaxGrid ? groups : kMaxGrid), block(pl.threads);
  switch (pl.c * 100 + pl.lanes) {
    case 116: launch.template operator()<1, 16>(grid, block); break;
    case 132: launch.template operator()<1, 32>(grid, block); break;
#define SPEAR_Q8_ROWS(C, LANES)                                                    \
  case C * 100 + LANES: launch.template operator()<C, LANES>(grid, block); break;
    SPEAR_Q8_ROWS(1, 64) SPEAR_Q8_ROWS(2, 64) SPEAR_Q8_ROWS(3, 64) SPEAR_Q8_ROWS(4, 64)
    SPEAR_Q8_ROWS(2, 0) SPEAR_Q8_ROWS(3, 0) SPEAR_Q8_ROWS(4, 0) SPEAR_Q8_ROWS(5, 0)
    SPEAR_Q8_ROWS(6, 0) SPEAR_Q8_ROWS(7, 0) SPEAR_Q8_ROWS(8, 0)
#undef SPEAR_Q8_ROWS
  }
  return hipGetLastError();
}

struct QuantizeLaunch {
  int rows, width;
  const void* x;
  bool x_f32;
  int64_t stride;
  int8_t* codes;
  float* scales;
  hipStream_t st;
  template <int C, int LANES>
  void operator()(dim3 grid, dim3 block) const {
    if (x_f32)
      hipLaunchKernelGGL((quantize_kernel<C, LANES, true>), grid, block, 0, st, x, stride, codes, scales, rows, width);
    else
      hipLaunchKernelGGL((quantize_kernel<C, LANES, false>), grid, block, 0, st, x, stride, codes, scales, rows,
                         width);
  }
};

// Results that the L2s (32 MB in all) would hold until the kernel's end, and only
// then write, leave it while the kernel runs.  That pays up to about 12 MB for each
// of sum and y, the next read of them included, and in part at 16; past that the next
// read is slower by more.  us, without and with, norm to bf16 alone, norm and a
// quantization of its result, two norms that pass a residual on:
//   512 x 8192 6.1 / 5.4, 11.0 / 10.7, 16.9 / 16.1    1333 x 4096 8.1 / 7.1, 13.1 / 12.4, 20.7 / 20.1
//   1024 x 8192 10.0 / 9.3, 16.4 / 15.9, 26.7 / 27.4  4096 x 8192 28.1 / 24.9, 45.9 / 47.9, 83.6 / 86.4
constexpr int64_t kEarly = 6 << 20;  // elements

struct NormLaunch {
  int rows, width;
  const Q8Norm& a;
  hipStream_t st;
  template <int C, int LANES>
  void operator()(dim3 grid, dim3 block) const {
    if ((int64_t)rows * width <= kEarly)
      hipLaunchKernelGGL((norm_kernel<C, LANES, true>), grid, block, 0, st, a, rows, width);
    else
      hipLaunchKernelGGL((norm_kernel<C, LANES, false>), grid, block, 0, st, a, rows, width);
  }
};

}  // namespace

hipError_t launch_q8_quantize(int rows, int width, const void* x, bool x_f32, int64_t x_stride,
                              int8_t* codes, float* scales, hipStream_t st) {
  return with_plan(rows, width, x_f32, QuantizeLaunch{rows, width, x, x_f32, x_stride, codes, scales, st});
}

hipError_t launch_q8_norm(int rows, int width, const Q8Norm& a, hipStream_t st) {
  return with_plan(rows, width, false, NormLaunch{rows, width, a, st});
}

hipError_t launch_q8_dequant(int rows, int width, const int8_t* codes, const float* scales,
                             float* out, hipStream_t st) {
  int share = 2;  // rows have at least 4 words
  while (share < 8 && (1 << share) < width / 4) ++share;
  const int groups = (int)(((int64_t)rows + (256 >> share) - 1) >> (8 - share));
  const dim3 grid((width / 4 + (1 << share) - 1) >> share, groups < 32768 ? groups : 32768);
  hipLaunchKernelGGL(dequant_kernel, grid, dim3(256), 0, st, codes, scales, out, rows, width, share);
  return hipGetLastError();
}

}  // namespace spear

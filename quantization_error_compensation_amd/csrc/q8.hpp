// The 8-bit path: shapes handed to the kernels and the launchers'
// declarations (q8_api.hip, k_q8_*.hip).
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace spear {

constexpr int kQ8MaxWidth = 65536;
constexpr int kQ8MaxRows = 262144;     // d_out
constexpr int kQ8MaxTokens = 1 << 20;

struct Q8Norm {
  const uint16_t* x;
  int64_t x_stride;
  const uint16_t *residual, *weight;  // residual NULL: nothing is added
  uint16_t *sum, *y;                  // y NULL: not written
  int8_t* codes;                      // NULL: not quantized
  float* scales;
  double eps;
};

struct Q8Shape {
  int K, N, T;
  bool gated, gelu, out_f32;
  int rows() const { return gated ? 2 * N : N; }  // of the weights
};

struct Q8Product {
  const int8_t* xq;
  const float* xs;
  const int8_t* wq;
  const float* ws;
  void* y;
};

hipError_t launch_q8_quantize(int rows, int width, const void* x, bool x_f32, int64_t x_stride,
                              int8_t* codes, float* scales, hipStream_t st);
hipError_t launch_q8_dequant(int rows, int width, const int8_t* codes, const float* scales,
                             float* out, hipStream_t st);
hipError_t launch_q8_norm(int rows, int width, const Q8Norm& a, hipStream_t st);
struct Q8Stream;  // q8_plan.hpp
hipError_t launch_q8_stream(const Q8Shape& s, const Q8Product& a, const Q8Stream& f, hipStream_t st);
// Bytes of workspace of calls of up to s.T tokens, and launch of the product.
size_t q8_product_workspace(const Q8Shape& s);
hipError_t launch_q8_product(const Q8Shape& s, const Q8Product& a, void* workspace, hipStream_t st);

}  // namespace spear

// Products of the 8-bit path: int8 codes on the matrix cores, exact 32-bit
// sums, scales and the gate in the epilogue.
#include "common.hpp"
#include "internal.hpp"
#include "q8_math.hpp"

namespace spear {
namespace {

// One wave per 16 weight rows (of each projection) x 16 tokens.
__global__ __launch_bounds__(64) void product_kernel(Q8Product a, Q8Shape s) {
  const int lane = threadIdx.x, i16 = lane & 15, q = lane >> 4;
  const int n0 = blockIdx.x * 16, t0 = blockIdx.y * 16;
  const int parts = s.gated ? 2 : 1;
  const rsrc_t xr = make_rsrc(a.xq + (size_t)t0 * s.K, (uint32_t)min(16, s.T - t0) * s.K);
  i32x4 acc[2] = {i32x4{0, 0, 0, 0}, i32x4{0, 0, 0, 0}};
  for (int k0 = 0; k0 < s.K; k0 += 64) {
    const int k = k0 + 16 * q;
    const uint32_t off = k < s.K ? (uint32_t)(i16 * s.K + k) : 0x7FFFFFFFu;
    const u32x4 x = bload16(xr, off, 0);
    for (int p = 0; p < parts; ++p) {
      const rsrc_t wr = make_rsrc(a.wq + (size_t)(n0 + p * s.N) * s.K, 16u * s.K);
      acc[p] = mfma16x16x64_i8(bload16(wr, off, 0), x, acc[p]);
    }
  }
  const int t = t0 + i16;
  if (t >= s.T) return;
  const float xs = a.xs[t];
  for (int i = 0; i < 4; ++i) {
    const int n = n0 + 4 * q + i;
    float v = (float)acc[0][i] * xs * a.ws[n];
    if (s.gated) v = gate(s.gelu, v, (float)acc[1][i] * xs * a.ws[n + s.N]);
    if (s.out_f32) static_cast<float*>(a.y)[(size_t)t * s.N + n] = v;
    else static_cast<uint16_t*>(a.y)[(size_t)t * s.N + n] = (uint16_t)f32_to_bf16_rne(v);
  }
}

}  // namespace

size_t q8_product_workspace(const Q8Shape&) { return kCounterSlots * 4; }

hipError_t launch_q8_product(const Q8Shape& s, const Q8Product& a, void*, hipStream_t st) {
  hipLaunchKernelGGL(product_kernel, dim3(s.N / 16, (s.T + 15) / 16), dim3(64), 0, st, a, s);
  return hipGetLastError();
}

}  // namespace spear

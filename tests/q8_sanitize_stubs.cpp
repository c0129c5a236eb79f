// Launch functions of the 8-bit path for a host-only build of its ABI
// (q8_api.hip without the kernel files), used by tests/test_q8_sanitizers.py.
// No check that runs there gets this far.
#include <hip/hip_runtime_api.h>

#include "internal.hpp"
#include "q8.hpp"

namespace spear {
hipError_t launch_q8_quantize(int, int, const void*, bool, int64_t, int8_t*, float*, hipStream_t) {
  return hipErrorNotSupported;
}
hipError_t launch_q8_dequant(int, int, const int8_t*, const float*, float*, hipStream_t) {
  return hipErrorNotSupported;
}
hipError_t launch_q8_norm(int, int, const Q8Norm&, hipStream_t) { return hipErrorNotSupported; }
hipError_t launch_q8_product(const Q8Shape&, const Q8Product&, void*, hipStream_t) {
  return hipErrorNotSupported;
}
size_t q8_product_workspace(const Q8Shape& s) { return 4096 * 4 + (size_t)(s.T < 1024 ? s.T : 1024) * 64; }
}  // namespace spear

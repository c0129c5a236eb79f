// Launch functions of the key/value cache for a host-only build of its ABI
// (kv_api.hip without the kernel files), used by tests/test_kv_sanitizers.py.
// No check that runs there gets this far.
#include <hip/hip_runtime_api.h>

#include "internal.hpp"
#include "kv.hpp"

namespace spear {
hipError_t launch_kv_append(const KvShape&, const KvBatch&, const KvAppendArgs&, hipStream_t) {
  return hipErrorNotSupported;
}
hipError_t launch_kv_dequant(const KvShape&, const KvBatch&, const KvCache&, float*, float*, hipStream_t) {
  return hipErrorNotSupported;
}
hipError_t launch_kv_prefill(const KvShape&, const KvBatch&, const KvAttentionArgs&, void*, hipStream_t) {
  return hipErrorNotSupported;
}
hipError_t launch_kv_decode(const KvShape&, const KvBatch&, const KvAttentionArgs&, void*, hipStream_t) {
  return hipErrorNotSupported;
}
size_t kv_prefill_workspace(const KvShape& s) { return 4096 * 4 + 1024 * (size_t)s.D; }
size_t kv_decode_workspace(const KvShape& s) { return 4096 * 4 + 512 * (size_t)s.D; }
}  // namespace spear

// What the entry-point files share: per-device state, argument checks and the
// driver's TMA descriptor encoder. Defined in abi.cu. Not part of the public ABI.
#pragma once

#include <cudaTypedefs.h>

#include <cstdint>

namespace skv {

struct DeviceInfo {
  uint32_t* status = nullptr;   // the device's status word (kernels OR their bits in)
  int num_sms = 0;
};
// The current device, set up on its first use; MLA_OK or MLA_ERR_NO_DEVICE / MLA_ERR_CUDA.
int current_device(DeviceInfo* out);
// The driver's cuTensorMapEncodeTiled, or null.
PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder();
// The limit of the kernels' pipeline waits (mla_set_wait_limit_ns) and of an aborting CTA's drains.
uint64_t wait_limit_ns();
uint64_t drain_limit_ns();

inline bool ptr_aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

}  // namespace skv

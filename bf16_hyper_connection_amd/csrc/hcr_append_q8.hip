// Append to pages of codes (hcr_append_device.h).

#include "hcr_append_device.h"

namespace hcr {

int launch_append_q8(const AppendArgs& a, void* stream) {
  return a.code.code == HCR_INT8 ? launch_append_of<HCR_INT8>(a, stream) : launch_append_of<HCR_E4M3>(a, stream);
}

}  // namespace hcr

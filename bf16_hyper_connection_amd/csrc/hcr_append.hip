// Append to BF16 pages (hcr_append_device.h).

#include "hcr_append_device.h"

namespace hcr {

int launch_append(const AppendArgs& a, void* stream) {
  return coded(a.code) ? launch_append_q8(a, stream) : launch_append_of<HCR_BF16>(a, stream);
}

}  // namespace hcr

// Attention over pages of int8 codes (hcr_attn_device.h).

#include "hcr_attn_launch.h"

namespace hcr {

int launch_attn_int8(const AttnArgs& a, void* stream) {
  if (a.window.size) return launch_seen<WINDOW, HCR_INT8>(a, stream);
  return a.sel ? launch_seen<LISTED, HCR_INT8>(a, stream) : launch_seen<DENSE, HCR_INT8>(a, stream);
}

}  // namespace hcr

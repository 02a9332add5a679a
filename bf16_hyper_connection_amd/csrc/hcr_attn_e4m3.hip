// Attention over pages of E4M3 codes (hcr_attn_device.h).

#include "hcr_attn_launch.h"

namespace hcr {

int launch_attn_e4m3(const AttnArgs& a, void* stream) {
  if (a.window.size) return launch_seen<WINDOW, HCR_E4M3>(a, stream);
  return a.sel ? launch_seen<LISTED, HCR_E4M3>(a, stream) : launch_seen<DENSE, HCR_E4M3>(a, stream);
}

}  // namespace hcr

// Attention over BF16 pages, all of a sequence's or the listed ones (hcr_attn_device.h).

#include "hcr_attn_launch.h"

namespace hcr {

int launch_attn(const AttnArgs& a, void* stream) {
  if (a.code.code == HCR_INT8) return launch_attn_int8(a, stream);
  if (a.code.code == HCR_E4M3) return launch_attn_e4m3(a, stream);
  if (a.window.size) return launch_attn_window(a, stream);
  return a.sel ? launch_seen<LISTED, HCR_BF16>(a, stream) : launch_seen<DENSE, HCR_BF16>(a, stream);
}

}  // namespace hcr

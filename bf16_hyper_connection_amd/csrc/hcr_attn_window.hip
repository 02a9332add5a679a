// Attention over BF16 pages through a sliding window (hcr_attn_device.h).

#include "hcr_attn_launch.h"

namespace hcr {

int launch_attn_window(const AttnArgs& a, void* stream) { return launch_seen<WINDOW, HCR_BF16>(a, stream); }

}  // namespace hcr

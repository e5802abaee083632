// device_status.h -- where the device status word lives (not part of the
// public ABI).
#pragma once

#include "attn_internal.h"

namespace attn {

// Address of the current device's status word (defined in block_mask.cu).
cudaError_t status_word_address(DeviceStatus** out);

}  // namespace attn

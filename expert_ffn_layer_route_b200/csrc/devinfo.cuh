// Limits of the current device, read once per device (defined in moe_api.cu).
#pragma once

namespace moe {

struct DevInfo {
  int sms = 0, smem_optin = 0, smem_per_sm = 0;
};

DevInfo dev_info();

}  // namespace moe

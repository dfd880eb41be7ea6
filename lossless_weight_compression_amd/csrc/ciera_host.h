// Shared by the host sides of the library.  Not part of the public ABI.
#pragma once
#include <hip/hip_runtime.h>

#include "ciera.h"

namespace ciera {

// Notes the HIP error behind the calling thread's last CIERA_ERR_DEVICE and
// returns that status.
ciera_status_t device_error(const char* what, hipError_t e);

}  // namespace ciera

// Host helpers shared by the library's translation units: device failures and their text, alignment.
#pragma once
#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "cdrge.h"

namespace cdrge {

constexpr size_t kAlign = 256;

inline size_t align_up(size_t x) { return (x + kAlign - 1) / kAlign * kAlign; }

// Notes a failed HIP call for cdrge_last_error_detail (per thread) and returns CDRGE_ERR_DEVICE.
cdrge_status device_error(const char* what, hipError_t e);
// Notes that `who` needs more workspace than it was given and returns CDRGE_ERR_WORKSPACE.
cdrge_status workspace_error(const char* who, size_t need, size_t have);

#define CDRGE_HIP(call)                                          \
  do {                                                           \
    const hipError_t _e = (call);                                \
    if (_e != hipSuccess) return device_error(#call, _e);        \
  } while (0)

}  // namespace cdrge

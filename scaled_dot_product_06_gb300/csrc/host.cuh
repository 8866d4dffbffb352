// Host-side parts that the C entry points share (defined in api.cu).
#pragma once
#include <cudaTypedefs.h>

#include "../../include/sdpa.h"

namespace sdpa {

constexpr float kSoftcapMost = 4096.f;  // see check_softcap

// The driver's tensor-map encoder (looked up once).
sdpa_status_t tensor_map_encoder(PFN_cuTensorMapEncodeTiled_v12000* out);
// The current device's error word (looked up once per device).
sdpa_status_t device_error_word(uint32_t** out);

}  // namespace sdpa

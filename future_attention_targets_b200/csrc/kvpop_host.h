// What the host sides of the C ABI share: error reporting, the device check
// and the debug build's word (defined in kvpop_api.cu).
#pragma once

#include <stdint.h>

#include "kvpop.h"

namespace kvpop {

kvpop_status host_fail(kvpop_status st, const char* message);   // records kvpop_last_error()
kvpop_status host_cuda_fail(int cuda_error, const char* what);
kvpop_status host_device();                                      // the current device is one this library runs on
int32_t* host_debug_word();
// Unique id of the calling thread's current CUDA context, or 0 when none is current or the driver cannot say
// (defined in static_cache.cu).
unsigned long long current_context_id();

}  // namespace kvpop

// What the C-ABI translation units (api.cu, api_paged.cu) share: the
// thread's error message, the device status word, the tensor-map encoder and
// the guard that keeps C++ exceptions inside the library.
#pragma once

#include <cudaTypedefs.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "infllmv2.h"

namespace infllmv2 {

// Records the message of a failed call and returns its code.
int fail(int code, const char* fmt, ...) __attribute__((format(printf, 2, 3)));
int cuda_fail(cudaError_t e, const char* where);

// The driver's tensor-map encoder, or null where it cannot be found.
PFN_cuTensorMapEncodeTiled_v12000 encode_fn();

// Device status word of the current device, or null.
uint32_t* status_ptr();

bool aligned16(const void* p);

}  // namespace infllmv2

#define INFLLMV2_GUARD(...)                                                   \
  try {                                                                       \
    __VA_ARGS__;                                                              \
  } catch (...) {                                                             \
    return INFLLMV2_INVALID_ARGUMENT;                                         \
  }

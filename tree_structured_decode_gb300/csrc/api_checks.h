// What the C ABI's entry points share: errors with their text, alignment, and
// nothing thrown.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>
#include <string>

#include "../../include/tree_attn.h"
#include "plan_state.h"

namespace ta {
namespace api {

inline tree_attn_status fail(tree_attn_status s, const std::string& msg) {
  set_last_error(msg);
  return s;
}
inline tree_attn_status launched(cudaError_t e, const char* what) {
  if (e == cudaSuccess) return TA_OK;
  return fail(TA_ERR_CUDA, std::string(what) + ": " + cudaGetErrorString(e));
}
inline bool off(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) != 0; }

// Nothing is thrown across the ABI.
template <class F>
tree_attn_status guarded(F&& f) {
  try {
    set_last_error("");
    return f();
  } catch (...) {
    return TA_ERR_OOM;
  }
}

// SMs of the current device (152 where there is none).
inline int device_sms() {
  int device = 0, sms = 0;
  if (cudaGetDevice(&device) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, device) != cudaSuccess || sms <= 0)
    return 152;
  return sms;
}

}  // namespace api
}  // namespace ta

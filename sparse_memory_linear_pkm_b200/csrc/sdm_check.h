// Argument checks, error reporting and device facts shared by the entry points
// of libsdm_b200.so (defined in sdm_api.cu; none of this is part of the C ABI).
#pragma once

#include <cuda_runtime.h>

#include <cstdint>
#include <string>

#include "sdm.h"

namespace sdm_host {

// Per-device facts and the device address of the error word.
struct DeviceInfo {
  int sms = 0;
  int max_smem_optin = 0;
  int smem_per_sm = 0;
  unsigned* err = nullptr;
  bool ready = false;
};

// Facts of the current device (looked up once per device).
sdm_status_t device_info(DeviceInfo** out);
// Records msg as the calling thread's last error and returns s.
sdm_status_t fail(sdm_status_t s, const std::string& msg);
// Clears the calling thread's last error; SDM_OK.
sdm_status_t ok();
// SDM_ERR_CUDA (with the launch error named after `what`) if the last launch failed.
sdm_status_t launch_status(const char* what);
// Raises a kernel's dynamic shared-memory limit to at least smem on the current device.
void set_smem(const void* kern, size_t smem);

// dtype is SDM_F32 or SDM_BF16.
sdm_status_t check_dtype(int32_t dtype, const char* name);
// A pointer of a call that is not empty: not NULL, 16-byte aligned.
sdm_status_t need_ptr(const void* p, const char* name, bool nonempty);
// The same for arrays read one element at a time: aligned to the element size.
sdm_status_t need_gate(const void* p, const char* name, bool nonempty, int32_t dtype);
bool aligned16(const void* p);
size_t in_size(int32_t dtype);
size_t align256(size_t x);

// A piece of memory by name, and whether two of them share a byte.
struct Piece {
  const char* name;
  const void* p;
  size_t bytes;
};
inline bool overlap(const Piece& a, const Piece& b) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
  return a.p != nullptr && b.p != nullptr && x < y + b.bytes && y < x + a.bytes;
}
// SDM_ERR_INVALID_ARGUMENT if an output shares a byte with an input or another output.
sdm_status_t check_apart(const Piece* outs, int n_outs, const Piece* ins, int n_ins);

}  // namespace sdm_host

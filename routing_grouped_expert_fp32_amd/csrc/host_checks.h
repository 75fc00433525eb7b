// Host-side checks and launch reporting shared by the C-ABI layers (api.cpp, api_train.cpp): buffer
// ranges, the device check, and the debugging synchronisation. Plain C++ on the HIP runtime API.
#pragma once

#include <hip/hip_runtime_api.h>

#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <mutex>
#include <vector>

#include "../../include/beam_moe.h"

namespace beam {
namespace host {

constexpr int kMaxDevices = 64;

inline size_t al256(size_t b) { return (b + 255) & ~size_t(255); }

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

inline size_t dtype_bytes(int32_t dt) {
  switch (dt) {
    case BEAM_F32: return 4;
    case BEAM_BF16: return 2;
    case BEAM_FP8_E4M3: return 1;
    default: return 0;
  }
}

struct Range {
  uintptr_t lo, hi;
};
inline Range rng(const void* p, size_t bytes) {
  const uintptr_t a = reinterpret_cast<uintptr_t>(p);
  return {a, a + bytes};
}
inline bool overlap(const Range& a, const Range& b) { return a.lo < b.hi && b.lo < a.hi; }

// every output must be disjoint from every input and every other output
inline bool any_alias(const std::vector<Range>& ins, const std::vector<Range>& outs) {
  for (size_t i = 0; i < outs.size(); ++i) {
    if (outs[i].lo == outs[i].hi) continue;
    for (const auto& r : ins)
      if (r.lo != r.hi && overlap(outs[i], r)) return true;
    for (size_t j = i + 1; j < outs.size(); ++j)
      if (outs[j].lo != outs[j].hi && overlap(outs[i], outs[j])) return true;
  }
  return false;
}

inline int g_cus[kMaxDevices];   // compute units per device, cached by check_device

inline beam_status_t check_device() {
  static int arch_ok[kMaxDevices];   // 0 unknown, 1 gfx950, 2 other
  static std::mutex mu;
  int dev = -1;
  if (hipGetDevice(&dev) != hipSuccess || dev < 0 || dev >= kMaxDevices) return BEAM_ERR_DEVICE;
  std::lock_guard<std::mutex> lock(mu);
  if (arch_ok[dev] == 0) {
    hipDeviceProp_t prop;
    if (hipGetDeviceProperties(&prop, dev) != hipSuccess) return BEAM_ERR_DEVICE;
    arch_ok[dev] = std::strncmp(prop.gcnArchName, "gfx950", 6) == 0 ? 1 : 2;
    g_cus[dev] = prop.multiProcessorCount;
  }
  return arch_ok[dev] == 1 ? BEAM_OK : BEAM_ERR_DEVICE;
}

// compute units of the current device (after a successful check_device)
inline int device_cus() {
  int dev = 0;
  if (hipGetDevice(&dev) != hipSuccess || dev < 0 || dev >= kMaxDevices) return 256;
  return g_cus[dev] > 0 ? g_cus[dev] : 256;
}

// BEAM_MOE_SYNC_CHECK set to anything but "0" (read once): every launch is followed by a
// synchronisation of its stream, and a kernel that failed is reported (stderr, naming the stage)
// as BEAM_ERR_LAUNCH from the call that launched it. A debugging aid: it serialises the host with
// the GPU and must not be used under stream capture.
inline bool sync_check() {
  static const bool on = [] {
    const char* v = std::getenv("BEAM_MOE_SYNC_CHECK");
    return v && *v && std::strcmp(v, "0") != 0;
  }();
  return on;
}

inline beam_status_t launched(hipError_t err, hipStream_t st, const char* what) {
  if (err == hipSuccess && sync_check()) err = hipStreamSynchronize(st);
  if (err == hipSuccess) return BEAM_OK;
  std::fprintf(stderr, "beam_moe: %s failed: %s\n", what, hipGetErrorString(err));
  return BEAM_ERR_LAUNCH;
}

}  // namespace host
}  // namespace beam

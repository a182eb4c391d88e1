// The context behind the C ABI, shared by the files that implement its entry points.
#pragma once

#include <vector>

#include "oscar.h"
#include "oscar_internal.h"

struct oscar_ctx {
  oscar_config cfg;
  int num_sms = 0;
  unsigned* d_err = nullptr;
  // per layer: R_K | R_V | R_V^T (3 * 128 * 128 floats), then the bf16
  // three-term splits of R_K^T and R_V^T (6 * 128 * 128 bf16)
  std::vector<float*> d_rot;
  std::vector<float> tau_k, tau_v;
  std::vector<uint32_t> rot_flags;
  std::vector<bool> loaded;
};

namespace oscar {

// Makes the context's device current for a call and puts the caller's back.
struct DeviceGuard {
  int prev = -1;
  explicit DeviceGuard(int dev) {
    if (cudaGetDevice(&prev) != cudaSuccess) prev = -1;
    if (prev != dev)
      cudaSetDevice(dev);
    else
      prev = -1;  // nothing to put back
  }
  ~DeviceGuard() {
    if (prev >= 0) cudaSetDevice(prev);
  }
};

}  // namespace oscar

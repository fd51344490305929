// train_launch.hpp -- internal launch interface of the operators around the linear layers
// (residual norm, gated scan, AdamW) between their argument checks (train_api.hip) and
// their kernels.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "nvfp4.h"

namespace nvfp4 {

// ---------------------------------------------------------------- residual norm
struct NormForward {
  nvfp4_norm_params p;
  nvfp4_norm_forward_args a;
};

struct NormBackward {
  nvfp4_norm_params p;
  nvfp4_norm_backward_args a;
  void *ws;
};

// Bytes of the backward workspace for parameters that passed the checks (rows, cols > 0).
size_t norm_workspace_bytes(const nvfp4_norm_params &p);

hipError_t launch_norm_forward(const NormForward &n, hipStream_t stream);
hipError_t launch_norm_backward(const NormBackward &n, hipStream_t stream);

// ---------------------------------------------------------------- gated scan
struct ScanLaunch {
  nvfp4_scan_args a;
  nvfp4_scan_grads d;   // backward only
  void *ws;
};

// Bytes of the workspace for sizes that passed the checks (all > 0).
size_t scan_workspace_bytes(int64_t batch, int64_t time, int64_t chan, bool backward);

hipError_t launch_scan_forward(const ScanLaunch &s, hipStream_t stream);
hipError_t launch_scan_backward(const ScanLaunch &s, hipStream_t stream);

// ---------------------------------------------------------------- AdamW
// Elements of a tensor that one workgroup updates (a multiple of NVFP4_ADAMW_BLOCK).
constexpr int kAdamChunk = 4096;
// Gradient pointers that travel with a launch, by value: 8 bytes each of the 4 KiB that a
// kernel's arguments may take.
constexpr int kAdamGrads = 440;

struct AdamRow {          // one tensor, in the table
  nvfp4_adamw_tensor t;
  int64_t first_chunk;    // chunks of the tensors before this one
};

struct AdamHeader {       // the table's beginning; AdamRow[count] follows
  uint64_t magic;
  int64_t count, chunks;
  int32_t state_bits, reserved;
};

constexpr uint64_t kAdamMagic = 0x61646177'34706676ull;

struct AdamScalars {
  float beta1, omb1, beta2, omb2;   // beta and 1 - beta, each rounded once from binary64
  float rate, root, eps;            // lr / (1 - beta1^step), 1 / sqrt(1 - beta2^step), eps
  double lr;                        // 1 - lr * weight_decay is formed in binary64
  uint32_t step, k0, k1;            // of the stochastic rounding
  int32_t stochastic_param;
  const float *grad_scale;
};

struct AdamLaunch {
  const AdamHeader *host;           // the host copy, for the launch geometry
  const void *device;               // the device copy
  const void *const *grads;
  AdamScalars s;
};

hipError_t launch_adamw(const AdamLaunch &l, hipStream_t stream);

struct AdamMoments {
  const uint8_t *m, *v;
  const float *ms, *vs;
  int64_t n;
  void *m_out, *v_out;
  int out_f32;
};

hipError_t launch_adamw_moments(const AdamMoments &l, hipStream_t stream);

}  // namespace nvfp4

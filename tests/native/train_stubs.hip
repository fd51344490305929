// train_stubs.hip -- stand-ins for the kernel launchers of the operators around the linear
// layers (test only): linked with their argument checks (train_api.hip) in a host-only build
// under UndefinedBehaviorSanitizer, so that every entry point can be driven on a machine
// without a GPU.  A call that passes the checks is counted here and launches nothing.
#include "train_launch.hpp"

extern "C" {
int stub_calls = 0;
int64_t stub_size = -1;
}

namespace nvfp4 {

static hipError_t record(int64_t size) {
  ++stub_calls;
  stub_size = size;
  return hipErrorNotSupported;
}

size_t norm_workspace_bytes(const nvfp4_norm_params &p) { return 8 * (size_t)p.rows; }
size_t scan_workspace_bytes(int64_t batch, int64_t, int64_t chan, bool) { return 4 * (size_t)(batch * chan); }
hipError_t launch_norm_forward(const NormForward &n, hipStream_t) { return record(n.p.rows); }
hipError_t launch_norm_backward(const NormBackward &n, hipStream_t) { return record(n.p.rows); }
hipError_t launch_scan_forward(const ScanLaunch &s, hipStream_t) { return record(s.a.time); }
hipError_t launch_scan_backward(const ScanLaunch &s, hipStream_t) { return record(s.a.time); }
hipError_t launch_adamw(const AdamLaunch &l, hipStream_t) { return record(l.host->chunks); }
hipError_t launch_adamw_moments(const AdamMoments &l, hipStream_t) { return record(l.n); }

}  // namespace nvfp4

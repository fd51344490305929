// scan.hip -- a gated linear recurrence over time, forward and backward.
//
//   s = sigmoid(g),  a = floor + (1 - floor) s  (0 at a reset),  h_t = a_t h_{t-1} + (1 - a_t) u_t
//
// 1 - a is formed as (1 - floor) sigmoid(-g), without cancellation.  Backward, from the end:
//   G_t = dy_t + a_{t+1} G_{t+1},  du = (1 - a) G,  da = G (h_{t-1} - u)  (0 at a reset),
//   dg = da (1 - floor) s (1 - s),  dfloor = sum da (1 - s),  dh0 = a_1 G_1
//
// Plain kernels: a thread per batch row and channel walks the time steps.
#include "nvfp4_device.hpp"
#include "train_launch.hpp"

namespace nvfp4 {
namespace {

template <bool F32>
__device__ __forceinline__ float load1(const void *p, int64_t i) {
  return F32 ? static_cast<const float *>(p)[i]
             : __uint_as_float((uint32_t) static_cast<const uint16_t *>(p)[i] << 16);
}

template <bool F32>
__device__ __forceinline__ void store1(void *p, int64_t i, float v) {
  if (F32) static_cast<float *>(p)[i] = v;
  else static_cast<uint16_t *>(p)[i] = bf16_bits_rn(v);
}

// sigmoid(g) and sigmoid(-g), each without cancellation: e = exp(-|g|) cannot overflow.
__device__ __forceinline__ void sigmoids(float g, float &s, float &sc) {
  const float e = __expf(-fabsf(g));
  const float r = 1.0f / (1.0f + e);
  s = g >= 0.0f ? r : e * r;
  sc = g >= 0.0f ? e * r : r;
  if (g != g) s = sc = g;
}

template <bool F32>
__global__ __launch_bounds__(64) void scan_forward_kernel(nvfp4_scan_args a) {
  const int64_t i = (int64_t)blockIdx.x * 64 + threadIdx.x;
  if (i >= a.batch * a.chan) return;
  const int64_t b = i / a.chan, c = i % a.chan;
  const float fl = a.floor ? a.floor[c] : 0.0f;
  float h = a.h0 ? a.h0[i] : 0.0f;
  for (int64_t t = 0; t < a.time; ++t) {
    const float g = load1<F32>(a.g, b * a.g_batch + t * a.g_time + c);
    const float u = load1<F32>(a.u, b * a.u_batch + t * a.u_time + c);
    float s, sc;
    sigmoids(g, s, sc);
    if (a.reset && a.reset[b * a.time + t])
      h = u;
    else
      h = (fl + (1.0f - fl) * s) * h + (1.0f - fl) * sc * u;
    store1<F32>(a.y, b * a.y_batch + t * a.y_time + c, h);
  }
  if (a.h_last) a.h_last[i] = h;
}

template <bool F32>
__global__ __launch_bounds__(64) void scan_backward_kernel(ScanLaunch l) {
  const nvfp4_scan_args &a = l.a;
  const nvfp4_scan_grads &d = l.d;
  const int64_t i = (int64_t)blockIdx.x * 64 + threadIdx.x;
  if (i >= a.batch * a.chan) return;
  const int64_t b = i / a.chan, c = i % a.chan;
  const float fl = a.floor ? a.floor[c] : 0.0f;
  float carry = d.dh_last ? d.dh_last[i] : 0.0f, dfl = 0.0f;
  for (int64_t t = a.time - 1; t >= 0; --t) {
    const float g = load1<F32>(a.g, b * a.g_batch + t * a.g_time + c);
    const float u = load1<F32>(a.u, b * a.u_batch + t * a.u_time + c);
    const float h = t > 0 ? load1<F32>(a.y, b * a.y_batch + (t - 1) * a.y_time + c)
                          : a.h0 ? a.h0[i] : 0.0f;
    const float grad = load1<F32>(d.dy, b * d.dy_batch + t * d.dy_time + c) + carry;
    float s, sc, dg = 0.0f, du = grad;
    sigmoids(g, s, sc);
    if (a.reset && a.reset[b * a.time + t]) {
      carry = 0.0f;
    } else {
      const float da = grad * (h - u);
      du = (1.0f - fl) * sc * grad;
      dg = da * ((1.0f - fl) * s * sc);
      dfl += da * sc;
      carry = (fl + (1.0f - fl) * s) * grad;
    }
    store1<F32>(d.du, b * d.du_batch + t * d.du_time + c, du);
    store1<F32>(d.dg, b * d.dg_batch + t * d.dg_time + c, dg);
  }
  if (d.dh0) d.dh0[i] = carry;
  if (d.dfloor) static_cast<float *>(l.ws)[i] = dfl;
}

__global__ __launch_bounds__(64) void scan_floor_kernel(ScanLaunch l) {
  const int64_t c = (int64_t)blockIdx.x * 64 + threadIdx.x;
  if (c >= l.a.chan) return;
  float s = 0.0f;
  if (l.a.time > 0)
    for (int64_t b = 0; b < l.a.batch; ++b) s += static_cast<const float *>(l.ws)[b * l.a.chan + c];
  l.d.dfloor[c] = s;
}

}  // namespace

size_t scan_workspace_bytes(int64_t batch, int64_t time, int64_t chan, bool backward) {
  return backward ? 4 * (size_t)(batch * chan) : 0;
}

hipError_t launch_scan_forward(const ScanLaunch &s, hipStream_t stream) {
  const uint32_t wgs = (uint32_t)((s.a.batch * s.a.chan + 63) / 64);
  if (s.a.dtype == NVFP4_DT_FP32)
    scan_forward_kernel<true><<<wgs, 64, 0, stream>>>(s.a);
  else
    scan_forward_kernel<false><<<wgs, 64, 0, stream>>>(s.a);
  return hipGetLastError();
}

hipError_t launch_scan_backward(const ScanLaunch &s, hipStream_t stream) {
  const uint32_t wgs = (uint32_t)((s.a.batch * s.a.chan + 63) / 64);
  ScanLaunch l = s;
  if (s.a.time == 0) l.ws = nullptr;
  if (wgs) {
    if (s.a.time == 0) l.d.dfloor = nullptr;
    if (s.a.dtype == NVFP4_DT_FP32)
      scan_backward_kernel<true><<<wgs, 64, 0, stream>>>(l);
    else
      scan_backward_kernel<false><<<wgs, 64, 0, stream>>>(l);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  if (s.d.dfloor) {
    scan_floor_kernel<<<(uint32_t)((s.a.chan + 63) / 64), 64, 0, stream>>>(s);
    return hipGetLastError();
  }
  return hipSuccess;
}

}  // namespace nvfp4

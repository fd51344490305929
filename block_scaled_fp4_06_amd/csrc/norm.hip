// norm.hip -- the norm after a block, its gate and the scaled residual sum, and the norm
// before the next block, forward and backward.
//
//   n2 = z rstd_post,  x_out = skip x + branch gate (n2 (c + post)),  h = x_out rstd (c + next)
//
// Backward, with n = x_out rstd, t = dh (c + next), G = branch gate (c + post):
//   D  = dx_out + rstd (t - n mean(t n))          dx = skip D
//   dz = rstd_post (G D - n2 mean(G D n2))
//   dnext = sum_rows dh n,  dpost = sum_rows branch gate D n2,
//   dgate = sum over its rows of branch D n2 (c + post)
//
// Plain kernels: a workgroup per row, a thread per column of the sums over rows.
#include "nvfp4_device.hpp"
#include "train_launch.hpp"

namespace nvfp4 {
namespace {

__device__ __forceinline__ float load1(const void *p, int f32, int64_t i) {
  return f32 ? static_cast<const float *>(p)[i]
             : __uint_as_float((uint32_t) static_cast<const uint16_t *>(p)[i] << 16);
}

__device__ __forceinline__ void store1(void *p, int f32, int64_t i, float v) {
  if (f32) static_cast<float *>(p)[i] = v;
  else static_cast<uint16_t *>(p)[i] = bf16_bits_rn(v);
}

__device__ __forceinline__ float round_to(int f32, float v) {
  return f32 ? v : __uint_as_float((uint32_t)bf16_bits_rn(v) << 16);
}

// Sum over the 256 threads of a workgroup, in every thread.
__device__ float wg_sum(float v) {
  __shared__ float part[4];
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) v += __shfl_xor(v, o, 64);
  __syncthreads();
  if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = v;
  __syncthreads();
  return (part[0] + part[1]) + (part[2] + part[3]);
}

__global__ __launch_bounds__(256) void norm_forward_kernel(NormForward n) {
  const nvfp4_norm_params &p = n.p;
  const nvfp4_norm_forward_args &a = n.a;
  const int64_t row = blockIdx.x;
  const int cols = (int)p.cols;
  float sum = 0.0f;
  if (a.z) {
    for (int c = threadIdx.x; c < cols; c += 256) {
      const float v = load1(a.z, p.z_dtype, row * a.ld_z + c);
      sum += v * v;
    }
    const float rp = 1.0f / sqrtf(wg_sum(sum) / (float)cols + p.eps);
    if (threadIdx.x == 0) a.rstd_post[row] = rp;
    const int64_t grow = row / (p.rows / p.gate_rows);
    sum = 0.0f;
    for (int c = threadIdx.x; c < cols; c += 256) {
      float v = load1(a.z, p.z_dtype, row * a.ld_z + c) * rp *
                (p.weight_offset + load1(a.post_weight, p.weight_dtype, c));
      if (a.gate) v *= load1(a.gate, p.gate_dtype, grow * a.ld_gate + c);
      v = round_to(p.x_dtype, p.skip_scale * load1(a.x, p.x_dtype, row * a.ld_x + c) + p.branch_scale * v);
      store1(a.x_out, p.x_dtype, row * a.ld_x_out + c, v);
      sum += v * v;
    }
  } else {
    for (int c = threadIdx.x; c < cols; c += 256) {
      const float v = load1(a.x, p.x_dtype, row * a.ld_x + c);
      sum += v * v;
    }
  }
  if (!a.next_weight) return;
  const float r = 1.0f / sqrtf(wg_sum(sum) / (float)cols + p.eps);
  if (threadIdx.x == 0) a.rstd[row] = r;
  const void *x = a.z ? a.x_out : a.x;
  const int64_t ld = a.z ? a.ld_x_out : a.ld_x;
  for (int c = threadIdx.x; c < cols; c += 256)
    store1(a.h, p.z_dtype, row * a.ld_h + c,
           load1(x, p.x_dtype, row * ld + c) * r *
               (p.weight_offset + load1(a.next_weight, p.weight_dtype, c)));
}

// The terms of one element of the backward pass.
struct Terms {
  float t, n, d0, n2, g, w;   // d0 = dx_out; g = branch * gate; w = c + post
};

__device__ __forceinline__ Terms terms(const NormBackward &b, int64_t row, int64_t grow, int c,
                                       float r, float rp) {
  const nvfp4_norm_params &p = b.p;
  const nvfp4_norm_backward_args &a = b.a;
  Terms e = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
  if (a.next_weight) {
    e.n = load1(a.x_out, p.x_dtype, row * a.ld_x_out + c) * r;
    e.t = load1(a.dh, p.z_dtype, row * a.ld_dh + c) *
          (p.weight_offset + load1(a.next_weight, p.weight_dtype, c));
  }
  if (a.dx_out) e.d0 = load1(a.dx_out, p.x_dtype, row * a.ld_dx_out + c);
  if (a.z) {
    e.n2 = load1(a.z, p.z_dtype, row * a.ld_z + c) * rp;
    e.w = p.weight_offset + load1(a.post_weight, p.weight_dtype, c);
    e.g = p.branch_scale * (a.gate ? load1(a.gate, p.gate_dtype, grow * a.ld_gate + c) : 1.0f);
  }
  return e;
}

// The two means of a row, into the workspace.
__global__ __launch_bounds__(256) void norm_means_kernel(NormBackward b) {
  const nvfp4_norm_params &p = b.p;
  const int64_t row = blockIdx.x, grow = row / (p.rows / p.gate_rows);
  const int cols = (int)p.cols;
  const float r = b.a.next_weight ? b.a.rstd[row] : 0.0f, rp = b.a.z ? b.a.rstd_post[row] : 0.0f;
  float s = 0.0f;
  for (int c = threadIdx.x; c < cols; c += 256) {
    const Terms e = terms(b, row, grow, c, r, rp);
    s += e.t * e.n;
  }
  const float m1 = wg_sum(s) / (float)cols;
  s = 0.0f;
  for (int c = threadIdx.x; c < cols; c += 256) {
    const Terms e = terms(b, row, grow, c, r, rp);
    s += e.g * e.w * (e.d0 + r * (e.t - e.n * m1)) * e.n2;
  }
  const float m2 = wg_sum(s) / (float)cols;
  if (threadIdx.x == 0) {
    static_cast<float *>(b.ws)[2 * row] = m1;
    static_cast<float *>(b.ws)[2 * row + 1] = m2;
  }
}

__global__ __launch_bounds__(64) void norm_columns_kernel(NormBackward b) {
  const nvfp4_norm_params &p = b.p;
  const nvfp4_norm_backward_args &a = b.a;
  const int c = blockIdx.x * 64 + threadIdx.x;
  if (c >= p.cols) return;
  const float *means = static_cast<const float *>(b.ws);
  const int64_t q = p.rows / p.gate_rows;
  float next = 0.0f, post = 0.0f, gate = 0.0f;
  for (int64_t row = 0; row < p.rows; ++row) {
    const float r = a.next_weight ? a.rstd[row] : 0.0f, rp = a.z ? a.rstd_post[row] : 0.0f;
    const Terms e = terms(b, row, row / q, c, r, rp);
    const float d = e.d0 + r * (e.t - e.n * means[2 * row]);
    if (a.next_weight) next += load1(a.dh, p.z_dtype, row * a.ld_dh + c) * e.n;
    post += e.g * d * e.n2;
    gate += p.branch_scale * d * (e.n2 * e.w);
    if ((row + 1) % q == 0) {
      if (a.dgate) store1(a.dgate, p.gate_dtype, row / q * a.ld_dgate + c, gate);
      gate = 0.0f;
    }
  }
  if (a.dnext_weight) store1(a.dnext_weight, p.weight_dtype, c, next);
  if (a.dpost_weight) store1(a.dpost_weight, p.weight_dtype, c, post);
  if (p.rows == 0 && a.dgate)
    for (int64_t g = 0; g < p.gate_rows; ++g) store1(a.dgate, p.gate_dtype, g * a.ld_dgate + c, 0.0f);
}

__global__ __launch_bounds__(256) void norm_backward_kernel(NormBackward b) {
  const nvfp4_norm_params &p = b.p;
  const nvfp4_norm_backward_args &a = b.a;
  const int64_t row = blockIdx.x, grow = row / (p.rows / p.gate_rows);
  const float r = a.next_weight ? a.rstd[row] : 0.0f, rp = a.z ? a.rstd_post[row] : 0.0f;
  const float m1 = static_cast<const float *>(b.ws)[2 * row], m2 = static_cast<const float *>(b.ws)[2 * row + 1];
  for (int c = threadIdx.x; c < p.cols; c += 256) {
    const Terms e = terms(b, row, grow, c, r, rp);
    const float d = e.d0 + r * (e.t - e.n * m1);
    store1(a.dx, p.x_dtype, row * a.ld_dx + c, a.z ? p.skip_scale * d : d);
    if (a.z) store1(a.dz, p.z_dtype, row * a.ld_dz + c, rp * (e.g * e.w * d - e.n2 * m2));
  }
}

}  // namespace

size_t norm_workspace_bytes(const nvfp4_norm_params &p) { return 8 * (size_t)p.rows; }

hipError_t launch_norm_forward(const NormForward &n, hipStream_t stream) {
  norm_forward_kernel<<<(uint32_t)n.p.rows, 256, 0, stream>>>(n);
  return hipGetLastError();
}

hipError_t launch_norm_backward(const NormBackward &n, hipStream_t stream) {
  hipError_t e = hipSuccess;
  if (n.p.rows > 0) {
    norm_means_kernel<<<(uint32_t)n.p.rows, 256, 0, stream>>>(n);
    if ((e = hipGetLastError()) != hipSuccess) return e;
  }
  if (n.a.dnext_weight || n.a.dpost_weight || n.a.dgate) {
    norm_columns_kernel<<<(uint32_t)((n.p.cols + 63) / 64), 64, 0, stream>>>(n);
    if ((e = hipGetLastError()) != hipSuccess) return e;
  }
  if (n.p.rows > 0) {
    norm_backward_kernel<<<(uint32_t)n.p.rows, 256, 0, stream>>>(n);
    e = hipGetLastError();
  }
  return e;
}

}  // namespace nvfp4

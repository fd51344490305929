// adamw.hip -- one AdamW step over many tensors, moments in 32 or in 8 bits.
//
//   m = beta1 m + (1 - beta1) g        v = beta2 v + (1 - beta2) g^2
//   w = w (1 - lr decay) - rate * m / (sqrt(v) * root + eps)
//
// (rate = lr / (1 - beta1^step), root = 1 / sqrt(1 - beta2^step), formed on the host in
// binary64 and rounded once.)  Everything is binary32, unfused, in the order written, with
// correctly rounded division and square root, so a plain evaluation gives the same bits.
//
// Bound: HBM.  Per element the step reads and writes the weight and both moments and reads
// the gradient once; no value is needed twice.
//
// Work division: a workgroup takes one chunk of kAdamChunk elements of one tensor, found by
// bisection in the table's running chunk counts; the launch covers every chunk of up to
// kAdamGrads tensors, whose gradient pointers travel in the kernel's arguments.
//
// 8-bit moments: a lane holds 8 consecutive elements, half a wave one block of 256; the
// block's two largest magnitudes are maxima over 32 lanes.
#include "nvfp4_device.hpp"
#include "train_launch.hpp"

namespace nvfp4 {
namespace {

// A block's scales: the powers of two that divide its largest magnitude into [2^7, 2^8) for
// the first moment (E4M3 reaches 448) and [2^18, 2^19) for the second's root (code 254 is
// 983040, and rounding up ends at 2^19 at most).
constexpr uint32_t kExpM = 7, kExpR = 18;
constexpr float kTiny = 0x1p-100f;    // blocks below it are held as zero

struct GradPointers {
  const void *p[kAdamGrads];
};

template <int E>
__device__ __forceinline__ void load_values(const void *p, bool f32, bool wide, int64_t i, int cnt,
                                            float (&out)[E]) {
  if (f32) {
    const float *q = static_cast<const float *>(p) + i;
    if (wide && cnt == E) {
#pragma unroll
      for (int j = 0; j < E; j += 4) {
        const float4 v = *reinterpret_cast<const float4 *>(q + j);
        out[j] = v.x; out[j + 1] = v.y; out[j + 2] = v.z; out[j + 3] = v.w;
      }
    } else {
#pragma unroll
      for (int j = 0; j < E; ++j) out[j] = j < cnt ? q[j] : 0.0f;
    }
  } else {
    const uint16_t *q = static_cast<const uint16_t *>(p) + i;
    if (wide && cnt == E) {
#pragma unroll
      for (int j = 0; j < E; j += 4) {
        const uint2 v = *reinterpret_cast<const uint2 *>(q + j);
        out[j] = bf16_lo(v.x); out[j + 1] = bf16_hi(v.x);
        out[j + 2] = bf16_lo(v.y); out[j + 3] = bf16_hi(v.y);
      }
    } else {
#pragma unroll
      for (int j = 0; j < E; ++j) out[j] = j < cnt ? __uint_as_float((uint32_t)q[j] << 16) : 0.0f;
    }
  }
}

template <int E>
__device__ __forceinline__ void store_f32(float *p, bool wide, int64_t i, int cnt,
                                          const float (&v)[E]) {
  float *q = p + i;
  if (wide && cnt == E) {
#pragma unroll
    for (int j = 0; j < E; j += 4)
      *reinterpret_cast<float4 *>(q + j) = make_float4(v[j], v[j + 1], v[j + 2], v[j + 3]);
  } else {
#pragma unroll
    for (int j = 0; j < E; ++j)
      if (j < cnt) q[j] = v[j];
  }
}

template <int E>
__device__ __forceinline__ void store_u16(uint16_t *p, bool wide, int64_t i, int cnt,
                                          const uint16_t (&v)[E]) {
  uint16_t *q = p + i;
  if (wide && cnt == E) {
#pragma unroll
    for (int j = 0; j < E; j += 4)
      *reinterpret_cast<uint2 *>(q + j) = make_uint2((uint32_t)v[j] | ((uint32_t)v[j + 1] << 16),
                                                     (uint32_t)v[j + 2] | ((uint32_t)v[j + 3] << 16));
  } else {
#pragma unroll
    for (int j = 0; j < E; ++j)
      if (j < cnt) q[j] = v[j];
  }
}

__device__ __forceinline__ bool finite_bits(float v) {
  return (__float_as_uint(v) & 0x7FFFFFFFu) < 0x7F800000u;
}

// Largest over the 32 lanes of a half wave.
__device__ __forceinline__ uint32_t half_max(uint32_t v) {
  v = row16_max_u32(v);
  return max(v, (uint32_t)__builtin_amdgcn_ds_swizzle((int)v, 0x401F));  // xor 16
}

// 16-bit draws of elements 8 j .. 8 j + 7 (two per word).
__device__ __forceinline__ Philox4 draws8(int64_t j, const AdamScalars &s, uint32_t tensor,
                                          uint32_t k) {
  return philox4x32_10((uint32_t)j, (uint32_t)(j >> 32), s.step, 2u * tensor + k, s.k0, s.k1);
}

__device__ __forceinline__ uint32_t lane_draw(const Philox4 &d, int j) {
  const uint32_t w = (j >> 1) == 0 ? d.x : (j >> 1) == 1 ? d.y : (j >> 1) == 2 ? d.z : d.w;
  return (j & 1) ? w >> 16 : w & 0xFFFFu;
}

__device__ __forceinline__ float root_decode(uint32_t c) {
  const uint32_t e = c >> 4, f = c & 15u;
  const float v = (float)(e ? (16u + f) << e : 2u * f);
  return c == 255u ? __uint_as_float(0x7FC00000u) : v;
}

// Scale and its inverse for a block whose largest finite magnitude has these bits.
struct BlockScale { float scale, inv; };
__device__ __forceinline__ BlockScale block_scale(uint32_t top, uint32_t exponent) {
  const uint32_t bits = (top & 0x7F800000u) - (exponent << 23);
  const bool live = __uint_as_float(top) >= kTiny;
  return BlockScale{live ? __uint_as_float(bits) : 0.0f,
                    live ? __uint_as_float((254u << 23) - bits) : 0.0f};
}

// Code of t = r / scale in [0, 2^19): below 32 the grid step is 2, so 32 is added and the
// mantissa of the sum counts steps; above, exponent and the four leading mantissa bits are
// the code.  The draw is added to the 19 bits that are dropped.
__device__ __forceinline__ uint32_t root_encode(float t, uint32_t draw) {
  const bool low = t < 32.0f;
  const uint32_t bits = __float_as_uint(low ? t + 32.0f : t);
  const uint32_t c = ((bits - 0x42000000u + 8u * draw + 4u) >> 19) + (low ? 0u : 16u);
  return t > 0.0f ? min(max(c, 1u), 254u) : 0u;
}

template <int BITS>
__global__ __launch_bounds__(256) void adamw_kernel(const uint8_t *__restrict__ table, int t0,
                                                    int t1, int64_t chunk0, AdamScalars s,
                                                    GradPointers grads) {
  constexpr int E = BITS == 8 ? 8 : 4;
  const AdamRow *rows = reinterpret_cast<const AdamRow *>(table + sizeof(AdamHeader));
  const int64_t chunk = chunk0 + blockIdx.x;
  int lo = t0, hi = t1;   // the last tensor whose first chunk is at most `chunk`
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (rows[mid].first_chunk <= chunk) lo = mid; else hi = mid;
  }
  const nvfp4_adamw_tensor &t = rows[lo].t;
  const void *g = grads.p[lo - t0];
  if (!g) return;
  const int64_t n = t.n;
  const bool pf = t.param_dtype == NVFP4_DT_FP32, gf = t.grad_dtype == NVFP4_DT_FP32;
  void *const param = t.param;
  float *const master = t.master;
  const bool pwide = ((uintptr_t)param & 15) == 0, gwide = ((uintptr_t)g & 15) == 0,
             mwide = ((uintptr_t)master & 15) == 0;
  const float keep = (float)(1.0 - s.lr * t.weight_decay);
  const float gs = s.grad_scale ? *s.grad_scale : 1.0f;
  const int64_t begin = (chunk - rows[lo].first_chunk) * kAdamChunk;
  const int64_t end = min(n, begin + kAdamChunk);

  for (int64_t i0 = begin + (threadIdx.x & ~63) * E; i0 < end; i0 += 256 * E) {
    const int64_t i = i0 + (threadIdx.x & 63) * E;
    const int cnt = (int)max((int64_t)0, min((int64_t)E, end - i));
    float gv[E], w[E], m[E], v[E], r[E];
    load_values<E>(g, gf, gwide, i, cnt, gv);
    if (master) load_values<E>(master, true, mwide, i, cnt, w);
    else load_values<E>(param, pf, pwide, i, cnt, w);
    if constexpr (BITS == 32) {
      load_values<E>(t.exp_avg, true, true, i, cnt, m);
      load_values<E>(t.exp_avg_sq, true, true, i, cnt, v);
    } else {
      uint32_t mc[2] = {0u, 0u}, vc[2] = {0u, 0u};
      float ms = 0.0f, vs = 0.0f;
      if (cnt == E) {
        const uint2 a = *reinterpret_cast<const uint2 *>(static_cast<const uint8_t *>(t.exp_avg) + i);
        const uint2 b = *reinterpret_cast<const uint2 *>(static_cast<const uint8_t *>(t.exp_avg_sq) + i);
        mc[0] = a.x; mc[1] = a.y;
        vc[0] = b.x; vc[1] = b.y;
      } else {
#pragma unroll
        for (int j = 0; j < E; ++j)
          if (j < cnt) {
            mc[j >> 2] |= (uint32_t) static_cast<const uint8_t *>(t.exp_avg)[i + j] << (8 * (j & 3));
            vc[j >> 2] |= (uint32_t) static_cast<const uint8_t *>(t.exp_avg_sq)[i + j] << (8 * (j & 3));
          }
      }
      if (cnt > 0) {
        ms = t.exp_avg_scale[i / NVFP4_ADAMW_BLOCK];
        vs = t.exp_avg_sq_scale[i / NVFP4_ADAMW_BLOCK];
      }
#pragma unroll
      for (int j = 0; j < E; ++j) {
        m[j] = e4m3_decode((mc[j >> 2] >> (8 * (j & 3))) & 0xFFu) * ms;
        const float q = root_decode((vc[j >> 2] >> (8 * (j & 3))) & 0xFFu) * vs;
        v[j] = q * q;
      }
    }
#pragma unroll
    for (int j = 0; j < E; ++j) {
      const float gj = s.grad_scale ? gv[j] * gs : gv[j];
      m[j] = s.beta1 * m[j] + s.omb1 * gj;
      v[j] = s.beta2 * v[j] + s.omb2 * (gj * gj);
      r[j] = sqrtf(v[j]);
      w[j] = w[j] * keep - s.rate * (m[j] / (r[j] * s.root + s.eps));
    }
    if (master) store_f32<E>(master, mwide, i, cnt, w);
    if (pf) {
      store_f32<E>(static_cast<float *>(param), pwide, i, cnt, w);
    } else {
      uint16_t b[E];
      if (s.stochastic_param) {
        const Philox4 d = draws8(i >> 3, s, (uint32_t)lo, 1u);
#pragma unroll
        for (int j = 0; j < E; ++j) {
          const uint32_t bits = __float_as_uint(w[j]) + lane_draw(d, (E == 8 ? 0 : (int)(i & 4)) + j);
          b[j] = finite_bits(w[j]) ? (uint16_t)(bits >> 16) : bf16_bits_rn(w[j]);
        }
      } else {
#pragma unroll
        for (int j = 0; j < E; ++j) b[j] = bf16_bits_rn(w[j]);
      }
      store_u16<E>(static_cast<uint16_t *>(param), pwide, i, cnt, b);
    }
    if constexpr (BITS == 32) {
      store_f32<E>(static_cast<float *>(t.exp_avg), true, i, cnt, m);
      store_f32<E>(static_cast<float *>(t.exp_avg_sq), true, i, cnt, v);
    } else {
      uint32_t topm = 0u, topr = 0u;
#pragma unroll
      for (int j = 0; j < E; ++j) {
        if (j < cnt && finite_bits(m[j])) topm = max(topm, __float_as_uint(m[j]) & 0x7FFFFFFFu);
        if (j < cnt && finite_bits(r[j])) topr = max(topr, __float_as_uint(r[j]));
      }
      const BlockScale bm = block_scale(half_max(topm), kExpM), br = block_scale(half_max(topr), kExpR);
      const Philox4 d = draws8(i >> 3, s, (uint32_t)lo, 0u);
      uint32_t mc[2] = {0u, 0u}, vc[2] = {0u, 0u};
#pragma unroll
      for (int j = 0; j < E; ++j) {
        uint32_t c = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(bm.scale > 0.0f ? m[j] * bm.inv : 0.0f, 0.0f, 0, false) & 0xFFu;
        if (!finite_bits(m[j])) c = 0x7Fu;
        mc[j >> 2] |= c << (8 * (j & 3));
        c = root_encode(r[j] * br.inv, lane_draw(d, j));
        if (!finite_bits(r[j])) c = 255u;
        vc[j >> 2] |= c << (8 * (j & 3));
      }
      uint8_t *pm = static_cast<uint8_t *>(t.exp_avg) + i, *pv = static_cast<uint8_t *>(t.exp_avg_sq) + i;
      if (cnt == E) {
        *reinterpret_cast<uint2 *>(pm) = make_uint2(mc[0], mc[1]);
        *reinterpret_cast<uint2 *>(pv) = make_uint2(vc[0], vc[1]);
      } else {
#pragma unroll
        for (int j = 0; j < E; ++j)
          if (j < cnt) {
            pm[j] = (uint8_t)(mc[j >> 2] >> (8 * (j & 3)));
            pv[j] = (uint8_t)(vc[j >> 2] >> (8 * (j & 3)));
          }
      }
      if (cnt > 0 && (threadIdx.x & 31) == 0) {
        t.exp_avg_scale[i / NVFP4_ADAMW_BLOCK] = bm.scale;
        t.exp_avg_sq_scale[i / NVFP4_ADAMW_BLOCK] = br.scale;
      }
    }
  }
}

// One thread per 8 codes of each moment.
template <bool F32>
__global__ __launch_bounds__(256) void moments_kernel(AdamMoments l) {
  const int64_t i = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 8;
  if (i >= l.n) return;
  const int cnt = (int)min((int64_t)8, l.n - i);
  const float ms = l.ms[i / NVFP4_ADAMW_BLOCK], vs = l.vs[i / NVFP4_ADAMW_BLOCK];
  float m[8], v[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    m[j] = j < cnt ? e4m3_decode(l.m[i + j]) * ms : 0.0f;
    const float q = j < cnt ? root_decode(l.v[i + j]) * vs : 0.0f;
    v[j] = q * q;
  }
  if constexpr (F32) {
    store_f32<8>(static_cast<float *>(l.m_out), true, i, cnt, m);
    store_f32<8>(static_cast<float *>(l.v_out), true, i, cnt, v);
  } else {
    uint16_t a[8], b[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      a[j] = bf16_bits_rn(m[j]);
      b[j] = bf16_bits_rn(v[j]);
    }
    store_u16<8>(static_cast<uint16_t *>(l.m_out), true, i, cnt, a);
    store_u16<8>(static_cast<uint16_t *>(l.v_out), true, i, cnt, b);
  }
}

}  // namespace

hipError_t launch_adamw(const AdamLaunch &l, hipStream_t stream) {
  const AdamRow *rows = reinterpret_cast<const AdamRow *>(l.host + 1);
  const int64_t count = l.host->count;
  for (int64_t t0 = 0; t0 < count; t0 += kAdamGrads) {
    const int64_t t1 = t0 + kAdamGrads < count ? t0 + kAdamGrads : count;
    const int64_t c0 = rows[t0].first_chunk;
    const int64_t c1 = t1 < count ? rows[t1].first_chunk : l.host->chunks;
    if (c1 == c0) continue;
    GradPointers g;
    for (int64_t i = 0; i < kAdamGrads; ++i) g.p[i] = t0 + i < t1 ? l.grads[t0 + i] : nullptr;
    const uint8_t *dev = static_cast<const uint8_t *>(l.device);
    if (l.host->state_bits == 8)
      adamw_kernel<8><<<(uint32_t)(c1 - c0), 256, 0, stream>>>(dev, (int)t0, (int)t1, c0, l.s, g);
    else
      adamw_kernel<32><<<(uint32_t)(c1 - c0), 256, 0, stream>>>(dev, (int)t0, (int)t1, c0, l.s, g);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

hipError_t launch_adamw_moments(const AdamMoments &l, hipStream_t stream) {
  const int64_t wgs = (l.n + 2047) / 2048;
  if (l.out_f32)
    moments_kernel<true><<<(uint32_t)wgs, 256, 0, stream>>>(l);
  else
    moments_kernel<false><<<(uint32_t)wgs, 256, 0, stream>>>(l);
  return hipGetLastError();
}

}  // namespace nvfp4

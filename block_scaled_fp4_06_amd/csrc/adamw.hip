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
// Work division: a workgroup takes one chunk of kAdamChunk elements of one tensor, found in
// the table's running chunk counts; the launch covers every chunk of up to
// kAdamGrads tensors, whose gradient pointers travel in the kernel's arguments.  (Chunks of
// 4096: 60 tensors of 9 million elements in all take 31 us, 39 with 16384; 2048 lose 2 % on
// large 8-bit tensors, the 30 small ones below take 5.1, 4.3 and with 16384 11.4 us.)
//
// 8-bit moments: a lane holds 8 consecutive elements, half a wave one block of 256; the
// block's two largest magnitudes are maxima over 32 lanes.
//
// Measured with 104857600 elements: bf16 weights with fp32 masters and moments 500-554 us,
// 5.3-5.9 TB/s (a copy reaches 5.4).  8-bit moments and stochastically rounded
// bf16 weights 253-283 us a step, 3.7-4.2 TB/s: the rounds of Philox and the correctly
// rounded roots and divisions bound it, not memory; both moments decoded to bf16 96 us, 6.6
// TB/s (the codes were just written).  30 tensors of 60001 elements in all: 5.1 us.
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

// 16 bytes at any element's alignment: a packed type makes them one instruction.
struct __attribute__((packed, aligned(2))) Four { uint32_t w[4]; };
struct __attribute__((packed, aligned(2))) Two { uint32_t w[2]; };

// p, known to point to global memory: pointers from a table are otherwise taken for any
// memory's, and accesses then wait for LDS too.
template <class T>
__device__ __forceinline__ T *global(T *p) {
  return (T *)(__attribute__((address_space(1))) T *)(uintptr_t)p;
}

// E consecutive values (4 or 8), all there.
template <bool F32, int E>
__device__ __forceinline__ void load_whole(const void *p, int64_t i, float (&out)[E]) {
  if constexpr (F32) {
#pragma unroll
    for (int j = 0; j < E; j += 4) {
      const Four v = *reinterpret_cast<const Four *>(static_cast<const float *>(p) + i + j);
#pragma unroll
      for (int l = 0; l < 4; ++l) out[j + l] = __uint_as_float(v.w[l]);
    }
  } else if constexpr (E == 8) {
    const Four v = *reinterpret_cast<const Four *>(static_cast<const uint16_t *>(p) + i);
#pragma unroll
    for (int l = 0; l < 4; ++l) {
      out[2 * l] = bf16_lo(v.w[l]);
      out[2 * l + 1] = bf16_hi(v.w[l]);
    }
  } else {
    const Two v = *reinterpret_cast<const Two *>(static_cast<const uint16_t *>(p) + i);
#pragma unroll
    for (int l = 0; l < 2; ++l) {
      out[2 * l] = bf16_lo(v.w[l]);
      out[2 * l + 1] = bf16_hi(v.w[l]);
    }
  }
}

template <bool F32, int E>
__device__ __forceinline__ void load_part(const void *p, int64_t i, int cnt, float (&out)[E]) {
#pragma unroll
  for (int j = 0; j < E; ++j) {
    out[j] = 0.0f;
    if (j >= cnt) continue;
    if constexpr (F32) out[j] = static_cast<const float *>(p)[i + j];
    else out[j] = __uint_as_float((uint32_t) static_cast<const uint16_t *>(p)[i + j] << 16);
  }
}

// WHOLE: all E are there; otherwise the first cnt.
template <bool WHOLE, bool F32, int E>
__device__ __forceinline__ void load_values(const void *p, int64_t i, int cnt, float (&out)[E]) {
  if constexpr (WHOLE) load_whole<F32, E>(p, i, out);
  else load_part<F32, E>(p, i, cnt, out);
}

template <bool WHOLE, int E>
__device__ __forceinline__ void store_f32(float *p, int64_t i, int cnt, const float (&v)[E]) {
  if constexpr (WHOLE) {
#pragma unroll
    for (int j = 0; j < E; j += 4)
      *reinterpret_cast<Four *>(p + i + j) = Four{{__float_as_uint(v[j]), __float_as_uint(v[j + 1]),
                                                   __float_as_uint(v[j + 2]), __float_as_uint(v[j + 3])}};
  } else {
#pragma unroll
    for (int j = 0; j < E; ++j)
      if (j < cnt) p[i + j] = v[j];
  }
}

// w: pairs of 16-bit values.
template <bool WHOLE, int E>
__device__ __forceinline__ void store_u16(uint16_t *p, int64_t i, int cnt, const uint32_t (&w)[E / 2]) {
  if constexpr (WHOLE) {
    if constexpr (E == 8) *reinterpret_cast<Four *>(p + i) = Four{{w[0], w[1], w[2], w[3]}};
    else *reinterpret_cast<Two *>(p + i) = Two{{w[0], w[1]}};
  } else {
#pragma unroll
    for (int j = 0; j < E; ++j)
      if (j < cnt) p[i + j] = (uint16_t)(w[j >> 1] >> (16 * (j & 1)));
  }
}

// Two bf16 values in a word, nearest-even.
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  typedef __bf16 Pair __attribute__((ext_vector_type(2)));
  return __builtin_bit_cast(uint32_t, Pair{(__bf16)lo, (__bf16)hi});
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

// Values of the 256 codes, in LDS: a read there costs the vector units less than forming the
// value (the 8-bit step is bound by their instructions).
__device__ __forceinline__ float root_value(uint32_t c) {
  const uint32_t e = c >> 4, f = c & 15u;
  const float v = (float)(e ? (16u + f) << e : 2u * f);
  return c == 255u ? __uint_as_float(0x7FC00000u) : v;
}

// By 256 threads; a barrier follows.
__device__ __forceinline__ void fill_roots(float *table) {
  table[threadIdx.x] = root_value(threadIdx.x);
  __syncthreads();
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
// the code.  The draw (of 16 bits, plus 1/2) is added to the 19 bits that are dropped.  A root
// above zero has code 1 at least.
__device__ __forceinline__ uint32_t root_encode(float t, uint32_t draw) {
  const bool low = t < 32.0f;
  const uint32_t bits = __float_as_uint(low ? t + 32.0f : t);
  const uint32_t base = low ? 4u - 0x42000000u : 4u - 0x42000000u + (16u << 19);
  const uint32_t c = (bits + (base + (draw << 3))) >> 19;
  return min(max(c, min(__float_as_uint(t), 1u)), 254u);
}

// What a chunk's elements need of their tensor.
struct Chunk {
  const nvfp4_adamw_tensor *t;
  const void *g;
  uint32_t tensor;
  int64_t begin, end;
  float keep, gs;
  const float *roots;   // fill_roots' table (8-bit moments)
};

// E elements per lane from i on.  WHOLE: the wave has all of them; otherwise every access is
// bounded element by element.
template <int BITS, bool PF, bool MASTER, bool GF, bool WHOLE>
__device__ __forceinline__ void update(const Chunk &ch, const AdamScalars &s, int64_t i) {
  constexpr int E = BITS == 8 ? 8 : 4;
  const nvfp4_adamw_tensor &t = *ch.t;
  char *const param = global(static_cast<char *>(t.param));
  char *const exp_avg = global(static_cast<char *>(t.exp_avg)), *const exp_avg_sq = global(static_cast<char *>(t.exp_avg_sq));
  float *const master = global(t.master), *const scale_m = global(t.exp_avg_scale), *const scale_r = global(t.exp_avg_sq_scale);
  const char *const grad = global(static_cast<const char *>(ch.g));
  const int cnt = WHOLE ? E : (int)max((int64_t)0, min((int64_t)E, ch.end - i));
  float g[E], w[E], m[E], v[E], r[E];
  load_values<WHOLE, GF, E>(grad, i, cnt, g);
  if constexpr (MASTER) load_values<WHOLE, true, E>(master, i, cnt, w);
  else load_values<WHOLE, PF, E>(param, i, cnt, w);
  if constexpr (BITS == 32) {
    load_values<WHOLE, true, E>(exp_avg, i, cnt, m);
    load_values<WHOLE, true, E>(exp_avg_sq, i, cnt, v);
  } else {
    const uint8_t *pm = reinterpret_cast<const uint8_t *>(exp_avg) + i, *pv = reinterpret_cast<const uint8_t *>(exp_avg_sq) + i;
    uint32_t mc[2] = {0u, 0u}, vc[2] = {0u, 0u};
    float ms = 0.0f, vs = 0.0f;
    if constexpr (WHOLE) {
      const uint2 a = *reinterpret_cast<const uint2 *>(pm), b = *reinterpret_cast<const uint2 *>(pv);
      mc[0] = a.x; mc[1] = a.y;
      vc[0] = b.x; vc[1] = b.y;
    } else {
#pragma unroll
      for (int j = 0; j < E; ++j)
        if (j < cnt) {
          mc[j >> 2] |= (uint32_t)pm[j] << (8 * (j & 3));
          vc[j >> 2] |= (uint32_t)pv[j] << (8 * (j & 3));
        }
    }
    if (WHOLE || cnt > 0) {
      ms = scale_m[i / NVFP4_ADAMW_BLOCK];
      vs = scale_r[i / NVFP4_ADAMW_BLOCK];
    }
#pragma unroll
    for (int j = 0; j < E; ++j) {
      m[j] = e4m3_decode((mc[j >> 2] >> (8 * (j & 3))) & 0xFFu) * ms;
      const float q = ch.roots[(vc[j >> 2] >> (8 * (j & 3))) & 0xFFu] * vs;
      v[j] = q * q;
    }
  }
#pragma unroll
  for (int j = 0; j < E; ++j) {
    const float gj = s.grad_scale ? g[j] * ch.gs : g[j];
    m[j] = s.beta1 * m[j] + s.omb1 * gj;
    v[j] = s.beta2 * v[j] + s.omb2 * (gj * gj);
    r[j] = sqrtf(v[j]);
    w[j] = w[j] * ch.keep - s.rate * (m[j] / (r[j] * s.root + s.eps));
  }
  if constexpr (MASTER) store_f32<WHOLE, E>(master, i, cnt, w);
  if constexpr (PF) {
    store_f32<WHOLE, E>(reinterpret_cast<float *>(param), i, cnt, w);
  } else {
    uint32_t b[E / 2];
    if (s.stochastic_param) {
      const Philox4 d = draws8(i >> 3, s, ch.tensor, 1u);
      // (E = 4: the lanes of the upper half of eight take the last two words)
      const uint32_t words[4] = {E == 4 && (i & 4) ? d.z : d.x, E == 4 && (i & 4) ? d.w : d.y, d.z, d.w};
#pragma unroll
      for (int j = 0; j < E / 2; ++j) {
        const float a = w[2 * j], c = w[2 * j + 1];
        const uint32_t lo = __float_as_uint(a) + (words[j] & 0xFFFFu), hi = __float_as_uint(c) + (words[j] >> 16);
        b[j] = (lo >> 16) | (hi & 0xFFFF0000u);
        if (!finite_bits(a) || !finite_bits(c)) {   // inf and NaN take no draw
          const uint32_t n = pack2(a, c);
          if (!finite_bits(a)) b[j] = (b[j] & 0xFFFF0000u) | (n & 0xFFFFu);
          if (!finite_bits(c)) b[j] = (b[j] & 0xFFFFu) | (n & 0xFFFF0000u);
        }
      }
    } else {
#pragma unroll
      for (int j = 0; j < E / 2; ++j) b[j] = pack2(w[2 * j], w[2 * j + 1]);
    }
    store_u16<WHOLE, E>(reinterpret_cast<uint16_t *>(param), i, cnt, b);
  }
  if constexpr (BITS == 32) {
    store_f32<WHOLE, E>(reinterpret_cast<float *>(exp_avg), i, cnt, m);
    store_f32<WHOLE, E>(reinterpret_cast<float *>(exp_avg_sq), i, cnt, v);
  } else {
    uint32_t topm = 0u, topr = 0u;
    bool odd = false;   // a moment that is not finite
#pragma unroll
    for (int j = 0; j < E; ++j) {
      if (!WHOLE && j >= cnt) continue;
      const uint32_t am = __float_as_uint(m[j]) & 0x7FFFFFFFu, ar = __float_as_uint(r[j]) & 0x7FFFFFFFu;
      odd |= max(am, ar) >= 0x7F800000u;
      topm = max(topm, am);
      topr = max(topr, ar);
    }
    if (__any(odd)) {   // (they do not enter the block's scale)
      topm = topr = 0u;
#pragma unroll
      for (int j = 0; j < E; ++j) {
        if (!WHOLE && j >= cnt) continue;
        if (finite_bits(m[j])) topm = max(topm, __float_as_uint(m[j]) & 0x7FFFFFFFu);
        if (finite_bits(r[j])) topr = max(topr, __float_as_uint(r[j]));
      }
    }
    const BlockScale bm = block_scale(half_max(topm), kExpM), br = block_scale(half_max(topr), kExpR);
    const bool live = bm.scale > 0.0f;
    const Philox4 d = draws8(i >> 3, s, ch.tensor, 0u);
    uint32_t mc[2] = {0u, 0u}, vc[2] = {0u, 0u};
#pragma unroll
    for (int j = 0; j < E; j += 4) {
      const float a = m[j] * bm.inv, b = m[j + 1] * bm.inv, c = m[j + 2] * bm.inv, e = m[j + 3] * bm.inv;
      uint32_t q = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
      q = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(c, e, (int)q, true);
      mc[j >> 2] = live ? q : 0u;
#pragma unroll
      for (int l = 0; l < 4; ++l) vc[j >> 2] |= root_encode(r[j + l] * br.inv, lane_draw(d, j + l)) << (8 * l);
    }
    if (__any(odd)) {
#pragma unroll
      for (int j = 0; j < E; ++j) {
        const uint32_t byte = 0xFFu << (8 * (j & 3));
        if (!finite_bits(m[j])) mc[j >> 2] = (mc[j >> 2] & ~byte) | (0x7Fu << (8 * (j & 3)));
        if (!finite_bits(r[j])) vc[j >> 2] |= byte;
      }
    }
    uint8_t *pm = reinterpret_cast<uint8_t *>(exp_avg) + i, *pv = reinterpret_cast<uint8_t *>(exp_avg_sq) + i;
    if constexpr (WHOLE) {
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
    if ((WHOLE || cnt > 0) && (threadIdx.x & 31) == 0) {
      scale_m[i / NVFP4_ADAMW_BLOCK] = bm.scale;
      scale_r[i / NVFP4_ADAMW_BLOCK] = br.scale;
    }
  }
}

template <int BITS, bool PF, bool MASTER, bool GF>
__device__ __forceinline__ void update_chunk(const Chunk &c, const AdamScalars &s) {
  constexpr int E = BITS == 8 ? 8 : 4;
  for (int64_t i = c.begin + (threadIdx.x & ~63) * E; i < c.end; i += 256 * E) {
    if (i + 64 * E <= c.end) update<BITS, PF, MASTER, GF, true>(c, s, i + (threadIdx.x & 63) * E);
    else update<BITS, PF, MASTER, GF, false>(c, s, i + (threadIdx.x & 63) * E);
  }
}

template <int BITS, bool PF, bool MASTER>
__device__ __forceinline__ void update_as(const Chunk &c, const AdamScalars &s) {
  if (c.t->grad_dtype == NVFP4_DT_FP32) update_chunk<BITS, PF, MASTER, true>(c, s);
  else update_chunk<BITS, PF, MASTER, false>(c, s);
}

template <int BITS>
__global__ __launch_bounds__(256) void adamw_kernel(const uint8_t *__restrict__ table, int t0, int t1,
                                                    int64_t chunk0, AdamScalars s, GradPointers grads) {
  const AdamRow *rows = reinterpret_cast<const AdamRow *>(table + sizeof(AdamHeader));
  const int64_t chunk = chunk0 + blockIdx.x;
  // the last tensor whose first chunk is at most `chunk`: the lanes of each wave look at 64
  // tensors at a time, all of whose loads are in flight together
  int lo = t0 - 1;
#pragma unroll
  for (int k = 0; k < (kAdamGrads + 63) / 64; ++k) {
    const int t = t0 + 64 * k + ((int)threadIdx.x & 63);
    if (t0 + 64 * k < t1) lo += __popcll(__ballot(t < t1 && rows[min(t, t1 - 1)].first_chunk <= chunk));
  }
  Chunk c;
  __shared__ float roots[BITS == 8 ? 256 : 1];
  if constexpr (BITS == 8) fill_roots(roots);
  c.roots = roots;
  c.t = &rows[lo].t;
  c.g = grads.p[lo - t0];
  if (!c.g) return;
  c.tensor = (uint32_t)lo;
  c.begin = (chunk - rows[lo].first_chunk) * kAdamChunk;
  c.end = min(c.t->n, c.begin + kAdamChunk);
  c.keep = (float)(1.0 - s.lr * c.t->weight_decay);
  c.gs = s.grad_scale ? *s.grad_scale : 1.0f;
  if (c.t->param_dtype == NVFP4_DT_FP32) update_as<BITS, true, false>(c, s);
  else if (c.t->master) update_as<BITS, false, true>(c, s);
  else update_as<BITS, false, false>(c, s);
}

// One thread per 8 codes of each moment (the last thread bounds its accesses).
template <bool F32>
__global__ __launch_bounds__(256) void moments_kernel(AdamMoments l) {
  __shared__ float roots[256];
  fill_roots(roots);
  for (int64_t i = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 8; i < l.n; i += (int64_t)gridDim.x * 2048) {
    const int cnt = (int)min((int64_t)8, l.n - i);
    const float ms = l.ms[i / NVFP4_ADAMW_BLOCK], vs = l.vs[i / NVFP4_ADAMW_BLOCK];
    uint32_t mc[2] = {0u, 0u}, vc[2] = {0u, 0u};
    if (cnt == 8) {
      const uint2 a = *reinterpret_cast<const uint2 *>(l.m + i), b = *reinterpret_cast<const uint2 *>(l.v + i);
      mc[0] = a.x; mc[1] = a.y;
      vc[0] = b.x; vc[1] = b.y;
    } else {
      for (int j = 0; j < cnt; ++j) {
        mc[j >> 2] |= (uint32_t)l.m[i + j] << (8 * (j & 3));
        vc[j >> 2] |= (uint32_t)l.v[i + j] << (8 * (j & 3));
      }
    }
    float m[8], v[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      m[j] = e4m3_decode((mc[j >> 2] >> (8 * (j & 3))) & 0xFFu) * ms;
      const float q = roots[(vc[j >> 2] >> (8 * (j & 3))) & 0xFFu] * vs;
      v[j] = q * q;
    }
    if constexpr (F32) {
      if (cnt == 8) {
        store_f32<true, 8>(static_cast<float *>(l.m_out), i, cnt, m);
        store_f32<true, 8>(static_cast<float *>(l.v_out), i, cnt, v);
      } else {
        store_f32<false, 8>(static_cast<float *>(l.m_out), i, cnt, m);
        store_f32<false, 8>(static_cast<float *>(l.v_out), i, cnt, v);
      }
    } else {
      uint32_t a[4], b[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        a[j] = pack2(m[2 * j], m[2 * j + 1]);
        b[j] = pack2(v[2 * j], v[2 * j + 1]);
      }
      if (cnt == 8) {
        store_u16<true, 8>(static_cast<uint16_t *>(l.m_out), i, cnt, a);
        store_u16<true, 8>(static_cast<uint16_t *>(l.v_out), i, cnt, b);
      } else {
        store_u16<false, 8>(static_cast<uint16_t *>(l.m_out), i, cnt, a);
        store_u16<false, 8>(static_cast<uint16_t *>(l.v_out), i, cnt, b);
      }
    }
  }
}

}  // namespace

constexpr int64_t kMaxGrid = 1 << 23;

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
    // (a grid's threads are counted in 32 bits)
    for (int64_t c = c0; c < c1; c += kMaxGrid) {
      const uint32_t grid = (uint32_t)(c1 - c < kMaxGrid ? c1 - c : kMaxGrid);
      if (l.host->state_bits == 8) adamw_kernel<8><<<grid, 256, 0, stream>>>(dev, (int)t0, (int)t1, c, l.s, g);
      else adamw_kernel<32><<<grid, 256, 0, stream>>>(dev, (int)t0, (int)t1, c, l.s, g);
      const hipError_t e = hipGetLastError();
      if (e != hipSuccess) return e;
    }
  }
  return hipSuccess;
}

hipError_t launch_adamw_moments(const AdamMoments &l, hipStream_t stream) {
  const int64_t need = (l.n + 2047) / 2048, most = 1 << 20;
  const int64_t wgs = need < most ? need : most;
  if (l.out_f32)
    moments_kernel<true><<<(uint32_t)wgs, 256, 0, stream>>>(l);
  else
    moments_kernel<false><<<(uint32_t)wgs, 256, 0, stream>>>(l);
  return hipGetLastError();
}

}  // namespace nvfp4

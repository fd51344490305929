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
// Bound: HBM.  Forward reads x and z and writes x_out and h; backward reads x_out, z, dx_out
// and dh and writes dx and dz: 8 and 12 bytes per element in bf16.  So a row is read once,
// into the registers of the threads that share it, and everything that depends on its
// statistics is formed from there.
//
//  * A row belongs to `waves` waves, V * K elements to a thread (V consecutive ones per
//    load).  Workgroups are persistent: they walk over rows, the next row's loads in flight
//    while the current one is reduced, and the weights stay in registers.
//  * Backward needs three sums over a row, of t x, G z (dx_out + rstd t) and G z x: with
//    them mean(t n) and mean(G D n2) follow from one reduction.
//  * Sums over rows: with s = sum D n2 over the rows that share a gate row, dgate is
//    branch (c + post) s and dpost gathers branch gate s, so a thread keeps s, dnext and
//    dpost for its columns.  Each slot (a range of rows, see split_rows) leaves its sums in
//    the workspace and a second kernel adds the slots in order: no atomics, the same bits
//    every time.
//  * Rows too long for that (over kMaxRow columns) take two passes: the row sums first, then
//    strips of columns that walk down the rows.
//
// Measured at 8192 x 5120 (bf16, fp32 weights, one gate row): forward 67 us, 5.0 TB/s (a
// copy reaches 5.4); backward 115 us, 4.4 TB/s, of which the sums over rows take 5.
// 2048 x 20480, two passes backward: 90 and 211 us.  One row of 5120: 4 us.
#include "norm_rows.hpp"
#include "nvfp4_device.hpp"
#include "train_launch.hpp"

namespace nvfp4 {
namespace {

// ---------------------------------------------------------------- loads and stores
// Every thread works on 8 consecutive elements at a time.  The 16-byte accesses are to
// packed types, so they are single instructions at any element's alignment (rows of odd
// length, views): one path for all strides.  Only a row's last, shorter piece goes element
// by element.
struct __attribute__((packed, aligned(2))) Four { uint32_t w[4]; };

template <bool F32>
struct Raw {              // 8 elements as loaded
  static constexpr int kWords = F32 ? 8 : 4;
  uint32_t w[kWords];

  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < kWords; ++i) w[i] = 0u;
  }
  __device__ __forceinline__ void load(const void *p, int64_t i, int cnt) {
    if (cnt >= 8) {
      const Four *q = reinterpret_cast<const Four *>(static_cast<const char *>(p) + i * (F32 ? 4 : 2));
#pragma unroll
      for (int j = 0; j < kWords / 4; ++j) {
        const Four v = q[j];
#pragma unroll
        for (int l = 0; l < 4; ++l) w[4 * j + l] = v.w[l];
      }
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        if (j >= cnt) continue;
        if constexpr (F32) w[j] = static_cast<const uint32_t *>(p)[i + j];
        else w[j >> 1] |= (uint32_t) static_cast<const uint16_t *>(p)[i + j] << (16 * (j & 1));
      }
    }
  }
  // All eight, without a branch.
  __device__ __forceinline__ void load8(const void *p, int64_t i) {
    const Four *q = reinterpret_cast<const Four *>(static_cast<const char *>(p) + i * (F32 ? 4 : 2));
#pragma unroll
    for (int j = 0; j < kWords / 4; ++j) {
      const Four v = q[j];
#pragma unroll
      for (int l = 0; l < 4; ++l) w[4 * j + l] = v.w[l];
    }
  }
  __device__ __forceinline__ float get(int j) const {
    if constexpr (F32) return __uint_as_float(w[j]);
    else return (j & 1) ? bf16_hi(w[j >> 1]) : bf16_lo(w[j >> 1]);
  }
};

// Two bf16 values in a word, nearest-even.
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  typedef __bf16 Two __attribute__((ext_vector_type(2)));
  return __builtin_bit_cast(uint32_t, Two{(__bf16)lo, (__bf16)hi});
}

// Elements from `own` to cnt - 1 of the 8 at p[i].
template <bool F32>
__device__ __forceinline__ void store(void *p, int64_t i, int cnt, const float (&v)[8], int own = 0) {
  if (own <= 0 && cnt >= 8) {
    Four *q = reinterpret_cast<Four *>(static_cast<char *>(p) + i * (F32 ? 4 : 2));
#pragma unroll
    for (int j = 0; j < (F32 ? 2 : 1); ++j) {
      Four f;
#pragma unroll
      for (int l = 0; l < 4; ++l)
        f.w[l] = F32 ? __float_as_uint(v[4 * j + l]) : pack2(v[2 * l], v[2 * l + 1]);
      q[j] = f;
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      if (j < own || j >= cnt) continue;
      if constexpr (F32) static_cast<float *>(p)[i + j] = v[j];
      else static_cast<uint16_t *>(p)[i + j] = bf16_bits_rn(v[j]);
    }
  }
}

template <bool F32>
__device__ __forceinline__ float rounded(float v) {
  return F32 ? v : __uint_as_float((uint32_t)bf16_bits_rn(v) << 16);
}

// Weights and gates: parameters of either type.
__device__ __forceinline__ void load_param(const void *p, int f32, int64_t i, int cnt, float (&v)[8]) {
  if (f32) {
    Raw<true> r;
    r.zero();
    r.load(p, i, cnt);
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = r.get(j);
  } else {
    Raw<false> r;
    r.zero();
    r.load(p, i, cnt);
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = r.get(j);
  }
}

__device__ __forceinline__ void store_param(void *p, int f32, int64_t i, float v) {
  if (f32) static_cast<float *>(p)[i] = v;
  else static_cast<uint16_t *>(p)[i] = bf16_bits_rn(v);
}

// threadIdx.y of a wave's lanes, which all have the same: the rows that follow from it, and
// their addresses, are then kept once per wave.
__device__ __forceinline__ int wave_y() { return (int)__builtin_amdgcn_readfirstlane(threadIdx.y); }

// ---------------------------------------------------------------- sums over a row
template <int CTRL, int ROWS>
__device__ __forceinline__ float dpp_add(float v) {
  return v + __uint_as_float((uint32_t)__builtin_amdgcn_update_dpp(0, (int)__float_as_uint(v), CTRL,
                                                                   ROWS, 0xF, false));
}

// Sum over the 64 lanes of a wave, in every lane.
__device__ __forceinline__ float wave_sum(float v) {
  v = dpp_add<0xB1, 0xF>(v);    // lane ^ 1
  v = dpp_add<0x4E, 0xF>(v);    // lane ^ 2
  v = dpp_add<0x141, 0xF>(v);   // the other half of 8 lanes
  v = dpp_add<0x140, 0xF>(v);   // the other half of 16
  v = dpp_add<0x142, 0xA>(v);   // rows 1 and 3 add rows 0 and 2
  v = dpp_add<0x143, 0xC>(v);   // rows 2 and 3 add row 1's sum
  return __uint_as_float((uint32_t)__builtin_amdgcn_readlane((int)__float_as_uint(v), 63));
}

// Sums of N values over the waves that share a row.  `part` is used in turns (turn flips): a
// wave writes a half again only after another sum's barrier, which every wave reaches after
// it has read that half.
template <int N>
__device__ __forceinline__ void row_sum(float (&v)[N], float (*part)[16][N], int &turn, int waves) {
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = wave_sum(v[i]);
  if (waves == 1) return;
  const int first = threadIdx.y * waves;
  if ((threadIdx.x & 63) == 0)
#pragma unroll
    for (int i = 0; i < N; ++i) part[turn][first + (threadIdx.x >> 6)][i] = v[i];
  __syncthreads();
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = part[turn][first][i];
  for (int w = 1; w < waves; ++w)
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] += part[turn][first + w][i];
  turn ^= 1;
}

// ---------------------------------------------------------------- columns of a thread
// Where a thread's 8 columns are.  Rows of 8 columns or more: the last threads of a row take
// its last 8 elements, so that no load depends on a branch; their own are the elements
// own .. 7 (none for a thread past the end), and the weights of the others are zero, which
// keeps them out of every sum.  PART (fewer than 8 columns): cnt elements exist.
template <bool PART>
struct Place {
  int col, own, cnt;
  __device__ __forceinline__ Place(int at, int cols) : col(at), own(0), cnt(8) {
    if constexpr (PART) {
      cnt = cols - at;
    } else if (at > cols - 8) {
      own = min(8, at - (cols - 8));
      col = cols - 8;
    }
  }
};

template <bool PART, bool F32>
__device__ __forceinline__ void fetch(const void *p, int64_t i, int cnt, Raw<F32> &r) {
  if constexpr (PART) {
    r.zero();
    r.load(p, i, cnt);
  } else {
    r.load8(p, i);
  }
}

// ---------------------------------------------------------------- forward
// blockDim = (64 waves, rows at a time); rows at a time is 1 unless waves is 1.  A row in
// registers is read once: 67 us at 8192 x 5120, where a second reading from the caches took
// 265.  HOLD: the
// weights (and a gate shared by all rows) stay in registers and the next row is fetched
// ahead; rows of more than 16384 columns leave no registers for either.  THREADS bounds the
// workgroup.
template <bool XF, bool ZF, int K, bool HOLD, int THREADS, bool PART>
__global__ __launch_bounds__(THREADS) void norm_forward_kernel(NormForward n) {
  __shared__ float part[2][16][1];
  const nvfp4_norm_params &p = n.p;
  const nvfp4_norm_forward_args &a = n.a;
  const int cols = (int)p.cols, waves = blockDim.x >> 6, tid = threadIdx.x;
  const int64_t rows = p.rows, step = (int64_t)gridDim.x * blockDim.y;
  const int64_t per_gate = rows / p.gate_rows;
  const bool branch = a.z != nullptr, next = a.next_weight != nullptr;
  const bool one_gate = a.gate && p.gate_rows == 1;
  const float scale = 1.0f / (float)cols;
  int turn = 0;

  int col[K], own[K], cnt[K];
#pragma unroll
  for (int k = 0; k < K; ++k) {
    const Place<PART> at((k * (int)blockDim.x + tid) * 8, cols);
    col[k] = at.col;
    own[k] = at.own;
    cnt[k] = at.cnt;
  }
  // sum of squares of the thread's own elements
  auto squares = [&](int k, float sum, auto &&value) {
    if (own[k] == 0) {
#pragma unroll
      for (int j = 0; j < 8; ++j) sum = __builtin_fmaf(value(j), value(j), sum);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) sum = j < own[k] ? sum : __builtin_fmaf(value(j), value(j), sum);
    }
    return sum;
  };
  // (c + post) branch [gate], and c + next
  float wp[HOLD ? K : 1][8], wn[HOLD ? K : 1][8];
  auto post_of = [&](int k, float (&w)[8]) {
    load_param(a.post_weight, p.weight_dtype, col[k], cnt[k], w);
    float g[8];
    if (one_gate) load_param(a.gate, p.gate_dtype, col[k], cnt[k], g);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      w[j] = p.branch_scale * (p.weight_offset + w[j]);
      if (one_gate) w[j] *= g[j];
    }
  };
  auto next_of = [&](int k, float (&w)[8]) {
    load_param(a.next_weight, p.weight_dtype, col[k], cnt[k], w);
#pragma unroll
    for (int j = 0; j < 8; ++j) w[j] += p.weight_offset;
  };
  if constexpr (HOLD) {
#pragma unroll
    for (int k = 0; k < K; ++k) {
      if (branch) post_of(k, wp[k]);
      if (next) next_of(k, wn[k]);
    }
  }

  Raw<XF> rx[K];
  Raw<ZF> rz[K];
  auto fetch_x_z = [&](int64_t row) {
#pragma unroll
    for (int k = 0; k < K; ++k) {
      rz[k].zero();
      fetch<PART>(a.x, row * a.ld_x + col[k], cnt[k], rx[k]);
      if (branch) fetch<PART>(a.z, row * a.ld_z + col[k], cnt[k], rz[k]);
    }
  };
  int64_t row = (int64_t)blockIdx.x * blockDim.y + wave_y();
  if (HOLD && row < rows) fetch_x_z(row);
  for (; row < rows; row += step) {
    if (!HOLD) fetch_x_z(row);
    float x[K][8];
    Raw<ZF> z[K];
#pragma unroll
    for (int k = 0; k < K; ++k) {
      z[k] = rz[k];
#pragma unroll
      for (int j = 0; j < 8; ++j) x[k][j] = rx[k].get(j);
    }
    if (HOLD && row + step < rows) fetch_x_z(row + step);
    if (branch) {
      float s[1] = {0.0f};
#pragma unroll
      for (int k = 0; k < K; ++k) s[0] = squares(k, s[0], [&](int j) { return z[k].get(j); });
      row_sum<1>(s, part, turn, waves);
      const float rp = 1.0f / sqrtf(s[0] * scale + p.eps);
      if (tid == 0) a.rstd_post[row] = rp;
      const int64_t grow = a.gate && !one_gate ? row / per_gate : 0;
#pragma unroll
      for (int k = 0; k < K; ++k) {
        float w[8], g[8];
        if constexpr (HOLD) {
#pragma unroll
          for (int j = 0; j < 8; ++j) w[j] = wp[k][j];
        } else {
          post_of(k, w);
        }
        if (a.gate && !one_gate) {
          load_param(a.gate, p.gate_dtype, grow * a.ld_gate + col[k], cnt[k], g);
#pragma unroll
          for (int j = 0; j < 8; ++j) w[j] *= g[j];
        }
#pragma unroll
        for (int j = 0; j < 8; ++j)
          x[k][j] = rounded<XF>(__builtin_fmaf(z[k].get(j) * rp, w[j], p.skip_scale * x[k][j]));
        if (own[k] < 8) store<XF>(a.x_out, row * a.ld_x_out + col[k], cnt[k], x[k], own[k]);
      }
    }
    if (!next) continue;
    float s[1] = {0.0f};
#pragma unroll
    for (int k = 0; k < K; ++k) s[0] = squares(k, s[0], [&](int j) { return x[k][j]; });
    row_sum<1>(s, part, turn, waves);
    const float r = 1.0f / sqrtf(s[0] * scale + p.eps);
    if (tid == 0) a.rstd[row] = r;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      float w[8];
      if constexpr (HOLD) {
#pragma unroll
        for (int j = 0; j < 8; ++j) w[j] = wn[k][j];
      } else {
        next_of(k, w);
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) w[j] = x[k][j] * r * w[j];
      if (own[k] < 8) store<ZF>(a.h, row * a.ld_h + col[k], cnt[k], w, own[k]);
    }
  }
}

// ---------------------------------------------------------------- backward
constexpr int kMaxRow = 8192;     // columns of a row that one workgroup holds: 1024 x 8

// What a thread keeps for its columns: c + next; G = branch gate (c + post) of the current
// group; and the sums over rows.
struct Columns {
  float wn[8], g[8];
  float next[8], post[8], s[8];
};

template <bool XF, bool ZF>
struct Operands {         // one row's
  Raw<XF> x, d;
  Raw<ZF> z, h;
  float r, rp;            // rstd and rstd_post
  // Makes the compiler unpack the words again where they are used next, instead of keeping
  // 32 unpacked values across the row's reduction.
  __device__ __forceinline__ void unpack_again() {
#pragma unroll
    for (int i = 0; i < Raw<XF>::kWords; ++i) asm volatile("" : "+v"(x.w[i]), "+v"(d.w[i]));
#pragma unroll
    for (int i = 0; i < Raw<ZF>::kWords; ++i) asm volatile("" : "+v"(z.w[i]), "+v"(h.w[i]));
  }
};

// Workgroups' sums in the workspace: [dnext, dpost, dgate][workgroup][column].
__device__ __forceinline__ float *sums_at(void *ws, const Split &s, int which, int64_t wg, int cols) {
  return static_cast<float *>(ws) + ((int64_t)which * s.sums + wg) * cols;
}

template <bool PART, bool XF, bool ZF>
__device__ __forceinline__ void fetch_row(const nvfp4_norm_backward_args &a, int64_t row,
                                          const Place<PART> &at, Operands<XF, ZF> &o) {
  o.d.zero(); o.z.zero(); o.h.zero();
  o.r = a.next_weight ? a.rstd[row] : 0.0f;
  o.rp = a.z ? a.rstd_post[row] : 0.0f;
  fetch<PART>(a.x_out, row * a.ld_x_out + at.col, at.cnt, o.x);
  if (a.z) fetch<PART>(a.z, row * a.ld_z + at.col, at.cnt, o.z);
  if (a.dx_out) fetch<PART>(a.dx_out, row * a.ld_dx_out + at.col, at.cnt, o.d);
  if (a.next_weight) fetch<PART>(a.dh, row * a.ld_dh + at.col, at.cnt, o.h);
}

// branch gate and c + post of a group (both zero without a branch).
template <bool PART>
__device__ __forceinline__ void gate_and_post(const NormBackward &b, int64_t group, const Place<PART> &at,
                                              float (&g)[8], float (&w)[8]) {
#pragma unroll
  for (int j = 0; j < 8; ++j) g[j] = w[j] = 0.0f;
  if (!b.a.z) return;
  load_param(b.a.post_weight, b.p.weight_dtype, at.col, at.cnt, w);
  if (b.a.gate) load_param(b.a.gate, b.p.gate_dtype, group * b.a.ld_gate + at.col, at.cnt, g);
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    w[j] += b.p.weight_offset;
    g[j] = b.a.gate ? b.p.branch_scale * g[j] : b.p.branch_scale;
  }
}

template <bool PART>
__device__ __forceinline__ void open_group(const NormBackward &b, int64_t group, const Place<PART> &at,
                                           Columns &c) {
  float g[8], w[8];
  gate_and_post(b, group, at, g, w);
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    c.g[j] = j < at.own ? 0.0f : g[j] * w[j];
    c.s[j] = 0.0f;
  }
}

template <bool PART>
__device__ __forceinline__ void open_slot(const NormBackward &b, int64_t group, const Place<PART> &at,
                                          Columns &c) {
#pragma unroll
  for (int j = 0; j < 8; ++j) c.wn[j] = c.next[j] = c.post[j] = 0.0f;
  if (b.a.next_weight) {
    load_param(b.a.next_weight, b.p.weight_dtype, at.col, at.cnt, c.wn);
#pragma unroll
    for (int j = 0; j < 8; ++j) c.wn[j] = j < at.own ? 0.0f : c.wn[j] + b.p.weight_offset;
  }
  open_group(b, group, at, c);
}

// The end of a group: s goes into dpost and, where the group was the slot's alone, the
// gate's gradient (a part of a group leaves its s for close_slots).
template <bool PART>
__device__ __forceinline__ void close_group(const NormBackward &b, const Split &s, int64_t group,
                                            const Place<PART> &at, Columns &c) {
  float g[8], w[8];
  gate_and_post(b, group, at, g, w);
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    c.post[j] += g[j] * c.s[j];
    c.s[j] *= b.p.branch_scale * w[j];
    if (s.parts == 0 && b.a.dgate && j >= at.own && j < at.cnt)
      store_param(b.a.dgate, b.p.gate_dtype, group * b.a.ld_dgate + at.col + j, c.s[j]);
  }
}

// A thread's share of three sums over a row: t x, G z (dx_out + rstd t) and G z x with
// t = dh (c + next); their factors rstd and rstd_post are the row's.
template <bool XF, bool ZF>
__device__ __forceinline__ void partial_sums(const Operands<XF, ZF> &o, const Columns &c, float (&s)[3]) {
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const float x = o.x.get(j), t = o.h.get(j) * c.wn[j], q = c.g[j] * o.z.get(j);
    s[0] = __builtin_fmaf(t, x, s[0]);
    s[1] = __builtin_fmaf(q, __builtin_fmaf(o.r, t, o.d.get(j)), s[1]);
    s[2] = __builtin_fmaf(q, x, s[2]);
  }
}

// The row's means m1 = mean(t n) and m2 = mean(G D n2) from those sums.
__device__ __forceinline__ void means_of(const float (&s)[3], float r, float rp, float scale, float &m1, float &m2) {
  m1 = r * s[0] * scale;
  m2 = rp * (s[1] - r * r * m1 * s[2]) * scale;
}

// dx and dz of one row, and its terms of the sums over rows.
template <bool PART, bool XF, bool ZF>
__device__ __forceinline__ void finish_row(const NormBackward &b, int64_t row, const Operands<XF, ZF> &o,
                                           const Place<PART> &at, float m1, float m2, Columns &c) {
  const float r = o.r, rp = o.rp;
  const float skip = b.a.z ? b.p.skip_scale : 1.0f, k1 = -r * m1, k2 = -rp * m2;
  float dx[8], dz[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const float x = o.x.get(j), dh = o.h.get(j), n2 = o.z.get(j) * rp;
    const float d = __builtin_fmaf(r, __builtin_fmaf(x, k1, dh * c.wn[j]), o.d.get(j));
    c.next[j] = __builtin_fmaf(dh, x * r, c.next[j]);
    c.s[j] = __builtin_fmaf(d, n2, c.s[j]);
    dx[j] = skip * d;
    dz[j] = __builtin_fmaf(c.g[j] * d, rp, n2 * k2);
  }
  if (at.own >= 8) return;
  store<XF>(b.a.dx, row * b.a.ld_dx + at.col, at.cnt, dx, at.own);
  if (b.a.z) store<ZF>(b.a.dz, row * b.a.ld_dz + at.col, at.cnt, dz, at.own);
}

// Walks over `count` rows from `row` on, R at a time (do_rows: the first one's index, which
// of them are before `end`, their operands; the streams of a workgroup take the same number
// of turns), the next R rows' operands in flight, and the groups' ends between them.  ONE:
// all rows are of one group, so nothing but s is kept for dpost and dgate along the way;
// otherwise R is 1.
template <int R, bool ONE, bool PART, bool XF, bool ZF, class Rows>
__device__ __forceinline__ void walk_rows(const NormBackward &b, const Split &sp, int64_t row, int64_t end,
                                          int64_t count, const Place<PART> &at, Columns &c, Rows &&do_rows) {
  static_assert(ONE || R == 1, "groups may end after any row");
  const int64_t per = sp.rows / sp.groups, last = max((int64_t)0, min(end, sp.rows) - 1);
  int64_t group = min(row, last) / per, left = (group + 1) * per - row;   // rows of the group from here on
  open_slot(b, group, at, c);
  Operands<XF, ZF> o[R], ahead[R];
#pragma unroll
  for (int k = 0; k < R; ++k) fetch_row<PART>(b.a, min(row + k, last), at, ahead[k]);
  for (int64_t i = 0; i < count; i += R, row += R) {
    int64_t rows[R];
    bool live[R];
#pragma unroll
    for (int k = 0; k < R; ++k) {
      o[k] = ahead[k];
      rows[k] = min(row + k, last);
      live[k] = row + k < end;
    }
    if (i + R < count)
#pragma unroll
      for (int k = 0; k < R; ++k) fetch_row<PART>(b.a, min(row + R + k, last), at, ahead[k]);
    do_rows(rows, live, o);
    if (!ONE && row < end && (--left == 0 || row + 1 == end)) {
      close_group(b, sp, group, at, c);
      if (row + 1 < end) {
        open_group(b, ++group, at, c);
        left = per;
      }
    }
  }
  if (ONE) close_group(b, sp, group, at, c);
}

// The sums of a workgroup's streams, added in order through LDS, into the workspace.  (A
// stream's s is its share of dgate here, where groups are split.)
template <bool PART>
__device__ __forceinline__ void close_slots(const NormBackward &b, const Split &sp, int64_t wg,
                                            const Place<PART> &at, Columns &c, float *lds) {
  const int cols = (int)b.p.cols, y = threadIdx.y, streams = blockDim.y, tid = threadIdx.x, width = blockDim.x;
#pragma unroll
  for (int what = 0; what < 3; ++what) {
    if (what == 0 ? !b.a.dnext_weight : what == 1 ? !b.a.dpost_weight : !(b.a.dgate && sp.parts)) continue;
    float (&v)[8] = what == 0 ? c.next : what == 1 ? c.post : c.s;
    if (streams > 1) {
      __syncthreads();
      if (y)
#pragma unroll
        for (int j = 0; j < 8; ++j) lds[((y - 1) * 8 + j) * width + tid] = v[j];
      __syncthreads();
      if (y) continue;
      for (int k = 1; k < streams; ++k)
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] += lds[((k - 1) * 8 + j) * width + tid];
    }
    if (at.own < 8) store<true>(sums_at(b.ws, sp, what, wg, cols), at.col, at.cnt, v, at.own);
  }
}

// blockDim = (64 waves, streams): R rows per stream at a time, whose sums share one
// reduction.  THREADS bounds the workgroup: fewer threads leave more registers to each (8192 x
// 5120 in binary32, ten waves: 211 us, 218 with 1024's bounds).
// What keeps it from a copy's rate is a row's way through the reduction with one workgroup
// to a CU; rstd fetched ahead with its row took 8192 x 5120 from 119 to 115 us (16384 x 2560
// from 127 to 110), and registers for a second workgroup spill (247 us).  Two rows at a time
// (one): 8192 x 2560 55 us (57), 16384 x 2560 110.5 (113), 65536 x 256 53.3 (54.3), but 8192 x
// 5120 115.3 (113.5), 16384 x 2048 90.9 (89.5); with 1024 threads they spill, 8192 x 6144 136
// us (287).
template <bool XF, bool ZF, int THREADS, int R, bool ONE, bool PART>
__global__ __launch_bounds__(THREADS) void norm_backward_kernel(NormBackward b, Split sp) {
  __shared__ float part[2][16][3 * R];
  extern __shared__ float lds[];
  const int cols = (int)b.p.cols, waves = blockDim.x >> 6, streams = blockDim.y;
  const int64_t slot = (int64_t)blockIdx.x * streams + wave_y();
  const float scale = 1.0f / (float)cols;
  const Place<PART> at((int)threadIdx.x * 8, cols);
  int turn = 0;
  int64_t row, end, count = 0;
  slot_rows(sp, slot, row, end);
  count = end - row;
  if (waves > 1)   // every stream takes as many turns as the longest: they share barriers
    for (int k = 0; k < streams; ++k) {
      int64_t r0, r1;
      slot_rows(sp, (int64_t)blockIdx.x * streams + k, r0, r1);
      count = max(count, r1 - r0);
    }
  Columns c;
  walk_rows<R, ONE, PART, XF, ZF>(b, sp, row, end, count, at, c,
                                  [&](const int64_t (&rows)[R], const bool (&live)[R], Operands<XF, ZF> (&o)[R]) {
    float s[3 * R];
#pragma unroll
    for (int k = 0; k < R; ++k) {
      float t[3] = {0.0f, 0.0f, 0.0f};
      partial_sums(o[k], c, t);
#pragma unroll
      for (int i = 0; i < 3; ++i) s[3 * k + i] = t[i];
    }
    row_sum<3 * R>(s, part, turn, waves);
#pragma unroll
    for (int k = 0; k < R; ++k) {
      const float t[3] = {s[3 * k], s[3 * k + 1], s[3 * k + 2]};
      float m1, m2;
      means_of(t, o[k].r, o[k].rp, scale, m1, m2);
      o[k].unpack_again();
      if (live[k]) finish_row(b, rows[k], o[k], at, m1, m2, c);
    }
  });
  close_slots(b, sp, blockIdx.x, at, c, lds);
}

// Long rows, first pass: m1 and m2 of every row, a workgroup per row at a time.  (HBM; both
// passes read everything, 20 bytes an element where one pass has 12: 205 us at 2048 x 20480.)
template <bool XF, bool ZF>
__global__ __launch_bounds__(512) void norm_means_kernel(NormBackward b, float *means) {
  __shared__ float part[2][16][3];
  const int cols = (int)b.p.cols, waves = blockDim.x >> 6;
  const int64_t per = b.p.rows / b.p.gate_rows;
  const float scale = 1.0f / (float)cols;
  int turn = 0;
  for (int64_t row = blockIdx.x; row < b.p.rows; row += gridDim.x) {
    float s[3] = {0.0f, 0.0f, 0.0f}, r = 0.0f, rp = 0.0f;
    for (int col = (int)threadIdx.x * 8; col < cols; col += (int)blockDim.x * 8) {
      const Place<false> at(col, cols);
      Operands<XF, ZF> o;
      fetch_row(b.a, row, at, o);
      Columns c;
      open_slot(b, row / per, at, c);
      partial_sums(o, c, s);
      r = o.r;
      rp = o.rp;
    }
    row_sum<3>(s, part, turn, waves);
    if (threadIdx.x == 0) means_of(s, r, rp, scale, means[2 * row], means[2 * row + 1]);
  }
}

// Long rows, second pass: a strip of 2048 columns of one slot's rows per workgroup.
template <bool XF, bool ZF>
__global__ __launch_bounds__(256) void norm_strips_kernel(NormBackward b, Split sp, const float *means,
                                                          int strips) {
  const int64_t slot = blockIdx.x / strips;
  const Place<false> at((int)((blockIdx.x % strips) * 256 + threadIdx.x) * 8, (int)b.p.cols);
  int64_t row, end;
  slot_rows(sp, slot, row, end);
  Columns c;
  walk_rows<1, false, false, XF, ZF>(b, sp, row, end, end - row, at, c,
                                     [&](const int64_t (&rows)[1], const bool (&)[1], Operands<XF, ZF> (&o)[1]) {
    const int64_t i = rows[0];
    finish_row(b, i, o[0], at, means[2 * i], means[2 * i + 1], c);
  });
  close_slots(b, sp, slot, at, c, nullptr);   // (one stream)
}

// The workgroups' sums added in order.  A workgroup has 32 columns of one result, 32 threads
// to a column, each with a consecutive share of the sums: results 0 and 1 are dnext and
// dpost, 2 + g the gate row g.  Where a gate row has few sums (kFew at most), a thread adds
// all of its column's instead, and a workgroup has 32 gate rows: 9 us for 11 gate rows of
// 14880 columns from 11 sums each, 24.7 with 32 threads to a column.  Latency: 4-5 us for 256
// sums of three times 5120 columns.
constexpr int64_t kFew = 32;
__global__ __launch_bounds__(1024) void norm_columns_kernel(NormBackward b, Split sp, int strips) {
  __shared__ float part[32][32];
  const int cols = (int)b.p.cols, lane = threadIdx.x & 31, share = threadIdx.x >> 5;
  const int c = (int)(blockIdx.x % strips) * 32 + lane;
  const int64_t what = blockIdx.x / strips;
  const int64_t per_group = sp.parts / sp.streams;
  if (what >= 2 && per_group <= kFew) {
    const int64_t g = (what - 2) * 32 + share;
    if (g >= sp.groups || c >= cols) return;   // (no barrier follows)
    const float *sums = sums_at(b.ws, sp, 2, g * per_group, cols);
    float v = 0.0f;
#pragma unroll 8
    for (int64_t i = 0; i < per_group; ++i) v += sums[i * cols + c];
    store_param(b.a.dgate, b.p.gate_dtype, g * b.a.ld_dgate + c, v);
    return;
  }
  void *out = what == 0 ? b.a.dnext_weight : what == 1 ? b.a.dpost_weight : b.a.dgate;
  if (!out) return;   // (the whole workgroup)
  const int64_t first = what < 2 ? 0 : (what - 2) * per_group, count = what < 2 ? sp.sums : per_group;
  const float *sums = sums_at(b.ws, sp, what < 2 ? (int)what : 2, first, cols);
  float v = 0.0f;
  if (c < cols) {
    const int64_t end = count * (share + 1) / 32;
#pragma unroll 8
    for (int64_t i = count * share / 32; i < end; ++i) v += sums[i * cols + c];
  }
  part[share][lane] = v;
  __syncthreads();
  if (share || c >= cols) return;
  v = 0.0f;
#pragma unroll
  for (int w = 0; w < 32; ++w) v += part[w][lane];
  if (what < 2) store_param(out, b.p.weight_dtype, c, v);
  else store_param(out, b.p.gate_dtype, (what - 2) * b.a.ld_dgate + c, v);
}

// No rows: every sum over rows is zero.
__global__ __launch_bounds__(256) void norm_zero_kernel(NormBackward b) {
  const int64_t n = b.p.cols;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n * b.p.gate_rows; i += 256 * (int64_t)gridDim.x) {
    if (b.a.dgate) store_param(b.a.dgate, b.p.gate_dtype, i / n * b.a.ld_dgate + i % n, 0.0f);
    if (i < n && b.a.dnext_weight) store_param(b.a.dnext_weight, b.p.weight_dtype, i, 0.0f);
    if (i < n && b.a.dpost_weight) store_param(b.a.dpost_weight, b.p.weight_dtype, i, 0.0f);
  }
}

// ---------------------------------------------------------------- launches
constexpr int kCus = 256;

// Waves that share a row of `cols` columns, `each` to a thread.
int waves_of(int64_t cols, int each) { return (int)((cols + 64 * each - 1) / (64 * each)); }

// Workgroups at a time on a CU of `threads` threads whose kernels use up to 128 registers.
int resident(int threads) { return threads >= 1024 ? 1 : 1024 / threads; }

// Short rows go several to a workgroup of up to 8 waves, so that their sums over rows are
// added there.
Split split_of(const nvfp4_norm_params &p) {
  if (p.cols > kMaxRow) return split_rows(p.rows, p.gate_rows, 1, 128);
  const int waves = waves_of(p.cols, 8), streams = waves <= 8 ? 8 / waves : 1;
  return split_rows(p.rows, p.gate_rows, streams, kCus);
}

template <bool XF, bool ZF, int K, bool HOLD, int THREADS, bool PART = false>
hipError_t run_forward(const NormForward &n, hipStream_t stream) {
  const int waves = waves_of(n.p.cols, 8 * K), y = waves == 1 ? 4 : 1;
  const int64_t want = (n.p.rows + y - 1) / y, most = (int64_t)kCus * 2 * resident(64 * waves * y);
  norm_forward_kernel<XF, ZF, K, HOLD, THREADS, PART>
      <<<(uint32_t)(want < most ? want : most), dim3(64 * waves, y), 0, stream>>>(n);
  return hipGetLastError();
}

template <bool XF, bool ZF>
hipError_t forward_of(const NormForward &n, hipStream_t stream) {
  // as few elements per thread as the workgroup's threads allow; up to 20480 columns, ten
  // waves' bounds, which leave more registers to each thread (2048 rows of 16400 columns 74
  // us, of 20480 90 us, with 1024 threads' bounds 88 and 104)
  const int64_t cols = n.p.cols;
  if (cols < 8) return run_forward<XF, ZF, 1, true, 1024, true>(n, stream);
  if (cols <= 8192) return run_forward<XF, ZF, 1, true, 1024>(n, stream);
  if (cols <= 16384) return run_forward<XF, ZF, 2, true, 1024>(n, stream);
  if (cols <= 20480) return run_forward<XF, ZF, 4, false, 640>(n, stream);
  return run_forward<XF, ZF, 4, false, 1024>(n, stream);
}

template <bool XF, bool ZF>
hipError_t backward_of(const NormBackward &b, const Split &sp, hipStream_t stream) {
  if (b.p.cols <= kMaxRow) {
    const int waves = waves_of(b.p.cols, 8);
    const dim3 block(64 * waves, sp.streams);
    const size_t lds = (size_t)(sp.streams - 1) * 8 * block.x * sizeof(float);
    const uint32_t grid = (uint32_t)sp.sums;
    const bool one = one_group(sp);
    if (b.p.cols < 8) norm_backward_kernel<XF, ZF, 640, 1, false, true><<<grid, block, lds, stream>>>(b, sp);
    else if (waves > 10) norm_backward_kernel<XF, ZF, 1024, 1, false, false><<<grid, block, lds, stream>>>(b, sp);
    else if (one) norm_backward_kernel<XF, ZF, 640, XF || ZF ? 1 : 2, true, false><<<grid, block, lds, stream>>>(b, sp);
    else norm_backward_kernel<XF, ZF, 640, 1, false, false><<<grid, block, lds, stream>>>(b, sp);
    return hipGetLastError();
  }
  float *means = static_cast<float *>(b.ws) + 3 * sp.sums * b.p.cols;
  const int64_t wgs = b.p.rows < 4 * kCus ? b.p.rows : 4 * kCus;
  norm_means_kernel<XF, ZF><<<(uint32_t)wgs, 512, 0, stream>>>(b, means);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  const int strips = (int)((b.p.cols + 2047) / 2048);
  norm_strips_kernel<XF, ZF><<<(uint32_t)(sp.slots * strips), 256, 0, stream>>>(b, sp, means, strips);
  return hipGetLastError();
}

}  // namespace

size_t norm_workspace_bytes(const nvfp4_norm_params &p) {
  const Split s = split_of(p);
  return 4 * (3 * (size_t)s.sums * (size_t)p.cols + (p.cols > kMaxRow ? 2 * (size_t)p.rows : 0));
}

hipError_t launch_norm_forward(const NormForward &n, hipStream_t stream) {
  if (n.p.x_dtype == NVFP4_DT_BF16) return forward_of<false, false>(n, stream);
  return n.p.z_dtype == NVFP4_DT_BF16 ? forward_of<true, false>(n, stream) : forward_of<true, true>(n, stream);
}

hipError_t launch_norm_backward(const NormBackward &b, hipStream_t stream) {
  const bool sums = b.a.dnext_weight || b.a.dpost_weight || b.a.dgate;
  if (b.p.rows == 0) {
    if (sums) norm_zero_kernel<<<64, 256, 0, stream>>>(b);
    return hipGetLastError();
  }
  const Split sp = split_of(b.p);
  const hipError_t e = b.p.x_dtype == NVFP4_DT_BF16   ? backward_of<false, false>(b, sp, stream)
                       : b.p.z_dtype == NVFP4_DT_BF16 ? backward_of<true, false>(b, sp, stream)
                                                      : backward_of<true, true>(b, sp, stream);
  if (e != hipSuccess || !sums) return e;
  const int strips = (int)((b.p.cols + 31) / 32);
  const int64_t gates = b.a.dgate && sp.parts ? sp.groups : 0;
  const int64_t results = 2 + (sp.parts / sp.streams <= kFew ? (gates + 31) / 32 : gates);
  norm_columns_kernel<<<(uint32_t)(results * strips), 1024, 0, stream>>>(b, sp, strips);
  return hipGetLastError();
}

}  // namespace nvfp4

// scan.hip -- a gated linear recurrence over time, forward and backward.
//
//   s = sigmoid(g),  a = floor + (1 - floor) s  (0 at a reset),  h_t = a_t h_{t-1} + (1 - a_t) u_t
//
// 1 - a is formed as (1 - floor) sigmoid(-g), without cancellation.  Backward, from the end,
// with c_t = a_t G_t carried towards the beginning:
//   G_t = dy_t + c_{t+1},  du = (1 - a) G,  da = G (h_{t-1} - u)  (0 at a reset),
//   dg = da (1 - floor) s (1 - s),  dfloor = sum da (1 - s),  dh0 = c_1
//
// Bound: HBM.  Forward reads g and u and writes y, 6 bytes per element in bf16; backward
// reads dy, g, u, y and writes dg and du, 12 bytes.  One pass over the data:
//
//  * A tile is 128 bytes of channels (8 lanes of 16 bytes) by kGroups x S time steps: each of
//    256 threads holds S consecutive steps of its channels in registers.  A run of steps acts
//    on the state as h -> A h + B; the threads' (A, B) are composed through LDS, and the tile
//    needs one state per channel from the tile before it.
//  * That state comes over a chain of tiles.  A tile publishes its own (A, B) as soon as it
//    has it, and its final state once it knows its first.  A tile that waits reads its last
//    kWindow predecessors at once, takes the nearest final state and applies the (A, B) of
//    the tiles since in order: h_j = A_j h_{j-1} + B_j whoever computes it, so the result does
//    not depend on timing.
//  * Workgroups take tiles from a counter, time-major, and wait only for tiles with a
//    smaller number, which another workgroup is working on already: some workgroup can
//    always go on, however many of them are resident.
//  * A reset is a cut, not a product with zero: (cut, B) composed with anything before it is
//    (cut, B), so inf and NaN end there.  A cut is held as A = -0.0, which no product of the
//    other factors (in [0, 1], or NaN) gives.
//
// Few steps (up to kShort) need no tiles: a thread walks over them.
#include "nvfp4_device.hpp"
#include "train_launch.hpp"

namespace nvfp4 {
namespace {

constexpr int kGroups = 32;          // time groups of a tile: 256 threads / 8 lanes of channels
constexpr int kSteps = 4;            // steps of a thread
constexpr int kTile = kGroups * kSteps;
constexpr int kWindow = 8;           // predecessors read at once
constexpr int kShort = 16;           // steps that one thread walks over by itself
constexpr uint64_t kWaitTicks = 500000000ull;   // last resort: 5 s of the 100 MHz clock

// ---------------------------------------------------------------- loads and stores
// 16 bytes of channels, at any element's alignment (the packed type makes them single
// instructions); `cnt` of them exist.
struct __attribute__((packed, aligned(2))) Four { uint32_t w[4]; };

template <bool F32>
struct Raw {
  static constexpr int V = F32 ? 4 : 8;
  uint32_t w[4];

  __device__ __forceinline__ void zero() { w[0] = w[1] = w[2] = w[3] = 0u; }
  __device__ __forceinline__ void load(const void *p, int64_t i, int cnt) {
    if (cnt >= V) {
      const Four v = *reinterpret_cast<const Four *>(static_cast<const char *>(p) + i * (F32 ? 4 : 2));
#pragma unroll
      for (int l = 0; l < 4; ++l) w[l] = v.w[l];
    } else {
#pragma unroll
      for (int j = 0; j < V; ++j) {
        if (j >= cnt) continue;
        if constexpr (F32) w[j] = static_cast<const uint32_t *>(p)[i + j];
        else w[j >> 1] |= (uint32_t) static_cast<const uint16_t *>(p)[i + j] << (16 * (j & 1));
      }
    }
  }
  __device__ __forceinline__ float get(int j) const {
    if constexpr (F32) return __uint_as_float(w[j]);
    else return (j & 1) ? bf16_hi(w[j >> 1]) : bf16_lo(w[j >> 1]);
  }
};

template <bool F32>
__device__ __forceinline__ void store(void *p, int64_t i, int cnt, const float (&v)[F32 ? 4 : 8]) {
  if (cnt >= (F32 ? 4 : 8)) {
    Four f;
#pragma unroll
    for (int l = 0; l < 4; ++l) {
      if constexpr (F32) f.w[l] = __float_as_uint(v[l]);
      else f.w[l] = (uint32_t)bf16_bits_rn(v[2 * l]) | ((uint32_t)bf16_bits_rn(v[2 * l + 1]) << 16);
    }
    *reinterpret_cast<Four *>(static_cast<char *>(p) + i * (F32 ? 4 : 2)) = f;
  } else {
#pragma unroll
    for (int j = 0; j < (F32 ? 4 : 8); ++j) {
      if (j >= cnt) continue;
      if constexpr (F32) static_cast<float *>(p)[i + j] = v[j];
      else static_cast<uint16_t *>(p)[i + j] = bf16_bits_rn(v[j]);
    }
  }
}

// V binary32 values (floor, states); zero where there are none.
template <int V>
__device__ __forceinline__ void load_f32(const float *p, int64_t i, int cnt, float (&v)[V]) {
#pragma unroll
  for (int j = 0; j < V; ++j) v[j] = p && j < cnt ? p[i + j] : 0.0f;
}

// ---------------------------------------------------------------- arithmetic
// sigmoid(g) and sigmoid(-g), each without cancellation: e = exp(-|g|) cannot overflow.
__device__ __forceinline__ void sigmoids(float g, float &s, float &sc) {
  const float e = __expf(-fabsf(g));
  const float r = __builtin_amdgcn_rcpf(1.0f + e), er = e * r;
  s = g >= 0.0f ? r : er;
  sc = g >= 0.0f ? er : r;
}

__device__ __forceinline__ float cut_mark() { return -0.0f; }
__device__ __forceinline__ bool is_cut(float a) { return __float_as_uint(a) == 0x80000000u; }

struct Pair { float a, b; };   // h -> a h + b, or h -> b behind a cut

__device__ __forceinline__ float apply(const Pair &p, float h) { return is_cut(p.a) ? p.b : __builtin_fmaf(p.a, h, p.b); }

// First p, then q.
__device__ __forceinline__ Pair then(const Pair &p, const Pair &q) {
  if (is_cut(q.a)) return q;
  return Pair{is_cut(p.a) ? p.a : q.a * p.a, __builtin_fmaf(q.a, p.b, q.b)};
}

// ---------------------------------------------------------------- the chain of tiles
// Words that have not been published are all ones; a published value that happens to be
// (a NaN) is replaced by another NaN.
struct Chain {
  uint32_t *ticket;
  uint64_t *pairs;      // [strip][chunk][channel]
  uint32_t *states;     // [strip][chunk][channel]
  int64_t strips, chunks, tiles, chan_strips;
};

constexpr uint64_t kNoPair = ~0ull;
constexpr uint32_t kNoState = ~0u;

__device__ __forceinline__ void publish(uint64_t *at, const Pair &p) {
  uint64_t w = ((uint64_t)__float_as_uint(p.b) << 32) | __float_as_uint(p.a);
  if (w == kNoPair) w = (0x7FC00000ull << 32) | 0x7FC00000ull;
  __hip_atomic_store(at, w, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

__device__ __forceinline__ void publish(uint32_t *at, float h) {
  uint32_t w = __float_as_uint(h);
  if (w == kNoState) w = 0x7FC00000u;
  __hip_atomic_store(at, w, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

// The state before chunk j (> 0) of a strip, in each lane for its channel; the lanes without
// one (live false) only take part in the votes.  Called by one whole wave.
template <int CH>
__device__ __forceinline__ float state_before(const Chain &c, int64_t strip, int64_t j, int ch, bool live) {
  const int64_t base = strip * c.chunks * CH + ch;
  const uint64_t start = wall_clock64();
  for (;;) {
    uint32_t st[kWindow];
    uint64_t pr[kWindow];
#pragma unroll
    for (int w = 0; w < kWindow; ++w) {
      st[w] = 0u;
      pr[w] = 0ull;
      const int64_t k = j - 1 - w;
      if (!live || k < 0) continue;
      st[w] = __hip_atomic_load(c.states + base + k * CH, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      pr[w] = __hip_atomic_load(c.pairs + base + k * CH, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
    int found = -1;
    bool open = true;   // every pair since is there
#pragma unroll
    for (int w = 0; w < kWindow; ++w) {
      if (found >= 0 || !open || j - 1 - w < 0) continue;
      if (__all(st[w] != kNoState)) found = w;
      else open = __all(pr[w] != kNoPair);
    }
    if (found >= 0) {
      float h = 0.0f;
#pragma unroll
      for (int w = kWindow - 1; w >= 0; --w) {
        if (w == found) h = __uint_as_float(st[w]);
        else if (w < found)
          h = apply(Pair{__uint_as_float((uint32_t)pr[w]), __uint_as_float((uint32_t)(pr[w] >> 32))}, h);
      }
      return h;
    }
    if (wall_clock64() - start > kWaitTicks) return __uint_as_float(0x7FC00000u);
    __builtin_amdgcn_s_sleep(1);
  }
}

// Clears the chain's words before a launch that uses them.
__global__ __launch_bounds__(256) void scan_clear_kernel(uint4 *p, int64_t n, uint32_t *ticket) {
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256)
    p[i] = make_uint4(~0u, ~0u, ~0u, ~0u);
  if (blockIdx.x == 0 && threadIdx.x == 0) *ticket = 0u;
}

// What the threads of a tile share.
template <int CH>
struct Shared {
  static constexpr int kSegs = 256 / CH, kPer = kGroups / kSegs;   // segments of time groups
  Pair group[kGroups][CH];     // a group's pair, then that of its segment's groups before it
  Pair seg[kSegs][CH];
  float first[kSegs][CH];      // the state before a segment
  uint32_t tile;
};

// From every thread's pair (for its V channels) to the state before its steps.  Two barriers
// between the pairs and the wait for the chain, one after it.
template <int V, int CH>
__device__ __forceinline__ void states_of_groups(Shared<CH> &sh, const Chain &c, int64_t strip, int64_t j,
                                                 int64_t c0, int64_t chan, const float *h0,
                                                 float *h_last, const Pair (&p)[V], float (&h)[V]) {
  const int tid = threadIdx.x, group = tid >> 3, lane = tid & 7;
#pragma unroll
  for (int i = 0; i < V; ++i) sh.group[group][lane * V + i] = p[i];
  __syncthreads();
  const int ch = tid % CH, seg = tid / CH;
  {
    Pair run = {1.0f, 0.0f};
#pragma unroll
    for (int i = 0; i < Shared<CH>::kPer; ++i) {
      const Pair q = sh.group[seg * Shared<CH>::kPer + i][ch];
      sh.group[seg * Shared<CH>::kPer + i][ch] = run;
      run = then(run, q);
    }
    sh.seg[seg][ch] = run;
  }
  __syncthreads();
  if (tid < 64) {
    const bool live = tid < CH && c0 + ch < chan;
    Pair all = sh.seg[0][ch];
#pragma unroll
    for (int s = 1; s < Shared<CH>::kSegs; ++s) all = then(all, sh.seg[s][ch]);
    const int64_t at = (strip * c.chunks + j) * CH + ch;
    float before = 0.0f;
    if (j == 0) {
      if (h0 && live) before = h0[strip / c.chan_strips * chan + c0 + ch];
    } else {
      if (live && j + 1 < c.chunks) publish(c.pairs + at, all);
      before = state_before<CH>(c, strip, j, ch, live);
    }
    const float after = apply(all, before);
    if (live) {
      if (j + 1 < c.chunks) publish(c.states + at, after);
      else if (h_last) h_last[strip / c.chan_strips * chan + c0 + ch] = after;
    }
    if (tid < CH) {
#pragma unroll
      for (int s = 0; s < Shared<CH>::kSegs; ++s) {
        sh.first[s][ch] = before;
        before = apply(sh.seg[s][ch], before);
      }
    }
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < V; ++i)
    h[i] = apply(sh.group[group][lane * V + i], sh.first[group / Shared<CH>::kPer][lane * V + i]);
}

// The next tile of this workgroup: from the counter, or in strides where no tile waits.
template <int CH>
__device__ __forceinline__ int64_t next_tile(Shared<CH> &sh, const Chain &c, int64_t turn) {
  if (c.chunks == 1) return (int64_t)blockIdx.x + turn * gridDim.x;
  __syncthreads();   // the tile before is done with the shared words
  if (threadIdx.x == 0)
    sh.tile = __hip_atomic_fetch_add(c.ticket, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  __syncthreads();
  return sh.tile;
}

// ---------------------------------------------------------------- forward
template <bool F32, bool RESET>
__global__ __launch_bounds__(256) void scan_forward_kernel(nvfp4_scan_args a, Chain c) {
  constexpr int V = Raw<F32>::V, CH = 8 * V;
  __shared__ Shared<CH> sh;
  const int group = threadIdx.x >> 3, lane = threadIdx.x & 7;
  for (int64_t turn = 0;; ++turn) {
    const int64_t tile = next_tile(sh, c, turn);
    if (tile >= c.tiles) return;
    const int64_t strip = tile % c.strips, j = tile / c.strips;
    const int64_t batch = strip / c.chan_strips, c0 = strip % c.chan_strips * CH, col = c0 + lane * V;
    const int cnt = (int)min((int64_t)V, max((int64_t)0, a.chan - col));
    const int64_t t0 = j * kTile + group * kSteps;
    Raw<F32> g[kSteps], u[kSteps];
#pragma unroll
    for (int s = 0; s < kSteps; ++s) {
      g[s].zero();
      u[s].zero();
      if (t0 + s >= a.time) continue;
      g[s].load(a.g, batch * a.g_batch + (t0 + s) * a.g_time + col, cnt);
      u[s].load(a.u, batch * a.u_batch + (t0 + s) * a.u_time + col, cnt);
    }
    float fl[V];
    load_f32<V>(a.floor, col, cnt, fl);
    float av[kSteps][V], bv[kSteps][V];
    Pair p[V];
#pragma unroll
    for (int i = 0; i < V; ++i) p[i] = Pair{1.0f, 0.0f};
#pragma unroll
    for (int s = 0; s < kSteps; ++s) {
      const bool in = t0 + s < a.time;
      const bool cut = RESET && in && a.reset[batch * a.time + t0 + s];
#pragma unroll
      for (int i = 0; i < V; ++i) {
        float sg, sc;
        sigmoids(g[s].get(i), sg, sc);
        const float uv = u[s].get(i), rest = 1.0f - fl[i];
        float x = __builtin_fmaf(rest, sg, fl[i]), y = rest * sc * uv;
        if (RESET && cut) {
          x = cut_mark();
          y = uv;
        }
        if (!in) {        // past the end: the state stays
          x = 1.0f;
          y = 0.0f;
        }
        av[s][i] = x;
        bv[s][i] = y;
        p[i] = RESET ? then(p[i], Pair{x, y}) : Pair{x * p[i].a, __builtin_fmaf(x, p[i].b, y)};
      }
    }
    float h[V];
    states_of_groups<V, CH>(sh, c, strip, j, c0, a.chan, a.h0, a.h_last, p, h);
#pragma unroll
    for (int s = 0; s < kSteps; ++s) {
      if (t0 + s >= a.time) break;
#pragma unroll
      for (int i = 0; i < V; ++i)
        h[i] = RESET ? apply(Pair{av[s][i], bv[s][i]}, h[i]) : __builtin_fmaf(av[s][i], h[i], bv[s][i]);
      store<F32>(a.y, batch * a.y_batch + (t0 + s) * a.y_time + col, cnt, h);
    }
    if (c.chunks == 1) __syncthreads();   // before the next tile writes the shared words
  }
}

// A thread per V channels walks over the steps.
template <bool F32>
__global__ __launch_bounds__(64) void scan_forward_short_kernel(nvfp4_scan_args a, int64_t threads) {
  constexpr int V = Raw<F32>::V;
  const int64_t per = (a.chan + V - 1) / V;
  for (int64_t i = (int64_t)blockIdx.x * 64 + threadIdx.x; i < threads; i += (int64_t)gridDim.x * 64) {
    const int64_t b = i / per, col = i % per * V;
    const int cnt = (int)min((int64_t)V, a.chan - col);
    float fl[V], h[V];
    load_f32<V>(a.floor, col, cnt, fl);
    load_f32<V>(a.h0, b * a.chan + col, cnt, h);
    for (int64_t t = 0; t < a.time; ++t) {
      Raw<F32> g, u;
      g.zero();
      u.zero();
      g.load(a.g, b * a.g_batch + t * a.g_time + col, cnt);
      u.load(a.u, b * a.u_batch + t * a.u_time + col, cnt);
      const bool cut = a.reset && a.reset[b * a.time + t];
#pragma unroll
      for (int k = 0; k < V; ++k) {
        float s, sc;
        sigmoids(g.get(k), s, sc);
        const float rest = 1.0f - fl[k];
        h[k] = cut ? u.get(k) : (fl[k] + rest * s) * h[k] + rest * sc * u.get(k);
      }
      store<F32>(a.y, b * a.y_batch + t * a.y_time + col, cnt, h);
    }
    if (a.h_last)
#pragma unroll
      for (int k = 0; k < V; ++k)
        if (k < cnt) a.h_last[b * a.chan + col + k] = h[k];
  }
}

// ---------------------------------------------------------------- backward
// One step: from dy and the carry c to dg, du and the next carry; adds to dfloor.
template <bool F32>
__device__ __forceinline__ void backward_step(const Raw<F32> &g, const Raw<F32> &u, const Raw<F32> &dy,
                                              const float (&before)[Raw<F32>::V], bool cut,
                                              const float (&fl)[Raw<F32>::V], float (&c)[Raw<F32>::V],
                                              float (&dg)[Raw<F32>::V], float (&du)[Raw<F32>::V],
                                              float (&dfl)[Raw<F32>::V]) {
#pragma unroll
  for (int i = 0; i < Raw<F32>::V; ++i) {
    float s, sc;
    sigmoids(g.get(i), s, sc);
    const float rest = 1.0f - fl[i], grad = dy.get(i) + c[i], w = rest * sc;
    const float da = grad * (before[i] - u.get(i));
    du[i] = cut ? grad : w * grad;
    dg[i] = cut ? 0.0f : da * (w * s);
    dfl[i] = __builtin_fmaf(cut ? 0.0f : da, sc, dfl[i]);
    c[i] = cut ? 0.0f : __builtin_fmaf(rest, s, fl[i]) * grad;
  }
}

template <bool F32>
__device__ __forceinline__ void state_before_step(const nvfp4_scan_args &a, int64_t b, int64_t t, int64_t col,
                                                  int cnt, float (&h)[Raw<F32>::V]) {
  if (t > 0) {
    Raw<F32> y;
    y.zero();
    y.load(a.y, b * a.y_batch + (t - 1) * a.y_time + col, cnt);
#pragma unroll
    for (int i = 0; i < Raw<F32>::V; ++i) h[i] = y.get(i);
  } else {
    load_f32<Raw<F32>::V>(a.h0, b * a.chan + col, cnt, h);
  }
}

// Time runs backward: a thread's step s is t = time - 1 - (j kTile + group kSteps + s).
template <bool F32, bool RESET>
__global__ __launch_bounds__(256) void scan_backward_kernel(ScanLaunch l, Chain c, float *floors) {
  constexpr int V = Raw<F32>::V, CH = 8 * V;
  __shared__ Shared<CH> sh;
  const nvfp4_scan_args &a = l.a;
  const nvfp4_scan_grads &d = l.d;
  const int group = threadIdx.x >> 3, lane = threadIdx.x & 7;
  for (int64_t turn = 0;; ++turn) {
    const int64_t tile = next_tile(sh, c, turn);
    if (tile >= c.tiles) return;
    const int64_t strip = tile % c.strips, j = tile / c.strips;
    const int64_t batch = strip / c.chan_strips, c0 = strip % c.chan_strips * CH, col = c0 + lane * V;
    const int cnt = (int)min((int64_t)V, max((int64_t)0, a.chan - col));
    const int64_t last = a.time - 1 - (j * kTile + group * kSteps);   // of the thread's steps
    Raw<F32> g[kSteps], u[kSteps], dy[kSteps], y[kSteps];
#pragma unroll
    for (int s = 0; s < kSteps; ++s) {
      g[s].zero(); u[s].zero(); dy[s].zero(); y[s].zero();
      const int64_t t = last - s;
      if (t < 0) continue;
      g[s].load(a.g, batch * a.g_batch + t * a.g_time + col, cnt);
      dy[s].load(d.dy, batch * d.dy_batch + t * d.dy_time + col, cnt);
      u[s].load(a.u, batch * a.u_batch + t * a.u_time + col, cnt);
      if (t > 0) y[s].load(a.y, batch * a.y_batch + (t - 1) * a.y_time + col, cnt);
    }
    float fl[V];
    load_f32<V>(a.floor, col, cnt, fl);
    Pair p[V];
#pragma unroll
    for (int i = 0; i < V; ++i) p[i] = Pair{1.0f, 0.0f};
    bool cut[kSteps];
#pragma unroll
    for (int s = 0; s < kSteps; ++s) {
      const bool in = last - s >= 0;
      cut[s] = RESET && in && a.reset[batch * a.time + last - s];
#pragma unroll
      for (int i = 0; i < V; ++i) {
        float sg, sc;
        sigmoids(g[s].get(i), sg, sc);
        const float x = in ? __builtin_fmaf(1.0f - fl[i], sg, fl[i]) : 1.0f;
        if (RESET && cut[s]) p[i] = Pair{cut_mark(), 0.0f};
        else p[i] = Pair{is_cut(p[i].a) ? p[i].a : x * p[i].a, x * (p[i].b + dy[s].get(i))};
      }
    }
    float h[V], dfl[V];
    states_of_groups<V, CH>(sh, c, strip, j, c0, a.chan, d.dh_last, d.dh0, p, h);
#pragma unroll
    for (int i = 0; i < V; ++i) dfl[i] = 0.0f;
#pragma unroll
    for (int s = 0; s < kSteps; ++s) {
      const int64_t t = last - s;
      if (t < 0) break;
      float before[V], dg[V], du[V];
#pragma unroll
      for (int i = 0; i < V; ++i) before[i] = y[s].get(i);
      if (t == 0) load_f32<V>(a.h0, batch * a.chan + col, cnt, before);
      backward_step<F32>(g[s], u[s], dy[s], before, RESET && cut[s], fl, h, dg, du, dfl);
      store<F32>(d.dg, batch * d.dg_batch + t * d.dg_time + col, cnt, dg);
      store<F32>(d.du, batch * d.du_batch + t * d.du_time + col, cnt, du);
    }
    if (d.dfloor) {   // the tile's sum over its steps, per channel
      __syncthreads();
#pragma unroll
      for (int i = 0; i < V; ++i) sh.group[group][lane * V + i].a = dfl[i];
      __syncthreads();
      const int ch = threadIdx.x % CH, seg = threadIdx.x / CH;
      float sum = 0.0f;
#pragma unroll
      for (int i = 0; i < Shared<CH>::kPer; ++i) sum += sh.group[seg * Shared<CH>::kPer + i][ch].a;
      sh.first[seg][ch] = sum;
      __syncthreads();
      if (threadIdx.x < CH && c0 + ch < a.chan) {
        sum = 0.0f;
#pragma unroll
        for (int s = 0; s < Shared<CH>::kSegs; ++s) sum += sh.first[s][ch];
        floors[(batch * c.chunks + j) * a.chan + c0 + ch] = sum;
      }
    }
    if (c.chunks == 1) __syncthreads();   // before the next tile writes the shared words
  }
}

template <bool F32>
__global__ __launch_bounds__(64) void scan_backward_short_kernel(ScanLaunch l, int64_t threads, float *floors) {
  constexpr int V = Raw<F32>::V;
  const nvfp4_scan_args &a = l.a;
  const nvfp4_scan_grads &d = l.d;
  const int64_t per = (a.chan + V - 1) / V;
  for (int64_t i = (int64_t)blockIdx.x * 64 + threadIdx.x; i < threads; i += (int64_t)gridDim.x * 64) {
    const int64_t b = i / per, col = i % per * V;
    const int cnt = (int)min((int64_t)V, a.chan - col);
    float fl[V], c[V], dfl[V];
    load_f32<V>(a.floor, col, cnt, fl);
    load_f32<V>(d.dh_last, b * a.chan + col, cnt, c);
#pragma unroll
    for (int k = 0; k < V; ++k) dfl[k] = 0.0f;
    for (int64_t t = a.time - 1; t >= 0; --t) {
      Raw<F32> g, u, dy;
      g.zero(); u.zero(); dy.zero();
      g.load(a.g, b * a.g_batch + t * a.g_time + col, cnt);
      u.load(a.u, b * a.u_batch + t * a.u_time + col, cnt);
      dy.load(d.dy, b * d.dy_batch + t * d.dy_time + col, cnt);
      float before[V], dg[V], du[V];
      state_before_step<F32>(a, b, t, col, cnt, before);
      backward_step<F32>(g, u, dy, before, a.reset && a.reset[b * a.time + t], fl, c, dg, du, dfl);
      store<F32>(d.dg, b * d.dg_batch + t * d.dg_time + col, cnt, dg);
      store<F32>(d.du, b * d.du_batch + t * d.du_time + col, cnt, du);
    }
#pragma unroll
    for (int k = 0; k < V; ++k) {
      if (k >= cnt) continue;
      if (d.dh0) d.dh0[b * a.chan + col + k] = c[k];
      if (floors) floors[b * a.chan + col + k] = dfl[k];
    }
  }
}

// dfloor: the sums of `rows` tiles (or batch rows) added in order, 32 threads to a channel.
__global__ __launch_bounds__(1024) void scan_floor_kernel(const float *sums, int64_t rows, int64_t chan,
                                                          float *dfloor) {
  __shared__ float part[32][32];
  const int lane = threadIdx.x & 31, share = threadIdx.x >> 5;
  const int64_t c = (int64_t)blockIdx.x * 32 + lane;
  float v = 0.0f;
  if (c < chan)
    for (int64_t i = rows * share / 32; i < rows * (share + 1) / 32; ++i) v += sums[i * chan + c];
  part[share][lane] = v;
  __syncthreads();
  if (share || c >= chan) return;
  v = 0.0f;
#pragma unroll
  for (int w = 0; w < 32; ++w) v += part[w][lane];
  dfloor[c] = v;
}

// ---------------------------------------------------------------- launches
constexpr int kCus = 256;

// Workspace: the ticket and the chain's words (more than one chunk), then the tiles' sums
// for dfloor (backward).
struct Layout {
  Chain c;
  size_t words;     // bytes to clear, after the ticket's 16
  size_t floors;    // offset of the sums
  size_t bytes;
};

Layout layout_of(int64_t batch, int64_t time, int64_t chan, bool f32, bool backward) {
  const int64_t ch = f32 ? 32 : 64;
  Layout l;
  l.c.chan_strips = (chan + ch - 1) / ch;
  l.c.strips = batch * l.c.chan_strips;
  l.c.chunks = time <= kShort ? 1 : (time + kTile - 1) / kTile;
  l.c.tiles = l.c.strips * l.c.chunks;
  l.words = l.c.chunks > 1 ? (size_t)l.c.tiles * ch * 12 : 0;
  l.floors = l.words ? 16 + ((l.words + 15) & ~(size_t)15) : 0;
  l.bytes = l.floors + (backward ? 4 * (size_t)(batch * l.c.chunks * chan) : 0);
  return l;
}

uint32_t grid_of(int64_t wgs, int64_t most) { return (uint32_t)(wgs < most ? wgs : most); }

// Clears the chain's words where there is a chain.
hipError_t prepare_chain(Layout &l, void *ws, hipStream_t stream) {
  if (!l.words) return hipSuccess;
  char *p = static_cast<char *>(ws);
  l.c.ticket = reinterpret_cast<uint32_t *>(p);
  l.c.pairs = reinterpret_cast<uint64_t *>(p + 16);
  l.c.states = reinterpret_cast<uint32_t *>(p + 16 + l.words / 12 * 8);
  const int64_t n = (int64_t)((l.words + 15) / 16);
  scan_clear_kernel<<<grid_of((n + 255) / 256, 4 * kCus), 256, 0, stream>>>(
      reinterpret_cast<uint4 *>(p + 16), n, l.c.ticket);
  return hipGetLastError();
}

template <bool F32>
hipError_t run_forward(const ScanLaunch &s, hipStream_t stream) {
  const nvfp4_scan_args &a = s.a;
  if (a.time <= kShort) {
    const int64_t threads = a.batch * ((a.chan + Raw<F32>::V - 1) / Raw<F32>::V);
    scan_forward_short_kernel<F32><<<grid_of((threads + 63) / 64, 64 * kCus), 64, 0, stream>>>(a, threads);
    return hipGetLastError();
  }
  Layout l = layout_of(a.batch, a.time, a.chan, F32, false);
  const hipError_t e = prepare_chain(l, s.ws, stream);
  if (e != hipSuccess) return e;
  const uint32_t grid = grid_of(l.c.tiles, 8 * kCus);
  if (a.reset) scan_forward_kernel<F32, true><<<grid, 256, 0, stream>>>(a, l.c);
  else scan_forward_kernel<F32, false><<<grid, 256, 0, stream>>>(a, l.c);
  return hipGetLastError();
}

template <bool F32>
hipError_t run_backward(const ScanLaunch &s, hipStream_t stream) {
  const nvfp4_scan_args &a = s.a;
  Layout l = layout_of(a.batch, a.time, a.chan, F32, true);
  float *floors = reinterpret_cast<float *>(static_cast<char *>(s.ws) + l.floors);
  hipError_t e = hipSuccess;
  if (a.batch > 0) {
    if (a.time <= kShort) {
      const int64_t threads = a.batch * ((a.chan + Raw<F32>::V - 1) / Raw<F32>::V);
      scan_backward_short_kernel<F32><<<grid_of((threads + 63) / 64, 64 * kCus), 64, 0, stream>>>(
          s, threads, a.time && s.d.dfloor ? floors : nullptr);   // (no steps: no workspace)
    } else {
      if ((e = prepare_chain(l, s.ws, stream)) != hipSuccess) return e;
      const uint32_t grid = grid_of(l.c.tiles, 8 * kCus);
      if (a.reset) scan_backward_kernel<F32, true><<<grid, 256, 0, stream>>>(s, l.c, floors);
      else scan_backward_kernel<F32, false><<<grid, 256, 0, stream>>>(s, l.c, floors);
    }
    if ((e = hipGetLastError()) != hipSuccess) return e;
  }
  if (!s.d.dfloor) return e;
  const int64_t rows = a.time ? a.batch * l.c.chunks : 0;
  scan_floor_kernel<<<(uint32_t)((a.chan + 31) / 32), 1024, 0, stream>>>(floors, rows, a.chan, s.d.dfloor);
  return hipGetLastError();
}

}  // namespace

size_t scan_workspace_bytes(int64_t batch, int64_t time, int64_t chan, bool backward) {
  // the larger of the two types' (binary32 strips are half as wide: their last one may
  // have fewer unused channels)
  const size_t a = layout_of(batch, time, chan, false, backward).bytes;
  const size_t b = layout_of(batch, time, chan, true, backward).bytes;
  return a > b ? a : b;
}

hipError_t launch_scan_forward(const ScanLaunch &s, hipStream_t stream) {
  return s.a.dtype == NVFP4_DT_FP32 ? run_forward<true>(s, stream) : run_forward<false>(s, stream);
}

hipError_t launch_scan_backward(const ScanLaunch &s, hipStream_t stream) {
  return s.a.dtype == NVFP4_DT_FP32 ? run_backward<true>(s, stream) : run_backward<false>(s, stream);
}

}  // namespace nvfp4

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
// reads dy, g, u, y and writes dg and du, 12 bytes.
//
//  * A tile is 128 bytes of channels (16 lanes of 8 bytes) by kTile time steps: each of 256
//    threads holds kSteps consecutive steps of its channels in registers.  A run of steps
//    acts on the state as h -> A h + B; the threads' (A, B) are composed through LDS.
//  * The tiles of a sequence run in one kernel, so everything is read once: the decoupled
//    look-back of Merrill and Garland, "Single-pass Parallel Prefix Scan with Decoupled
//    Look-back" (2016), over maps of a state instead of sums.  A workgroup
//    takes the next tile of its strip (a count in memory), so that it only ever waits for
//    tiles that workgroups already run; it tells the others the tile's (A, B) if it has to
//    wait, and the state behind the tile as soon as it knows it, each in one 64-bit word.
//    The state before a tile is the nearest known one with the (A, B) of the tiles since
//    applied to it in order: the same operations whoever was first, so results are the same
//    every time.  (Three kernels, (A, B) of all tiles, then states, then tiles, read part of
//    the inputs twice: 108 us forward, 152 us backward at the sizes below.)
//  * A reset is a cut, not a product with zero: (cut, B) composed with anything before it is
//    (cut, B), so inf and NaN end there.  A cut is held as A = -0.0, which no product of the
//    other factors (in [0, 1], or NaN) gives.
//
// Few steps (up to kShort) need no tiles: a thread walks over them.
//
// Measured in bf16: forward with resets 8192 x 5120 in 68 us, 3.7 TB/s; backward with a
// floor, 4 x 2048 x 5120, in 112 us, 4.5 TB/s (a copy reaches 5.4); forward with a floor, 6 x
// 800 x 8031, 52 us, 4.4 TB/s.  The rest is one tile's way through load, LDS, chain and store
// with 3 workgroups to a CU: 4 gain nothing, tiles of half the steps took a third longer, and
// more steps a thread do not fit in its registers.  16 bytes a lane, 4 steps: as fast, with
// twice the LDS and 20 registers more.  One step of 64 x 5120 takes 3.7 us.
#include "nvfp4_device.hpp"
#include "train_launch.hpp"

namespace nvfp4 {
namespace {

constexpr int kWords = 2;            // words of an access
constexpr int kLanes = 16;           // lanes of channels
constexpr int kGroups = 256 / kLanes;   // time groups of a tile
constexpr int kSteps = 8;            // steps of a thread
constexpr int kTile = kGroups * kSteps;
constexpr int kFirst = 1;            // tiles before its own that a tile looks at first
constexpr int kWindow = 8;           // ... and while it waits (65536 x 128: 1 tile 287 us, 2 156,
                                     // 4 94, 8 61, 16 49, but 8192 x 5120 with 16 70, with 8 68)
constexpr int kLooks = 1 << 22;      // how often a tile looks before it gives up: seconds
constexpr int kShort = 16;           // steps that one thread walks over by itself

// ---------------------------------------------------------------- loads and stores
// 8 bytes of channels, at any element's alignment (the packed type makes them single
// instructions).  PART: only `cnt` of the elements exist (fewer channels than one access
// covers); otherwise a strip's last lanes take the last whole access, so that no load
// depends on a branch, and store their own channels alone.
struct __attribute__((packed, aligned(2))) Words { uint32_t w[kWords]; };

template <bool F32>
struct Raw {
  static constexpr int V = F32 ? kWords : 2 * kWords;
  uint32_t w[kWords];

  template <bool PART>
  __device__ __forceinline__ void load(const char *p, int cnt) {
    if constexpr (!PART) {
      const Words v = *reinterpret_cast<const Words *>(p);
#pragma unroll
      for (int l = 0; l < kWords; ++l) w[l] = v.w[l];
    } else {
      for (int l = 0; l < kWords; ++l) w[l] = 0u;
#pragma unroll
      for (int j = 0; j < V; ++j) {
        if (j >= cnt) continue;
        if constexpr (F32) w[j] = reinterpret_cast<const uint32_t *>(p)[j];
        else w[j >> 1] |= (uint32_t) reinterpret_cast<const uint16_t *>(p)[j] << (16 * (j & 1));
      }
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

// Elements from .. to - 1 of the V at p; WHOLE: all of them.
template <bool WHOLE, bool F32>
__device__ __forceinline__ void store(char *p, int from, int to, const float (&v)[F32 ? kWords : 2 * kWords]) {
  constexpr int V = F32 ? kWords : 2 * kWords;
  if (WHOLE || (from <= 0 && to >= V)) {
    Words f;
#pragma unroll
    for (int l = 0; l < kWords; ++l) f.w[l] = F32 ? __float_as_uint(v[l % V]) : pack2(v[(2 * l) % V], v[(2 * l + 1) % V]);
    *reinterpret_cast<Words *>(p) = f;
  } else {
#pragma unroll
    for (int j = 0; j < V; ++j) {
      if (j < from || j >= to) continue;
      if constexpr (F32) reinterpret_cast<float *>(p)[j] = v[j];
      else reinterpret_cast<uint16_t *>(p)[j] = bf16_bits_rn(v[j]);
    }
  }
}

template <bool F32>
__device__ __forceinline__ const char *at(const void *p, int64_t i) {
  return static_cast<const char *>(p) + i * (F32 ? 4 : 2);
}
template <bool F32>
__device__ __forceinline__ char *at(void *p, int64_t i) {
  return static_cast<char *>(p) + i * (F32 ? 4 : 2);
}

// V binary32 values (floor, states); zero where there are none.
template <int V, bool PART>
__device__ __forceinline__ void load_f32(const float *p, int64_t i, int cnt, float (&v)[V]) {
#pragma unroll
  for (int j = 0; j < V; ++j) v[j] = p && (!PART || j < cnt) ? p[i + j] : 0.0f;
}

// ---------------------------------------------------------------- arithmetic
// exp(-g).  A product with log2(e) in 24 bits is off by up to |g| 2^-24 before the
// exponential, which bf16 results do not notice (4e-6 of the result at most where it is not
// zero, their own rounding 2e-3).  binary32 gets the product's error back as a factor: for
// |g| of 20 to 40 sigmoid(-g) is off by 3.6e-8 (rms), 8.4e-7 without.  (Clamped to where it
// is zero, and to log(2^128), where it is infinite: both products stay finite and the factor
// of the infinite one positive.)
template <bool F32>
__device__ __forceinline__ float exp_minus(float g) {
  if constexpr (!F32) return __expf(-g);
  constexpr float kLog2e = 0x1.715476p+0f, kRest = 0x1.4ae0cp-26f, kLn2 = 0x1.62e43p-1f;
  const float x = __builtin_elementwise_maximum(__builtin_elementwise_minimum(-g, 0x1.62e43p+6f), -150.0f);
  const float t = x * kLog2e, r = __builtin_fmaf(x, kRest, __builtin_fmaf(x, kLog2e, -t));
  const float e = __builtin_amdgcn_exp2f(t);
  return __builtin_fmaf(e, r * kLn2, e);
}

// sigmoid(g) and sigmoid(-g), neither by a difference of near equals: for g < 0, where
// exp(-g) may overflow (then sigmoid(g) is zero), 1 - sigmoid(g) loses nothing.
template <bool F32>
__device__ __forceinline__ void sigmoids(float g, float &s, float &sc) {
  const float e = exp_minus<F32>(g);
  s = __builtin_amdgcn_rcpf(1.0f + e);
  sc = g < 0.0f ? 1.0f - s : e * s;
}

// The decay a = floor + (1 - floor) sigmoid(g) and 1 - a.  For bf16 without a selection (6 x
// 800 x 8031 forward 63 us, 64.5 with): 4 exp(-g) is infinite from where the quotient would
// be subnormal, which the instruction flushes to zero, so exp(-g) sigmoid(g) is either right
// or NaN, infinity times zero, which the minimum takes for its end.  (A NaN gate is one in a.)
template <bool F32, bool FLOOR>
__device__ __forceinline__ void decay(float g, float fl, float &a, float &w) {
  const float rest = 1.0f - fl;
  float s;
  if constexpr (F32) {
    float sc;
    sigmoids<F32>(g, s, sc);
    w = FLOOR ? rest * sc : sc;
  } else {
    const float e4 = __builtin_amdgcn_exp2f(__builtin_fmaf(g, -0x1.715476p+0f, 2.0f));
    s = __builtin_amdgcn_rcpf(__builtin_fmaf(e4, 0.25f, 1.0f));
    w = (FLOOR ? 0.25f * rest : 0.25f) * __builtin_fminf(e4 * s, 4.0f);
  }
  a = FLOOR ? __builtin_fmaf(rest, s, fl) : s;
}

__device__ __forceinline__ float cut_mark() { return -0.0f; }
__device__ __forceinline__ bool is_cut(float a) { return __float_as_uint(a) == 0x80000000u; }

struct Pair { float a, b; };   // h -> a h + b, or h -> b behind a cut

__device__ __forceinline__ float apply(const Pair &p, float h) {
  return is_cut(p.a) ? p.b : __builtin_fmaf(p.a, h, p.b);
}

// First p, then q.  (A factor in [0, 1] times -0.0 is -0.0: what follows a cut keeps it.)
__device__ __forceinline__ Pair then(const Pair &p, const Pair &q) {
  return is_cut(q.a) ? q : Pair{q.a * p.a, __builtin_fmaf(q.a, p.b, q.b)};
}

// ---------------------------------------------------------------- tiles
// Tiles along time of every sequence, and what passes between them.  A strip (of one batch
// row) counts its tiles as they are taken; a tile has a word per place: its pair, later
// the state after it as the pair that leads there from anywhere.  Zero: neither yet.
struct Tiling {
  int64_t chunks;
  int64_t chunk0, strip0;   // the launch's first tile and strip (grids are bounded)
  uint32_t across;          // strips of a batch row
  uint32_t strips, each;    // the launch's strips; how many of them a die has at most (0: any die has any)
  uint32_t *taken;          // [strip][kLine]
  uint64_t *words;          // [strip][tile][place]
};

constexpr uint32_t kDies = 8;   // consecutive workgroups go to the dies in turn

// The strip of a workgroup, and the tile that its place in the grid suggests.  A die gets a
// run of strips: neighbouring ones share cache lines where rows do not begin at one.
struct Spot {
  int64_t strip, batch, tile;
  int32_t at;   // the strip's place in its row
  bool none;    // no strip: the dies' shares differ by one
  __device__ __forceinline__ explicit Spot(const Tiling &t) {
    const uint32_t n = blockIdx.x;
    uint32_t k, turn;
    none = false;
    if (t.each) {
      const uint32_t die = n % kDies, q = n / kDies;
      const uint32_t from = (uint32_t)((uint64_t)die * t.strips / kDies), to = (uint32_t)((uint64_t)(die + 1) * t.strips / kDies);
      turn = q / t.each;
      k = from + (q - turn * t.each);
      none = k >= to;
    } else {
      turn = n / t.strips;
      k = n - turn * t.strips;
    }
    tile = t.chunk0 + turn;
    strip = t.strip0 + k;
    if (t.strip0 == 0) {   // (almost always: a division of 32 bits)
      batch = k / t.across;
      at = (int32_t)(k - (uint32_t)batch * t.across);
    } else {
      batch = strip / t.across;
      at = (int32_t)(strip - batch * t.across);
    }
  }
};

constexpr int kLine = 32;   // (128 bytes: strips do not share lines)

// A word holds both numbers at once, so nothing has to be ordered around it.  The factor's
// bits are inverted: no word is then zero, given that a NaN comes in one form.
__device__ __forceinline__ uint64_t word_of(const Pair &p) {
  const uint32_t a = p.a == p.a ? __float_as_uint(p.a) : 0x7FC00000u;
  return ((uint64_t)__float_as_uint(p.b) << 32) | (uint32_t)~a;
}
__device__ __forceinline__ Pair pair_of(uint64_t w) {
  return Pair{__uint_as_float(~(uint32_t)w), __uint_as_float((uint32_t)(w >> 32))};
}

// Stores and loads that go past the caches of one die.
__device__ __forceinline__ uint64_t load_agent(const uint64_t *p) {
  return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ void store_agent(uint64_t *p, uint64_t v) {
  __hip_atomic_store(p, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

// Where a thread's V channels are, in the strip of kLanes V at `at`.
// Its own are the elements own .. cnt - 1 of the access at col.
template <int V, bool PART>
struct Place {
  int64_t first, col;   // the strip's first channel; the thread's access
  int own, cnt;
  __device__ __forceinline__ Place(int64_t at, int64_t chan) {
    first = at * (kLanes * V);
    col = first + (threadIdx.x % kLanes) * V;
    own = 0;
    cnt = V;
    if constexpr (PART) {
      cnt = (int)min((int64_t)V, max((int64_t)0, chan - col));
    } else if (col > chan - V) {   // (chan >= V)
      own = (int)min((int64_t)V, col - (chan - V));
      col = chan - V;
    }
  }
};

// The channel of a strip's place tid < kLanes V (element tid % V of lane tid / V), whether there
// is one, and whether it is that lane's own.
template <int V, bool PART>
__device__ __forceinline__ int64_t channel_of(int tid, int64_t first, int64_t chan, bool &own) {
  const int64_t c = first + tid;
  if constexpr (PART) {
    own = c < chan;
    return c;
  } else {
    const int64_t lane = first + tid / V * V, moved = max((int64_t)0, lane - (chan - V));
    own = tid % V >= moved;
    return c - moved;
  }
}

// Whether all of a tile's steps and of its strip's channels exist.
template <int V>
__device__ __forceinline__ bool whole_tile(const nvfp4_scan_args &a, int64_t j, int64_t first) {
  return (j + 1) * kTile <= a.time && first + kLanes * V <= a.chan;
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

// The threads' pairs (one per channel) into segments' pairs; each group's place then holds
// the pair of its segment's groups before it.
template <int V, int CH>
__device__ __forceinline__ void compose(Shared<CH> &sh, const Pair (&p)[V]) {
  const int tid = threadIdx.x, group = tid / kLanes, lane = tid % kLanes;
#pragma unroll
  for (int i = 0; i < V; ++i) sh.group[group][lane * V + i] = p[i];
  __syncthreads();
  const int ch = tid % CH, seg = tid / CH;
  Pair run = {1.0f, 0.0f};
#pragma unroll
  for (int i = 0; i < Shared<CH>::kPer; ++i) {
    const Pair q = sh.group[seg * Shared<CH>::kPer + i][ch];
    sh.group[seg * Shared<CH>::kPer + i][ch] = run;
    run = then(run, q);
  }
  sh.seg[seg][ch] = run;
  __syncthreads();
}

// The state before tile j > 0 (whose words are at `own`) as far as it follows from the W tiles
// before: whether it does in all lanes.
template <int CH, int W>
__device__ __forceinline__ bool look(const uint64_t *own, int64_t j, float &before) {
  const int reach = (int)min((int64_t)W, j);
  uint64_t w[W];
#pragma unroll
  for (int k = 0; k < W; ++k) w[k] = load_agent(own - (int64_t)min(k + 1, reach) * CH);
  // from the nearest state on (which needs none before it)
  bool gap = true;
#pragma unroll
  for (int k = W - 1; k >= 0; --k) {
    const Pair p = pair_of(w[k]);
    gap = w[k] == 0ull || (gap && !is_cut(p.a));
    before = apply(p, before);
  }
  return !__any(gap);
}

// The chain.  In wave 0, lane = place: from the tile's pair to the state before it, and what
// other tiles need to know of both.  `given` is the state before the first tile.  States
// follow from the one before by one pair, in order, however many of those a tile applies
// itself: results do not depend on who was first.
template <int CH>
__device__ __forceinline__ float state_before_tile(const Tiling &t, int64_t strip, int64_t j, const Pair &all,
                                                   float given) {
  const bool live = threadIdx.x < CH, more = j + 1 < t.chunks;
  uint64_t *own = t.words + (strip * t.chunks + j) * CH + threadIdx.x % CH;
  float before = given;
  if (j > 0) {
    if (!look<CH, kFirst>(own, j, before)) {
      if (live && more) store_agent(own, word_of(all));   // (a pair is for those who wait with this tile)
      int looks = 0;
      while (!look<CH, kWindow>(own, j, before)) {
        if (++looks == kLooks) {   // (never: see the order of the tiles)
          before = __uint_as_float(0x7FC00000u);
          break;
        }
        __builtin_amdgcn_s_sleep(1);
      }
    }
  }
  if (live && more) store_agent(own, word_of(Pair{cut_mark(), apply(all, before)}));
  return before;
}

// Whether (it waits until) the first tile of the strip has told its words of this thread's
// channels: it then has read the state before it, which is told after that.  For a last tile
// that puts the state after it in that state's place; behind a cut nothing else makes it wait.
template <int V>
__device__ __forceinline__ bool first_tile_has_read(const Tiling &t, int64_t strip) {
  const uint64_t *w = t.words + strip * t.chunks * (kLanes * V) + (threadIdx.x % kLanes) * V;
  for (int looks = 0; looks < kLooks; ++looks) {   // (ends as the chain's waits do)
    bool all = true;
#pragma unroll
    for (int i = 0; i < V; ++i) all &= load_agent(w + i) != 0ull;
    if (all) return true;
    __builtin_amdgcn_s_sleep(1);
  }
  return false;
}

// The state before each thread's steps from compose()'s result and the state before the
// first tile (per channel).
template <int V, bool PART>
__device__ __forceinline__ void states_of_groups(Shared<kLanes * V> &sh, const Tiling &t, const float *given,
                                                 const Spot &at, int64_t j, int64_t first, int64_t chan,
                                                 float (&h)[V]) {
  constexpr int CH = kLanes * V, kSegs = Shared<CH>::kSegs;
  const int tid = threadIdx.x, group = tid / kLanes, lane = tid % kLanes;
  if (tid < 64) {
    Pair all = sh.seg[0][tid % CH];
#pragma unroll
    for (int s = 1; s < kSegs; ++s) all = then(all, sh.seg[s][tid % CH]);
    float before = 0.0f;
    if (j == 0 && given && tid < CH) {
      bool own;
      const int64_t c = channel_of<V, PART>(tid, first, chan, own);
      if (!PART || own) before = given[at.batch * chan + c];
      asm volatile("" : "+v"(before) : : "memory");   // (waits here: the chain's stores come after)
    }
    if (t.chunks > 1) before = state_before_tile<CH>(t, at.strip, j, all, before);
    if (tid < CH) {
#pragma unroll
      for (int s = 0; s < kSegs; ++s) {
        sh.first[s][tid] = before;
        before = apply(sh.seg[s][tid], before);
      }
    }
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < V; ++i)
    h[i] = apply(sh.group[group][lane * V + i], sh.first[group / Shared<CH>::kPer][lane * V + i]);
}

// The tile a workgroup takes: the next of its strip.  That is the one its place in the grid
// suggests wherever workgroups begin in order, so the loads of that one can be on their way
// while the count is asked for.
template <int CH>
struct Taken {
  uint32_t number = 0;
  __device__ __forceinline__ void ask(const Tiling &t, int64_t strip) {
    if (t.chunks > 1 && threadIdx.x == 0)
      number = __hip_atomic_fetch_add(t.taken + strip * kLine, 1u,
                                      __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  }
  __device__ __forceinline__ int64_t tell(Shared<CH> &sh, const Tiling &t, int64_t guess) {
    if (t.chunks == 1) return guess;
    if (threadIdx.x == 0) sh.tile = number;
    __syncthreads();
    return (int64_t)__builtin_amdgcn_readfirstlane((int)sh.tile);
  }
};

// Clears counts and words before a launch, by the same way as they are used.
__global__ __launch_bounds__(256) void scan_clear_kernel(uint64_t *p, int64_t n) {
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256)
    store_agent(p + i, 0ull);
}

// ---------------------------------------------------------------- forward
// A thread's steps of tile j.  WHOLE: all the tile's steps and channels exist.  Otherwise
// steps past the end (all in the last tile) read the last one again and lead nowhere.
template <bool WHOLE>
struct ForwardSteps {
  int64_t at, t0;   // the first one, and the first one read
  int more, last;   // how many there are; the last one read, from t0
  __device__ __forceinline__ ForwardSteps(int64_t j, int64_t time) {
    at = j * kTile + (threadIdx.x / kLanes) * kSteps;
    t0 = WHOLE ? at : min(at, time - 1);
    more = WHOLE ? kSteps : (int)min((int64_t)kSteps, time - at);
    last = max(0, more - 1);
  }
  __device__ __forceinline__ int step(int s) const { return WHOLE ? s : min(s, last); }
};

template <bool F32, bool RESET>
struct ForwardLoads {
  Raw<F32> g[kSteps], u[kSteps];
  uint8_t reset[kSteps];
  template <bool PART, bool WHOLE>
  __device__ __forceinline__ void fetch(const nvfp4_scan_args &a, int64_t batch, int64_t j,
                                        const Place<Raw<F32>::V, PART> &pl) {
    const ForwardSteps<WHOLE> st(j, a.time);
    const char *pg = at<F32>(a.g, batch * a.g_batch + st.t0 * a.g_time + pl.col);
    const char *pu = at<F32>(a.u, batch * a.u_batch + st.t0 * a.u_time + pl.col);
#pragma unroll
    for (int s = 0; s < kSteps; ++s) {
      g[s].template load<PART>(at<F32>(pg, st.step(s) * a.g_time), pl.cnt);
      u[s].template load<PART>(at<F32>(pu, st.step(s) * a.u_time), pl.cnt);
    }
    if (RESET && (!PART || a.reset))
#pragma unroll
      for (int s = 0; s < kSteps; ++s) reset[s] = a.reset[batch * a.time + st.t0 + st.step(s)];
  }
};

template <bool F32, bool RESET, bool FLOOR, bool PART, bool WHOLE>
__device__ __forceinline__ void forward_tile(const nvfp4_scan_args &a, const Tiling &tl, const Spot &spot,
                                             int64_t j, const Place<Raw<F32>::V, PART> &pl,
                                             ForwardLoads<F32, RESET> &in, Shared<kLanes * Raw<F32>::V> &sh) {
  constexpr int V = Raw<F32>::V, CH = kLanes * V;
  Raw<F32>(&g)[kSteps] = in.g, (&u)[kSteps] = in.u;
  const int64_t batch = spot.batch;
  const ForwardSteps<WHOLE> st(j, a.time);
  float fl[V];
  if constexpr (FLOOR) load_f32<V, PART>(a.floor, pl.col, pl.cnt, fl);
  float av[kSteps][V], bv[kSteps][V];
  Pair p[V];
#pragma unroll
  for (int i = 0; i < V; ++i) p[i] = Pair{1.0f, 0.0f};
  bool cut[kSteps];
#pragma unroll
  for (int s = 0; s < kSteps; ++s) {
    cut[s] = RESET && (!PART || a.reset) && in.reset[s];
#pragma unroll
    for (int i = 0; i < V; ++i) {
      float w;
      decay<F32, FLOOR>(g[s].get(i), fl[i], av[s][i], w);
      bv[s][i] = w * u[s].get(i);
      p[i] = Pair{av[s][i] * p[i].a, __builtin_fmaf(av[s][i], p[i].b, bv[s][i])};
    }
    if (RESET && __any(cut[s])) {   // (one branch for the wave: resets are few)
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (cut[s]) {
          bv[s][i] = u[s].get(i);
          p[i] = Pair{cut_mark(), bv[s][i]};
        }
    }
  }
  compose<V, CH>(sh, p);
  float h[V];
  states_of_groups<V, PART>(sh, tl, a.h0, spot, j, pl.first, a.chan, h);
  char *py = at<F32>(a.y, batch * a.y_batch + st.t0 * a.y_time + pl.col);
#pragma unroll
  for (int s = 0; s < kSteps; ++s) {
    if (!WHOLE && s >= st.more) break;
#pragma unroll
    for (int i = 0; i < V; ++i) h[i] = __builtin_fmaf(av[s][i], h[i], bv[s][i]);
    if (RESET && __any(cut[s])) {
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (cut[s]) h[i] = bv[s][i];
    }
    store<WHOLE, F32>(at<F32>(py, s * a.y_time), pl.own, pl.cnt, h);
  }
  if (a.h_last && st.more > 0 && st.at + st.more == a.time) {
    if (a.h_last == a.h0 && j > 0 && !first_tile_has_read<V>(tl, spot.strip))
#pragma unroll
      for (int i = 0; i < V; ++i) h[i] = __uint_as_float(0x7FC00000u);
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (i >= pl.own && i < pl.cnt) a.h_last[batch * a.chan + pl.col + i] = h[i];
  }
}

// (One branch for a workgroup: no lane of most tiles has anything to check.)
template <bool F32, bool RESET, bool FLOOR, bool PART>
__global__ __launch_bounds__(256) __attribute__((amdgpu_waves_per_eu(3)))
void scan_forward_kernel(nvfp4_scan_args a, Tiling tl) {
  constexpr int V = Raw<F32>::V;
  __shared__ Shared<kLanes * V> sh;
  const Spot at(tl);
  if (at.none) return;
  const int64_t batch = at.batch, guess = at.tile;
  const Place<V, PART> pl(at.at, a.chan);
  ForwardLoads<F32, RESET> in;
  Taken<kLanes * V> taken;
  taken.ask(tl, at.strip);
  int64_t j = guess;
  for (bool asked = false;;) {
    in.template fetch<PART, false>(a, batch, j, pl);
    if (asked) break;
    const int64_t mine = taken.tell(sh, tl, guess);
    if (mine == j) break;
    asked = true;
    j = mine;
  }
  if (!PART && whole_tile<V>(a, j, pl.first)) {
    forward_tile<F32, RESET, FLOOR, PART, true>(a, tl, at, j, pl, in, sh);
  } else {
    forward_tile<F32, RESET, FLOOR, PART, false>(a, tl, at, j, pl, in, sh);
  }
}

// A thread per V channels walks over the steps (the last thread of a row has the rest).
template <bool F32, bool PART>
__global__ __launch_bounds__(64) void scan_forward_short_kernel(nvfp4_scan_args a, int64_t threads) {
  constexpr int V = Raw<F32>::V;
  const int64_t per = PART ? (a.chan + V - 1) / V : a.chan / V;
  for (int64_t i = (int64_t)blockIdx.x * 64 + threadIdx.x; i < threads; i += (int64_t)gridDim.x * 64) {
    const int64_t b = i / per, col = i % per * V;
    const int cnt = (int)min((int64_t)V, a.chan - col);
    float fl[V], h[V];
    load_f32<V, PART>(a.floor, col, cnt, fl);
    load_f32<V, PART>(a.h0, b * a.chan + col, cnt, h);
    for (int64_t t = 0; t < a.time; ++t) {
      Raw<F32> g, u;
      g.template load<PART>(at<F32>(a.g, b * a.g_batch + t * a.g_time + col), cnt);
      u.template load<PART>(at<F32>(a.u, b * a.u_batch + t * a.u_time + col), cnt);
      const bool cut = a.reset && a.reset[b * a.time + t];
#pragma unroll
      for (int k = 0; k < V; ++k) {
        float s, sc;
        sigmoids<F32>(g.get(k), s, sc);
        const float rest = 1.0f - fl[k], x = __builtin_fmaf(rest, s, fl[k]);
        h[k] = cut ? u.get(k) : __builtin_fmaf(x, h[k], rest * sc * u.get(k));
      }
      store<false, F32>(at<F32>(a.y, b * a.y_batch + t * a.y_time + col), 0, cnt, h);
    }
    if (a.h_last)
#pragma unroll
      for (int k = 0; k < V; ++k)
        if (k < cnt) a.h_last[b * a.chan + col + k] = h[k];
  }
}

// ---------------------------------------------------------------- backward
// One step: from dy and the carry c to dg, du and the next carry; adds to dfloor.  CUTS: it
// may be a reset.
template <bool F32, bool FLOOR, bool CUTS>
__device__ __forceinline__ void backward_step(const Raw<F32> &g, const Raw<F32> &u, const Raw<F32> &dy,
                                              const float (&before)[Raw<F32>::V], bool cut,
                                              const float (&fl)[Raw<F32>::V], float (&c)[Raw<F32>::V],
                                              float (&dg)[Raw<F32>::V], float (&du)[Raw<F32>::V],
                                              float (&dfl)[Raw<F32>::V]) {
#pragma unroll
  for (int i = 0; i < Raw<F32>::V; ++i) {
    float s, sc;
    sigmoids<F32>(g.get(i), s, sc);
    const float rest = 1.0f - fl[i], grad = dy.get(i) + c[i], w = FLOOR ? rest * sc : sc;
    float da = grad * (before[i] - u.get(i));
    du[i] = w * grad;
    dg[i] = da * (w * s);
    c[i] = (FLOOR ? __builtin_fmaf(rest, s, fl[i]) : s) * grad;
    if (CUTS && cut) {
      du[i] = grad;
      dg[i] = da = c[i] = 0.0f;
    }
    if constexpr (FLOOR) dfl[i] = __builtin_fmaf(da, sc, dfl[i]);
  }
}

// Time runs backward: a thread's step s is t = time - 1 - (j kTile + group kSteps + s).
// WHOLE: all the tile's steps and channels exist, and a step before each of them.  Otherwise
// steps before the beginning (all in the last tile) read the first one again and lead nowhere.
template <bool WHOLE>
struct BackwardSteps {
  int64_t steps, t0;       // how many from the first one on to the beginning; the first one read
  int more, last, prior;   // how many there are; the last one read, from t0; steps before t0
  __device__ __forceinline__ BackwardSteps(int64_t j, int64_t time) {
    steps = time - (j * kTile + (threadIdx.x / kLanes) * kSteps);
    t0 = WHOLE ? steps - 1 : max((int64_t)0, steps - 1);
    more = WHOLE ? kSteps : (int)min((int64_t)kSteps, steps);
    last = max(0, more - 1);
    prior = WHOLE ? kSteps : (int)min((int64_t)kSteps, t0);
  }
  __device__ __forceinline__ int step(int s) const { return WHOLE ? s : min(s, last); }
  __device__ __forceinline__ int before(int s) const { return WHOLE ? s + 1 : min(s + 1, prior); }
};

template <bool F32, bool RESET>
struct BackwardLoads {
  Raw<F32> g[kSteps], dy[kSteps], u[kSteps], y[kSteps];
  uint8_t reset[kSteps];
  template <bool PART, bool WHOLE>
  __device__ __forceinline__ void fetch(const nvfp4_scan_args &a, const nvfp4_scan_grads &d, int64_t batch,
                                        int64_t j, const Place<Raw<F32>::V, PART> &pl) {
    const BackwardSteps<WHOLE> st(j, a.time);
    const char *pg = at<F32>(a.g, batch * a.g_batch + st.t0 * a.g_time + pl.col);
    const char *pdy = at<F32>(d.dy, batch * d.dy_batch + st.t0 * d.dy_time + pl.col);
#pragma unroll
    for (int s = 0; s < kSteps; ++s) {
      g[s].template load<PART>(at<F32>(pg, -st.step(s) * a.g_time), pl.cnt);
      dy[s].template load<PART>(at<F32>(pdy, -st.step(s) * d.dy_time), pl.cnt);
    }
    if (RESET && (!PART || a.reset))
#pragma unroll
      for (int s = 0; s < kSteps; ++s) reset[s] = a.reset[batch * a.time + st.t0 - st.step(s)];
  }
  // What the second half needs, on its way while the first half's results are composed.
  template <bool PART, bool WHOLE>
  __device__ __forceinline__ void fetch_more(const nvfp4_scan_args &a, int64_t batch,
                                             const BackwardSteps<WHOLE> &st,
                                             const Place<Raw<F32>::V, PART> &pl) {
    const char *pu = at<F32>(a.u, batch * a.u_batch + st.t0 * a.u_time + pl.col);
    const char *py = at<F32>(a.y, batch * a.y_batch + st.t0 * a.y_time + pl.col);
    asm volatile("" ::: "memory");
#pragma unroll
    for (int s = 0; s < kSteps; ++s) {
      u[s].template load<PART>(at<F32>(pu, -st.step(s) * a.u_time), pl.cnt);
      y[s].template load<PART>(at<F32>(py, -st.before(s) * a.y_time), pl.cnt);
    }
  }
};

template <bool F32, bool RESET, bool FLOOR, bool PART, bool WHOLE>
__device__ __forceinline__ void backward_tile(const ScanLaunch &l, const Tiling &tl, float *floors,
                                              const Spot &spot, int64_t j, const Place<Raw<F32>::V, PART> &pl,
                                              BackwardLoads<F32, RESET> &in, Shared<kLanes * Raw<F32>::V> &sh) {
  constexpr int V = Raw<F32>::V, CH = kLanes * V;
  const nvfp4_scan_args &a = l.a;
  const nvfp4_scan_grads &d = l.d;
  const int group = threadIdx.x / kLanes, lane = threadIdx.x % kLanes;
  Raw<F32>(&g)[kSteps] = in.g, (&dy)[kSteps] = in.dy, (&u)[kSteps] = in.u, (&y)[kSteps] = in.y;
  const int64_t batch = spot.batch;
  const BackwardSteps<WHOLE> st(j, a.time);
  float fl[V];
#pragma unroll
  for (int i = 0; i < V; ++i) fl[i] = 0.0f;
  if constexpr (FLOOR) load_f32<V, PART>(a.floor, pl.col, pl.cnt, fl);
  Pair p[V];
#pragma unroll
  for (int i = 0; i < V; ++i) p[i] = Pair{1.0f, 0.0f};
  bool cut[kSteps];
#pragma unroll
  for (int s = 0; s < kSteps; ++s) {
    cut[s] = RESET && (!PART || a.reset) && in.reset[s];
#pragma unroll
    for (int i = 0; i < V; ++i) {
      float x, w;
      decay<F32, FLOOR>(g[s].get(i), fl[i], x, w);
      p[i] = Pair{x * p[i].a, x * (p[i].b + dy[s].get(i))};
    }
    if (RESET && __any(cut[s])) {   // (one branch for the wave: resets are few)
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (cut[s]) p[i] = Pair{cut_mark(), 0.0f};
    }
  }
  if constexpr (FLOOR) {
#pragma unroll
    for (int i = 0; i < V; ++i) asm volatile("" : "+v"(fl[i]));
  }
  in.template fetch_more<PART, WHOLE>(a, batch, st, pl);
  compose<V, CH>(sh, p);
  float c[V], dfl[V];
  states_of_groups<V, PART>(sh, tl, d.dh_last, spot, j, pl.first, a.chan, c);
  // (the gates' sigmoids are formed again: kept, they would take 64 registers a thread)
#pragma unroll
  for (int s = 0; s < kSteps; ++s)
#pragma unroll
    for (int w = 0; w < kWords; ++w) asm volatile("" : "+v"(g[s].w[w]), "+v"(dy[s].w[w]));
  char *pdg = at<F32>(d.dg, batch * d.dg_batch + st.t0 * d.dg_time + pl.col);
  char *pdu = at<F32>(d.du, batch * d.du_batch + st.t0 * d.du_time + pl.col);
#pragma unroll
  for (int i = 0; i < V; ++i) dfl[i] = 0.0f;
#pragma unroll
  for (int s = 0; s < kSteps; ++s) {
    if (!WHOLE && s >= st.more) break;
    float prior_h[V], dg[V], du[V];
#pragma unroll
    for (int i = 0; i < V; ++i) prior_h[i] = y[s].get(i);
    if (!WHOLE && st.t0 == s) load_f32<V, PART>(a.h0, batch * a.chan + pl.col, pl.cnt, prior_h);
    backward_step<F32, FLOOR, RESET>(g[s], u[s], dy[s], prior_h, RESET && cut[s], fl, c, dg, du, dfl);
    store<WHOLE, F32>(at<F32>(pdg, -s * d.dg_time), pl.own, pl.cnt, dg);
    store<WHOLE, F32>(at<F32>(pdu, -s * d.du_time), pl.own, pl.cnt, du);
  }
  if (!WHOLE && d.dh0 && st.steps > 0 && st.steps <= kSteps)   // the thread with the first step
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (i >= pl.own && i < pl.cnt) d.dh0[batch * a.chan + pl.col + i] = c[i];
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
    if (threadIdx.x < CH) {
      bool own;
      const int64_t chan = channel_of<V, PART>(threadIdx.x, pl.first, a.chan, own);
      sum = 0.0f;
#pragma unroll
      for (int s = 0; s < Shared<CH>::kSegs; ++s) sum += sh.first[s][ch];
      if (own) floors[(batch * tl.chunks + j) * a.chan + chan] = sum;
    }
  }
}

template <bool F32, bool RESET, bool FLOOR, bool PART>
__global__ __launch_bounds__(256) __attribute__((amdgpu_waves_per_eu(3)))
void scan_backward_kernel(ScanLaunch l, Tiling tl, float *floors) {
  constexpr int V = Raw<F32>::V;
  __shared__ Shared<kLanes * V> sh;
  const Spot at(tl);
  if (at.none) return;
  const int64_t batch = at.batch, guess = at.tile;
  const Place<V, PART> pl(at.at, l.a.chan);
  BackwardLoads<F32, RESET> in;
  Taken<kLanes * V> taken;
  taken.ask(tl, at.strip);
  auto whole = [&](int64_t j) { return !PART && j + 1 < tl.chunks && whole_tile<V>(l.a, j, pl.first); };
  int64_t j = guess;
  for (bool asked = false;;) {
    in.template fetch<PART, false>(l.a, l.d, batch, j, pl);
    if (asked) break;
    const int64_t mine = taken.tell(sh, tl, guess);
    if (mine == j) break;
    asked = true;
    j = mine;
  }
  if (whole(j)) {
    backward_tile<F32, RESET, FLOOR, PART, true>(l, tl, floors, at, j, pl, in, sh);
  } else {
    backward_tile<F32, RESET, FLOOR, PART, false>(l, tl, floors, at, j, pl, in, sh);
  }
}

template <bool F32, bool PART>
__global__ __launch_bounds__(64) void scan_backward_short_kernel(ScanLaunch l, int64_t threads, float *floors) {
  constexpr int V = Raw<F32>::V;
  const nvfp4_scan_args &a = l.a;
  const nvfp4_scan_grads &d = l.d;
  const int64_t per = PART ? (a.chan + V - 1) / V : a.chan / V;
  for (int64_t i = (int64_t)blockIdx.x * 64 + threadIdx.x; i < threads; i += (int64_t)gridDim.x * 64) {
    const int64_t b = i / per, col = i % per * V;
    const int cnt = (int)min((int64_t)V, a.chan - col);
    float fl[V], c[V], dfl[V];
    load_f32<V, PART>(a.floor, col, cnt, fl);
    load_f32<V, PART>(d.dh_last, b * a.chan + col, cnt, c);
#pragma unroll
    for (int k = 0; k < V; ++k) dfl[k] = 0.0f;
    for (int64_t t = a.time - 1; t >= 0; --t) {
      Raw<F32> g, u, dy, y;
      g.template load<PART>(at<F32>(a.g, b * a.g_batch + t * a.g_time + col), cnt);
      u.template load<PART>(at<F32>(a.u, b * a.u_batch + t * a.u_time + col), cnt);
      dy.template load<PART>(at<F32>(d.dy, b * d.dy_batch + t * d.dy_time + col), cnt);
      float before[V], dg[V], du[V];
      if (t > 0) {
        y.template load<PART>(at<F32>(a.y, b * a.y_batch + (t - 1) * a.y_time + col), cnt);
#pragma unroll
        for (int k = 0; k < V; ++k) before[k] = y.get(k);
      } else {
        load_f32<V, PART>(a.h0, b * a.chan + col, cnt, before);
      }
      backward_step<F32, true, true>(g, u, dy, before, a.reset && a.reset[b * a.time + t], fl, c, dg, du, dfl);
      store<false, F32>(at<F32>(d.dg, b * d.dg_batch + t * d.dg_time + col), 0, cnt, dg);
      store<false, F32>(at<F32>(d.du, b * d.du_batch + t * d.du_time + col), 0, cnt, du);
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

// Workspace (more than one tile): the strips' counts, the tiles' words; then the tiles' sums
// for dfloor (backward).
struct Layout {
  int64_t chunks;
  size_t words, floors, bytes;   // offsets, and the whole
};

Layout layout_of(int64_t batch, int64_t time, int64_t chan, int place, bool backward) {
  Layout l;
  l.chunks = time <= kShort ? 1 : (time + kTile - 1) / kTile;
  const int64_t strips = l.chunks > 1 ? batch * ((chan + place - 1) / place) : 0;
  l.words = 4 * (size_t)(strips * kLine);
  l.floors = l.words + 8 * (size_t)(strips * l.chunks * place);
  l.bytes = l.floors + (backward ? 4 * (size_t)(batch * l.chunks * chan) : 0);
  return l;
}

Tiling tiling_of(const Layout &l, void *ws) {
  char *p = static_cast<char *>(ws);
  return Tiling{l.chunks, 0, 0, 0, 0, 0, reinterpret_cast<uint32_t *>(p), reinterpret_cast<uint64_t *>(p + l.words)};
}

uint32_t at_most(int64_t n, int64_t most) { return (uint32_t)(n < most ? n : most); }

// Launches over all strips of `ch` channels and their tiles, in slices that a grid can count.
// Dies get runs of strips where that leaves none with much less than another (9 x 6143 x 468
// backward 100 us, 119 without; 4 x 2048 x 5120, whose rows begin at cache lines, 120 and
// 129).  launch(grid, tiling).
template <class Launch>
hipError_t over_tiles(const nvfp4_scan_args &a, Tiling t, int ch, Launch &&launch) {
  constexpr int64_t most = 1 << 20, grid = 1 << 23;
  t.across = (uint32_t)((a.chan + ch - 1) / ch);
  const int64_t strips = a.batch * t.across;
  for (; t.strip0 < strips; t.strip0 += most) {
    t.strips = at_most(strips - t.strip0, most);
    t.each = (t.strips + kDies - 1) / kDies;
    if (t.each * kDies > t.strips + t.strips / 8) t.each = 0;
    const int64_t row = t.each ? t.each * kDies : t.strips, turns = grid / row;
    for (t.chunk0 = 0; t.chunk0 < t.chunks; t.chunk0 += turns) {
      launch((uint32_t)(row * at_most(t.chunks - t.chunk0, turns)), t);
      const hipError_t e = hipGetLastError();
      if (e != hipSuccess) return e;
    }
  }
  return hipSuccess;
}

hipError_t clear_words(const Layout &l, void *ws, hipStream_t stream) {
  if (l.chunks == 1) return hipSuccess;
  const int64_t n = (int64_t)(l.floors / 8);
  scan_clear_kernel<<<at_most((n + 255) / 256, 8 * kCus), 256, 0, stream>>>(static_cast<uint64_t *>(ws), n);
  return hipGetLastError();
}

template <bool F32, bool RESET, bool FLOOR, bool PART>
hipError_t forward_tiles(const ScanLaunch &s, const Layout &l, hipStream_t stream) {
  const hipError_t e = clear_words(l, s.ws, stream);
  if (e != hipSuccess) return e;
  return over_tiles(s.a, tiling_of(l, s.ws), kLanes * Raw<F32>::V, [&](uint32_t grid, const Tiling &t) {
    scan_forward_kernel<F32, RESET, FLOOR, PART><<<grid, 256, 0, stream>>>(s.a, t);
  });
}

template <bool F32, bool RESET, bool FLOOR, bool PART>
hipError_t backward_tiles(const ScanLaunch &s, const Layout &l, float *floors, hipStream_t stream) {
  const hipError_t e = clear_words(l, s.ws, stream);
  if (e != hipSuccess) return e;
  return over_tiles(s.a, tiling_of(l, s.ws), kLanes * Raw<F32>::V, [&](uint32_t grid, const Tiling &t) {
    scan_backward_kernel<F32, RESET, FLOOR, PART><<<grid, 256, 0, stream>>>(s, t, floors);
  });
}

template <bool F32>
hipError_t run_forward(const ScanLaunch &s, hipStream_t stream) {
  constexpr int V = Raw<F32>::V;
  const nvfp4_scan_args &a = s.a;
  const bool few = a.chan < V;   // fewer channels than one access covers
  if (a.time <= kShort) {   // (threads of whole accesses: where channels are left over, all in parts)
    const int64_t threads = a.batch * ((a.chan + V - 1) / V);
    const uint32_t grid = at_most((threads + 63) / 64, 64 * kCus);
    if (a.chan % V) scan_forward_short_kernel<F32, true><<<grid, 64, 0, stream>>>(a, threads);
    else scan_forward_short_kernel<F32, false><<<grid, 64, 0, stream>>>(a, threads);
    return hipGetLastError();
  }
  const Layout l = layout_of(a.batch, a.time, a.chan, kLanes * V, false);
  if (few) return forward_tiles<F32, true, true, true>(s, l, stream);
  if (a.reset)
    return a.floor ? forward_tiles<F32, true, true, false>(s, l, stream)
                   : forward_tiles<F32, true, false, false>(s, l, stream);
  return a.floor ? forward_tiles<F32, false, true, false>(s, l, stream)
                 : forward_tiles<F32, false, false, false>(s, l, stream);
}

template <bool F32>
hipError_t run_backward(const ScanLaunch &s, hipStream_t stream) {
  constexpr int V = Raw<F32>::V;
  const nvfp4_scan_args &a = s.a;
  const bool few = a.chan < V;
  const Layout l = layout_of(a.batch, a.time, a.chan, kLanes * V, true);
  float *floors = reinterpret_cast<float *>(static_cast<char *>(s.ws) + l.floors);
  hipError_t e = hipSuccess;
  if (a.batch > 0) {
    if (a.time <= kShort) {
      const int64_t threads = a.batch * ((a.chan + V - 1) / V);
      const uint32_t grid = at_most((threads + 63) / 64, 64 * kCus);
      float *sums = a.time && s.d.dfloor ? floors : nullptr;   // (no steps: no workspace)
      if (a.chan % V) scan_backward_short_kernel<F32, true><<<grid, 64, 0, stream>>>(s, threads, sums);
      else scan_backward_short_kernel<F32, false><<<grid, 64, 0, stream>>>(s, threads, sums);
      e = hipGetLastError();
    } else if (few) {
      e = backward_tiles<F32, true, true, true>(s, l, floors, stream);
    } else if (a.reset) {
      e = a.floor ? backward_tiles<F32, true, true, false>(s, l, floors, stream)
                  : backward_tiles<F32, true, false, false>(s, l, floors, stream);
    } else {
      e = a.floor ? backward_tiles<F32, false, true, false>(s, l, floors, stream)
                  : backward_tiles<F32, false, false, false>(s, l, floors, stream);
    }
    if (e != hipSuccess) return e;
  }
  if (!s.d.dfloor) return e;
  const int64_t rows = a.time ? a.batch * l.chunks : 0;
  scan_floor_kernel<<<(uint32_t)((a.chan + 31) / 32), 1024, 0, stream>>>(floors, rows, a.chan, s.d.dfloor);
  return hipGetLastError();
}

}  // namespace

size_t scan_workspace_bytes(int64_t batch, int64_t time, int64_t chan, bool backward) {
  const size_t a = layout_of(batch, time, chan, kLanes * Raw<false>::V, backward).bytes;
  const size_t b = layout_of(batch, time, chan, kLanes * Raw<true>::V, backward).bytes;
  return a > b ? a : b;   // (of either type)
}

hipError_t launch_scan_forward(const ScanLaunch &s, hipStream_t stream) {
  return s.a.dtype == NVFP4_DT_FP32 ? run_forward<true>(s, stream) : run_forward<false>(s, stream);
}

hipError_t launch_scan_backward(const ScanLaunch &s, hipStream_t stream) {
  return s.a.dtype == NVFP4_DT_FP32 ? run_backward<true>(s, stream) : run_backward<false>(s, stream);
}

}  // namespace nvfp4

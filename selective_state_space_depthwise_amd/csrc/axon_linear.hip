// Gated linear recurrence: one state a channel (see axonscan.h).
//
//   h_t = a_t h_{t-1} + m_t u_t,   log a_t = -exp(A_log) dt_t,   dt = sigmoid or softplus of a gate
//
// Backward, with k the gradient that a token hands to the one before it (dstate_out behind the last):
//   g_t = dy_t + k_{t+1},  k_t = a_t g_t
//   G_t = g_t (a_t L_t h_{t-1} + u_t L_t dm/dL),  L = log a:   sqrt: dm/dL = -a^2 / m, complement: -a
//   dA_log = sum G;  ddt_raw = G (1 - sigmoid) or G sigmoid / softplus;  du = g m.
// L dm/dL = -a^2 L / m stays bounded where m goes to zero (m^2 = 1 - a^2 is about -2 L there), which
// dm/dL does not: only the product is formed.
//
// One pass over the data. A workgroup takes a tile (192 tokens forward, 64 backward, of the block tables) of 64
// channels, a lane a channel, a wave 8 or 16 of its tokens in registers: a wave finds its decay and own part, the
// waves are joined in LDS, and tiles hand on what leaves them in the order in which workgroups start (below). Only
// then are the states found and stored, so that every value is read and written once.
//
// Bound by memory and by latency: rows of 128 bytes, four streams in and three out, reach 4.6 to 4.8 TB/s by themselves
// in this order of workgroups (5.5 where each die takes the same neighbouring groups of every tile, which made the
// kernels no faster), and a wave does not load while it computes. 16384 x 2560 bf16 (336 MB) 84-92 us, fp32 127 us;
// packed 32768 x 2560 159-168 us; training of 8 x 2048 x 2560 (336 + 587 MB) 242 us; backward of 16384 x 2560 fp32
// (1.17 GB) 207-230 us. From the first kernel, one channel
// of a sequence a lane, of 16384 tokens 21.7 ms. What it took: tiles that hand on; 12 waves of 16 tokens; gates,
// input scale and what is gated as template arguments, since loads behind branches are waited for at once (101 ->
// 90 us); plain decays inside a wave; rows at a scalar offset; stores past the caches. Tried and dropped: two channels
// a lane, persistent workgroups (117 us; that ask for the next tile's rows early 122-193 us), eight tokens a wave.
#include <hip/hip_runtime.h>

#include <cmath>
#include <cstdint>
#include <type_traits>

#include "axon_device.h"
#include "axon_packed.h"
#include "axon_wide.h"

namespace axon {
namespace {

struct LinearArgs {
  const void *x, *dt_raw, *in_raw, *dy;
  const float *A_log, *dt_bias, *in_bias;
  Packed p;
  int64_t x_stride, dt_stride, in_stride, dy_stride;
  int channels, gate, input_scale, clear_behind;
  bool past;      // y and the gradients are stored past the caches
  bool together;  // all waves of a tile look at the tiles in front
  int tiles, groups;  // tiles of blocks, groups of 64 channels
  // scan, step
  const float* state_in;
  const int32_t *in_slots, *out_slots;
  int64_t in_count, out_count;
  float *state_out, *checkpoints;
  void* y;
  // backward
  const float *points, *dstate_out;
  void *dx, *ddt_raw, *din_raw;
  float *dA_log, *ddt_bias, *din_bias, *dstate_in;
  float* partial;  // (tiles, 3, channels)
  // What tiles tell each other (tiles, 64 groups): all bits set where nothing is told yet.
  uint32_t* ticket;  // null: one tile
  uint64_t* sums;    // decay over a tile, and its own part
  uint32_t* carry;   // what leaves it
};

// Gates take v = raw + bias, added before it is scaled: a bias scaled by itself would be rounded at its own size, which
// counts where the two cancel (raw of -4000, bias of 4000: 2840 2^-24 of the gate).
__device__ __forceinline__ float sigmoid_f32(float v) {
  return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(v * -kLog2e));
}

// sigmoid(v) and 1 - sigmoid(v), each with a relative error of (3 |v| + 8) 2^-24 at most (the roundings of v, of
// log2 e and of their product in the exponent; exponential, sum, reciprocal and product); the first is no less
// than 2^-126.
struct Gate {
  float on, off;
  __device__ __forceinline__ explicit Gate(float v) {
    const float x = __builtin_amdgcn_exp2f(v * -kLog2e);
    const float e = __builtin_elementwise_minimum(x, 8.5e37f);  // keeps NaN
    on = __builtin_amdgcn_rcpf(1.0f + e);
    off = e * on;
  }
};
// softplus, NaN kept.
__device__ __forceinline__ float softplus_nan(float v) { return v != v ? v : softplus_f32(v); }

// expm1(log a) from log2 a (<= 0) and a. Below log2 a = -0.36, a - 1 cancels two bits at most; above it
// the series up to (log a)^6 / 720 leaves a relative 5e-8.
__device__ __forceinline__ float expm1_of(float l2, float a) {
  float p = fmaf(l2, 1.54035304e-4f, 1.33335581e-3f);
  p = fmaf(l2, p, 9.61812911e-3f);
  p = fmaf(l2, p, 5.55041087e-2f);
  p = fmaf(l2, p, 2.40226507e-1f);
  p = fmaf(l2, p, 6.93147181e-1f) * l2;
  return l2 > -0.36f ? p : a - 1.0f;
}

// A state over several tokens, from the sum of their log2 a and their own part: a h + part. Rounding a
// close to 1 would be the same error for every block of a slow channel, 2^-24 against 1 - a, so that for
// a >= 1/2 it is h + expm1(log a) h; below, that would lose the part beside a larger h. Whatever outlives
// a wave's tokens goes this way: what waves and tiles hand on, from the state that a sequence begins with to
// the one that it hands back (and so for its gradients), else scans of a few tokens that continue one another
// would lose the decay (300 of 16 tokens at log a = -1e-6 to -1e-7: nine roundings of the state a call, now
// one). Only the outputs in between multiply by the plain a, up to 16 times from what entered the wave: off by
// 32 2^-24 of h at most, which ends with the wave. `carry` holds a, or expm1(log a) with the sign bit set.
__device__ __forceinline__ float carry_of(float l2) {
  const float a = __builtin_amdgcn_exp2f(l2);
  return l2 < -1.0f ? a : __uint_as_float(__float_as_uint(expm1_of(l2, a)) | 0x80000000u);
}
__device__ __forceinline__ float advance(float carry, float h, float part) {
  return fmaf(carry, h, part) + (__float_as_int(carry) < 0 ? h : 0.0f);
}

// m from log2 a and a.
template <int SCALE>
__device__ __forceinline__ float input_factor(float l2, float a) {
  if constexpr (SCALE == AXON_INPUT_PLAIN) return 1.0f;
  const float em1 = expm1_of(l2, a);
  if constexpr (SCALE == AXON_INPUT_COMPLEMENT) return -em1;
  return __builtin_amdgcn_sqrtf(-em1 * (2.0f + em1));
}

// log2 a; rate: -exp(A_log) log2 e.
template <int GATE>
__device__ __forceinline__ float log2_decay(float rate, float raw, float bias) {
  if constexpr (GATE == AXON_LINEAR_SIGMOID) return rate * sigmoid_f32(raw + bias);
  return rate * softplus_nan(raw + bias);
}

// A wave's share of a tile: P tokens of one block, a channel a lane.
struct Share {
  int seq, first, count;   // count 0: none; rows first .. first + count - 1
  int row;                 // of the block tables
  bool begins, ends;       // holds the sequence's first / last token
  bool opens;              // holds the block's first token
};

template <int P, int WAVES>
__device__ __forceinline__ Share share_of(const Packed& p, int tile, int wave) {
  const int at = (tile * WAVES + wave) * P;  // tokens in front, were all blocks full
  Share s{};
  s.row = at / kBlock;
  const int sub = at - s.row * kBlock;
  const BlockAt b = block_at(p, s.row);
  s.seq = b.seq;
  s.first = b.first + sub;
  s.count = b.seq < 0 ? 0 : min(max(b.count - sub, 0), P);
  s.opens = s.count > 0 && sub == 0;
  s.begins = s.opens && b.begins;
  s.ends = s.count > 0 && b.ends && sub + s.count == b.count;
  return s;
}

// A channel's parameters, asked for before the rows so that nothing waits for them alone.
template <bool GATED>
struct Channel {
  float A_log, dt_bias, in_bias = 0.0f;
  __device__ __forceinline__ Channel(const LinearArgs& g, int e) {
    A_log = g.A_log[e];
    dt_bias = (g.dt_bias ? g.dt_bias : g.A_log)[e];
    if constexpr (GATED) in_bias = (g.in_bias ? g.in_bias : g.A_log)[e];
    if (!g.dt_bias) dt_bias = 0.0f;
    if (!g.in_bias) in_bias = 0.0f;
  }
  __device__ __forceinline__ float rate() const { return -expf(A_log) * kLog2e; }
};

// P rows of a wave as loaded; rows behind the last repeat it.
template <typename Act, int P>
struct Rows {
  typename RawOf<Act>::type v[P];
  __device__ __forceinline__ void load(const void* base, int64_t stride, const Share& s, int e) {
    const rsrc_t r = make_rsrc(static_cast<const Act*>(base) + s.first * stride);
    const uint32_t step = static_cast<uint32_t>(stride) * sizeof(Act), off = e * sizeof(Act);
#pragma unroll
    for (int j = 0; j < P; ++j) {
      const uint32_t row = static_cast<uint32_t>(min(j, s.count - 1)) * step;
      if constexpr (sizeof(Act) == 4) v[j] = __builtin_amdgcn_raw_buffer_load_b32(r, off, row, 0);
      else v[j] = __builtin_amdgcn_raw_buffer_load_b16(r, off, row, 0);
    }
  }
  __device__ __forceinline__ float operator[](int j) const { return widen(v[j]); }
};

// A value of the row at the scalar offset `row`; PAST: not kept in the caches (past_caches).
template <bool PAST>
__device__ __forceinline__ void store_row(const float*, rsrc_t r, uint32_t off, uint32_t row, float v) {
  __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(v), r, off, row, PAST ? 2 : 0);
}
template <bool PAST>
__device__ __forceinline__ void store_row(const bf16_bits*, rsrc_t r, uint32_t off, uint32_t row, float v) {
  __builtin_amdgcn_raw_buffer_store_b16(f32_to_bf16(v), r, off, row, PAST ? 2 : 0);
}
using Past = std::true_type;
using Kept = std::false_type;

// ---- What tiles tell each other -----------------------------------------------------------------
// A tile first publishes its own part (its decay, as for advance, and h from zero), then, once it knows what
// enters it, what leaves it. A reader takes the nearest tile that has published the latter and applies
// the parts between in the order in which those tiles do it themselves, so that the result does not
// depend on who was first. Both are one atomic of the value itself: a NaN with all bits set stands for
// nothing, and stored NaNs are others.
__device__ __forceinline__ uint32_t told(float v) {
  return v != v ? 0x7FC00000u : __float_as_uint(v);
}
__device__ __forceinline__ void tell_part(uint64_t* p, float decay, float h) {
  __hip_atomic_store(p, static_cast<uint64_t>(told(h)) << 32 | told(decay), __ATOMIC_RELAXED,
                     __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ void tell_carry(uint32_t* p, float h) {
  __hip_atomic_store(p, told(h), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
constexpr int kWindow = 2;  // tiles looked at

// Waits for what tile `from` hands on; tiles go down from it (DIR -1) or up (DIR 1), `left` of them.
// `column`: of the lane, among the `columns` of a tile. Every tile's workgroup has started once a later
// ticket is out, and none of them waits for a later one, so that the wait ends. (Two calls at once in one
// workspace, which no caller may make, could wipe what was told: the wait is given up after seconds, as NaN.)
constexpr int kPatience = 1 << 22;
template <int DIR>
__device__ __forceinline__ float hear(const LinearArgs& g, int from, int left, int64_t columns,
                                      int64_t column) {
  const int n = min(left, kWindow);
  for (int looks = 0; looks < kPatience; ++looks) {
    uint32_t c[kWindow];
    uint64_t s[kWindow];
#pragma unroll
    for (int k = 0; k < kWindow; ++k) {
      const int64_t at = (from + DIR * min(k, n - 1)) * columns + column;
      c[k] = __hip_atomic_load(g.carry + at, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      s[k] = __hip_atomic_load(g.sums + at, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
    int found = -1;
    bool between = true;  // all sums up to here are told
#pragma unroll
    for (int k = 0; k < kWindow; ++k) {
      if (found < 0 && k < n && between) {
        if (__all(c[k] != ~0u)) found = k;
        else between = __all(s[k] != ~uint64_t(0));
      }
    }
    if (found >= 0) {
      float h = 0.0f;
#pragma unroll
      for (int k = kWindow - 1; k >= 0; --k) {
        if (k == found) h = __uint_as_float(c[k]);
        else if (k < found)
          h = advance(__uint_as_float(static_cast<uint32_t>(s[k])), h,
                      __uint_as_float(static_cast<uint32_t>(s[k] >> 32)));
      }
      return h;
    }
    __builtin_amdgcn_s_sleep(2);
  }
  return __builtin_nanf("");
}

__global__ __launch_bounds__(256) void linear_clear_kernel(uint4* p, int64_t count) {
  const int64_t step = int64_t(gridDim.x) * 256;
  for (int64_t i = int64_t(blockIdx.x) * 256 + threadIdx.x; i < count; i += step)
    p[i] = make_uint4(~0u, ~0u, ~0u, ~0u);
}

// All loads so far have come. They have been used where they were asked for, but not on every path that the compiler
// sees, and what it takes for open it waits for between the stores (training of 8 x 2048 x 2560 bf16 259 us, with this
// 242 us; packed 32768 x 2560 forward 160 us, 158.6 us).
__device__ __forceinline__ void loads_done() { __builtin_amdgcn_s_waitcnt(0x0F70); }  // vmcnt(0) alone

// What a tile's waves leave for each other, a channel a lane.
template <int WAVES>
struct Parts {
  float logs[WAVES][64], decay[WAVES][64], part[WAVES][64], enter[64];
  int fresh[WAVES];  // nothing from in front (behind, backwards) reaches the wave's end

  __device__ __forceinline__ void put(int wave, int lane, float log, float own, bool starts) {
    logs[wave][lane] = log;
    decay[wave][lane] = carry_of(log);
    part[wave][lane] = own;
    if (lane == 0) fresh[wave] = starts;
  }
};

// The tile's waves in front of a wave (behind it for DIR 1): their decay and own part.
template <int DIR, int WAVES>
struct Front {
  float log = 0.0f, part = 0.0f;
  bool closed = false;  // a sequence begins (ends) among them
  __device__ __forceinline__ Front(const Parts<WAVES>& sh, int wave, int lane) {
    for (int w = DIR < 0 ? 0 : WAVES - 1; w != wave; w -= DIR) {
      const bool f = sh.fresh[w];
      part = f ? sh.part[w][lane] : advance(sh.decay[w][lane], part, sh.part[w][lane]);
      log += sh.logs[w][lane];
      closed |= f;
    }
  }
  __device__ __forceinline__ float enter(float h) const {
    return closed ? part : advance(carry_of(log), h, part);
  }
};

// Tiles looked at by each wave, where all do: with four waves three of them (131072 tokens x 64 bf16 backward
// 229 us, two 302 us; four cost registers, 16384 x 2560 157 -> 165 us).
template <int WAVES>
constexpr int kLook = WAVES == 4 ? 3 : 2;
// What all waves of a tile have read for each other.
template <int WAVES>
struct Look {
  uint32_t carry[kLook<WAVES> * WAVES][64];
  uint64_t sums[kLook<WAVES> * WAVES][64];
  int told[kLook<WAVES> * WAVES];  // bit 0: the carry, bit 1: the sums
};

// As hear, by all waves of a tile.
template <int DIR, int WAVES>
__device__ __forceinline__ float hear_all(const LinearArgs& g, Look<WAVES>& look, int wave, int lane, int from,
                                          int left, int64_t columns, int64_t column) {
  const int n = min(left, kLook<WAVES> * WAVES);
  for (int looks = 0; looks < kPatience; ++looks) {
#pragma unroll
    for (int i = 0; i < kLook<WAVES>; ++i) {
      const int k = wave * kLook<WAVES> + i;
      const int64_t at = (from + DIR * min(k, n - 1)) * columns + column;
      const uint32_t c = __hip_atomic_load(g.carry + at, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      const uint64_t s = __hip_atomic_load(g.sums + at, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      look.carry[k][lane] = c;
      look.sums[k][lane] = s;
      const int told = (__all(c != ~0u) ? 1 : 0) | (__all(s != ~uint64_t(0)) ? 2 : 0);
      if (lane == 0) look.told[k] = told;
    }
    __syncthreads();
    const int told = lane < n ? look.told[lane] : 0;
    const uint64_t carries = __ballot(told & 1), sums = __ballot(told & 2);
    const int found = carries ? __builtin_ctzll(carries) : -1;
    if (found >= 0 && (~sums & ((uint64_t(1) << found) - 1)) == 0) {
      float h = __uint_as_float(look.carry[found][lane]);
#pragma unroll 8
      for (int k = found - 1; k >= 0; --k) {
        const uint64_t s = look.sums[k][lane];
        h = advance(__uint_as_float(static_cast<uint32_t>(s)), h, __uint_as_float(static_cast<uint32_t>(s >> 32)));
      }
      return h;
    }
    __syncthreads();
    __builtin_amdgcn_s_sleep(2);
  }
  return __builtin_nanf("");
}

// The tile's own part is told, and what enters it is found, by the wave that it enters first; where channels
// are few by all waves, since then the chain of tiles is what takes the time. left as for hear.
template <int DIR, int WAVES>
__device__ __forceinline__ void exchange(const LinearArgs& g, Parts<WAVES>& sh, Look<WAVES>& look, int wave,
                                         int lane, int tile, int grp, int left) {
  constexpr int kFirst = DIR < 0 ? 0 : WAVES - 1;
  if (wave != kFirst && !g.together) return;
  float sum = 0.0f, own = 0.0f;
  bool closed = false;  // a sequence begins (ends) in the tile: nothing passes through it
#pragma unroll
  for (int n = 0; n < WAVES; ++n) {
    const int w = DIR < 0 ? n : WAVES - 1 - n;
    const bool f = sh.fresh[w];
    own = f ? sh.part[w][lane] : advance(sh.decay[w][lane], own, sh.part[w][lane]);
    sum += sh.logs[w][lane];
    closed |= f;
  }
  float before = 0.0f;
  if (g.ticket) {
    const bool alone = left == 0 || sh.fresh[kFirst];  // nothing enters
    const int64_t columns = int64_t(g.groups) * 64, column = int64_t(grp) * 64 + lane;
    const int64_t at = tile * columns + column;
    const float decay = carry_of(sum);
    if (wave == kFirst) {
      if (closed || alone) tell_carry(g.carry + at, own);
      else tell_part(g.sums + at, decay, own);
    }
    if (!alone) {
      before = g.together ? hear_all<DIR>(g, look, wave, lane, tile + DIR, left, columns, column)
                          : hear<DIR>(g, tile + DIR, left, columns, column);
      if (wave == kFirst && !closed) tell_carry(g.carry + at, advance(decay, before, own));
    }
  }
  if (wave == kFirst) sh.enter[lane] = before;
}

// The unit (tile and channel group) of this workgroup: in the order in which workgroups start.
__device__ __forceinline__ uint32_t take_ticket(const LinearArgs& g, uint32_t* shared) {
  if (!g.ticket) return blockIdx.x;
  if (threadIdx.x == 0)
    *shared = 1 + __hip_atomic_fetch_add(g.ticket, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  __syncthreads();
  return __builtin_amdgcn_readfirstlane(*shared);
}

// ---- The scan -----------------------------------------------------------------------------------
// Waves to a workgroup and registers are chosen for 24 waves a CU.
template <typename Act, int P, int WAVES, int GATE, int SCALE, bool GATED>
__global__ __launch_bounds__(64 * WAVES, 6) void linear_tile_kernel(LinearArgs g) {
  __shared__ uint32_t ticket;
  __shared__ Parts<WAVES> sh;
  __shared__ Look<WAVES> look;
  const uint32_t t = take_ticket(g, &ticket);
  const int tile = t / g.groups, grp = t - tile * g.groups;
  if (static_cast<uint32_t>(tile) >= static_cast<uint32_t>(g.tiles)) return;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const bool in_range = grp * 64 + lane < g.channels;
  const int e = min(grp * 64 + lane, g.channels - 1);
  const Channel<GATED> channel(g, e);
  const Share s = share_of<P, WAVES>(g.p, tile, wave);
  float a[P], b[P];
  float h0 = 0.0f;  // what enters the wave, where it begins a sequence
  float L = 0.0f, h = 0.0f;
  if (s.count > 0) {
    Rows<Act, P> x, raw, in;
    raw.load(g.dt_raw, g.dt_stride, s, e);
    x.load(g.x, g.x_stride, s, e);
    if constexpr (GATED) in.load(g.in_raw, g.in_stride, s, e);
    if (s.begins && g.state_in) {
      const int64_t slot = g.in_slots ? table_at(g.in_slots, s.seq) : s.seq;
      if (slot >= 0 && slot < g.in_count) h0 = g.state_in[slot * g.channels + e];
    }
    const float rate = channel.rate(), bias = channel.dt_bias, ib = channel.in_bias;
    // a: log2 a first
#pragma unroll
    for (int j = 0; j < P; ++j) a[j] = log2_decay<GATE>(rate, raw[j], bias);
    if (s.count < P) {
#pragma unroll
      for (int j = 0; j < P; ++j)
        if (j >= s.count) a[j] = 0.0f;
    }
#pragma unroll
    for (int j = 0; j < P; ++j) {
      const float l2 = a[j];
      L += l2;
      a[j] = __builtin_amdgcn_exp2f(l2);
      b[j] = x[j] * input_factor<SCALE>(l2, a[j]);
    }
    if constexpr (GATED) {
#pragma unroll
      for (int j = 0; j < P; ++j) b[j] *= sigmoid_f32(in[j] + ib);
    }
    if (s.count < P) {
#pragma unroll
      for (int j = 0; j < P; ++j)
        if (j >= s.count) b[j] = 0.0f;
    }
#pragma unroll
    for (int j = 0; j < P; ++j) h = fmaf(a[j], h, b[j]);
    if (s.begins) h = advance(carry_of(L), h0, h);
  }
  loads_done();
  sh.put(wave, lane, L, h, s.begins);
  __syncthreads();
  exchange<-1, WAVES>(g, sh, look, wave, lane, tile, grp, tile);
  const Front<-1, WAVES> front(sh, wave, lane);
  __syncthreads();
  if (s.count > 0) {
    h = s.begins ? h0 : front.enter(sh.enter[lane]);
    const float enters = h;
    const int plain = s.count - (s.ends ? 1 : 0);  // tokens whose output is the plain product
    if (in_range) {
      if (s.opens && g.checkpoints) g.checkpoints[int64_t(s.row) * g.channels + e] = h;
      const rsrc_t y = make_rsrc(static_cast<Act*>(g.y) + int64_t(s.first) * g.channels);
      const uint32_t step = static_cast<uint32_t>(g.channels) * sizeof(Act), off = e * sizeof(Act);
      auto states = [&](auto past) {
#pragma unroll
        for (int j = 0; j < P; ++j) {
          h = fmaf(a[j], h, b[j]);
          if (j < plain) store_row<decltype(past)::value>(static_cast<Act*>(nullptr), y, off, j * step, h);
        }
      };
      if (g.past) states(Past{});
      else states(Kept{});
      if (s.ends) {
        // the final state is the last output too
        const float own = sh.part[wave][lane], last = s.begins ? own : advance(sh.decay[wave][lane], enters, own);
        store_row<false>(static_cast<Act*>(nullptr), y, off, (s.count - 1) * step, last);
        const int64_t slot = g.out_slots ? table_at(g.out_slots, s.seq) : s.seq;
        if (g.state_out && slot >= 0 && slot < g.out_count) g.state_out[slot * g.channels + e] = last;
      }
    }
  }
  if (!in_range) return;
  // Sequences without tokens, and rows behind the last one: shared out to the tiles' waves.
  for (int n = tile * WAVES + wave; n < g.p.sequences; n += g.tiles * WAVES) {
    if (!g.state_out || packed_start(g.p, n) < packed_start(g.p, n + 1)) continue;
    const int64_t from = g.in_slots ? table_at(g.in_slots, n) : n;
    const int64_t to = g.out_slots ? table_at(g.out_slots, n) : n;
    if (to >= 0 && to < g.out_count)
      g.state_out[to * g.channels + e] =
          g.state_in && from >= 0 && from < g.in_count ? g.state_in[from * g.channels + e] : 0.0f;
  }
  if (g.clear_behind)
    for (int64_t r = int64_t(packed_start(g.p, g.p.sequences)) + tile * WAVES + wave; r < g.p.tokens;
         r += int64_t(g.tiles) * WAVES)
      store_act(static_cast<Act*>(g.y), r * g.channels + e, 0.0f);
}

// ---- Its backward pass --------------------------------------------------------------------------
// The same from the last tile to the first. A wave finds its block's states again from the block's
// checkpoint and the parts of the waves in front of it.
template <typename Act, int P, int WAVES, int GATE, int SCALE, bool GATED>
__global__ __launch_bounds__(64 * WAVES, WAVES == 4 ? 3 : 5) void linear_tile_back_kernel(LinearArgs g) {
  static_assert(WAVES * P % kBlock == 0, "a tile holds whole blocks");
  constexpr int kBlockWaves = kBlock / P;
  __shared__ uint32_t ticket;
  __shared__ Parts<WAVES> sh;
  __shared__ Look<WAVES> look;
  __shared__ float states[WAVES][64], totals[WAVES][3][64];
  const uint32_t t = take_ticket(g, &ticket);
  const int turn = t / g.groups, grp = t - turn * g.groups;
  if (static_cast<uint32_t>(turn) >= static_cast<uint32_t>(g.tiles)) return;
  const int tile = g.tiles - 1 - turn;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const bool in_range = grp * 64 + lane < g.channels;
  const int e = min(grp * 64 + lane, g.channels - 1);
  const Channel<GATED> channel(g, e);
  const Share s = share_of<P, WAVES>(g.p, tile, wave);
  // Per token: a, what the gate's slope makes of G, m times the input's gate, m u (1 - gate), dy. G is
  // g (aL h - w): first aL, w and the inputs m u, then, once the states are known, aL h - w in their place.
  float av[P], slope[P], mo[P], mz[P], dy[P], aL[P], w[P], hb[P];
  float L = 0.0f, h = 0.0f, k = 0.0f, k0 = 0.0f, point = 0.0f;
  if (s.count > 0) {
    Rows<Act, P> x, raw, in, d;
    raw.load(g.dt_raw, g.dt_stride, s, e);
    x.load(g.x, g.x_stride, s, e);
    if constexpr (GATED) in.load(g.in_raw, g.in_stride, s, e);
    d.load(g.dy, g.dy_stride, s, e);
    if (s.opens) point = g.points[int64_t(s.row) * g.channels + e];
    if (s.ends && g.dstate_out) k0 = g.dstate_out[int64_t(s.seq) * g.channels + e];
    const float rate = channel.rate(), bias = channel.dt_bias, ib = channel.in_bias;
    // mo: the input's gate, mz: u (1 - gate), hb: u at first
    if constexpr (GATED) {
#pragma unroll
      for (int j = 0; j < P; ++j) {
        const Gate q(in[j] + ib);
        mo[j] = q.on;
        hb[j] = x[j] * q.on;
        mz[j] = hb[j] * q.off;
      }
    } else {
#pragma unroll
      for (int j = 0; j < P; ++j) mo[j] = 1.0f, hb[j] = x[j], mz[j] = 0.0f;
    }
    h = point;
#pragma unroll
    for (int j = 0; j < P; ++j) {
      const bool held = j < s.count;
      float l2;
      if constexpr (GATE == AXON_LINEAR_SIGMOID) {
        const Gate q(raw[j] + bias);
        l2 = rate * q.on;
        slope[j] = q.off;
      } else {
        const float v = raw[j] + bias, sp = softplus_nan(v);
        l2 = rate * sp;
        slope[j] = v < -20.0f ? 1.0f : sigmoid_f32(v) * __builtin_amdgcn_rcpf(sp);
      }
      l2 = held ? l2 : 0.0f;
      L += l2;
      const float u = held ? hb[j] : 0.0f;
      av[j] = __builtin_amdgcn_exp2f(l2);
      aL[j] = av[j] * (fmaxf(l2, -200.0f) * kLn2);  // 0 for log a = -inf
      float m = 1.0f;
      w[j] = 0.0f;
      if constexpr (SCALE == AXON_INPUT_SQRT) {
        // m = sqrt(q) and 1 / m, of q 2^64 so that the least q keep their root
        const float em1 = expm1_of(l2, av[j]), q = -em1 * (2.0f + em1), big = q * 0x1p64f;
        const float rm = big == 0.0f ? 0.0f : __builtin_amdgcn_rsqf(big) * 0x1p32f;
        m = q * rm;
        w[j] = aL[j] * (av[j] * u * rm);
      } else if constexpr (SCALE == AXON_INPUT_COMPLEMENT) {
        m = -expm1_of(l2, av[j]);
        w[j] = aL[j] * u;
      }
      mo[j] *= m;
      mz[j] *= m;
      hb[j] = m * u;
      dy[j] = held ? d[j] : 0.0f;
      h = fmaf(av[j], h, hb[j]);
    }
#pragma unroll
    for (int j = P - 1; j >= 0; --j) k = av[j] * (k + dy[j]);
  }
  if (s.ends) k = advance(carry_of(L), k0, k);
  loads_done();
  sh.put(wave, lane, L, k, s.ends);
  states[wave][lane] = h;
  __syncthreads();
  exchange<1, WAVES>(g, sh, look, wave, lane, tile, grp, turn);
  // The states in front of the wave's tokens.
  if (s.count > 0) {
    const int w0 = wave / kBlockWaves * kBlockWaves;
    h = s.opens ? point : states[w0][lane];
    for (int n = w0 + 1; n < wave; ++n) h = advance(sh.decay[n][lane], h, states[n][lane]);
#pragma unroll
    for (int j = 0; j < P; ++j) {
      w[j] = fmaf(aL[j], h, -w[j]);
      h = fmaf(av[j], h, hb[j]);
    }
  }
  const Front<1, WAVES> behind(sh, wave, lane);
  __syncthreads();
  float sA = 0.0f, sdt = 0.0f, sin = 0.0f;
  if (s.count > 0) {
    k = s.ends ? k0 : behind.enter(sh.enter[lane]);
    const float enters = k;
    const int64_t first = int64_t(s.first) * g.channels;
    const rsrc_t dx = make_rsrc(static_cast<Act*>(g.dx) + first);
    const rsrc_t ddt = make_rsrc(static_cast<Act*>(g.ddt_raw) + first);
    const rsrc_t din = make_rsrc(static_cast<Act*>(g.din_raw) + (GATED ? first : 0));
    const uint32_t step = static_cast<uint32_t>(g.channels) * sizeof(Act), off = e * sizeof(Act);
    auto grads = [&](auto past) {
      constexpr Act* kType = nullptr;
      constexpr bool kPast = decltype(past)::value;
#pragma unroll
      for (int j = P - 1; j >= 0; --j) {
        if (j >= s.count) continue;
        const float gt = dy[j] + k;
        k = av[j] * gt;
        const float G = gt * w[j], odt = G * slope[j], oin = gt * mz[j];
        sA += G;
        sdt += odt;
        sin += oin;
        store_row<kPast>(kType, ddt, off, j * step, odt);
        store_row<kPast>(kType, dx, off, j * step, gt * mo[j]);
        if constexpr (GATED) store_row<kPast>(kType, din, off, j * step, oin);
      }
    };
    if (in_range) {
      if (g.past) grads(Past{});
      else grads(Kept{});
    }
    if (s.begins && g.dstate_in && in_range)
      g.dstate_in[int64_t(s.seq) * g.channels + e] =
          s.ends ? sh.part[wave][lane] : advance(sh.decay[wave][lane], enters, sh.part[wave][lane]);
  }
  totals[wave][0][lane] = sA;
  totals[wave][1][lane] = sdt;
  totals[wave][2][lane] = sin;
  __syncthreads();
  if (!in_range) return;
  for (int q = wave; q < 3; q += WAVES) {
    float sum = 0.0f;
#pragma unroll
    for (int n = 0; n < WAVES; ++n) sum += totals[n][q][lane];
    g.partial[(int64_t(tile) * 3 + q) * g.channels + e] = sum;
  }
  if (g.dstate_in)
    for (int n = tile * WAVES + wave; n < g.p.sequences; n += g.tiles * WAVES) {
      if (packed_start(g.p, n) < packed_start(g.p, n + 1)) continue;
      const int64_t at = int64_t(n) * g.channels + e;
      g.dstate_in[at] = g.dstate_out ? g.dstate_out[at] : 0.0f;
    }
  for (int64_t r = int64_t(packed_start(g.p, g.p.sequences)) + tile * WAVES + wave; r < g.p.tokens;
       r += int64_t(g.tiles) * WAVES) {
    const int64_t at = r * g.channels + e;
    store_act(static_cast<Act*>(g.dx), at, 0.0f);
    store_act(static_cast<Act*>(g.ddt_raw), at, 0.0f);
    if constexpr (GATED) store_act(static_cast<Act*>(g.din_raw), at, 0.0f);
  }
}

// Sums of the tiles' parts in 64 bits: a channel a lane, each wave takes every 16th tile.
constexpr int kSumWaves = 16;
__global__ __launch_bounds__(64 * kSumWaves) void linear_sum_kernel(LinearArgs g, int parts) {
  __shared__ double sums[kSumWaves][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int e = blockIdx.x * 64 + lane, which = blockIdx.y;
  double s = 0.0;
  if (e < g.channels) {
    const float* from = g.partial + int64_t(which) * g.channels + e;
#pragma unroll 8
    for (int j = wave; j < parts; j += kSumWaves) s += from[int64_t(j) * 3 * g.channels];
  }
  sums[wave][lane] = s;
  __syncthreads();
  if (wave || e >= g.channels) return;
#pragma unroll
  for (int w = 1; w < kSumWaves; ++w) s += sums[w][lane];
  float* out = which == 0 ? g.dA_log : which == 1 ? g.ddt_bias : g.din_bias;
  out[e] = static_cast<float>(s);
}

// V channels of a row a thread, all asked for before the first is used.
template <typename Act, int V>
__global__ __launch_bounds__(256) void linear_step_kernel(LinearArgs g) {
  const int e = (blockIdx.x * 256 + threadIdx.x) * V, n = blockIdx.y;
  if (e >= g.channels) return;
  const int64_t slot = g.in_slots ? g.in_slots[n] : n;
  if (slot < 0 || slot >= g.in_count) return;
  float* state = g.state_out + slot * g.channels + e;
  Raw<Act, V> x, raw, in;
  Raw<float, V> old, A_log, bias, in_bias;
  raw.load(static_cast<const Act*>(g.dt_raw) + n * g.dt_stride + e);
  x.load(static_cast<const Act*>(g.x) + n * g.x_stride + e);
  if (g.in_raw) in.load(static_cast<const Act*>(g.in_raw) + n * g.in_stride + e);
  old.load(state);
  A_log.load(g.A_log + e);
  if (g.dt_bias) bias.load(g.dt_bias + e);
  if (g.in_raw && g.in_bias) in_bias.load(g.in_bias + e);
  float u[V], v[V], i_raw[V], h[V], rate[V], b[V] = {}, ib[V] = {};
  x.get(u);
  raw.get(v);
  old.get(h);
  A_log.get(rate);
  if (g.in_raw) in.get(i_raw);
  if (g.dt_bias) bias.get(b);
  if (g.in_raw && g.in_bias) in_bias.get(ib);
#pragma unroll
  for (int i = 0; i < V; ++i) {
    rate[i] = -expf(rate[i]) * kLog2e;
    const float l2 = g.gate == AXON_LINEAR_SIGMOID
                         ? log2_decay<AXON_LINEAR_SIGMOID>(rate[i], v[i], b[i])
                         : log2_decay<AXON_LINEAR_SOFTPLUS>(rate[i], v[i], b[i]);
    const float a = __builtin_amdgcn_exp2f(l2);
    if (g.input_scale == AXON_INPUT_COMPLEMENT) u[i] *= input_factor<AXON_INPUT_COMPLEMENT>(l2, a);
    if (g.input_scale == AXON_INPUT_SQRT) u[i] *= input_factor<AXON_INPUT_SQRT>(l2, a);
    if (g.in_raw) u[i] *= sigmoid_f32(i_raw[i] + ib[i]);
    h[i] = advance(carry_of(l2), h[i], u[i]);
  }
  Raw<float, V>::template store<false>(state, h);
  Raw<Act, V>::template store<false>(static_cast<Act*>(g.y) + int64_t(n) * g.channels + e, h);
}

axon_status check_shape(const axon_linear_shape* s, bool backward) {
  if (!s) return AXON_ERR_INVALID_ARGUMENT;
  const int64_t strides[] = {s->x_stride, s->dt_stride, s->in_stride, s->dy_stride};
  const axon_status why =
      check_packed(s->sequences, s->tokens, s->channels, strides, backward ? 4 : 3, s->channels,
                   backward ? 0 : s->state_slots, backward ? 0 : s->out_slots, s->act_dtype);
  if (why != AXON_OK) return why;
  if ((s->gate != AXON_LINEAR_SIGMOID && s->gate != AXON_LINEAR_SOFTPLUS) ||
      (s->input_scale != AXON_INPUT_PLAIN && s->input_scale != AXON_INPUT_COMPLEMENT &&
       s->input_scale != AXON_INPUT_SQRT) ||
      (s->clear_behind != 0 && s->clear_behind != 1))
    return AXON_ERR_UNSUPPORTED;
  return AXON_OK;
}

bool bad(const void* p, size_t a) { return !p || !aligned_to(p, a); }
bool off(const void* p, size_t a) { return p && !aligned_to(p, a); }

axon_status check_params(const axon_linear_params* p, const void* in_raw) {
  if (!p || bad(p->A_log, 4) || off(p->dt_bias, 4) || (in_raw && off(p->in_bias, 4)))
    return AXON_ERR_INVALID_ARGUMENT;
  return AXON_OK;
}

LinearArgs make_args(const axon_linear_shape& s, const axon_linear_params& p, const void* x,
                     const void* dt_raw, const void* in_raw, const int32_t* tables) {
  LinearArgs a{};
  a.x = x, a.dt_raw = dt_raw, a.in_raw = in_raw;
  a.A_log = p.A_log, a.dt_bias = p.dt_bias, a.in_bias = p.in_bias;
  a.p = make_packed(s.sequences, s.tokens, tables);
  a.x_stride = s.x_stride ? s.x_stride : s.channels;
  a.dt_stride = s.dt_stride ? s.dt_stride : s.channels;
  a.in_stride = s.in_stride ? s.in_stride : s.channels;
  a.dy_stride = s.dy_stride ? s.dy_stride : s.channels;
  a.channels = static_cast<int>(s.channels);
  a.gate = s.gate, a.input_scale = s.input_scale, a.clear_behind = s.clear_behind;
  a.past = past_caches(size_t(s.tokens * s.channels) * (s.act_dtype == AXON_BF16 ? 2 : 4));
  return a;
}

// Byte ranges of the inputs that every form reads.
void input_spans(const LinearArgs& a, int64_t tokens, size_t es, Span out[6]) {
  const size_t c4 = 4 * size_t(a.channels);
  out[0] = rows_span(a.x, tokens, a.x_stride, a.channels, es);
  out[1] = rows_span(a.dt_raw, tokens, a.dt_stride, a.channels, es);
  out[2] = rows_span(a.in_raw, tokens, a.in_stride, a.channels, es);
  out[3] = span(a.A_log, c4);
  out[4] = span(a.dt_bias, c4);
  out[5] = a.in_raw ? span(a.in_bias, c4) : Span{};
}

size_t tables_bytes(const Packed& p) {
  return p.starts ? 4 * (2 * (size_t(p.sequences) + 1) + 2 * size_t(p.rows)) : 0;
}

// Tokens a wave and waves a tile. Forward: 12 waves of 16 tokens, two workgroups a CU (16384 tokens x 2560 bf16 92 us;
// 8 waves 94 us, 4 waves 147 us). Backward bf16: 4 waves of 16 tokens, three workgroups a CU (8 x 2048 tokens x 2560,
// with the forward pass, 242 us; 8 waves of 8 tokens 264 us; a softplus gate with a gated input spills 8 to 12 of 168
// registers); fp32: 8 waves of 8 (3 x 1999 tokens x 1001 79 us against 86 us).
constexpr int kTokens = 16, kWaves = 12;
constexpr int kBackTokens = 16, kBackWaves = 4;      // bf16
constexpr int kBackTokens32 = 8, kBackWaves32 = 8;   // fp32

// Rows x channels from which a step takes four channels a thread: 512 rows x 7680 bf16 16.4 -> 12.0 us from
// memory; in the caches 256 rows x 2560 4.0 and 4.1 us, one row 2.1 and 2.9 us.
constexpr int64_t kStepWide = 1 << 20;

// Groups of channels up to which all waves of a tile look at the tiles in front, and tiles in a row from which
// they do. Forward, bf16: 131072 tokens x 64 200 -> 60 us, 16384 x 512 44 -> 37 us, x 1024 48 -> 50 us. Backward:
// 131072 x 64 581 -> 229 us, 16384 x 1024 109 -> 81 us, x 2560 151 -> 166 us, 16 tiles in a row x 1024 54 -> 58 us.
// Between: 16384 x 768 forward 47 -> 42 us, x 1280 backward 111 -> 95 us, x 1536 127 -> 118 us; backward, tiles in a row
// of 8 sequences x 1024, 24 67 -> 69 us, 32 82 -> 81 us, 64 150 -> 133 us. fp32: 131072 x 64 205 -> 63 us and 568 -> 196
// us, 16384 x 512 forward 49 -> 41 us, x 768 52 -> 51 us, x 1024 56 -> 60 us, backward x 1024 107 -> 94 us, x 1280 111
// and 111 us, x 1536 143 -> 146 us; 24 tiles in a row x 1024 85 -> 87 us, 32 91 -> 94 us, 64 202 -> 195 us.
constexpr int kFewGroups = 8, kFewGroupsBack = 16, kLongChain = 32;

// Tiles, and what of the workspace they use.
struct Plan {
  int64_t tiles, groups;
  size_t sums, carry, ticket, chain;  // offsets and bytes of what tiles tell each other; chain 0: nothing
  size_t bytes;
  bool together;
};

Plan plan_linear(const axon_linear_shape& s, bool packed, bool backward) {
  Plan p{};
  // rows of the tables, or sequences without tokens, at least one tile
  const int64_t rows = std::max<int64_t>(packed_rows(s.sequences, s.tokens, packed), 1);
  static_assert(kBackTokens * kBackWaves == kBackTokens32 * kBackWaves32, "tiles of one size");
  const int64_t blocks = (backward ? kBackTokens * kBackWaves : kTokens * kWaves) / kBlock;
  p.tiles = (rows + blocks - 1) / blocks;
  p.groups = (s.channels + 63) / 64;
  // few packed sequences may be long ones; where it would cost most they are taken as alike
  const int64_t in_a_row = packed && p.groups <= kFewGroups ? p.tiles : p.tiles / s.sequences;
  p.together = p.groups <= (backward ? kFewGroupsBack : kFewGroups) && in_a_row >= kLongChain;
  const size_t cells = size_t(p.tiles) * size_t(p.groups) * 64;
  if (p.tiles > 1) {
    p.sums = 0;
    p.carry = 8 * cells;
    p.ticket = 12 * cells;
    p.chain = p.ticket + 16;
  }
  p.bytes = p.chain + (backward ? 4 * 3 * size_t(p.tiles) * size_t(s.channels) : 0);
  return p;
}

// The workspace holds for either kind of batch: a uniform one has no more blocks than a packed one can.
size_t workspace_of(const axon_linear_shape& s, bool backward) {
  return plan_linear(s, true, backward).bytes;
}

void use_plan(LinearArgs* a, const Plan& p, void* workspace) {
  a->tiles = static_cast<int>(p.tiles), a->groups = static_cast<int>(p.groups);
  a->together = p.together;
  char* w = static_cast<char*>(workspace);
  if (p.chain) {
    a->sums = reinterpret_cast<uint64_t*>(w + p.sums);
    a->carry = reinterpret_cast<uint32_t*>(w + p.carry);
    a->ticket = reinterpret_cast<uint32_t*>(w + p.ticket);
  }
  a->partial = reinterpret_cast<float*>(w + p.chain);
}

void clear_chain(const Plan& p, void* workspace, hipStream_t st) {
  if (!p.chain) return;
  const int64_t count = static_cast<int64_t>(p.chain / 16), wgs = (count + 1023) / 1024;
  hipLaunchKernelGGL(linear_clear_kernel, dim3(static_cast<unsigned>(std::min<int64_t>(wgs, 2048))), dim3(256),
                     0, st, static_cast<uint4*>(workspace), count);
}

// Workgroups along x, beyond 2^20 of them (a launch holds fewer than 2^32 threads along x) along y.
dim3 tile_grid(const Plan& p) {
  const int64_t n = p.tiles * p.groups, x = std::min<int64_t>(n, 1 << 20);
  return dim3(static_cast<unsigned>(x), static_cast<unsigned>((n + x - 1) / x));
}

template <bool BACK, typename Act, int GATE, int SCALE>
void launch_gated(const LinearArgs& a, dim3 grid, hipStream_t st) {
  constexpr bool kWide = sizeof(Act) == 4;
  constexpr int P = !BACK ? kTokens : kWide ? kBackTokens32 : kBackTokens;
  constexpr int W = !BACK ? kWaves : kWide ? kBackWaves32 : kBackWaves;
  auto launch = [&](auto gated) {
    constexpr bool kGated = decltype(gated)::value;
    if constexpr (BACK)
      hipLaunchKernelGGL((linear_tile_back_kernel<Act, P, W, GATE, SCALE, kGated>), grid, dim3(64 * W), 0, st, a);
    else
      hipLaunchKernelGGL((linear_tile_kernel<Act, P, W, GATE, SCALE, kGated>), grid, dim3(64 * W), 0, st, a);
  };
  a.in_raw ? launch(std::true_type()) : launch(std::false_type());
}

template <bool BACK, typename Act, int GATE>
void launch_scale(const LinearArgs& a, dim3 grid, hipStream_t st) {
  if (a.input_scale == AXON_INPUT_SQRT) launch_gated<BACK, Act, GATE, AXON_INPUT_SQRT>(a, grid, st);
  else if (a.input_scale == AXON_INPUT_COMPLEMENT) launch_gated<BACK, Act, GATE, AXON_INPUT_COMPLEMENT>(a, grid, st);
  else launch_gated<BACK, Act, GATE, AXON_INPUT_PLAIN>(a, grid, st);
}

template <bool BACK>
void launch_tiles(const LinearArgs& a, const Plan& plan, bool bf, hipStream_t st) {
  const dim3 grid = tile_grid(plan);
  const bool sigmoid = a.gate == AXON_LINEAR_SIGMOID;
  if (bf)
    sigmoid ? launch_scale<BACK, bf16_bits, AXON_LINEAR_SIGMOID>(a, grid, st)
            : launch_scale<BACK, bf16_bits, AXON_LINEAR_SOFTPLUS>(a, grid, st);
  else
    sigmoid ? launch_scale<BACK, float, AXON_LINEAR_SIGMOID>(a, grid, st)
            : launch_scale<BACK, float, AXON_LINEAR_SOFTPLUS>(a, grid, st);
}

unsigned channel_groups(int channels, int width) {
  return static_cast<unsigned>((channels + width - 1) / width);
}

// Four channels a thread where alignment allows it and there are threads enough.
template <typename Act>
void launch_step(const LinearArgs& a, hipStream_t st) {
  const size_t wide = 4 * sizeof(Act);
  const int64_t values = int64_t(a.channels) * a.p.sequences;
  if (values >= kStepWide && a.channels % 4 == 0 && a.x_stride % 4 == 0 && a.dt_stride % 4 == 0 &&
      a.in_stride % 4 == 0 && aligned_to(a.x, wide) && aligned_to(a.dt_raw, wide) && aligned_to(a.in_raw, wide) &&
      aligned_to(a.y, wide) && aligned_to(a.state_out, 16) && aligned_to(a.A_log, 16) &&
      aligned_to(a.dt_bias, 16) && aligned_to(a.in_bias, 16))
    hipLaunchKernelGGL((linear_step_kernel<Act, 4>), dim3(channel_groups(a.channels, 1024), a.p.sequences),
                       dim3(256), 0, st, a);
  else
    hipLaunchKernelGGL((linear_step_kernel<Act, 1>), dim3(channel_groups(a.channels, 256), a.p.sequences),
                       dim3(256), 0, st, a);
}

}  // namespace
}  // namespace axon

extern "C" {

size_t axon_linear_checkpoint_rows(int64_t sequences, int64_t tokens, int32_t packed) {
  if (sequences < 1 || sequences > 65535 || tokens < 0 || tokens >= (int64_t(1) << 29) ||
      (packed != 0 && packed != 1) || (!packed && tokens % sequences))
    return 0;
  return size_t(axon::packed_rows(sequences, tokens, packed != 0));
}

size_t axon_linear_scan_workspace_bytes(const axon_linear_shape* shape) {
  if (axon::check_shape(shape, false) != AXON_OK) return 0;
  return axon::workspace_of(*shape, false);
}

axon_status axon_linear_scan(const axon_linear_shape* shape, const axon_linear_params* params,
                             const void* x, const void* dt_raw, const void* in_raw,
                             const int32_t* tables, const float* state_in, const int32_t* in_slots,
                             void* y, float* state_out, const int32_t* out_slots,
                             float* checkpoints, void* workspace, size_t workspace_bytes,
                             void* stream) {
  using namespace axon;
  axon_status why = check_shape(shape, false);
  if (why != AXON_OK) return why;
  why = check_params(params, in_raw);
  if (why != AXON_OK) return why;
  const axon_linear_shape& s = *shape;
  if (!tables && s.tokens % s.sequences) return AXON_ERR_INVALID_ARGUMENT;
  if (off(tables, 4) || off(in_slots, 4) || off(out_slots, 4) || off(state_in, 4) ||
      off(state_out, 4) || off(checkpoints, 4))
    return AXON_ERR_INVALID_ARGUMENT;
  if ((state_in && !in_slots && s.state_slots < s.sequences) ||
      (state_out && !out_slots && s.out_slots < s.sequences) ||
      (state_in && state_in == state_out && s.state_slots != s.out_slots))
    return AXON_ERR_INVALID_ARGUMENT;
  const bool bf = s.act_dtype == AXON_BF16;
  const size_t es = bf ? 2 : 4;
  if (s.tokens && (bad(x, es) || bad(dt_raw, es) || off(in_raw, es) || bad(y, es)))
    return AXON_ERR_INVALID_ARGUMENT;
  const size_t need = axon_linear_scan_workspace_bytes(shape);
  if (workspace_bytes < need) return AXON_ERR_WORKSPACE_TOO_SMALL;
  if (need && bad(workspace, 16)) return AXON_ERR_INVALID_ARGUMENT;

  LinearArgs a = make_args(s, *params, x, dt_raw, in_raw, tables);
  const size_t row4 = 4 * size_t(s.channels), seq4 = 4 * size_t(s.sequences);
  Span reads[9];
  input_spans(a, s.tokens, es, reads);
  reads[6] = span(tables, tables_bytes(a.p));
  reads[7] = span(in_slots, seq4);
  reads[8] = span(out_slots, seq4);
  const Span in_state = span(state_in, row4 * size_t(s.state_slots));
  const Span outs[] = {s.tokens ? span(y, es * size_t(s.tokens * s.channels)) : Span{},
                       span(state_out, row4 * size_t(s.out_slots)),
                       span(checkpoints, row4 * size_t(a.p.rows)), span(workspace, need)};
  for (int i = 0; i < 4; ++i) {
    for (const Span& r : reads)
      if (overlaps(outs[i], r)) return AXON_ERR_INVALID_ARGUMENT;
    for (int j = 0; j < i; ++j)
      if (overlaps(outs[i], outs[j])) return AXON_ERR_INVALID_ARGUMENT;
    if (!(i == 1 && state_in == state_out) && overlaps(outs[i], in_state))
      return AXON_ERR_INVALID_ARGUMENT;
  }
  a.state_in = state_in, a.in_slots = in_slots, a.in_count = s.state_slots;
  a.state_out = state_out, a.out_slots = out_slots, a.out_count = s.out_slots;
  a.y = y, a.checkpoints = checkpoints;
  const Plan plan = plan_linear(s, tables != nullptr, false);
  use_plan(&a, plan, workspace);
  hipStream_t st = static_cast<hipStream_t>(stream);
  clear_chain(plan, workspace, st);
  launch_tiles<false>(a, plan, bf, st);
  return hipGetLastError() == hipSuccess ? AXON_OK : AXON_ERR_HIP;
}

size_t axon_linear_scan_backward_workspace_bytes(const axon_linear_shape* shape) {
  if (axon::check_shape(shape, true) != AXON_OK) return 0;
  return axon::workspace_of(*shape, true);
}

axon_status axon_linear_scan_backward(const axon_linear_shape* shape,
                                      const axon_linear_params* params, const void* dy,
                                      const void* x, const void* dt_raw, const void* in_raw,
                                      const int32_t* tables, const float* checkpoints,
                                      const float* dstate_out, void* dx, void* ddt_raw,
                                      void* din_raw, float* dA_log, float* ddt_bias,
                                      float* din_bias, float* dstate_in, void* workspace,
                                      size_t workspace_bytes, void* stream) {
  using namespace axon;
  axon_status why = check_shape(shape, true);
  if (why != AXON_OK) return why;
  why = check_params(params, in_raw);
  if (why != AXON_OK) return why;
  const axon_linear_shape& s = *shape;
  if (!tables && s.tokens % s.sequences) return AXON_ERR_INVALID_ARGUMENT;
  const bool bf = s.act_dtype == AXON_BF16;
  const size_t es = bf ? 2 : 4;
  if (off(tables, 4) || off(dstate_out, 4) || off(dstate_in, 4) || bad(dA_log, 4) ||
      bad(ddt_bias, 4) || off(din_bias, 4))
    return AXON_ERR_INVALID_ARGUMENT;
  if (s.tokens && (bad(dy, es) || bad(x, es) || bad(dt_raw, es) || off(in_raw, es) ||
                   bad(checkpoints, 4) || bad(dx, es) || bad(ddt_raw, es)))
    return AXON_ERR_INVALID_ARGUMENT;
  // All three or none; without tokens in_raw and din_raw may be empty arrays' null.
  if (s.tokens && (in_raw ? bad(din_raw, es) || !din_bias : din_raw || din_bias))
    return AXON_ERR_INVALID_ARGUMENT;
  const size_t need = axon_linear_scan_backward_workspace_bytes(shape);
  if (workspace_bytes < need) return AXON_ERR_WORKSPACE_TOO_SMALL;
  if (need && bad(workspace, 16)) return AXON_ERR_INVALID_ARGUMENT;

  LinearArgs a = make_args(s, *params, x, dt_raw, in_raw, tables);
  const size_t row4 = 4 * size_t(s.channels), seqs4 = row4 * size_t(s.sequences);
  const size_t act = s.tokens ? es * size_t(s.tokens * s.channels) : 0;
  Span reads[10];
  input_spans(a, s.tokens, es, reads);
  reads[6] = span(tables, tables_bytes(a.p));
  reads[7] = rows_span(dy, s.tokens, a.dy_stride, s.channels, es);
  reads[8] = span(checkpoints, row4 * size_t(a.p.rows));
  reads[9] = span(dstate_out, seqs4);
  const Span outs[] = {span(dx, act), span(ddt_raw, act), span(din_raw, act), span(dA_log, row4),
                       span(ddt_bias, row4), span(din_bias, row4), span(dstate_in, seqs4),
                       span(workspace, need)};
  for (int i = 0; i < 8; ++i) {
    for (const Span& r : reads)
      if (overlaps(outs[i], r)) return AXON_ERR_INVALID_ARGUMENT;
    for (int j = 0; j < i; ++j)
      if (overlaps(outs[i], outs[j])) return AXON_ERR_INVALID_ARGUMENT;
  }
  a.dy = dy, a.points = checkpoints, a.dstate_out = dstate_out;
  a.dx = dx, a.ddt_raw = ddt_raw, a.din_raw = din_raw;
  a.dA_log = dA_log, a.ddt_bias = ddt_bias, a.din_bias = din_bias, a.dstate_in = dstate_in;
  const Plan plan = plan_linear(s, tables != nullptr, true);
  use_plan(&a, plan, workspace);
  hipStream_t st = static_cast<hipStream_t>(stream);
  clear_chain(plan, workspace, st);
  launch_tiles<true>(a, plan, bf, st);
  hipLaunchKernelGGL(linear_sum_kernel, dim3(channel_groups(a.channels, 64), din_bias ? 3 : 2),
                     dim3(64 * kSumWaves), 0, st, a, a.tiles);
  return hipGetLastError() == hipSuccess ? AXON_OK : AXON_ERR_HIP;
}

axon_status axon_linear_step(const axon_linear_shape* shape, const axon_linear_params* params,
                             const void* x, const void* dt_raw, const void* in_raw, float* state,
                             const int32_t* slots, void* y, void* stream) {
  using namespace axon;
  axon_status why = check_shape(shape, false);
  if (why != AXON_OK) return why;
  why = check_params(params, in_raw);
  if (why != AXON_OK) return why;
  const axon_linear_shape& s = *shape;
  if (s.tokens != s.sequences) return AXON_ERR_INVALID_ARGUMENT;
  const bool bf = s.act_dtype == AXON_BF16;
  const size_t es = bf ? 2 : 4;
  if (bad(x, es) || bad(dt_raw, es) || off(in_raw, es) || bad(y, es) || bad(state, 4) ||
      (slots ? off(slots, 4) : s.state_slots < s.sequences))
    return AXON_ERR_INVALID_ARGUMENT;
  LinearArgs a = make_args(s, *params, x, dt_raw, in_raw, nullptr);
  Span reads[7];
  input_spans(a, s.tokens, es, reads);
  reads[6] = span(slots, 4 * size_t(s.sequences));
  const Span pool = span(state, 4 * size_t(s.state_slots * s.channels));
  const Span out = span(y, es * size_t(s.tokens * s.channels));
  for (const Span& r : reads)
    if (overlaps(out, r) || overlaps(pool, r)) return AXON_ERR_INVALID_ARGUMENT;
  if (overlaps(out, pool)) return AXON_ERR_INVALID_ARGUMENT;
  a.state_out = state, a.in_slots = slots, a.in_count = s.state_slots, a.y = y;
  bf ? launch_step<bf16_bits>(a, static_cast<hipStream_t>(stream))
     : launch_step<float>(a, static_cast<hipStream_t>(stream));
  return hipGetLastError() == hipSuccess ? AXON_OK : AXON_ERR_HIP;
}

}  // extern "C"

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
#include <hip/hip_runtime.h>

#include <cmath>
#include <cstdint>

#include "axon_device.h"
#include "axon_packed.h"

namespace axon {
namespace {

struct LinearArgs {
  const void *x, *dt_raw, *in_raw, *dy;
  const float *A_log, *dt_bias, *in_bias;
  Packed p;
  int64_t x_stride, dt_stride, in_stride, dy_stride;
  int channels, gate, input_scale, clear_behind;
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
  float* partial;  // (sequences, 3, channels)
};

// expm1(v) for v <= 0 (and NaN). Below -1/4 exp(v) - 1 cancels two bits at most; above it the series
// up to v^6 / 720 leaves a relative 5e-8.
__device__ __forceinline__ float expm1_neg(float v, float e) {
  float p = fmaf(v, 1.0f / 720.0f, 1.0f / 120.0f);
  p = fmaf(v, p, 1.0f / 24.0f);
  p = fmaf(v, p, 1.0f / 6.0f);
  p = fmaf(v, p, 0.5f);
  p = fmaf(v * v, p, v);
  return v > -0.25f ? p : e - 1.0f;
}

// sigmoid(v) and 1 - sigmoid(v), each with a relative error of a few 2^-24.
struct Sigmoid {
  float on, off;
  __device__ __forceinline__ explicit Sigmoid(float v) {
    const float e = __builtin_amdgcn_exp2f(-fabsf(v) * kLog2e);
    const float big = __builtin_amdgcn_rcpf(1.0f + e), small = e * big;
    on = v < 0.0f ? small : big;
    off = v < 0.0f ? big : small;
  }
};

// What a token's gate makes of its channel: log a, a, expm1(log a), m.
struct Decay {
  float L, a, em1, m;
  __device__ __forceinline__ Decay(float v, float rate, int gate, int input_scale) {
    L = -rate * (gate == AXON_LINEAR_SIGMOID ? Sigmoid(v).on : softplus_f32(v));
    if (v != v) L = v;
    a = __builtin_amdgcn_exp2f(L * kLog2e);
    em1 = expm1_neg(L, a);
    m = input_scale == AXON_INPUT_PLAIN ? 1.0f
        : input_scale == AXON_INPUT_COMPLEMENT
            ? -em1
            : __builtin_amdgcn_sqrtf(-em1 * (2.0f + em1));
  }
  // a h + b. For a >= 1/2 the rounding of a would be a systematic error of the decay, 2^-25 against
  // 1 - a; below, h + expm1(log a) h would lose b beside a larger h.
  __device__ __forceinline__ float advance(float h, float b) const {
    return a < 0.5f ? fmaf(a, h, b) : h + fmaf(em1, h, b);
  }
};

// The simple form: a lane walks one channel of one sequence.
template <typename Act>
__global__ __launch_bounds__(64) void linear_walk_kernel(LinearArgs g) {
  const int e = blockIdx.x * 64 + threadIdx.x, n = blockIdx.y;
  if (e >= g.channels) return;
  const Act* x = static_cast<const Act*>(g.x);
  const Act* raw = static_cast<const Act*>(g.dt_raw);
  const Act* in = static_cast<const Act*>(g.in_raw);
  const float rate = expf(g.A_log[e]);
  const float bias = g.dt_bias ? g.dt_bias[e] : 0.0f, ib = in && g.in_bias ? g.in_bias[e] : 0.0f;
  const int s0 = packed_start(g.p, n), s1 = packed_start(g.p, n + 1);
  float h = 0.0f;
  if (g.state_in) {
    const int64_t slot = g.in_slots ? g.in_slots[n] : n;
    if (slot >= 0 && slot < g.in_count) h = g.state_in[slot * g.channels + e];
  }
  const int64_t row0 = g.p.starts ? max(g.p.block_starts[n], 0) : int64_t(n) * g.p.blocks_per_seq;
  for (int t = s0; t < s1; ++t) {
    const int64_t row = row0 + (t - s0) / kBlock;
    if (g.checkpoints && (t - s0) % kBlock == 0 && row < g.p.rows)
      g.checkpoints[row * g.channels + e] = h;
    const Decay d(load_act(raw, t * g.dt_stride + e) + bias, rate, g.gate, g.input_scale);
    float u = load_act(x, t * g.x_stride + e);
    if (in) u *= Sigmoid(load_act(in, t * g.in_stride + e) + ib).on;
    h = d.advance(h, d.m * u);
    store_act(static_cast<Act*>(g.y), int64_t(t) * g.channels + e, h);
  }
  if (g.state_out) {
    const int64_t slot = g.out_slots ? g.out_slots[n] : n;
    if (slot >= 0 && slot < g.out_count) g.state_out[slot * g.channels + e] = h;
  }
  if (g.clear_behind)
    for (int t = packed_start(g.p, g.p.sequences) + n; t < g.p.tokens; t += g.p.sequences)
      store_act(static_cast<Act*>(g.y), int64_t(t) * g.channels + e, 0.0f);
}

// The same backwards, a block at a time: the block's states are found again from its checkpoint.
template <typename Act>
__global__ __launch_bounds__(64) void linear_walk_back_kernel(LinearArgs g) {
  const int e = blockIdx.x * 64 + threadIdx.x, n = blockIdx.y;
  if (e >= g.channels) return;
  const Act* x = static_cast<const Act*>(g.x);
  const Act* raw = static_cast<const Act*>(g.dt_raw);
  const Act* in = static_cast<const Act*>(g.in_raw);
  const float rate = expf(g.A_log[e]);
  const float bias = g.dt_bias ? g.dt_bias[e] : 0.0f, ib = in && g.in_bias ? g.in_bias[e] : 0.0f;
  const int s0 = packed_start(g.p, n), s1 = packed_start(g.p, n + 1);
  const int64_t row0 = g.p.starts ? max(g.p.block_starts[n], 0) : int64_t(n) * g.p.blocks_per_seq;
  float k = g.dstate_out ? g.dstate_out[int64_t(n) * g.channels + e] : 0.0f;
  double sA = 0.0, sdt = 0.0, sin = 0.0;
  float before[kBlock];
  for (int first = s0 + (s1 - s0 - 1) / kBlock * kBlock; s1 > s0 && first >= s0; first -= kBlock) {
    const int count = min(kBlock, s1 - first);
    const int64_t row = row0 + (first - s0) / kBlock;
    float h = row < g.p.rows ? g.points[row * g.channels + e] : 0.0f;
    for (int j = 0; j < count; ++j) {
      const int64_t t = first + j;
      before[j] = h;
      const Decay d(load_act(raw, t * g.dt_stride + e) + bias, rate, g.gate, g.input_scale);
      float u = load_act(x, t * g.x_stride + e);
      if (in) u *= Sigmoid(load_act(in, t * g.in_stride + e) + ib).on;
      h = d.advance(h, d.m * u);
    }
    for (int j = count - 1; j >= 0; --j) {
      const int64_t t = first + j;
      const float v = load_act(raw, t * g.dt_stride + e) + bias;
      const Decay d(v, rate, g.gate, g.input_scale);
      const float xv = load_act(x, t * g.x_stride + e);
      const Sigmoid i(in ? load_act(in, t * g.in_stride + e) + ib : 0.0f);
      const float u = in ? xv * i.on : xv;
      const float gt = load_act(static_cast<const Act*>(g.dy), t * g.dy_stride + e) + k;
      const float aL = d.a == 0.0f ? 0.0f : d.a * d.L;
      float G = aL * before[j];
      if (g.input_scale == AXON_INPUT_COMPLEMENT) G -= aL * u;
      if (g.input_scale == AXON_INPUT_SQRT && d.m != 0.0f) G -= d.a * (aL * u) / d.m;
      G *= gt;
      const Sigmoid s(v);
      const float slope = g.gate == AXON_LINEAR_SIGMOID ? s.off : (v < -20.0f ? 1.0f : s.on / softplus_f32(v));
      const float draw = G * slope, du = gt * d.m;
      sA += G, sdt += draw;
      const int64_t at = t * g.channels + e;
      store_act(static_cast<Act*>(g.ddt_raw), at, draw);
      store_act(static_cast<Act*>(g.dx), at, in ? du * i.on : du);
      if (in) {
        const float di = du * xv * i.on * i.off;
        sin += di;
        store_act(static_cast<Act*>(g.din_raw), at, di);
      }
      k = d.advance(gt, 0.0f);
    }
  }
  if (g.dstate_in) g.dstate_in[int64_t(n) * g.channels + e] = k;
  float* part = g.partial + int64_t(n) * 3 * g.channels + e;
  part[0] = static_cast<float>(sA);
  part[g.channels] = static_cast<float>(sdt);
  part[2 * int64_t(g.channels)] = static_cast<float>(sin);
  for (int t = packed_start(g.p, g.p.sequences) + n; t < g.p.tokens; t += g.p.sequences) {
    const int64_t at = int64_t(t) * g.channels + e;
    store_act(static_cast<Act*>(g.dx), at, 0.0f);
    store_act(static_cast<Act*>(g.ddt_raw), at, 0.0f);
    if (in) store_act(static_cast<Act*>(g.din_raw), at, 0.0f);
  }
}

__global__ __launch_bounds__(64) void linear_sum_kernel(LinearArgs g, int parts) {
  const int e = blockIdx.x * 64 + threadIdx.x, which = blockIdx.y;
  if (e >= g.channels) return;
  double s = 0.0;
  for (int j = 0; j < parts; ++j) s += g.partial[(int64_t(j) * 3 + which) * g.channels + e];
  float* out = which == 0 ? g.dA_log : which == 1 ? g.ddt_bias : g.din_bias;
  out[e] = static_cast<float>(s);
}

template <typename Act>
__global__ __launch_bounds__(256) void linear_step_kernel(LinearArgs g) {
  const int e = blockIdx.x * 256 + threadIdx.x, n = blockIdx.y;
  if (e >= g.channels) return;
  const int64_t slot = g.in_slots ? g.in_slots[n] : n;
  if (slot < 0 || slot >= g.in_count) return;
  const Act* in = static_cast<const Act*>(g.in_raw);
  const float v = load_act(static_cast<const Act*>(g.dt_raw), n * g.dt_stride + e);
  float u = load_act(static_cast<const Act*>(g.x), n * g.x_stride + e);
  const Decay d(v + (g.dt_bias ? g.dt_bias[e] : 0.0f), expf(g.A_log[e]), g.gate, g.input_scale);
  if (in) u *= Sigmoid(load_act(in, n * g.in_stride + e) + (g.in_bias ? g.in_bias[e] : 0.0f)).on;
  float* state = g.state_out + slot * g.channels + e;
  const float h = d.advance(*state, d.m * u);
  *state = h;
  store_act(static_cast<Act*>(g.y), int64_t(n) * g.channels + e, h);
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

unsigned channel_groups(int channels, int width) {
  return static_cast<unsigned>((channels + width - 1) / width);
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

size_t axon_linear_scan_workspace_bytes(const axon_linear_shape*) { return 0; }

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
  const dim3 grid(channel_groups(a.channels, 64), a.p.sequences);
  hipStream_t st = static_cast<hipStream_t>(stream);
  if (bf)
    hipLaunchKernelGGL(linear_walk_kernel<bf16_bits>, grid, dim3(64), 0, st, a);
  else
    hipLaunchKernelGGL(linear_walk_kernel<float>, grid, dim3(64), 0, st, a);
  return hipGetLastError() == hipSuccess ? AXON_OK : AXON_ERR_HIP;
}

size_t axon_linear_scan_backward_workspace_bytes(const axon_linear_shape* shape) {
  if (axon::check_shape(shape, true) != AXON_OK) return 0;
  return 4 * 3 * size_t(shape->sequences) * size_t(shape->channels);
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
  a.partial = static_cast<float*>(workspace);
  const dim3 grid(channel_groups(a.channels, 64), a.p.sequences);
  hipStream_t st = static_cast<hipStream_t>(stream);
  if (bf)
    hipLaunchKernelGGL(linear_walk_back_kernel<bf16_bits>, grid, dim3(64), 0, st, a);
  else
    hipLaunchKernelGGL(linear_walk_back_kernel<float>, grid, dim3(64), 0, st, a);
  hipLaunchKernelGGL(linear_sum_kernel, dim3(channel_groups(a.channels, 64), din_bias ? 3 : 2),
                     dim3(64), 0, st, a, a.p.sequences);
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
  const dim3 grid(channel_groups(a.channels, 256), a.p.sequences);
  hipStream_t st = static_cast<hipStream_t>(stream);
  if (bf)
    hipLaunchKernelGGL(linear_step_kernel<bf16_bits>, grid, dim3(256), 0, st, a);
  else
    hipLaunchKernelGGL(linear_step_kernel<float>, grid, dim3(256), 0, st, a);
  return hipGetLastError() == hipSuccess ? AXON_OK : AXON_ERR_HIP;
}

}  // extern "C"

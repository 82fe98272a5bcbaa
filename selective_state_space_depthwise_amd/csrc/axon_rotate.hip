// Head norm with position rotation (see axonscan.h), forward and backward.
//
// With r = 1 / sqrt(mean(x^2) + eps), n = x r, z = n w and R the rotation: out = R z. Backward, with
// d = R^T dout: dw = sum d n, dn = d w, dx = r (dn - n mean(n dn)).
//
// A head is held by LANES lanes (a power of two), a lane holds up to UNITS pieces of 2 V of its
// channels: V of the first and V of the second halves of V pairs, or 2 V channels that are not
// turned. A wave takes 64 / LANES heads at a time and one row's heads one group after the other, so
// that its angles are found once a row. Angles: p freqs / (2 pi) turns in 64 bits, of which only the
// fraction goes to 32 bits.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "axon_device.h"
#include "axon_packed.h"

namespace axon {
namespace {

constexpr int kWaves = 4;   // of a workgroup
constexpr int kFlush = 32;  // rows

struct RotateArgs {
  const void *q, *k, *dq_out, *dk_out;
  const int32_t* positions;
  const double* freqs;
  const float *q_weight, *k_weight;
  void *q_out, *k_out;  // dq, dk in the backward pass
  int64_t rows, q_stride, k_stride, dq_stride, dk_stride;
  int q_heads, heads, dim, rotary, lanes, interleaved;
  int splits;  // forward: waves that share a row's heads
  float eps, inv_dim;
  float* partial;  // backward: (workgroups, 2, dim)
};

template <typename Act, int V>
__device__ __forceinline__ void load_v(const Act* p, float* v) {
  if constexpr (V == 1) {
    v[0] = load_act(p, 0);
  } else if constexpr (sizeof(Act) == 4) {
    const float4 t = *reinterpret_cast<const float4*>(p);
    v[0] = t.x, v[1] = t.y, v[2] = t.z, v[3] = t.w;
  } else {
    const uint2 t = *reinterpret_cast<const uint2*>(p);
    v[0] = __uint_as_float(t.x << 16), v[1] = __uint_as_float(t.x & 0xFFFF0000u);
    v[2] = __uint_as_float(t.y << 16), v[3] = __uint_as_float(t.y & 0xFFFF0000u);
  }
}
template <typename Act, int V>
__device__ __forceinline__ void store_v(Act* p, const float* v) {
  if constexpr (V == 1) {
    store_act(p, 0, v[0]);
  } else if constexpr (sizeof(Act) == 4) {
    *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
  } else {
    uint2 t;
    t.x = static_cast<uint32_t>(f32_to_bf16(v[0])) | static_cast<uint32_t>(f32_to_bf16(v[1])) << 16;
    t.y = static_cast<uint32_t>(f32_to_bf16(v[2])) | static_cast<uint32_t>(f32_to_bf16(v[3])) << 16;
    *reinterpret_cast<uint2*>(p) = t;
  }
}

// Where a unit's two pieces of V channels lie, and its first pair (turned units only).
template <int V>
struct Unit {
  int lo, hi, pair;
  bool live, turned;
  __device__ __forceinline__ Unit(const RotateArgs& g, int u) {
    live = 2 * V * u < g.dim;
    turned = 2 * V * u < g.rotary;
    pair = V * u;
    const bool split = turned && !g.interleaved;
    lo = split ? V * u : 2 * V * u;
    hi = split ? V * u + g.rotary / 2 : 2 * V * u + V;
  }
};

template <int V>
__device__ __forceinline__ void angles(const RotateArgs& g, const Unit<V>& u, const double* turns,
                                       int position, float* c, float* s) {
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const double t = position * turns[i];
    const float part = static_cast<float>(t - rint(t));
    sincospif(2.0f * part, &s[i], &c[i]);
    if (!u.turned) c[i] = 1.0f, s[i] = 0.0f;
  }
}

// (lo, hi) turned by the angle whose cosine and sine are c and s.
template <int V>
__device__ __forceinline__ void turn(bool interleaved, const float* c, const float* s, float* lo,
                                     float* hi) {
  if (V > 1 && interleaved) {  // the 2 V channels in order, pairs side by side
    float z[2 * V];
#pragma unroll
    for (int i = 0; i < V; ++i) z[i] = lo[i], z[V + i] = hi[i];
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const float a = z[2 * i], b = z[2 * i + 1];
      z[2 * i] = a * c[i] - b * s[i];
      z[2 * i + 1] = b * c[i] + a * s[i];
    }
#pragma unroll
    for (int i = 0; i < V; ++i) lo[i] = z[i], hi[i] = z[V + i];
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const float a = lo[i], b = hi[i];
      lo[i] = a * c[i] - b * s[i];
      hi[i] = b * c[i] + a * s[i];
    }
  }
}

template <int V>
__device__ __forceinline__ void load_weight(const float* w, const Unit<V>& u, float* lo, float* hi) {
#pragma unroll
  for (int i = 0; i < V; ++i) {
    lo[i] = w && u.live ? w[u.lo + i] : 1.0f;
    hi[i] = w && u.live ? w[u.hi + i] : 1.0f;
  }
}

__device__ __forceinline__ float sum_lanes(float v, int lanes) {
  for (int d = lanes >> 1; d > 0; d >>= 1) v += __shfl_xor(v, d, 64);
  return v;
}

template <typename Act, int V, int UNITS, bool BACK>
__global__ __launch_bounds__(64 * kWaves) void rotate_kernel(RotateArgs g) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int l = lane & (g.lanes - 1), sub = lane / g.lanes, per = 64 / g.lanes;
  const int groups = (g.heads + per - 1) / per;
  float wq[UNITS][2][V], wk[UNITS][2][V], sq[UNITS][2][V], sk[UNITS][2][V];
  double turns[UNITS][V];
#pragma unroll
  for (int n = 0; n < UNITS; ++n) {
    const Unit<V> u(g, l + n * g.lanes);
    load_weight<V>(g.q_weight, u, wq[n][0], wq[n][1]);
    load_weight<V>(g.k_weight, u, wk[n][0], wk[n][1]);
#pragma unroll
    for (int i = 0; i < V; ++i) {
      turns[n][i] = u.turned ? g.freqs[u.pair + i] * 0.15915494309189533577 : 0.0;
      sq[n][0][i] = sq[n][1][i] = sk[n][0][i] = sk[n][1][i] = 0.0f;
    }
  }
  // Weight gradients: fp32 over up to kFlush rows a lane, 64 bits beyond.
  __shared__ double part[BACK ? kWaves : 1][2][BACK ? 256 : 1];
  auto flush = [&] {
#pragma unroll
    for (int n = 0; n < UNITS; ++n) {
      const Unit<V> u(g, l + n * g.lanes);
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int i = 0; i < V; ++i) {
          // lanes that hold the same channels of other heads, in a fixed order
          for (int d = g.lanes; d < 64; d <<= 1) {
            sq[n][j][i] += __shfl_xor(sq[n][j][i], d, 64);
            sk[n][j][i] += __shfl_xor(sk[n][j][i], d, 64);
          }
          if (sub == 0 && u.live) {
            part[wave][0][(j ? u.hi : u.lo) + i] += sq[n][j][i];
            part[wave][1][(j ? u.hi : u.lo) + i] += sk[n][j][i];
          }
          sq[n][j][i] = sk[n][j][i] = 0.0f;
        }
    }
  };
  if constexpr (BACK) {
    for (int t = threadIdx.x; t < kWaves * 2 * 256; t += 64 * kWaves) (&part[0][0][0])[t] = 0.0;
    __syncthreads();
  }
  int pending = 0;
  const int64_t items = g.rows * g.splits, step = int64_t(gridDim.x) * kWaves;
  for (int64_t item = int64_t(blockIdx.x) * kWaves + wave; item < items; item += step) {
    const int64_t row = item / g.splits;
    const int split = static_cast<int>(item - row * g.splits);
    const int position = g.positions[row];
    float c[UNITS][V], s[UNITS][V];
#pragma unroll
    for (int n = 0; n < UNITS; ++n)
      angles<V>(g, Unit<V>(g, l + n * g.lanes), turns[n], position, c[n], s[n]);
    for (int grp = split; grp < groups; grp += g.splits) {
      const int head = grp * per + sub;
      const bool in = head < g.heads, is_q = head < g.q_heads;
      const int h = is_q ? head : head - g.q_heads;
      const Act* x = is_q ? static_cast<const Act*>(g.q) + row * g.q_stride
                          : static_cast<const Act*>(g.k) + row * g.k_stride;
      Act* out = is_q ? static_cast<Act*>(g.q_out) + (row * g.q_heads + h) * g.dim
                      : static_cast<Act*>(g.k_out) + (row * (g.heads - g.q_heads) + h) * g.dim;
      x += int64_t(h) * g.dim;
      float v[UNITS][2][V];
      float sum = 0.0f;
#pragma unroll
      for (int n = 0; n < UNITS; ++n) {
        const Unit<V> u(g, l + n * g.lanes);
#pragma unroll
        for (int i = 0; i < V; ++i) v[n][0][i] = v[n][1][i] = 0.0f;
        if (in && u.live) {
          load_v<Act, V>(x + u.lo, v[n][0]);
          load_v<Act, V>(x + u.hi, v[n][1]);
        }
#pragma unroll
        for (int i = 0; i < V; ++i) {
          sum = fmaf(v[n][0][i], v[n][0][i], sum);
          sum = fmaf(v[n][1][i], v[n][1][i], sum);
        }
      }
      const float r = 1.0f / sqrtf(sum_lanes(sum, g.lanes) * g.inv_dim + g.eps);
      if constexpr (!BACK) {
#pragma unroll
        for (int n = 0; n < UNITS; ++n) {
          const Unit<V> u(g, l + n * g.lanes);
#pragma unroll
          for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int i = 0; i < V; ++i) v[n][j][i] *= r * (is_q ? wq[n][j][i] : wk[n][j][i]);
          if (u.turned) turn<V>(g.interleaved, c[n], s[n], v[n][0], v[n][1]);
          if (in && u.live) {
            store_v<Act, V>(out + u.lo, v[n][0]);
            store_v<Act, V>(out + u.hi, v[n][1]);
          }
        }
      } else {
        const Act* dy = is_q ? static_cast<const Act*>(g.dq_out) + row * g.dq_stride
                             : static_cast<const Act*>(g.dk_out) + row * g.dk_stride;
        dy += int64_t(h) * g.dim;
        float d[UNITS][2][V];
        float dot = 0.0f;
#pragma unroll
        for (int n = 0; n < UNITS; ++n) {
          const Unit<V> u(g, l + n * g.lanes);
#pragma unroll
          for (int i = 0; i < V; ++i) d[n][0][i] = d[n][1][i] = 0.0f;
          if (in && u.live) {
            load_v<Act, V>(dy + u.lo, d[n][0]);
            load_v<Act, V>(dy + u.hi, d[n][1]);
          }
          float back[V];
#pragma unroll
          for (int i = 0; i < V; ++i) back[i] = -s[n][i];
          if (u.turned) turn<V>(g.interleaved, c[n], back, d[n][0], d[n][1]);
#pragma unroll
          for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int i = 0; i < V; ++i) {
              v[n][j][i] *= r;  // n
              const float dw = d[n][j][i] * v[n][j][i];
              if (in && u.live) {
                if (is_q) sq[n][j][i] += dw;
                else sk[n][j][i] += dw;
              }
              d[n][j][i] *= is_q ? wq[n][j][i] : wk[n][j][i];
              dot = fmaf(d[n][j][i], v[n][j][i], dot);
            }
        }
        const float mean = sum_lanes(dot, g.lanes) * g.inv_dim;
#pragma unroll
        for (int n = 0; n < UNITS; ++n) {
          const Unit<V> u(g, l + n * g.lanes);
#pragma unroll
          for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int i = 0; i < V; ++i) d[n][j][i] = r * fmaf(-v[n][j][i], mean, d[n][j][i]);
          if (in && u.live) {
            store_v<Act, V>(out + u.lo, d[n][0]);
            store_v<Act, V>(out + u.hi, d[n][1]);
          }
        }
      }
    }
    if constexpr (BACK) {
      if (++pending == kFlush) flush(), pending = 0;
    }
  }
  if constexpr (BACK) {
    flush();
    __syncthreads();
    for (int t = threadIdx.x; t < 2 * g.dim; t += 64 * kWaves) {
      const int which = t >= g.dim, at = which ? t - g.dim : t;
      double a = 0.0;
#pragma unroll
      for (int w = 0; w < kWaves; ++w) a += part[w][which][at];
      g.partial[int64_t(blockIdx.x) * 2 * g.dim + t] = static_cast<float>(a);
    }
  }
}

// Sums of the workgroups' parts: a wave for each of 2 D values.
__global__ __launch_bounds__(64) void rotate_sum_kernel(const float* partial, int parts, int dim,
                                                        float* dq_weight, float* dk_weight) {
  const int t = blockIdx.x;
  float* out = t < dim ? dq_weight : dk_weight;
  if (!out) return;
  double s = 0.0;
  for (int p = threadIdx.x; p < parts; p += 64) s += partial[int64_t(p) * 2 * dim + t];
  for (int d = 32; d > 0; d >>= 1) s += __shfl_xor(s, d, 64);
  if (threadIdx.x == 0) out[t < dim ? t : t - dim] = static_cast<float>(s);
}

constexpr int kBackWorkgroups = 1024;
int back_workgroups(int64_t rows) {
  return static_cast<int>(std::min<int64_t>((rows + kWaves - 1) / kWaves, kBackWorkgroups));
}

template <typename Act, int V, int UNITS, bool BACK>
void launch_units(RotateArgs a, hipStream_t st) {
  if (BACK) {
    a.splits = 1;
    hipLaunchKernelGGL((rotate_kernel<Act, V, UNITS, true>), dim3(back_workgroups(a.rows)),
                       dim3(64 * kWaves), 0, st, a);
  } else {
    a.splits = 1;
    const int64_t wgs = std::min<int64_t>((a.rows * a.splits + kWaves - 1) / kWaves, 1 << 20);
    hipLaunchKernelGGL((rotate_kernel<Act, V, UNITS, false>), dim3(static_cast<unsigned>(wgs)),
                       dim3(64 * kWaves), 0, st, a);
  }
}

template <typename Act, bool BACK>
void launch_rotate(RotateArgs a, bool wide, hipStream_t st) {
  const int units = a.dim / (wide ? 8 : 2);
  a.lanes = 1;
  while (a.lanes < 64 && a.lanes < units) a.lanes *= 2;
  if (wide) launch_units<Act, 4, 1, BACK>(a, st);
  else if (units <= 64) launch_units<Act, 1, 1, BACK>(a, st);
  else launch_units<Act, 1, 2, BACK>(a, st);
}

axon_status check_desc(const axon_norm_rotate_desc* d, bool backward) {
  if (!d) return AXON_ERR_INVALID_ARGUMENT;
  if (d->rows < 0 || d->q_heads < 1 || d->k_heads < 0 || d->head_dim < 2 || d->rotary_dim < 2 ||
      d->rotary_dim > d->head_dim || d->q_stride < 0 || d->k_stride < 0 ||
      (backward && (d->dq_stride < 0 || d->dk_stride < 0)) || !std::isfinite(d->eps) ||
      d->eps < 0.0f)
    return AXON_ERR_INVALID_ARGUMENT;
  if (d->q_heads > 65535 || d->k_heads > 65535 || d->head_dim > 256 || d->head_dim % 2 ||
      d->rotary_dim % 2 || d->rows >= (int64_t(1) << 31) ||
      (d->act_dtype != AXON_F32 && d->act_dtype != AXON_BF16) ||
      (d->interleaved != 0 && d->interleaved != 1))
    return AXON_ERR_UNSUPPORTED;
  const int64_t own[] = {d->q_heads * d->head_dim, d->k_heads * d->head_dim,
                         d->q_heads * d->head_dim, d->k_heads * d->head_dim};
  const int64_t strides[] = {d->q_stride, d->k_stride, d->dq_stride, d->dk_stride};
  for (int j = 0; j < (backward ? 4 : 2); ++j) {
    if (strides[j] > (int64_t(1) << 31)) return AXON_ERR_UNSUPPORTED;
    if (strides[j] && strides[j] < own[j]) return AXON_ERR_INVALID_ARGUMENT;
    int64_t t;
    if (__builtin_mul_overflow(d->rows, strides[j] ? strides[j] : own[j], &t) || t > kMaxTotal)
      return AXON_ERR_UNSUPPORTED;
  }
  return AXON_OK;
}

bool bad(const void* p, size_t a) { return !p || !aligned_to(p, a); }
bool off(const void* p, size_t a) { return p && !aligned_to(p, a); }

RotateArgs make_args(const axon_norm_rotate_desc& d) {
  RotateArgs a{};
  const int64_t qw = d.q_heads * d.head_dim, kw = d.k_heads * d.head_dim;
  a.rows = d.rows;
  a.q_stride = d.q_stride ? d.q_stride : qw, a.k_stride = d.k_stride ? d.k_stride : kw;
  a.dq_stride = d.dq_stride ? d.dq_stride : qw, a.dk_stride = d.dk_stride ? d.dk_stride : kw;
  a.q_heads = static_cast<int>(d.q_heads), a.heads = static_cast<int>(d.q_heads + d.k_heads);
  a.dim = static_cast<int>(d.head_dim), a.rotary = static_cast<int>(d.rotary_dim);
  a.interleaved = d.interleaved, a.eps = d.eps, a.inv_dim = 1.0f / static_cast<float>(d.head_dim);
  return a;
}

// Four channels a load: heads and halves of four, rows and pointers that keep them aligned.
bool wide_ok(const RotateArgs& a, size_t es, bool backward, bool k) {
  const size_t align = 4 * es;
  if (a.dim % 8 || a.rotary % 8 || a.q_stride % 4 || !aligned_to(a.q, align) ||
      !aligned_to(a.q_out, align))
    return false;
  if (k && (a.k_stride % 4 || !aligned_to(a.k, align) || !aligned_to(a.k_out, align))) return false;
  if (!backward) return true;
  if (a.dq_stride % 4 || !aligned_to(a.dq_out, align)) return false;
  return !k || (a.dk_stride % 4 == 0 && aligned_to(a.dk_out, align));
}

}  // namespace
}  // namespace axon

extern "C" {

axon_status axon_norm_rotate(const axon_norm_rotate_desc* desc, const void* q, const void* k,
                             const int32_t* positions, const double* freqs, const float* q_weight,
                             const float* k_weight, void* q_out, void* k_out, void* stream) {
  using namespace axon;
  const axon_status why = check_desc(desc, false);
  if (why != AXON_OK) return why;
  const axon_norm_rotate_desc& d = *desc;
  if (d.rows == 0) return AXON_OK;
  const bool bf = d.act_dtype == AXON_BF16, with_k = d.k_heads > 0;
  const size_t es = bf ? 2 : 4;
  if (bad(q, es) || bad(q_out, es) || (with_k && (bad(k, es) || bad(k_out, es))) ||
      bad(positions, 4) || bad(freqs, 8) || off(q_weight, 4) || (with_k && off(k_weight, 4)))
    return AXON_ERR_INVALID_ARGUMENT;
  RotateArgs a = make_args(d);
  a.q = q, a.k = k, a.positions = positions, a.freqs = freqs;
  a.q_weight = q_weight, a.k_weight = with_k ? k_weight : nullptr;
  a.q_out = q_out, a.k_out = k_out;
  const int64_t qw = d.q_heads * d.head_dim, kw = d.k_heads * d.head_dim;
  const size_t d4 = 4 * size_t(d.head_dim);
  const Span in_q = rows_span(q, d.rows, a.q_stride, qw, es);
  const Span in_k = with_k ? rows_span(k, d.rows, a.k_stride, kw, es) : Span{};
  const Span out_q = span(q_out, es * size_t(d.rows * qw));
  const Span out_k = with_k ? span(k_out, es * size_t(d.rows * kw)) : Span{};
  const Span reads[] = {span(positions, 4 * size_t(d.rows)), span(freqs, 4 * size_t(d.rotary_dim)),
                        span(q_weight, d4), span(a.k_weight, d4)};
  for (const Span& r : reads)
    if (overlaps(out_q, r) || overlaps(out_k, r)) return AXON_ERR_INVALID_ARGUMENT;
  if (overlaps(out_q, out_k) || overlaps(out_q, in_k) || overlaps(out_k, in_q) ||
      (!(q == q_out && a.q_stride == qw) && overlaps(out_q, in_q)) ||
      (with_k && !(k == k_out && a.k_stride == kw) && overlaps(out_k, in_k)))
    return AXON_ERR_INVALID_ARGUMENT;
  hipStream_t st = static_cast<hipStream_t>(stream);
  const bool wide = wide_ok(a, es, false, with_k);
  bf ? launch_rotate<bf16_bits, false>(a, wide, st) : launch_rotate<float, false>(a, wide, st);
  return hipGetLastError() == hipSuccess ? AXON_OK : AXON_ERR_HIP;
}

size_t axon_norm_rotate_backward_workspace_bytes(const axon_norm_rotate_desc* desc) {
  if (axon::check_desc(desc, true) != AXON_OK) return 0;
  return 4 * 2 * size_t(axon::back_workgroups(desc->rows)) * size_t(desc->head_dim);
}

axon_status axon_norm_rotate_backward(const axon_norm_rotate_desc* desc, const void* dq_out,
                                      const void* dk_out, const void* q, const void* k,
                                      const int32_t* positions, const double* freqs,
                                      const float* q_weight, const float* k_weight, void* dq,
                                      void* dk, float* dq_weight, float* dk_weight,
                                      void* workspace, size_t workspace_bytes, void* stream) {
  using namespace axon;
  const axon_status why = check_desc(desc, true);
  if (why != AXON_OK) return why;
  const axon_norm_rotate_desc& d = *desc;
  const bool bf = d.act_dtype == AXON_BF16, with_k = d.k_heads > 0, any = d.rows > 0;
  const size_t es = bf ? 2 : 4;
  if (off(dq_weight, 4) || off(dk_weight, 4) || off(q_weight, 4) || (with_k && off(k_weight, 4)) ||
      (any && (bad(q, es) || bad(dq_out, es) || bad(dq, es) || bad(positions, 4) ||
               bad(freqs, 8) || (with_k && (bad(k, es) || bad(dk_out, es) || bad(dk, es))))))
    return AXON_ERR_INVALID_ARGUMENT;
  if (!with_k && dk_weight) return AXON_ERR_INVALID_ARGUMENT;
  const size_t need = axon_norm_rotate_backward_workspace_bytes(desc);
  if (workspace_bytes < need) return AXON_ERR_WORKSPACE_TOO_SMALL;
  if (need && bad(workspace, 16)) return AXON_ERR_INVALID_ARGUMENT;
  RotateArgs a = make_args(d);
  a.q = q, a.k = k, a.dq_out = dq_out, a.dk_out = dk_out, a.positions = positions, a.freqs = freqs;
  a.q_weight = q_weight, a.k_weight = with_k ? k_weight : nullptr;
  a.q_out = dq, a.k_out = dk, a.partial = static_cast<float*>(workspace);
  const int64_t qw = d.q_heads * d.head_dim, kw = d.k_heads * d.head_dim;
  const size_t d4 = 4 * size_t(d.head_dim);
  const Span in_dq = any ? rows_span(dq_out, d.rows, a.dq_stride, qw, es) : Span{};
  const Span in_dk = any && with_k ? rows_span(dk_out, d.rows, a.dk_stride, kw, es) : Span{};
  const Span reads[] = {any ? rows_span(q, d.rows, a.q_stride, qw, es) : Span{},
                        any && with_k ? rows_span(k, d.rows, a.k_stride, kw, es) : Span{},
                        span(positions, 4 * size_t(d.rows)),
                        span(freqs, any ? 4 * size_t(d.rotary_dim) : 0), span(q_weight, d4),
                        span(a.k_weight, d4)};
  const Span outs[] = {span(dq, es * size_t(d.rows * qw)),
                       with_k ? span(dk, es * size_t(d.rows * kw)) : Span{}, span(dq_weight, d4),
                       span(dk_weight, d4), span(workspace, need)};
  for (int i = 0; i < 5; ++i) {
    for (const Span& r : reads)
      if (overlaps(outs[i], r)) return AXON_ERR_INVALID_ARGUMENT;
    for (int j = 0; j < i; ++j)
      if (overlaps(outs[i], outs[j])) return AXON_ERR_INVALID_ARGUMENT;
    if (!(i == 0 && dq == dq_out && a.dq_stride == qw) && overlaps(outs[i], in_dq))
      return AXON_ERR_INVALID_ARGUMENT;
    if (!(i == 1 && dk == dk_out && a.dk_stride == kw) && overlaps(outs[i], in_dk))
      return AXON_ERR_INVALID_ARGUMENT;
  }
  hipStream_t st = static_cast<hipStream_t>(stream);
  if (any) {
    const bool wide = wide_ok(a, es, true, with_k);
    bf ? launch_rotate<bf16_bits, true>(a, wide, st) : launch_rotate<float, true>(a, wide, st);
  }
  if (dq_weight || dk_weight)
    hipLaunchKernelGGL(rotate_sum_kernel, dim3(static_cast<unsigned>(2 * d.head_dim)), dim3(64), 0,
                       st, a.partial, back_workgroups(d.rows), a.dim, dq_weight, dk_weight);
  return hipGetLastError() == hipSuccess ? AXON_OK : AXON_ERR_HIP;
}

}  // extern "C"

// Head norm with position rotation (see axonscan.h), forward and backward.
//
// With r = 1 / sqrt(mean(x^2) + eps), n = x r, z = n w and R the rotation: out = R z. Backward, with
// d = R^T dout: dw = sum d n, dn = d w, dx = r (dn - n mean(n dn)).
//
// A head is held by LANES lanes (a power of two), a lane holds up to UNITS pieces of 2 V of its
// channels: V of the first and V of the second halves of V pairs, or 2 V channels in order (pairs side
// by side, or not turned). A wave takes 64 / LANES heads at a time and one row's heads one group after
// the other, so that its angles are found once a row; where heads are few, the heads of several rows (ROWS).
// Angles: p freqs / (2 pi) turns in 64 bits, of which only the fraction goes to 32 bits: off by 2^-26 turns at most, 9e-8
// rad whatever the position, beside sine and cosine of 32 bits (a product in 64 bits a pair and row is what costs).
//
// Bound by memory: 16384 rows of 40 heads of 128 bf16 (336 MB) in 65-68 us, 5.0 TB/s where a copy of that
// type reaches 5.4. What it took from 81 us: groups of one tensor (pointers and weights the same in all
// lanes), sums whose exchanges are part of the addition, the values of five groups asked for before the
// first is used and without branches, stores past the caches.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <type_traits>

#include "axon_device.h"
#include "axon_packed.h"
#include "axon_wide.h"

namespace axon {
namespace {

constexpr int kWaves = 4;   // of a workgroup
constexpr int kFlush = 32;  // items: rows, or several rows where heads are few

// Backward workgroups that a CU holds at once, as registers allow; as many are started, since a second
// round of them finds the CUs half empty (16384 rows of 40 heads of 128 bf16 with four a CU 111 us, of which
// one head group a wave is asked for at a time; three a CU and two groups 120 us, and 150 us with four started.
// fp32, 8192 rows of 20 heads: 54 us and 48 us, for four spill). Of the 128 registers that four leave, one row a wave
// takes 125 or 127; several rows a wave spill two (pairs apart) or four (side by side).
template <typename Act>
constexpr int kBackFit = sizeof(Act) == 2 ? 4 : 3;
constexpr int kCus = 256;

struct RotateArgs {
  const void *q, *k, *dq_out, *dk_out;
  const int32_t* positions;
  const double* freqs;
  const float *q_weight, *k_weight;
  void *q_out, *k_out;  // dq, dk in the backward pass
  int64_t rows, q_stride, k_stride, dq_stride, dk_stride;
  int q_heads, heads, dim, rotary, lanes, interleaved;
  int splits;  // forward: waves that share a row's heads
  int group;   // heads of a row that a wave takes at a time; lanes beyond take other rows
  bool past;   // outputs are stored past the caches
  float eps, inv_dim;
  float* partial;  // backward: (workgroups, 2, dim)
};

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

// A unit's values as pairs (first[i], second[i]) that are turned together. SIDE: they lie side by side in
// the 2 V channels (where V is 1 they are the two pieces in any case).
template <typename Act, int V, bool SIDE>
struct Pairs {
  float first[V], second[V];
  __device__ __forceinline__ void set(const float* lo, const float* hi) {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      if constexpr (SIDE) {
        first[i] = 2 * i < V ? lo[2 * i] : hi[2 * i - V];
        second[i] = 2 * i < V ? lo[2 * i + 1] : hi[2 * i + 1 - V];
      } else {
        first[i] = lo[i], second[i] = hi[i];
      }
    }
  }
  __device__ __forceinline__ void take(const Raw<Act, V>* r) {
    float lo[V], hi[V];
    r[0].get(lo);
    r[1].get(hi);
    set(lo, hi);
  }
  template <bool PAST>
  __device__ __forceinline__ void store(Act* p, const Unit<V>& u) const {
    float z[2 * V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
      z[SIDE ? 2 * i : i] = first[i];
      z[SIDE ? 2 * i + 1 : V + i] = second[i];
    }
    Raw<Act, V>::template store<PAST>(p + u.lo, z);
    Raw<Act, V>::template store<PAST>(p + u.hi, z + V);
  }
};

// Sum over aligned groups of `lanes` lanes (a power of two): exchanges inside 16 lanes are part of the
// addition (neighbours, pairs, then mirrored halves, whose lanes hold the same sums already).
template <int CTRL>
__device__ __forceinline__ float add_dpp(float v) {
  return v + __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), CTRL, 0xF, 0xF, true));
}
__device__ __forceinline__ float sum_lanes(float v, int lanes) {
  if (lanes > 1) v = add_dpp<0xB1>(v);    // quad_perm [1,0,3,2]
  if (lanes > 2) v = add_dpp<0x4E>(v);    // quad_perm [2,3,0,1]
  if (lanes > 4) v = add_dpp<0x141>(v);   // row_half_mirror
  if (lanes > 8) v = add_dpp<0x140>(v);   // row_mirror
  if (lanes > 16) v += __shfl_xor(v, 16, 64);
  if (lanes > 32) v += __shfl_xor(v, 32, 64);
  return v;
}

// One tensor (q or k) of the call.
template <typename Act>
struct Tensor {
  const Act *x, *dy;
  Act* out;
  int64_t x_stride, dy_stride, out_stride;
  int heads;
  __device__ __forceinline__ Tensor(const RotateArgs& g, bool q)
      : x(static_cast<const Act*>(q ? g.q : g.k)),
        dy(static_cast<const Act*>(q ? g.dq_out : g.dk_out)),
        out(static_cast<Act*>(q ? g.q_out : g.k_out)),
        x_stride(q ? g.q_stride : g.k_stride),
        dy_stride(q ? g.dq_stride : g.dk_stride),
        heads(q ? g.q_heads : g.heads - g.q_heads) {
    out_stride = int64_t(heads) * g.dim;
  }
};

// Groups of heads are of q or of k, so that a wave's pointers and weights do not differ between lanes.
template <typename Act, int V, int UNITS, int G, bool SIDE, bool PAST, bool BACK, bool ROWS>
__global__ __launch_bounds__(64 * kWaves, BACK ? kBackFit<Act> : 1) void rotate_kernel(RotateArgs g) {
  using P = Pairs<Act, V, SIDE>;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int l = lane & (g.lanes - 1), place = lane / g.lanes, per = ROWS ? g.group : 64 / g.lanes;
  const int sub = ROWS ? place & (per - 1) : place;           // head of a group
  const int ahead = ROWS ? place / per : 0;                   // row of an item's
  const uint32_t together = ROWS ? 64 / (g.lanes * per) : 1;  // rows of an item
  const int q_groups = (g.q_heads + per - 1) / per, groups = q_groups + (g.heads - g.q_heads + per - 1) / per;
  P wq[UNITS], wk[UNITS], sq[BACK ? UNITS : 1], sk[BACK ? UNITS : 1];
  double turns[UNITS][V];
#pragma unroll
  for (int n = 0; n < UNITS; ++n) {
    const Unit<V> u(g, l + n * g.lanes);
    float lo[V], hi[V];
    auto weights = [&](const float* w, P& to) {
#pragma unroll
      for (int i = 0; i < V; ++i) {
        lo[i] = w ? w[min(u.lo + i, g.dim - 1)] : 1.0f;
        hi[i] = w ? w[min(u.hi + i, g.dim - 1)] : 1.0f;
      }
      to.set(lo, hi);
    };
    weights(g.q_weight, wq[n]);
    weights(g.k_weight, wk[n]);
#pragma unroll
    for (int i = 0; i < V; ++i) {
      turns[n][i] = g.freqs[min(u.pair + i, g.rotary / 2 - 1)] * 0.15915494309189533577;
      if constexpr (BACK) sq[n].first[i] = sq[n].second[i] = sk[n].first[i] = sk[n].second[i] = 0.0f;
    }
  }
  // Weight gradients: fp32 over up to kFlush items a lane, all head groups of their rows, 64 bits beyond; a
  // workgroup's part is rounded once to fp32.
  __shared__ double part[BACK ? kWaves : 1][2][BACK ? 256 : 1];
  auto flush = [&] {
#pragma unroll
    for (int n = 0; n < UNITS; ++n) {
      const Unit<V> u(g, l + n * g.lanes);
#pragma unroll
      for (int i = 0; i < V; ++i) {
        // lanes that hold the same channels of other heads, in a fixed order
        auto add = [&](float& v, int which, int at) {
          for (int d = g.lanes; d < 64; d <<= 1) v += __shfl_xor(v, d, 64);
          if (place == 0 && u.live) part[wave][which][at] += v;
          v = 0.0f;
        };
        const int first = SIDE ? (2 * i < V ? u.lo + 2 * i : u.hi + 2 * i - V) : u.lo + i;
        const int second = SIDE ? (2 * i < V ? u.lo + 2 * i + 1 : u.hi + 2 * i + 1 - V) : u.hi + i;
        add(sq[n].first[i], 0, first);
        add(sq[n].second[i], 0, second);
        add(sk[n].first[i], 1, first);
        add(sk[n].second[i], 1, second);
      }
    }
  };
  if constexpr (BACK) {
    for (int t = threadIdx.x; t < kWaves * 2 * 256; t += 64 * kWaves) (&part[0][0][0])[t] = 0.0;
    __syncthreads();
  }
  int pending = 0;
  // rows * splits < 2^31
  const uint32_t rows = static_cast<uint32_t>(g.rows), step = gridDim.x * kWaves;
  const uint32_t items = (ROWS ? (rows + together - 1) / together : rows) * g.splits;
  for (uint32_t item = blockIdx.x * kWaves + wave; item < items; item += step) {
    const uint32_t which = g.splits == 1 ? item : item / g.splits;
    const int split = static_cast<int>(item - which * g.splits);
    const bool held = !ROWS || which * together + ahead < rows;
    const uint32_t row = ROWS ? min(which * together + ahead, rows - 1) : which;
    P c[UNITS];  // cosines and sines of the row
    for (int first = split; first < groups; first += g.splits * G) {
      // The values of G groups are asked for before the first is used (and before the row's angles); places
      // that hold none read others' again, since loads behind branches wait for each other.
      const int position = g.positions[row];
      Raw<Act, V> rx[G][UNITS][2], rd[BACK ? G : 1][UNITS][2];
#pragma unroll
      for (int k = 0; k < G; ++k) {
        const int grp = min(first + k * g.splits, groups - 1);
        const Tensor<Act> t(g, grp < q_groups);
        const int head = min((grp < q_groups ? grp : grp - q_groups) * per + sub, t.heads - 1);
        const Act* x = t.x + row * t.x_stride;
        const Act* dy = t.dy + row * t.dy_stride;
#pragma unroll
        for (int n = 0; n < UNITS; ++n) {
          const Unit<V> u(g, l + n * g.lanes);
          const int lo = head * g.dim + (u.live ? u.lo : 0), hi = head * g.dim + (u.live ? u.hi : 0);
          rx[k][n][0].load(x + lo);
          rx[k][n][1].load(x + hi);
          if constexpr (BACK) {
            rd[k][n][0].load(dy + lo);
            rd[k][n][1].load(dy + hi);
          }
        }
      }
      if (first == split) {
#pragma unroll
        for (int n = 0; n < UNITS; ++n) {
          const bool turned = Unit<V>(g, l + n * g.lanes).turned;
#pragma unroll
          for (int i = 0; i < V; ++i) {
            const double t = position * turns[n][i];
            sincospif(2.0f * static_cast<float>(t - rint(t)), &c[n].second[i], &c[n].first[i]);
            if (!turned) c[n].first[i] = 1.0f, c[n].second[i] = 0.0f;
          }
        }
      }
#pragma unroll
      for (int k = 0; k < G; ++k) {
        const int grp = first + k * g.splits;
        if (grp >= groups) break;
        const bool is_q = grp < q_groups;
        const Tensor<Act> t(g, is_q);
        const int head = (is_q ? grp : grp - q_groups) * per;
        const bool in = held && head + sub < t.heads;
        Act* out = t.out + row * t.out_stride + int64_t(head) * g.dim;
        P v[UNITS];
        float sum = 0.0f;
#pragma unroll
        for (int n = 0; n < UNITS; ++n) {
          const Unit<V> u(g, l + n * g.lanes);
#pragma unroll
          for (int i = 0; i < V; ++i) v[n].first[i] = v[n].second[i] = 0.0f;
          if (in && u.live) v[n].take(rx[k][n]);
#pragma unroll
          for (int i = 0; i < V; ++i) {
            sum = fmaf(v[n].first[i], v[n].first[i], sum);
            sum = fmaf(v[n].second[i], v[n].second[i], sum);
          }
        }
        const float r = __builtin_amdgcn_rsqf(fmaf(sum_lanes(sum, g.lanes), g.inv_dim, g.eps));
        auto head_of = [&](const P* w, P* total) {
          if constexpr (!BACK) {
#pragma unroll
            for (int n = 0; n < UNITS; ++n) {
              const Unit<V> u(g, l + n * g.lanes);
#pragma unroll
              for (int i = 0; i < V; ++i) {
                const float a = v[n].first[i] * (r * w[n].first[i]), b = v[n].second[i] * (r * w[n].second[i]);
                v[n].first[i] = a * c[n].first[i] - b * c[n].second[i];
                v[n].second[i] = b * c[n].first[i] + a * c[n].second[i];
              }
              if (in && u.live) v[n].template store<PAST>(out + sub * g.dim, u);
            }
          } else {
            P d[UNITS];
            float dot = 0.0f;
#pragma unroll
            for (int n = 0; n < UNITS; ++n) {
              const Unit<V> u(g, l + n * g.lanes);
              const bool live = in && u.live;
#pragma unroll
              for (int i = 0; i < V; ++i) d[n].first[i] = d[n].second[i] = 0.0f;
              if (live) d[n].take(rd[k][n]);
#pragma unroll
              for (int i = 0; i < V; ++i) {
                const float a = d[n].first[i], b = d[n].second[i];
                float da = a * c[n].first[i] + b * c[n].second[i];
                float db = b * c[n].first[i] - a * c[n].second[i];
                v[n].first[i] *= r, v[n].second[i] *= r;  // n
                if (live) {
                  total[n].first[i] = fmaf(da, v[n].first[i], total[n].first[i]);
                  total[n].second[i] = fmaf(db, v[n].second[i], total[n].second[i]);
                }
                da *= w[n].first[i], db *= w[n].second[i];
                dot = fmaf(da, v[n].first[i], dot);
                dot = fmaf(db, v[n].second[i], dot);
                d[n].first[i] = da, d[n].second[i] = db;
              }
            }
            const float mean = sum_lanes(dot, g.lanes) * g.inv_dim;
#pragma unroll
            for (int n = 0; n < UNITS; ++n) {
              const Unit<V> u(g, l + n * g.lanes);
#pragma unroll
              for (int i = 0; i < V; ++i) {
                d[n].first[i] = r * fmaf(-v[n].first[i], mean, d[n].first[i]);
                d[n].second[i] = r * fmaf(-v[n].second[i], mean, d[n].second[i]);
              }
              if (in && u.live) d[n].template store<PAST>(out + sub * g.dim, u);
            }
          }
        };
        if (is_q) head_of(wq, sq);
        else head_of(wk, sk);
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

// Sums of the workgroups' parts, 16 of the 2 D values a workgroup: 64 threads take a value's parts in turn,
// in 64 bits, joined in a fixed order.
constexpr int kSumWaves = 16, kSumValues = 16;
__global__ __launch_bounds__(64 * kSumWaves) void rotate_sum_kernel(const float* partial, int parts, int dim,
                                                                    float* dq_weight, float* dk_weight) {
  __shared__ double part[kSumWaves][kSumValues];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int t = blockIdx.x * kSumValues + (threadIdx.x & (kSumValues - 1));
  double s = 0.0;
  if (t < 2 * dim) {
#pragma unroll 8
    for (int p = threadIdx.x / kSumValues; p < parts; p += 64 * kSumWaves / kSumValues)
      s += partial[int64_t(p) * 2 * dim + t];
  }
  for (int d = kSumValues; d < 64; d <<= 1) s += __shfl_xor(s, d, 64);
  if (lane < kSumValues) part[wave][lane] = s;
  __syncthreads();
  if (threadIdx.x >= kSumValues || t >= 2 * dim) return;
  s = 0.0;
#pragma unroll
  for (int w = 0; w < kSumWaves; ++w) s += part[w][threadIdx.x];
  float* out = t < dim ? dq_weight : dk_weight;
  if (out) out[t < dim ? t : t - dim] = static_cast<float>(s);
}

// Workgroups that run at once and take item after item, so that weights and frequencies are read seldom. Forward
// five a CU, of fp32 or of several rows four (16384 rows of 40 heads of 128 bf16 67 us, six 69 us; fp32, 32768 rows
// of 16 heads of 64: four 45 us, five 49 us).
int64_t forward_workgroups(bool bf16, bool rows) { return kCus * (bf16 && !rows ? 5 : 4); }
int back_workgroups(int64_t rows, bool bf16) {
  const int64_t most = kCus * (bf16 ? kBackFit<bf16_bits> : kBackFit<float>);
  return static_cast<int>(std::min((rows + kWaves - 1) / kWaves, most));
}

template <typename Act, int V, int UNITS, bool SIDE, bool BACK>
void launch_units(RotateArgs a, hipStream_t st) {
  constexpr bool bf16 = sizeof(Act) == 2;
  constexpr int G = BACK ? (bf16 ? 1 : 2) : V == 1 ? 2 : 5;
  const int per = 64 / a.lanes, k_heads = a.heads - a.q_heads;
  auto groups_of = [&](int n) { return (a.q_heads + n - 1) / n + (k_heads + n - 1) / n; };
  // Heads of a wave at a time: as many as leave no more than a quarter of its places empty. Where one row cannot
  // fill them a wave takes several (131072 rows of 1 + 1 heads of 64 bf16 93 -> 21 us, backward 136 -> 34 us).
  a.group = per;
  while (a.group > 1 && 4 * groups_of(a.group) * a.group > 5 * a.heads) a.group /= 2;
  const int groups = groups_of(a.group), together = per / a.group;
  const int64_t items = (a.rows + together - 1) / together;
  int64_t wgs = back_workgroups(a.rows, bf16);
  a.splits = 1;
  if constexpr (!BACK) {
    // A row's heads are shared out to as many waves as keep G groups each: more even than whole rows (73 us
    // against 77 us), and a decode batch has as many waves as it can.
    a.splits = static_cast<int>(std::min<int64_t>((groups + G - 1) / G, ((int64_t(1) << 31) - 1) / a.rows));
    wgs = std::min<int64_t>((items * a.splits + kWaves - 1) / kWaves,
                            forward_workgroups(bf16, together > 1));
  }
  const dim3 grid(static_cast<unsigned>(wgs)), threads(64 * kWaves);
  auto launch = [&](auto past, auto rows) {
    hipLaunchKernelGGL((rotate_kernel<Act, V, UNITS, G, SIDE, decltype(past)::value, BACK, decltype(rows)::value>),
                       grid, threads, 0, st, a);
  };
  const std::bool_constant<V == 4> past;  // one channel at a time is not stored so
  const std::true_type yes;
  const std::false_type no;
  if (past && a.past) together > 1 ? launch(past, yes) : launch(past, no);
  else together > 1 ? launch(no, yes) : launch(no, no);
}

template <typename Act, bool BACK>
void launch_rotate(RotateArgs a, bool wide, hipStream_t st) {
  const int units = a.dim / (wide ? 8 : 2);
  a.lanes = 1;
  while (a.lanes < 64 && a.lanes < units) a.lanes *= 2;
  if (wide && a.interleaved) launch_units<Act, 4, 1, true, BACK>(a, st);
  else if (wide) launch_units<Act, 4, 1, false, BACK>(a, st);
  else if (units <= 64) launch_units<Act, 1, 1, false, BACK>(a, st);
  else launch_units<Act, 1, 2, false, BACK>(a, st);
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
  a.past = past_caches(es * size_t(d.rows * (qw + kw)));
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
  return 4 * 2 * size_t(axon::back_workgroups(desc->rows, desc->act_dtype == AXON_BF16)) * size_t(desc->head_dim);
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
  a.past = past_caches(es * size_t(d.rows * (qw + kw)));
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
    hipLaunchKernelGGL(rotate_sum_kernel, dim3(static_cast<unsigned>((2 * d.head_dim + kSumValues - 1) / kSumValues)),
                       dim3(64 * kSumWaves), 0, st, a.partial, back_workgroups(d.rows, bf), a.dim, dq_weight, dk_weight);
  return hipGetLastError() == hipSuccess ? AXON_OK : AXON_ERR_HIP;
}

}  // extern "C"

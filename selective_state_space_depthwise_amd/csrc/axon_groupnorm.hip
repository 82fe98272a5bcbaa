// Group norm over the channels of one token, with its activation and gate (see axonscan.h).
//
// A group's values are read once, kept in registers as fp32 and written once, so HBM traffic is the
// tensors themselves; mean and variance are two passes over the registers (the variance of values
// already centred, which does not cancel). Two kernels:
//   norm_lanes_kernel   groups of up to 2048 channels: LPG lanes (a power of two, 4 .. 64) hold a
//                       group, up to 32 values each, reduced by lane exchanges; a workgroup of 4
//                       waves holds 256 / LPG groups.
//   norm_wide_kernel    a workgroup holds a group: up to 32 values a thread in registers, and
//                       groups beyond that are read again for the second and third pass (from L2).
// Values are read 16 bytes a lane where rows, width and alignment allow (VEC = 4 fp32, 8 bf16),
// else one by one. Bound by HBM: 16384 rows x 7680 bf16 with a gate (755 MB) 132 us, 5.7 TB/s;
// 5001 x 8 groups of 236 fp32 (75 MB) 19 us, 4.0 TB/s. One by one 16384 rows x 1004 bf16 take 78 us
// (x 1008: 12 us).
#include <hip/hip_runtime.h>

#include <cmath>
#include <cstdint>

#include "axon_device.h"
#include "axon_internal.h"

namespace axon {
namespace {

constexpr int kMaxValues = 32;  // of a group, held by one lane

struct NormArgs {
  const void *x, *z;
  const float *weight, *bias;
  void* y;
  int64_t total;  // rows * groups
  int64_t x_stride, z_stride;
  int groups, width, lanes;  // lanes: of one group (norm_lanes_kernel)
  float eps, inv_width;
  int centered, silu_out, gate, shared;
};

// VEC consecutive values as loaded, and as fp32. Loads are issued for everything a lane holds before
// the first value is used (their addresses are clamped instead of branched around).
template <typename Act, int VEC>
struct Raw;
template <typename Act>
struct Raw<Act, 1> {
  Act v;
  __device__ __forceinline__ void load(const Act* p) { v = *p; }
  __device__ __forceinline__ void get(float* out) const {
    if constexpr (sizeof(Act) == 4) out[0] = v;
    else out[0] = bf16_to_f32(v);
  }
};
template <>
struct Raw<float, 4> {
  float4 v;
  __device__ __forceinline__ void load(const float* p) { v = *reinterpret_cast<const float4*>(p); }
  __device__ __forceinline__ void get(float* out) const { out[0] = v.x, out[1] = v.y, out[2] = v.z, out[3] = v.w; }
};
template <>
struct Raw<bf16_bits, 8> {
  uint4 v;
  __device__ __forceinline__ void load(const bf16_bits* p) { v = *reinterpret_cast<const uint4*>(p); }
  __device__ __forceinline__ void get(float* out) const {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      out[2 * i] = __uint_as_float(w[i] << 16);
      out[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
  }
};
template <int VEC>
__device__ __forceinline__ void load_params(const float* p, float* v) {
  if constexpr (VEC == 1) {
    v[0] = p[0];
  } else {
#pragma unroll
    for (int j = 0; j < VEC; j += 4) {
      const float4 t = *reinterpret_cast<const float4*>(p + j);
      v[j] = t.x, v[j + 1] = t.y, v[j + 2] = t.z, v[j + 3] = t.w;
    }
  }
}
template <int VEC>
__device__ __forceinline__ void store_vec(float* p, const float* v) {
  if constexpr (VEC == 4)
    *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
  else
    p[0] = v[0];
}
template <int VEC>
__device__ __forceinline__ void store_vec(bf16_bits* p, const float* v) {
  if constexpr (VEC == 8) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      w[i] = static_cast<uint32_t>(f32_to_bf16(v[2 * i])) |
             static_cast<uint32_t>(f32_to_bf16(v[2 * i + 1])) << 16;
    *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
  } else {
    p[0] = f32_to_bf16(v[0]);
  }
}

// A launch holds fewer than 2^32 threads along x, so workgroups beyond kGridX go along y.
constexpr int64_t kGridX = 1 << 20;

dim3 grid_of(int64_t wgs) {
  if (wgs <= kGridX) return dim3(static_cast<unsigned>(wgs));
  return dim3(static_cast<unsigned>(kGridX), static_cast<unsigned>((wgs + kGridX - 1) / kGridX));
}
__device__ __forceinline__ int64_t wg_index() {
  return int64_t(blockIdx.y) * gridDim.x + blockIdx.x;
}

template <typename Act, int VEC>
__device__ __forceinline__ void finish(const NormArgs& a, int64_t row, int grp, int c, float* n,
                                       const float* gz) {
  const int wi = (a.shared ? 0 : grp * a.width) + c;
  float t[VEC];
  if (a.weight) {
    load_params<VEC>(a.weight + wi, t);
#pragma unroll
    for (int e = 0; e < VEC; ++e) n[e] *= t[e];
  }
  if (a.bias) {
    load_params<VEC>(a.bias + wi, t);
#pragma unroll
    for (int e = 0; e < VEC; ++e) n[e] += t[e];
  }
  if (a.silu_out) {
#pragma unroll
    for (int e = 0; e < VEC; ++e) n[e] = silu(n[e]);
  }
  if (a.gate == AXON_GATE_AFTER) {
#pragma unroll
    for (int e = 0; e < VEC; ++e) n[e] *= gz[e];
  }
  Act* y = static_cast<Act*>(a.y) + (row * a.groups + grp) * int64_t(a.width) + c;
  store_vec<VEC>(y, n);
}

// x and z of VEC channels from c on, and then u (gated before) and SiLU(z).
template <typename Act, int VEC>
struct Fetched {
  Raw<Act, VEC> x, z;
  __device__ __forceinline__ void load(const NormArgs& a, int64_t row, int grp, int c) {
    const int64_t off = int64_t(grp) * a.width + c;
    x.load(static_cast<const Act*>(a.x) + row * a.x_stride + off);
    if (a.gate != AXON_GATE_NONE) z.load(static_cast<const Act*>(a.z) + row * a.z_stride + off);
  }
  __device__ __forceinline__ void get(const NormArgs& a, float* u, float* gz) const {
    x.get(u);
    if (a.gate != AXON_GATE_NONE) {
      z.get(gz);
#pragma unroll
      for (int e = 0; e < VEC; ++e) gz[e] = silu(gz[e]);
      if (a.gate == AXON_GATE_BEFORE) {
#pragma unroll
        for (int e = 0; e < VEC; ++e) u[e] *= gz[e];
      }
    }
  }
};

__device__ __forceinline__ float reduce_lanes(float v, int lanes) {
  for (int d = lanes >> 1; d > 0; d >>= 1) v += __shfl_xor(v, d, 64);
  return v;
}

// (Four groups a lane set, all loaded before the first is reduced, gained nothing: 5001 x 8 groups of
// 236 fp32 take 20 us either way.)
template <typename Act, int VEC, int R>
__global__ __launch_bounds__(256) void norm_lanes_kernel(NormArgs a) {
  const int l = threadIdx.x & (a.lanes - 1);
  const int64_t gi = wg_index() * (256 / a.lanes) + threadIdx.x / a.lanes;
  // Lanes without a group take part in the exchanges with the last one's values.
  const bool live = gi < a.total;
  const int64_t row = (live ? gi : a.total - 1) / a.groups;
  const int grp = static_cast<int>((live ? gi : a.total - 1) - row * a.groups);
  Fetched<Act, VEC> f[R];
#pragma unroll
  for (int j = 0; j < R; ++j) {
    const int c = (j * a.lanes + l) * VEC;
    f[j].load(a, row, grp, c < a.width ? c : 0);
  }
  float u[R * VEC], gz[R * VEC];
#pragma unroll
  for (int j = 0; j < R; ++j) {
    f[j].get(a, u + j * VEC, gz + j * VEC);
    if ((j * a.lanes + l) * VEC >= a.width) {
#pragma unroll
      for (int e = 0; e < VEC; ++e) u[j * VEC + e] = 0.0f;
    }
  }
  if (a.centered) {
    float s = 0.0f;
#pragma unroll
    for (int j = 0; j < R * VEC; ++j) s += u[j];
    const float mean = reduce_lanes(s, a.lanes) * a.inv_width;
#pragma unroll
    for (int j = 0; j < R; ++j) {
      const bool in = (j * a.lanes + l) * VEC < a.width;
#pragma unroll
      for (int e = 0; e < VEC; ++e) u[j * VEC + e] = in ? u[j * VEC + e] - mean : 0.0f;
    }
  }
  float q = 0.0f;
#pragma unroll
  for (int j = 0; j < R * VEC; ++j) q = fmaf(u[j], u[j], q);
  const float rs = 1.0f / sqrtf(reduce_lanes(q, a.lanes) * a.inv_width + a.eps);
#pragma unroll
  for (int j = 0; j < R; ++j) {
    const int c = (j * a.lanes + l) * VEC;
    if (live && c < a.width) {
      float n[VEC];
#pragma unroll
      for (int e = 0; e < VEC; ++e) n[e] = u[j * VEC + e] * rs;
      finish<Act, VEC>(a, row, grp, c, n, gz + j * VEC);
    }
  }
}

template <int THREADS>
__device__ __forceinline__ float reduce_wg(float v, float* part) {
  v = reduce_lanes(v, 64);
  if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = v;
  __syncthreads();
  float s = 0.0f;
#pragma unroll
  for (int w = 0; w < THREADS / 64; ++w) s += part[w];
  __syncthreads();
  return s;
}

template <typename Act, int VEC, int R, int THREADS, bool HELD>
__global__ __launch_bounds__(THREADS) void norm_wide_kernel(NormArgs a) {
  __shared__ float part[THREADS / 64];
  const int64_t gi = wg_index();
  if (gi >= a.total) return;
  const int64_t row = gi / a.groups;
  const int grp = static_cast<int>(gi - row * a.groups);
  const int step = THREADS * VEC, first = threadIdx.x * VEC;
  float u[R * VEC], gz[R * VEC];
  float mean = 0.0f;
  Fetched<Act, VEC> f[R];
  if constexpr (HELD) {
    float s = 0.0f;
#pragma unroll
    for (int j = 0; j < R; ++j) {
      const int c = j * step + first;
      f[j].load(a, row, grp, c < a.width ? c : 0);
    }
#pragma unroll
    for (int j = 0; j < R; ++j) {
      f[j].get(a, u + j * VEC, gz + j * VEC);
      if (j * step + first >= a.width) {
#pragma unroll
        for (int e = 0; e < VEC; ++e) u[j * VEC + e] = 0.0f;
      }
    }
    if (a.centered) {
#pragma unroll
      for (int j = 0; j < R * VEC; ++j) s += u[j];
      mean = reduce_wg<THREADS>(s, part) * a.inv_width;
#pragma unroll
      for (int j = 0; j < R; ++j)
#pragma unroll
        for (int e = 0; e < VEC; ++e)
          u[j * VEC + e] = j * step + first < a.width ? u[j * VEC + e] - mean : 0.0f;
    }
    float q = 0.0f;
#pragma unroll
    for (int j = 0; j < R * VEC; ++j) q = fmaf(u[j], u[j], q);
    const float rs = 1.0f / sqrtf(reduce_wg<THREADS>(q, part) * a.inv_width + a.eps);
#pragma unroll
    for (int j = 0; j < R; ++j) {
      const int c = j * step + first;
      if (c < a.width) {
        float n[VEC];
#pragma unroll
        for (int e = 0; e < VEC; ++e) n[e] = u[j * VEC + e] * rs;
        finish<Act, VEC>(a, row, grp, c, n, gz + j * VEC);
      }
    }
  } else {
    // A thread adds up to 2^20 values here, often alike, where the roundings of an fp32 sum would not
    // average out: its own part of a sum is held in 64 bits (8192 x 8201 bf16: 149 -> 151 us).
    if (a.centered) {
      double sum = 0.0;
      for (int64_t c = first; c < a.width; c += step) {
        f[0].load(a, row, grp, static_cast<int>(c));
        f[0].get(a, u, gz);
#pragma unroll
        for (int e = 0; e < VEC; ++e) sum += u[e];
      }
      mean = reduce_wg<THREADS>(static_cast<float>(sum), part) * a.inv_width;
    }
    double q = 0.0;
    for (int64_t c = first; c < a.width; c += step) {
      f[0].load(a, row, grp, static_cast<int>(c));
      f[0].get(a, u, gz);
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        const float d = u[e] - mean;
        q += static_cast<double>(d) * d;
      }
    }
    const float rs = 1.0f / sqrtf(reduce_wg<THREADS>(static_cast<float>(q), part) * a.inv_width + a.eps);
    // In place a thread overwrites only what it alone reads in this pass; the passes before it
    // ended at the barriers of the sums.
    for (int64_t c = first; c < a.width; c += step) {
      f[0].load(a, row, grp, static_cast<int>(c));
      f[0].get(a, u, gz);
      float n[VEC];
#pragma unroll
      for (int e = 0; e < VEC; ++e) n[e] = (u[e] - mean) * rs;
      finish<Act, VEC>(a, row, grp, static_cast<int>(c), n, gz);
    }
  }
}

template <typename Act, int VEC>
void launch_norm(NormArgs a, hipStream_t st) {
  const int64_t vecs = (int64_t(a.width) + VEC - 1) / VEC;
  constexpr int kMaxR = kMaxValues / VEC;
  if (vecs <= 64 * (VEC == 1 ? 8 : kMaxR)) {
    // One vector a lane where 64 lanes suffice (more lanes in flight), then up to kMaxR.
    int lanes = 4;
    while (lanes < 64 && lanes < vecs) lanes *= 2;
    a.lanes = lanes;
    const int64_t r = (vecs + lanes - 1) / lanes;
    const int64_t per = 256 / lanes;
    const dim3 grid = grid_of((a.total + per - 1) / per);
    if (r <= 1)
      hipLaunchKernelGGL((norm_lanes_kernel<Act, VEC, 1>), grid, dim3(256), 0, st, a);
    else if (r <= 2)
      hipLaunchKernelGGL((norm_lanes_kernel<Act, VEC, 2>), grid, dim3(256), 0, st, a);
    else if (VEC == 8 || r <= 4)
      hipLaunchKernelGGL((norm_lanes_kernel<Act, VEC, 4>), grid, dim3(256), 0, st, a);
    else
      hipLaunchKernelGGL((norm_lanes_kernel<Act, VEC, VEC == 8 ? 4 : 8>), grid, dim3(256), 0, st, a);
    return;
  }
  const dim3 grid = grid_of(a.total);
  if (vecs <= 256 * kMaxR)
    hipLaunchKernelGGL((norm_wide_kernel<Act, VEC, kMaxR, 256, true>), grid, dim3(256), 0, st, a);
  else
    hipLaunchKernelGGL((norm_wide_kernel<Act, VEC, 1, 1024, false>), grid, dim3(1024), 0, st, a);
}

template <typename Act>
void launch_norm_act(const NormArgs& a, hipStream_t st) {
  constexpr int VEC = 16 / sizeof(Act);
  auto even = [](const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; };
  const bool z = a.gate != AXON_GATE_NONE;
  const bool wide = a.width % VEC == 0 && a.x_stride % VEC == 0 && even(a.x) && even(a.y) &&
                    even(a.weight) && even(a.bias) && (!z || (a.z_stride % VEC == 0 && even(a.z)));
  if (wide)
    launch_norm<Act, VEC>(a, st);
  else
    launch_norm<Act, 1>(a, st);
}

}  // namespace
}  // namespace axon

extern "C" {

axon_status axon_group_norm(const axon_group_norm_desc* d, const void* x, const void* z,
                            const float* weight, const float* bias, void* y, void* stream) {
  using namespace axon;
  if (!d) return AXON_ERR_INVALID_ARGUMENT;
  if (d->rows < 0 || d->groups < 1 || d->width < 1 || d->x_stride < 0 || d->z_stride < 0)
    return AXON_ERR_INVALID_ARGUMENT;
  if ((d->act_dtype != AXON_F32 && d->act_dtype != AXON_BF16) ||
      (d->activation != AXON_ACT_NONE && d->activation != AXON_ACT_SILU) ||
      (d->gate != AXON_GATE_NONE && d->gate != AXON_GATE_BEFORE && d->gate != AXON_GATE_AFTER) ||
      (d->centered != 0 && d->centered != 1) || (d->shared_weights != 0 && d->shared_weights != 1))
    return AXON_ERR_UNSUPPORTED;
  if (!std::isfinite(d->eps) || d->eps < 0.0f) return AXON_ERR_INVALID_ARGUMENT;
  int64_t chans, total, elems;
  if (__builtin_mul_overflow(d->groups, d->width, &chans) || chans > (int64_t(1) << 30) ||
      __builtin_mul_overflow(d->rows, d->groups, &total) || total >= (int64_t(1) << 31) ||
      __builtin_mul_overflow(d->rows, chans, &elems) || elems > (int64_t(1) << 40))
    return AXON_ERR_UNSUPPORTED;
  const int64_t xs = d->x_stride ? d->x_stride : chans, zs = d->z_stride ? d->z_stride : chans;
  const bool gated = d->gate != AXON_GATE_NONE;
  if (xs < chans || (gated && zs < chans)) return AXON_ERR_INVALID_ARGUMENT;
  if (xs > (int64_t(1) << 31) || (gated && zs > (int64_t(1) << 31))) return AXON_ERR_UNSUPPORTED;
  if (d->rows == 0) return AXON_OK;
  const size_t es = d->act_dtype == AXON_BF16 ? 2 : 4;
  auto bad = [](const void* p, size_t a) { return !p || (reinterpret_cast<uintptr_t>(p) & (a - 1)); };
  if (bad(x, es) || bad(y, es) || (gated && bad(z, es)) || (weight && bad(weight, 4)) ||
      (bias && bad(bias, 4)))
    return AXON_ERR_INVALID_ARGUMENT;
  const size_t wn = 4 * size_t(d->shared_weights ? d->width : chans);
  const Span out = span(y, es * size_t(elems));
  const Span in_x = span(x, es * size_t((d->rows - 1) * xs + chans));
  const bool in_place = x == y && xs == chans;
  if (!in_place && overlaps(out, in_x)) return AXON_ERR_INVALID_ARGUMENT;
  if (gated && overlaps(out, span(z, es * size_t((d->rows - 1) * zs + chans))))
    return AXON_ERR_INVALID_ARGUMENT;
  if (overlaps(out, span(weight, wn)) || overlaps(out, span(bias, wn)))
    return AXON_ERR_INVALID_ARGUMENT;
  NormArgs a;
  a.x = x, a.z = z, a.weight = weight, a.bias = bias, a.y = y;
  a.total = total, a.x_stride = xs, a.z_stride = zs;
  a.groups = static_cast<int>(d->groups), a.width = static_cast<int>(d->width), a.lanes = 0;
  a.eps = d->eps, a.inv_width = 1.0f / static_cast<float>(d->width);
  a.centered = d->centered, a.silu_out = d->activation == AXON_ACT_SILU, a.gate = d->gate;
  a.shared = d->shared_weights;
  hipStream_t st = static_cast<hipStream_t>(stream);
  if (d->act_dtype == AXON_BF16)
    launch_norm_act<bf16_bits>(a, st);
  else
    launch_norm_act<float>(a, st);
  return hipGetLastError() == hipSuccess ? AXON_OK : AXON_ERR_HIP;
}

}  // extern "C"

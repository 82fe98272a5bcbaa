// Several channels of a row at once (gfx950).
#pragma once

#include <hip/hip_runtime.h>

#include "axon_device.h"

namespace axon {

// V channels as loaded, and as fp32.
template <typename Act, int V>
struct Raw {
  Act v;
  __device__ __forceinline__ void load(const Act* p) { v = *p; }
  __device__ __forceinline__ void get(float* o) const { o[0] = load_act(&v, 0); }
  template <bool>
  static __device__ __forceinline__ void store(Act* p, const float* o) { store_act(p, 0, o[0]); }
};
template <>
struct Raw<float, 4> {
  float4 v;
  __device__ __forceinline__ void load(const float* p) { v = *reinterpret_cast<const float4*>(p); }
  __device__ __forceinline__ void get(float* o) const { o[0] = v.x, o[1] = v.y, o[2] = v.z, o[3] = v.w; }
  template <bool PAST>
  static __device__ __forceinline__ void store(float* p, const float* o) { store4<PAST>(p, o); }
};
__device__ __forceinline__ void widen2(uint32_t w, float* o) {
  o[0] = __uint_as_float(w << 16), o[1] = __uint_as_float(w & 0xFFFF0000u);
}
template <>
struct Raw<bf16_bits, 2> {
  uint32_t v;
  __device__ __forceinline__ void load(const bf16_bits* p) { v = *reinterpret_cast<const uint32_t*>(p); }
  __device__ __forceinline__ void get(float* o) const { widen2(v, o); }
  template <bool>
  static __device__ __forceinline__ void store(bf16_bits* p, const float* o) {
    *reinterpret_cast<uint32_t*>(p) = f32_to_bf16x2(o[0], o[1]);
  }
};
template <>
struct Raw<bf16_bits, 4> {
  uint2 v;
  __device__ __forceinline__ void load(const bf16_bits* p) { v = *reinterpret_cast<const uint2*>(p); }
  __device__ __forceinline__ void get(float* o) const { widen2(v.x, o), widen2(v.y, o + 2); }
  template <bool PAST>
  static __device__ __forceinline__ void store(bf16_bits* p, const float* o) { store4<PAST>(p, o); }
};

}  // namespace axon

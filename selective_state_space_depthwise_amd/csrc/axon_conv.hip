// Causal depthwise convolution of width 4 over packed or uniform sequences (see axonscan.h).
//
// A thread walks one channel of a block of 64 tokens with the last three inputs in registers.
// Only a sequence's first block reads its cache, and the same thread then writes the final cache from
// the sequence's last inputs, so that a cache may be updated in place without a wait between threads.
//
// Backward, with s_t = dy_t act'(p_t):  dxx_t = sum_k w[k] s_{t+3-k} + what dcache_out has for t,
// dw[k] = sum_t s_t xx_{t-3+k},  db = sum_t s_t.  A block finds s of the three tokens behind it again.
#include <hip/hip_runtime.h>

#include <cmath>
#include <cstdint>

#include "axon_device.h"
#include "axon_packed.h"

namespace axon {
namespace {

constexpr int kSums = kConv + 1;  // dw and db

struct ConvArgs {
  const void *x, *dy;
  const float *w, *b;
  Packed p;
  int64_t x_stride, dy_stride;
  int channels, silu, clear_behind;
  const float* cache_in;
  const int32_t *in_slots, *out_slots;
  int64_t in_count, out_count;
  float* cache_out;
  void* y;
  // backward
  const float* dcache_out;
  void* dx;
  float *dw, *db, *dcache_in;
  float* partial;  // (rows, kSums, channels)
};

// The cache of sequence n at channel e, zeros where there is none.
__device__ __forceinline__ void load_cache(const ConvArgs& g, int n, int e, float* c) {
  c[0] = c[1] = c[2] = 0.0f;
  if (!g.cache_in) return;
  const int64_t slot = g.in_slots ? g.in_slots[n] : n;
  if (slot < 0 || slot >= g.in_count) return;
#pragma unroll
  for (int j = 0; j < kHalo; ++j) c[j] = g.cache_in[(slot * kHalo + j) * g.channels + e];
}
__device__ __forceinline__ void store_cache(const ConvArgs& g, int n, int e, const float* c) {
  if (!g.cache_out) return;
  const int64_t slot = g.out_slots ? g.out_slots[n] : n;
  if (slot < 0 || slot >= g.out_count) return;
#pragma unroll
  for (int j = 0; j < kHalo; ++j) g.cache_out[(slot * kHalo + j) * g.channels + e] = c[j];
}

__device__ __forceinline__ float convolve(const float* w, float b, float x0, float x1, float x2,
                                          float x3) {
  return fmaf(w[3], x3, fmaf(w[2], x2, fmaf(w[1], x1, fmaf(w[0], x0, b))));
}

template <typename Act>
__global__ __launch_bounds__(64) void conv_kernel(ConvArgs g) {
  const int e = blockIdx.x * 64 + threadIdx.x, row = blockIdx.y + blockIdx.z * gridDim.y;
  const int rows = gridDim.y * gridDim.z;
  if (e >= g.channels) return;
  const Act* x = static_cast<const Act*>(g.x) + e;
  Act* y = static_cast<Act*>(g.y) + e;
  const BlockAt b = block_at(g.p, row);
  if (b.seq >= 0) {
    float w[kConv], h[kHalo];
#pragma unroll
    for (int k = 0; k < kConv; ++k) w[k] = g.w[int64_t(e) * kConv + k];
    const float bias = g.b ? g.b[e] : 0.0f;
    if (b.begins) {
      load_cache(g, b.seq, e, h);
      const int len = packed_start(g.p, b.seq + 1) - b.first;
      float c[kHalo];
#pragma unroll
      for (int j = 0; j < kHalo; ++j) {
        const int at = len - kHalo + j;  // -2 .. of the sequence
        c[j] = at >= 0 ? load_act(x, (b.first + at) * g.x_stride) : at == -2 ? h[1] : h[2];
      }
      store_cache(g, b.seq, e, c);
    } else {
#pragma unroll
      for (int j = 0; j < kHalo; ++j) h[j] = load_act(x, (b.first - kHalo + j) * g.x_stride);
    }
    for (int j = 0; j < b.count; ++j) {
      const float v = load_act(x, (int64_t(b.first) + j) * g.x_stride);
      float p = convolve(w, bias, h[0], h[1], h[2], v);
      if (g.silu) p = silu(p);
      store_act(y, (int64_t(b.first) + j) * g.channels, p);
      h[0] = h[1], h[1] = h[2], h[2] = v;
    }
  }
  for (int n = row; n < g.p.sequences; n += rows)
    if (packed_start(g.p, n) >= packed_start(g.p, n + 1)) {
      float c[kHalo];
      load_cache(g, n, e, c);
      store_cache(g, n, e, c);
    }
  if (g.clear_behind)
    for (int64_t t = int64_t(packed_start(g.p, g.p.sequences)) + row; t < g.p.tokens; t += rows)
      store_act(y, t * g.channels, 0.0f);
}

template <typename Act>
__global__ __launch_bounds__(64) void conv_back_kernel(ConvArgs g) {
  const int e = blockIdx.x * 64 + threadIdx.x, row = blockIdx.y + blockIdx.z * gridDim.y;
  const int rows = gridDim.y * gridDim.z;
  if (e >= g.channels) return;
  const Act* x = static_cast<const Act*>(g.x) + e;
  const Act* dy = static_cast<const Act*>(g.dy) + e;
  Act* dx = static_cast<Act*>(g.dx) + e;
  const BlockAt b = block_at(g.p, row);
  float sum[kSums] = {};
  if (b.seq >= 0) {
    float w[kConv], h[kHalo];
#pragma unroll
    for (int k = 0; k < kConv; ++k) w[k] = g.w[int64_t(e) * kConv + k];
    const float bias = g.b ? g.b[e] : 0.0f;
    if (b.begins) {
      load_cache(g, b.seq, e, h);
    } else {
#pragma unroll
      for (int j = 0; j < kHalo; ++j) h[j] = load_act(x, (b.first - kHalo + j) * g.x_stride);
    }
    const int64_t s1 = packed_start(g.p, b.seq + 1), len = s1 - packed_start(g.p, b.seq);
    const float* dco = g.dcache_out ? g.dcache_out + int64_t(b.seq) * kHalo * g.channels + e : nullptr;
    float s1d = 0.0f, s2d = 0.0f, s3d = 0.0f;  // s one, two and three tokens earlier
    float begin[kHalo] = {};                   // s of the sequence's first tokens
    for (int j = 0; j < b.count + kHalo; ++j) {
      const int64_t t = int64_t(b.first) + j;
      float s = 0.0f;
      if (t < s1) {
        const float v = load_act(x, t * g.x_stride);
        s = load_act(dy, t * g.dy_stride);
        if (g.silu) {
          const float p = convolve(w, bias, h[0], h[1], h[2], v);
          const float e2 = __builtin_amdgcn_exp2f(-fabsf(p) * kLog2e);
          const float big = __builtin_amdgcn_rcpf(1.0f + e2), small = e2 * big;
          const float on = p < 0.0f ? small : big, off = p < 0.0f ? big : small;
          s *= on * fmaf(p, off, 1.0f);
        }
        if (j < b.count) {
          sum[0] = fmaf(s, h[0], sum[0]);
          sum[1] = fmaf(s, h[1], sum[1]);
          sum[2] = fmaf(s, h[2], sum[2]);
          sum[3] = fmaf(s, v, sum[3]);
          sum[4] += s;
        }
        h[0] = h[1], h[1] = h[2], h[2] = v;
      }
      if (j == 0) begin[0] = s;
      if (j == 1) begin[1] = s;
      if (j == 2) begin[2] = s;
      if (j >= kHalo) {
        float d = fmaf(w[3], s3d, fmaf(w[2], s2d, fmaf(w[1], s1d, w[0] * s)));
        const int64_t at = t - kHalo, kept = at - (s1 - kHalo);  // which row of the final cache
        if (dco && kept >= 0) d += dco[kept * g.channels];
        store_act(dx, at * g.channels, d);
      }
      s3d = s2d, s2d = s1d, s1d = s;
    }
    if (b.begins && g.dcache_in) {
      float* out = g.dcache_in + int64_t(b.seq) * kHalo * g.channels + e;
#pragma unroll
      for (int c = 0; c < kHalo; ++c) {
        float d = 0.0f;
#pragma unroll
        for (int k = 0; k <= c; ++k) d = fmaf(w[k], begin[c - k], d);
        if (dco && c >= len) d += dco[(c - len) * g.channels];
        out[int64_t(c) * g.channels] = d;
      }
    }
  }
  if (row < g.p.rows)
#pragma unroll
    for (int k = 0; k < kSums; ++k) g.partial[(int64_t(row) * kSums + k) * g.channels + e] = sum[k];
  if (g.dcache_in)
    for (int n = row; n < g.p.sequences; n += rows)
      if (packed_start(g.p, n) >= packed_start(g.p, n + 1))
        for (int c = 0; c < kHalo; ++c) {
          const int64_t at = (int64_t(n) * kHalo + c) * g.channels + e;
          g.dcache_in[at] = g.dcache_out ? g.dcache_out[at] : 0.0f;
        }
  for (int64_t t = int64_t(packed_start(g.p, g.p.sequences)) + row; t < g.p.tokens; t += rows)
    store_act(dx, t * g.channels, 0.0f);
}

__global__ __launch_bounds__(64) void conv_sum_kernel(ConvArgs g, int parts) {
  const int e = blockIdx.x * 64 + threadIdx.x, k = blockIdx.y;
  if (e >= g.channels) return;
  double s = 0.0;
  for (int j = 0; j < parts; ++j) s += g.partial[(int64_t(j) * kSums + k) * g.channels + e];
  if (k < kConv)
    g.dw[int64_t(e) * kConv + k] = static_cast<float>(s);
  else
    g.db[e] = static_cast<float>(s);
}

template <typename Act>
__global__ __launch_bounds__(256) void conv_step_kernel(ConvArgs g) {
  const int e = blockIdx.x * 256 + threadIdx.x, n = blockIdx.y;
  if (e >= g.channels) return;
  const int64_t slot = g.in_slots ? g.in_slots[n] : n;
  if (slot < 0 || slot >= g.in_count) return;
  float* c = g.cache_out + slot * kHalo * g.channels + e;
  const float h0 = c[0], h1 = c[g.channels], h2 = c[2 * int64_t(g.channels)];
  const float v = load_act(static_cast<const Act*>(g.x), n * g.x_stride + e);
  float w[kConv];
#pragma unroll
  for (int k = 0; k < kConv; ++k) w[k] = g.w[int64_t(e) * kConv + k];
  float p = convolve(w, g.b ? g.b[e] : 0.0f, h0, h1, h2, v);
  if (g.silu) p = silu(p);
  store_act(static_cast<Act*>(g.y), int64_t(n) * g.channels + e, p);
  c[0] = h1, c[g.channels] = h2, c[2 * int64_t(g.channels)] = v;
}

axon_status check_shape(const axon_conv_shape* s, bool backward) {
  if (!s) return AXON_ERR_INVALID_ARGUMENT;
  const int64_t strides[] = {s->x_stride, s->dy_stride};
  const axon_status why = check_packed(
      s->sequences, s->tokens, s->channels, strides, backward ? 2 : 1, kHalo * s->channels,
      backward ? 0 : s->cache_slots, backward ? 0 : s->out_slots, s->act_dtype);
  if (why != AXON_OK) return why;
  if ((s->activation != AXON_CONV_NONE && s->activation != AXON_CONV_SILU) ||
      (s->clear_behind != 0 && s->clear_behind != 1))
    return AXON_ERR_UNSUPPORTED;
  return AXON_OK;
}

bool bad(const void* p, size_t a) { return !p || !aligned_to(p, a); }
bool off(const void* p, size_t a) { return p && !aligned_to(p, a); }

ConvArgs make_args(const axon_conv_shape& s, const void* x, const float* w, const float* b,
                   const int32_t* tables) {
  ConvArgs a{};
  a.x = x, a.w = w, a.b = b;
  a.p = make_packed(s.sequences, s.tokens, tables);
  a.x_stride = s.x_stride ? s.x_stride : s.channels;
  a.dy_stride = s.dy_stride ? s.dy_stride : s.channels;
  a.channels = static_cast<int>(s.channels);
  a.silu = s.activation == AXON_CONV_SILU, a.clear_behind = s.clear_behind;
  return a;
}

size_t tables_bytes(const Packed& p) {
  return p.starts ? 4 * (2 * (size_t(p.sequences) + 1) + 2 * size_t(p.rows)) : 0;
}

// Blocks along y and z (y holds 65535 of them at most).
dim3 block_grid(int channels, int width, int rows) {
  const unsigned r = static_cast<unsigned>(std::max(rows, 1)), z = (r + 32767) / 32768;
  return dim3(static_cast<unsigned>((channels + width - 1) / width), (r + z - 1) / z, z);
}

}  // namespace
}  // namespace axon

extern "C" {

axon_status axon_causal_conv(const axon_conv_shape* shape, const void* x, const float* conv_w,
                             const float* conv_b, const int32_t* tables, const float* cache_in,
                             const int32_t* in_slots, void* y, float* cache_out,
                             const int32_t* out_slots, void* stream) {
  using namespace axon;
  const axon_status why = check_shape(shape, false);
  if (why != AXON_OK) return why;
  const axon_conv_shape& s = *shape;
  if (!tables && s.tokens % s.sequences) return AXON_ERR_INVALID_ARGUMENT;
  const bool bf = s.act_dtype == AXON_BF16;
  const size_t es = bf ? 2 : 4;
  if (bad(conv_w, 4) || off(conv_b, 4) || off(tables, 4) || off(in_slots, 4) || off(out_slots, 4) ||
      off(cache_in, 4) || off(cache_out, 4) || (s.tokens && (bad(x, es) || bad(y, es))))
    return AXON_ERR_INVALID_ARGUMENT;
  if ((cache_in && !in_slots && s.cache_slots < s.sequences) ||
      (cache_out && !out_slots && s.out_slots < s.sequences) ||
      (cache_in && cache_in == cache_out && s.cache_slots != s.out_slots))
    return AXON_ERR_INVALID_ARGUMENT;
  ConvArgs a = make_args(s, x, conv_w, conv_b, tables);
  const size_t row4 = 4 * size_t(s.channels), seq4 = 4 * size_t(s.sequences);
  const Span reads[] = {rows_span(x, s.tokens, a.x_stride, s.channels, es),
                        span(conv_w, kConv * row4), span(conv_b, row4),
                        span(tables, tables_bytes(a.p)), span(in_slots, seq4),
                        span(out_slots, seq4)};
  const Span in_cache = span(cache_in, kHalo * row4 * size_t(s.cache_slots));
  const Span out_cache = span(cache_out, kHalo * row4 * size_t(s.out_slots));
  const Span out_y = s.tokens ? span(y, es * size_t(s.tokens * s.channels)) : Span{};
  for (const Span& r : reads)
    if (overlaps(out_y, r) || overlaps(out_cache, r)) return AXON_ERR_INVALID_ARGUMENT;
  if (overlaps(out_y, in_cache) || overlaps(out_y, out_cache) ||
      (cache_in != cache_out && overlaps(in_cache, out_cache)))
    return AXON_ERR_INVALID_ARGUMENT;
  a.cache_in = cache_in, a.in_slots = in_slots, a.in_count = s.cache_slots;
  a.cache_out = cache_out, a.out_slots = out_slots, a.out_count = s.out_slots, a.y = y;
  const dim3 grid = block_grid(a.channels, 64, a.p.rows);
  hipStream_t st = static_cast<hipStream_t>(stream);
  if (bf)
    hipLaunchKernelGGL(conv_kernel<bf16_bits>, grid, dim3(64), 0, st, a);
  else
    hipLaunchKernelGGL(conv_kernel<float>, grid, dim3(64), 0, st, a);
  return hipGetLastError() == hipSuccess ? AXON_OK : AXON_ERR_HIP;
}

size_t axon_causal_conv_backward_workspace_bytes(const axon_conv_shape* shape) {
  if (axon::check_shape(shape, true) != AXON_OK) return 0;
  // as many block rows as packed sequences can have
  return 4 * axon::kSums * size_t(shape->tokens / axon::kBlock + shape->sequences) *
         size_t(shape->channels);
}

axon_status axon_causal_conv_backward(const axon_conv_shape* shape, const void* dy, const void* x,
                                      const float* conv_w, const float* conv_b,
                                      const int32_t* tables, const float* cache_in,
                                      const float* dcache_out, void* dx, float* dconv_w,
                                      float* dconv_b, float* dcache_in, void* workspace,
                                      size_t workspace_bytes, void* stream) {
  using namespace axon;
  const axon_status why = check_shape(shape, true);
  if (why != AXON_OK) return why;
  const axon_conv_shape& s = *shape;
  if (!tables && s.tokens % s.sequences) return AXON_ERR_INVALID_ARGUMENT;
  const bool bf = s.act_dtype == AXON_BF16;
  const size_t es = bf ? 2 : 4;
  if (bad(conv_w, 4) || off(conv_b, 4) || off(tables, 4) || off(cache_in, 4) ||
      off(dcache_out, 4) || bad(dconv_w, 4) || bad(dconv_b, 4) || off(dcache_in, 4) ||
      (s.tokens && (bad(dy, es) || bad(x, es) || bad(dx, es))))
    return AXON_ERR_INVALID_ARGUMENT;
  const size_t need = axon_causal_conv_backward_workspace_bytes(shape);
  if (workspace_bytes < need) return AXON_ERR_WORKSPACE_TOO_SMALL;
  if (need && bad(workspace, 16)) return AXON_ERR_INVALID_ARGUMENT;
  ConvArgs a = make_args(s, x, conv_w, conv_b, tables);
  const size_t row4 = 4 * size_t(s.channels), caches = kHalo * row4 * size_t(s.sequences);
  const Span reads[] = {rows_span(x, s.tokens, a.x_stride, s.channels, es),
                        rows_span(dy, s.tokens, a.dy_stride, s.channels, es),
                        span(conv_w, kConv * row4), span(conv_b, row4),
                        span(tables, tables_bytes(a.p)), span(cache_in, caches),
                        span(dcache_out, caches)};
  const Span outs[] = {s.tokens ? span(dx, es * size_t(s.tokens * s.channels)) : Span{},
                       span(dconv_w, kConv * row4), span(dconv_b, row4), span(dcache_in, caches),
                       span(workspace, need)};
  for (int i = 0; i < 5; ++i) {
    for (const Span& r : reads)
      if (overlaps(outs[i], r)) return AXON_ERR_INVALID_ARGUMENT;
    for (int j = 0; j < i; ++j)
      if (overlaps(outs[i], outs[j])) return AXON_ERR_INVALID_ARGUMENT;
  }
  a.dy = dy, a.cache_in = cache_in, a.in_count = s.sequences;
  a.dcache_out = dcache_out, a.dx = dx, a.dw = dconv_w, a.db = dconv_b, a.dcache_in = dcache_in;
  a.partial = static_cast<float*>(workspace);
  const dim3 grid = block_grid(a.channels, 64, a.p.rows);
  hipStream_t st = static_cast<hipStream_t>(stream);
  if (bf)
    hipLaunchKernelGGL(conv_back_kernel<bf16_bits>, grid, dim3(64), 0, st, a);
  else
    hipLaunchKernelGGL(conv_back_kernel<float>, grid, dim3(64), 0, st, a);
  hipLaunchKernelGGL(conv_sum_kernel, dim3((a.channels + 63) / 64, kSums), dim3(64), 0, st, a,
                     a.p.rows);
  return hipGetLastError() == hipSuccess ? AXON_OK : AXON_ERR_HIP;
}

axon_status axon_causal_conv_step(const axon_conv_shape* shape, const void* x, const float* conv_w,
                                  const float* conv_b, float* cache, const int32_t* slots, void* y,
                                  void* stream) {
  using namespace axon;
  const axon_status why = check_shape(shape, false);
  if (why != AXON_OK) return why;
  const axon_conv_shape& s = *shape;
  if (s.tokens != s.sequences) return AXON_ERR_INVALID_ARGUMENT;
  const bool bf = s.act_dtype == AXON_BF16;
  const size_t es = bf ? 2 : 4;
  if (bad(x, es) || bad(y, es) || bad(conv_w, 4) || off(conv_b, 4) || bad(cache, 4) ||
      (slots ? off(slots, 4) : s.cache_slots < s.sequences))
    return AXON_ERR_INVALID_ARGUMENT;
  ConvArgs a = make_args(s, x, conv_w, conv_b, nullptr);
  const size_t row4 = 4 * size_t(s.channels);
  const Span reads[] = {rows_span(x, s.tokens, a.x_stride, s.channels, es),
                        span(conv_w, kConv * row4), span(conv_b, row4),
                        span(slots, 4 * size_t(s.sequences))};
  const Span pool = span(cache, kHalo * row4 * size_t(s.cache_slots));
  const Span out = span(y, es * size_t(s.tokens * s.channels));
  for (const Span& r : reads)
    if (overlaps(out, r) || overlaps(pool, r)) return AXON_ERR_INVALID_ARGUMENT;
  if (overlaps(out, pool)) return AXON_ERR_INVALID_ARGUMENT;
  a.cache_out = cache, a.in_slots = slots, a.in_count = s.cache_slots, a.y = y;
  const dim3 grid((a.channels + 255) / 256, a.p.sequences);
  hipStream_t st = static_cast<hipStream_t>(stream);
  if (bf)
    hipLaunchKernelGGL(conv_step_kernel<bf16_bits>, grid, dim3(256), 0, st, a);
  else
    hipLaunchKernelGGL(conv_step_kernel<float>, grid, dim3(256), 0, st, a);
  return hipGetLastError() == hipSuccess ? AXON_OK : AXON_ERR_HIP;
}

}  // extern "C"

// Causal depthwise convolution of width 4 over packed or uniform sequences (see axonscan.h).
//
// A wave walks a block of 64 tokens, V channels a lane, with the last three inputs in registers and the next
// rows on their way. Only a sequence's first block reads its cache, and the same thread then writes the final
// cache from the sequence's last inputs, so that a cache may be updated in place without a wait between threads.
//
// Bound by memory: packed 32768 x 7680 bf16 (1007 MB) in 207-210 us, 4.8-4.9 TB/s; a copy of as much takes
// 187-207 us. What it took: four channels a lane (one: 380 us), eight rows ahead, stores past the caches
// (219 -> 212 us); loads past the caches cost 224 us.
//
// Backward, with s_t = dy_t act'(p_t):  dxx_t = sum_k w[k] s_{t+3-k} + what dcache_out has for t,
// dw[k] = sum_t s_t xx_{t-3+k},  db = sum_t s_t.  A block finds s of the three tokens behind it again, and four
// blocks join their sums before they leave a part: fp32 over 256 tokens, 64 bits over the parts (with the forward pass
// 8 x 2048 x 7680 262 us; 134 registers, three waves a SIMD). fp32, 16384 x 2560: 68 us forward (336 MB), 113 us backward.
// A step is bound by memory from a large batch on (512 rows x 7680 bf16 22 us, 110 MB; fp32 24 us, 126 MB).
#include <hip/hip_runtime.h>

#include <cmath>
#include <cstdint>

#include "axon_device.h"
#include "axon_packed.h"
#include "axon_wide.h"

namespace axon {
namespace {

constexpr int kSums = kConv + 1;  // dw and db

struct ConvArgs {
  const void *x, *dy;
  const float *w, *b;
  Packed p;
  int64_t x_stride, dy_stride;
  int channels, silu, clear_behind;
  bool past;  // y, dx are stored past the caches
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

// The cache of sequence n at V channels from e on, zeros where there is none.
template <int V>
__device__ __forceinline__ void load_cache(const ConvArgs& g, int n, int e, float (*c)[V]) {
#pragma unroll
  for (int j = 0; j < kHalo; ++j)
#pragma unroll
    for (int i = 0; i < V; ++i) c[j][i] = 0.0f;
  if (!g.cache_in) return;
  const int64_t slot = g.in_slots ? g.in_slots[n] : n;
  if (slot < 0 || slot >= g.in_count) return;
#pragma unroll
  for (int j = 0; j < kHalo; ++j)
#pragma unroll
    for (int i = 0; i < V; ++i) c[j][i] = g.cache_in[(slot * kHalo + j) * g.channels + e + i];
}
template <int V>
__device__ __forceinline__ void store_cache(const ConvArgs& g, int n, int e, const float (*c)[V]) {
  if (!g.cache_out) return;
  const int64_t slot = g.out_slots ? g.out_slots[n] : n;
  if (slot < 0 || slot >= g.out_count) return;
#pragma unroll
  for (int j = 0; j < kHalo; ++j)
#pragma unroll
    for (int i = 0; i < V; ++i) g.cache_out[(slot * kHalo + j) * g.channels + e + i] = c[j][i];
}

template <int V>
struct Taps {
  float w[kConv][V], b[V];
  __device__ __forceinline__ void load(const ConvArgs& g, int e) {
#pragma unroll
    for (int i = 0; i < V; ++i) {
#pragma unroll
      for (int k = 0; k < kConv; ++k) w[k][i] = g.w[int64_t(e + i) * kConv + k];
      b[i] = (g.b ? g.b : g.w)[e + i];
      if (!g.b) b[i] = 0.0f;
    }
  }
  __device__ __forceinline__ float at(int i, float x0, float x1, float x2, float x3) const {
    return fmaf(w[3][i], x3, fmaf(w[2][i], x2, fmaf(w[1][i], x1, fmaf(w[0][i], x0, b[i]))));
  }
};

// Block rows go along y and z; with several waves a workgroup, each takes one.
__device__ __forceinline__ int block_row() {
  return __builtin_amdgcn_readfirstlane(
      static_cast<int>((blockIdx.y + blockIdx.z * gridDim.y) * (blockDim.x >> 6) + (threadIdx.x >> 6)));
}
__device__ __forceinline__ int block_rows() {
  return static_cast<int>(gridDim.y * gridDim.z * (blockDim.x >> 6));
}

// A wave: 64 V channels of one block. The next kAhead rows are on their way while kAhead are computed.
template <typename Act, int V, bool PAST>
__global__ __launch_bounds__(64) void conv_kernel(ConvArgs g) {
  constexpr int kAhead = 8;
  const int e = (blockIdx.x * 64 + threadIdx.x) * V;
  const int row = block_row(), rows = block_rows();
  if (e >= g.channels) return;
  const Act* x = static_cast<const Act*>(g.x) + e;
  Act* y = static_cast<Act*>(g.y) + e;
  const BlockAt b = block_at(g.p, row);
  if (b.seq >= 0) {
    const Act* xb = x + b.first * g.x_stride;
    Act* yb = y + int64_t(b.first) * g.channels;
    Raw<Act, V> next[kAhead];
#pragma unroll
    for (int j = 0; j < kAhead; ++j) next[j].load(xb + min(j, b.count - 1) * g.x_stride);
    Taps<V> taps;
    taps.load(g, e);
    float h[kHalo][V];
    if (b.begins) {
      load_cache<V>(g, b.seq, e, h);
      const int len = packed_start(g.p, b.seq + 1) - b.first;
      float c[kHalo][V];
#pragma unroll
      for (int j = 0; j < kHalo; ++j) {
        const int at = len - kHalo + j;  // -2 .. of the sequence
        if (at >= 0) {
          Raw<Act, V> last;
          last.load(xb + at * g.x_stride);
          last.get(c[j]);
        } else {
#pragma unroll
          for (int i = 0; i < V; ++i) c[j][i] = at == -2 ? h[1][i] : h[2][i];
        }
      }
      store_cache<V>(g, b.seq, e, c);
    } else {
#pragma unroll
      for (int j = 0; j < kHalo; ++j) {
        Raw<Act, V> r;
        r.load(xb + (j - kHalo) * g.x_stride);
        r.get(h[j]);
      }
    }
    for (int j0 = 0; j0 < b.count; j0 += kAhead) {
      Raw<Act, V> now[kAhead];
#pragma unroll
      for (int j = 0; j < kAhead; ++j) now[j] = next[j];
#pragma unroll
      for (int j = 0; j < kAhead; ++j)
        next[j].load(xb + min(j0 + kAhead + j, b.count - 1) * g.x_stride);
#pragma unroll
      for (int j = 0; j < kAhead; ++j) {
        float v[V], p[V];
        now[j].get(v);
#pragma unroll
        for (int i = 0; i < V; ++i) {
          p[i] = taps.at(i, h[0][i], h[1][i], h[2][i], v[i]);
          if (g.silu) p[i] = silu(p[i]);
          h[0][i] = h[1][i], h[1][i] = h[2][i], h[2][i] = v[i];
        }
        if (j0 + j < b.count) Raw<Act, V>::template store<PAST>(yb + int64_t(j0 + j) * g.channels, p);
      }
    }
  }
  for (int n = row; n < g.p.sequences; n += rows)
    if (packed_start(g.p, n) >= packed_start(g.p, n + 1)) {
      float c[kHalo][V];
      load_cache<V>(g, n, e, c);
      store_cache<V>(g, n, e, c);
    }
  if (g.clear_behind) {
    const float zero[V] = {};
    for (int64_t t = int64_t(packed_start(g.p, g.p.sequences)) + row; t < g.p.tokens; t += rows)
      Raw<Act, V>::template store<false>(y + t * g.channels, zero);
  }
}

constexpr int kBackWaves = 4;  // blocks of a workgroup, whose sums are joined

template <typename Act, int V, bool PAST>
__global__ __launch_bounds__(64 * kBackWaves) void conv_back_kernel(ConvArgs g) {
  constexpr int kAhead = 4;
  __shared__ float joined[kBackWaves][kSums * V][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int e = (blockIdx.x * 64 + lane) * V;
  const int row = block_row(), rows = block_rows();
  const bool live = e < g.channels;
  const BlockAt b = block_at(g.p, row);
  float sum[kSums][V] = {};
  if (live && b.seq >= 0) {
    const Act* xb = static_cast<const Act*>(g.x) + e + b.first * g.x_stride;
    const Act* dyb = static_cast<const Act*>(g.dy) + e + b.first * g.dy_stride;
    Act* dxb = static_cast<Act*>(g.dx) + e + int64_t(b.first) * g.channels;
    const int s0 = packed_start(g.p, b.seq), s1 = packed_start(g.p, b.seq + 1);
    const int have = min(b.count + kHalo, s1 - b.first);  // tokens of the block and behind it
    Raw<Act, V> nx[kAhead], nd[kAhead];
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      nx[j].load(xb + min(j, have - 1) * g.x_stride);
      nd[j].load(dyb + min(j, have - 1) * g.dy_stride);
    }
    Taps<V> taps;
    taps.load(g, e);
    float h[kHalo][V];
    if (b.begins) {
      load_cache<V>(g, b.seq, e, h);
    } else {
#pragma unroll
      for (int j = 0; j < kHalo; ++j) {
        Raw<Act, V> r;
        r.load(xb + (j - kHalo) * g.x_stride);
        r.get(h[j]);
      }
    }
    const float* dco = g.dcache_out ? g.dcache_out + int64_t(b.seq) * kHalo * g.channels + e : nullptr;
    float s1d[V] = {}, s2d[V] = {}, s3d[V] = {};  // s one, two and three tokens earlier
    float begin[kHalo][V] = {};                   // s of the sequence's first tokens
    for (int j0 = 0; j0 < b.count + kHalo; j0 += kAhead) {
      Raw<Act, V> cx[kAhead], cd[kAhead];
#pragma unroll
      for (int j = 0; j < kAhead; ++j) cx[j] = nx[j], cd[j] = nd[j];
#pragma unroll
      for (int j = 0; j < kAhead; ++j) {
        nx[j].load(xb + min(j0 + kAhead + j, have - 1) * g.x_stride);
        nd[j].load(dyb + min(j0 + kAhead + j, have - 1) * g.dy_stride);
      }
#pragma unroll
      for (int jj = 0; jj < kAhead; ++jj) {
        const int j = j0 + jj;
        float s[V] = {};
        if (j < have) {
          float v[V];
          cx[jj].get(v);
          cd[jj].get(s);
#pragma unroll
          for (int i = 0; i < V; ++i) {
            if (g.silu) {
              const float p = taps.at(i, h[0][i], h[1][i], h[2][i], v[i]);
              // sigmoid(p) and 1 - sigmoid(p), neither from the other by a subtraction
              const float x2 = __builtin_amdgcn_exp2f(-fabsf(p) * kLog2e);
              const float big = __builtin_amdgcn_rcpf(1.0f + x2), small = x2 * big;
              const float on = p < 0.0f ? small : big, off = p < 0.0f ? big : small;
              s[i] *= on * fmaf(p, off, 1.0f);
            }
            if (j < b.count) {
              sum[0][i] = fmaf(s[i], h[0][i], sum[0][i]);
              sum[1][i] = fmaf(s[i], h[1][i], sum[1][i]);
              sum[2][i] = fmaf(s[i], h[2][i], sum[2][i]);
              sum[3][i] = fmaf(s[i], v[i], sum[3][i]);
              sum[4][i] += s[i];
            }
            h[0][i] = h[1][i], h[1][i] = h[2][i], h[2][i] = v[i];
          }
        }
        if (j0 == 0 && jj < kHalo)
#pragma unroll
          for (int i = 0; i < V; ++i) begin[jj][i] = s[i];
        if (j >= kHalo && j < b.count + kHalo) {
          const int kept = b.first + j - s1;  // which row of the final cache this token is
          float d[V];
#pragma unroll
          for (int i = 0; i < V; ++i) {
            d[i] = fmaf(taps.w[3][i], s3d[i],
                        fmaf(taps.w[2][i], s2d[i], fmaf(taps.w[1][i], s1d[i], taps.w[0][i] * s[i])));
            if (dco && kept >= 0) d[i] += dco[int64_t(kept) * g.channels + i];
          }
          Raw<Act, V>::template store<PAST>(dxb + int64_t(j - kHalo) * g.channels, d);
        }
#pragma unroll
        for (int i = 0; i < V; ++i) s3d[i] = s2d[i], s2d[i] = s1d[i], s1d[i] = s[i];
      }
    }
    if (b.begins && g.dcache_in) {
      const int len = s1 - s0;
      float* out = g.dcache_in + int64_t(b.seq) * kHalo * g.channels + e;
#pragma unroll
      for (int c = 0; c < kHalo; ++c)
#pragma unroll
        for (int i = 0; i < V; ++i) {
          float d = 0.0f;
#pragma unroll
          for (int k = 0; k <= c; ++k) d = fmaf(taps.w[k][i], begin[c - k][i], d);
          if (dco && c >= len) d += dco[int64_t(c - len) * g.channels + i];
          out[int64_t(c) * g.channels + i] = d;
        }
    }
  }
#pragma unroll
  for (int k = 0; k < kSums; ++k)
#pragma unroll
    for (int i = 0; i < V; ++i) joined[wave][k * V + i][lane] = sum[k][i];
  __syncthreads();
  const int64_t part = blockIdx.y + int64_t(blockIdx.z) * gridDim.y;
  for (int t = wave; t < kSums * V; t += kBackWaves) {
    float a = 0.0f;
#pragma unroll
    for (int w = 0; w < kBackWaves; ++w) a += joined[w][t][lane];
    if (live) g.partial[(part * kSums + t / V) * g.channels + e + t % V] = a;
  }
  if (!live) return;
  if (g.dcache_in)
    for (int n = row; n < g.p.sequences; n += rows)
      if (packed_start(g.p, n) >= packed_start(g.p, n + 1))
        for (int c = 0; c < kHalo * V; ++c) {
          const int64_t at = (int64_t(n) * kHalo + c / V) * g.channels + e + c % V;
          g.dcache_in[at] = g.dcache_out ? g.dcache_out[at] : 0.0f;
        }
  const float zero[V] = {};
  for (int64_t t = int64_t(packed_start(g.p, g.p.sequences)) + row; t < g.p.tokens; t += rows)
    Raw<Act, V>::template store<false>(static_cast<Act*>(g.dx) + e + t * g.channels, zero);
}

// Sums of the workgroups' parts in 64 bits: a lane a sum, each wave takes every 16th part.
constexpr int kSumWaves = 16;
__global__ __launch_bounds__(64 * kSumWaves) void conv_sum_kernel(ConvArgs g, int parts) {
  __shared__ double sums[kSumWaves][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int e = blockIdx.x * 64 + lane, k = blockIdx.y;
  double s = 0.0;
  if (e < g.channels) {
    const float* from = g.partial + int64_t(k) * g.channels + e;
#pragma unroll 8
    for (int j = wave; j < parts; j += kSumWaves) s += from[int64_t(j) * kSums * g.channels];
  }
  sums[wave][lane] = s;
  __syncthreads();
  if (wave || e >= g.channels) return;
#pragma unroll
  for (int w = 1; w < kSumWaves; ++w) s += sums[w][lane];
  const float all = static_cast<float>(s);
  if (k < kConv)
    g.dw[int64_t(e) * kConv + k] = all;
  else
    g.db[e] = all;
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
  float p = fmaf(w[3], v, fmaf(w[2], h2, fmaf(w[1], h1, fmaf(w[0], h0, g.b ? g.b[e] : 0.0f))));
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
  a.past = past_caches(size_t(s.tokens * s.channels) * (s.act_dtype == AXON_BF16 ? 2 : 4));
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

// Parts that conv_back_kernel leaves: its workgroups of one channel group.
int64_t back_parts(int64_t rows) {
  const int64_t r = std::max<int64_t>((rows + kBackWaves - 1) / kBackWaves, 1), z = (r + 32767) / 32768;
  return (r + z - 1) / z * z;
}

// Channels a lane takes at once: as many as width, rows and pointers keep aligned.
bool vectors_ok(const ConvArgs& a, int v, size_t es, bool backward) {
  return a.channels % v == 0 && a.x_stride % v == 0 && aligned_to(a.x, v * es) &&
         (backward ? a.dy_stride % v == 0 && aligned_to(a.dy, v * es) && aligned_to(a.dx, v * es)
                   : aligned_to(a.y, v * es));
}

// Channels a lane: as many as alignment allows, fill a wave's lanes and leave waves enough for the card, since a
// wave of four walks its tokens for longer than one of one (bf16: 32768 tokens x 256 14 -> 11 us, backward 42 ->
// 21 us; 131072 x 64 19 -> 11 us, 48 -> 23 us; where there are many, 32768 x 2560, four 54 us, two 73 us).
constexpr int64_t kManyWaves = 2048;
int channels_a_lane(const ConvArgs& a, size_t es, bool backward) {
  int v = vectors_ok(a, 4, es, backward) ? 4 : es == 2 && vectors_ok(a, 2, es, backward) ? 2 : 1;
  while (v > 1 && (a.channels <= 32 * v || int64_t(a.p.rows) * ((a.channels + 64 * v - 1) / (64 * v)) < kManyWaves))
    v = es == 4 ? 1 : v / 2;
  return v;
}

template <typename Act, int V>
void launch_conv(const ConvArgs& a, hipStream_t st) {
  const dim3 grid = block_grid(a.channels, 64 * V, a.p.rows);
  if (V == 4 && a.past)
    hipLaunchKernelGGL((conv_kernel<Act, V, V == 4>), grid, dim3(64), 0, st, a);
  else
    hipLaunchKernelGGL((conv_kernel<Act, V, false>), grid, dim3(64), 0, st, a);
}
template <typename Act, int V>
void launch_back(const ConvArgs& a, hipStream_t st) {
  const dim3 grid = block_grid(a.channels, 64 * V, (a.p.rows + kBackWaves - 1) / kBackWaves);
  if (V == 4 && a.past)
    hipLaunchKernelGGL((conv_back_kernel<Act, V, V == 4>), grid, dim3(64 * kBackWaves), 0, st, a);
  else
    hipLaunchKernelGGL((conv_back_kernel<Act, V, false>), grid, dim3(64 * kBackWaves), 0, st, a);
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
  hipStream_t st = static_cast<hipStream_t>(stream);
  const int v = channels_a_lane(a, es, false);
  if (v == 4) bf ? launch_conv<bf16_bits, 4>(a, st) : launch_conv<float, 4>(a, st);
  else if (v == 2) launch_conv<bf16_bits, 2>(a, st);
  else bf ? launch_conv<bf16_bits, 1>(a, st) : launch_conv<float, 1>(a, st);
  return hipGetLastError() == hipSuccess ? AXON_OK : AXON_ERR_HIP;
}

size_t axon_causal_conv_backward_workspace_bytes(const axon_conv_shape* shape) {
  if (axon::check_shape(shape, true) != AXON_OK) return 0;
  // as many block rows as packed sequences can have
  return 4 * axon::kSums *
         size_t(axon::back_parts(axon::packed_rows(shape->sequences, shape->tokens, true))) *
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
  hipStream_t st = static_cast<hipStream_t>(stream);
  const int v = channels_a_lane(a, es, true);
  if (v == 4) bf ? launch_back<bf16_bits, 4>(a, st) : launch_back<float, 4>(a, st);
  else if (v == 2) launch_back<bf16_bits, 2>(a, st);
  else bf ? launch_back<bf16_bits, 1>(a, st) : launch_back<float, 1>(a, st);
  hipLaunchKernelGGL(conv_sum_kernel, dim3((a.channels + 63) / 64, kSums), dim3(64 * kSumWaves), 0, st, a,
                     static_cast<int>(back_parts(a.p.rows)));
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

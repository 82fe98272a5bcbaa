// The gated delta rule on gfx950: packed or uniform sequences in chunks of 64 tokens, and the
// single-token step (definitions in axonscan.h).
//
// Inside a chunk, with g_t the inclusive sum of dt A from the chunk's start and S0 (V x K) the
// entering state, the recurrence S_t = a_t S_{t-1} + D_t k^_t^T, D_t = beta_t (v_t - a_t S_{t-1} k^_t)
// unrolls to
//   D_t + beta_t sum_{s<t} e^{g_t-g_s} (k^_t.k^_s) D_s = beta_t (v_t - e^{g_t} S0 k^_t),
// a unit lower triangular system (I + M) D = diag(beta) X. Its inverse does not depend on the
// state, so it is computed for all chunks at once; the walk over the chunks is products only:
//   X = v - e^g (S0 k^),  D = T X with T = (I + M)^-1 diag(beta),
//   y = scale (e^g S0 q^ + A D),  A[t,s] = e^{g_t-g_s} q^_t.k^_s (s <= t),
//   S <- e^{g_last} S0 + sum_t e^{g_last-g_t} D_t k^_t^T.
// Every exponent is <= 0; the sums are compensated (head and tail) because steps near dt_max push
// g to thousands, where the plain fp32 sum's ulp would be the error of later differences. The
// norms of q and k multiply rows of the products instead of the operands.
//
//   prep_kernel  per chunk and key head: the Gram products, then per value head T (16 x 16 diagonal
//                blocks by substitution, which stays accurate where keys are alike and powers of M
//                would cancel; the blocks below by matrix products), A and the row factors.
//   walk_kernel  per sequence, value head and 16 columns of V one wave walks the chunks with its
//                slice of the state in registers. The state is held transposed (S^T, K x 16): the
//                result layout of a 16 x 16 product (lane (g, i): rows 4 g + r, column i) is also
//                the layout of the right operand of the next one when the contraction index is
//                taken as 4 g + r, so state, X and D go from product to product without leaving
//                their lanes.
// Products run on v_mfma_f32_16x16x4f32 (layout in axon_ssd.hip's head comment).
#include <hip/hip_runtime.h>

#include <cmath>
#include <cstdint>

#include "axon_device.h"
#include "axon_internal.h"

namespace axon {
namespace {

constexpr int kQ = 64;  // tokens of a chunk
constexpr int kThreads = 256;
constexpr int kMS = kQ + 4;  // LDS row stride of 64 x 64 matrices

typedef float f4 __attribute__((ext_vector_type(4)));

// What prep leaves for each (chunk, value head), in floats: T and A as ten 16 x 16 blocks on and
// below the diagonal (block I (I + 1) / 2 + J), each as 64 lanes x 4 in left-operand order (lane
// (g, i): row i, columns 4 g .. 4 g + 3), then the row factors e^g / |k|, e^{g_last-g} / |k|,
// scale e^g / |q| of the 64 tokens and e^{g_last}.
constexpr int kBlocks = 10;
constexpr int kOffA = kBlocks * 256;
constexpr int kOffRows = 2 * kBlocks * 256;
constexpr int kRecord = kOffRows + 256;

struct DeltaArgs {
  const void *q, *k, *v, *dt_raw, *beta_raw;
  const float *A_log, *dt_bias;
  float dt_min, dt_max, scale, eps;
  const int32_t *starts, *block_starts, *block_seq, *block_first;  // null: uniform batch
  const float* state_in;
  const int32_t* in_slots;
  void* y;
  float* state_out;
  const int32_t* out_slots;
  float* records;
  int64_t tokens, seqlen, q_stride, k_stride, v_stride, in_count, out_count;
  int sequences, hk, hv, ratio, value_dim, col_groups;
  int rows;             // chunk rows of the workspace
  int chunks_per_seq;   // uniform batch
};

__device__ __forceinline__ f4 mfma4(float a, float b, f4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x4f32(a, b, c, 0, 0, 0);
}

__device__ __forceinline__ float4 load4(const float* p) {
  return *reinterpret_cast<const float4*>(p);
}
__device__ __forceinline__ float4 load4(const bf16_bits* p) {
  const uint2 v = *reinterpret_cast<const uint2*>(p);
  return make_float4(__uint_as_float(v.x << 16), __uint_as_float(v.x & 0xFFFF0000u),
                     __uint_as_float(v.y << 16), __uint_as_float(v.y & 0xFFFF0000u));
}

// softplus to the last bits: the step enters the exponent of the decay multiplied by the rate.
__device__ __forceinline__ float gate_step(float v, float lo, float hi) {
  return fminf(fmaxf(fmaxf(v, 0.0f) + log1pf(expf(-fabsf(v))), lo), hi);
}
__device__ __forceinline__ float sigmoid(float v) { return 1.0f / (1.0f + expf(-v)); }

__device__ __forceinline__ float exp2_diff(float hi_a, float lo_a, float hi_b, float lo_b) {
  return __builtin_amdgcn_exp2f((hi_a - hi_b) + (lo_a - lo_b));
}

// The tokens of chunk row c: false where there are none. Table values are taken as given by the
// caller's array, so they are cut to the buffers' ranges here.
__device__ __forceinline__ bool chunk_of(const DeltaArgs& a, int c, int64_t* first, int* count) {
  int64_t begin, end;
  if (a.block_seq) {
    const int n = a.block_seq[c];
    if (n < 0 || n >= a.sequences) return false;
    begin = a.block_first[c];
    end = a.starts[n + 1];
  } else {
    const int n = c / a.chunks_per_seq;
    begin = n * a.seqlen + int64_t(c - n * a.chunks_per_seq) * kQ;
    end = (n + 1) * a.seqlen;
  }
  if (begin < 0 || begin >= a.tokens) return false;
  if (end > a.tokens) end = a.tokens;
  if (end <= begin) return false;
  *first = begin;
  *count = end - begin < kQ ? static_cast<int>(end - begin) : kQ;
  return true;
}

// ---- T, A and the row factors of every chunk ----------------------------------------------------
// Grid (chunk rows, key heads), 4 waves. Wave w owns rows 16 w .. 16 w + 15 of the Gram products
// and column block w of the inverse.
template <typename Act, int K>
__global__ __launch_bounds__(kThreads) void prep_kernel(DeltaArgs a) {
  constexpr int NB = K / 16;
  __shared__ float Ms[kQ * kMS];
  __shared__ float As[kQ * kMS];
  __shared__ float Ds[4][16 * 20];
  __shared__ float hi_s[kQ], lo_s[kQ], beta_s[kQ], rk_s[kQ], rq_s[kQ];
  int64_t first;
  int count;
  if (!chunk_of(a, blockIdx.x, &first, &count)) return;
  const int hk = blockIdx.y;
  const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6, g = lane >> 4, i = lane & 15;
  const Act* kp = static_cast<const Act*>(a.k) + first * a.k_stride + int64_t(hk) * K;
  const Act* qp = static_cast<const Act*>(a.q) + first * a.q_stride + int64_t(hk) * K;
  f4 gk[4], gq[4];
  {
    float4 krow[NB], qrow[NB];
    const int t = 16 * w + i;
    float sk = 0.0f, sq = 0.0f;
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      krow[b] = t < count ? load4(kp + t * a.k_stride + 16 * b + 4 * g) : float4{};
      qrow[b] = t < count ? load4(qp + t * a.q_stride + 16 * b + 4 * g) : float4{};
    }
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      sk += krow[b].x * krow[b].x + krow[b].y * krow[b].y + krow[b].z * krow[b].z +
            krow[b].w * krow[b].w;
      sq += qrow[b].x * qrow[b].x + qrow[b].y * qrow[b].y + qrow[b].z * qrow[b].z +
            qrow[b].w * qrow[b].w;
    }
    sk += __shfl_xor(sk, 16, 64);
    sk += __shfl_xor(sk, 32, 64);
    sq += __shfl_xor(sq, 16, 64);
    sq += __shfl_xor(sq, 32, 64);
    if (g == 0) {
      rk_s[t] = 1.0f / sqrtf(sk + a.eps);
      rq_s[t] = 1.0f / sqrtf(sq + a.eps);
    }
#pragma unroll
    for (int st = 0; st < 4; ++st) {
      gk[st] = f4{0.0f, 0.0f, 0.0f, 0.0f};
      gq[st] = f4{0.0f, 0.0f, 0.0f, 0.0f};
      if (st > w) continue;
      const int ts = 16 * st + i;
      float4 col[NB];
#pragma unroll
      for (int b = 0; b < NB; ++b)
        col[b] = ts < count ? load4(kp + ts * a.k_stride + 16 * b + 4 * g) : float4{};
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        gk[st] = mfma4(krow[b].x, col[b].x, gk[st]);
        gq[st] = mfma4(qrow[b].x, col[b].x, gq[st]);
        gk[st] = mfma4(krow[b].y, col[b].y, gk[st]);
        gq[st] = mfma4(qrow[b].y, col[b].y, gq[st]);
        gk[st] = mfma4(krow[b].z, col[b].z, gk[st]);
        gq[st] = mfma4(qrow[b].z, col[b].z, gq[st]);
        gk[st] = mfma4(krow[b].w, col[b].w, gk[st]);
        gq[st] = mfma4(qrow[b].w, col[b].w, gq[st]);
      }
    }
  }
  for (int vh = 0; vh < a.ratio; ++vh) {
    const int h = hk * a.ratio + vh;
    float* rec = a.records + (int64_t(blockIdx.x) * a.hv + h) * kRecord;
    __syncthreads();  // the previous head's matrices and factors have been read; rk_s, rq_s ready
    if (w == 0) {
      float dt = 0.0f, beta = 0.0f;
      if (lane < count) {
        const int64_t at = (first + lane) * a.hv + h;
        dt = gate_step(load_act(static_cast<const Act*>(a.dt_raw), at) + a.dt_bias[h], a.dt_min,
                       a.dt_max);
        beta = sigmoid(load_act(static_cast<const Act*>(a.beta_raw), at));
      }
      // No decay below 2^-16384 differs from 0: the bound keeps the sums finite for any dt_max.
      float hi = fmaxf(dt * decay_rate_log2(a.A_log[h]), -16384.0f), lo = 0.0f;
#pragma unroll
      for (int d = 1; d < 64; d <<= 1) {
        const float oh = __shfl_up(hi, d, 64), ol = __shfl_up(lo, d, 64);
        if (lane >= d) {
          const float s = hi + oh;
          const float bv = s - hi;
          const float err = (hi - (s - bv)) + (oh - bv);
          hi = s;
          lo = lo + ol + err;
        }
      }
      hi_s[lane] = hi, lo_s[lane] = lo, beta_s[lane] = beta;
      const float last_hi = __shfl(hi, 63, 64), last_lo = __shfl(lo, 63, 64);
      const float e = __builtin_amdgcn_exp2f(hi + lo);
      rec[kOffRows + lane] = e * rk_s[lane];
      rec[kOffRows + 64 + lane] = exp2_diff(last_hi, last_lo, hi, lo) * rk_s[lane];
      rec[kOffRows + 128 + lane] = a.scale * e * rq_s[lane];
      if (lane == 63) rec[kOffRows + 192] = e;
    }
    __syncthreads();
#pragma unroll
    for (int st = 0; st < 4; ++st) {
      if (st > w) continue;
      const int s = 16 * st + i;
      const float hs = hi_s[s], ls = lo_s[s], rks = rk_s[s];
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int t = 16 * w + 4 * g + r;
        const float e = exp2_diff(hi_s[t], lo_s[t], hs, ls) * rks;
        Ms[t * kMS + s] = s < t ? beta_s[t] * rk_s[t] * e * gk[st][r] : 0.0f;
        As[t * kMS + s] = s <= t ? a.scale * rq_s[t] * e * gq[st][r] : 0.0f;
      }
    }
    __syncthreads();
    // Diagonal block w: column i of (I + M_ww)^-1 by substitution (the four lane groups alike).
    {
      float x[16];
#pragma unroll
      for (int r = 0; r < 16; ++r) {
        float acc = r == i ? 1.0f : 0.0f;
#pragma unroll
        for (int s = 0; s < r; ++s) acc = fmaf(-Ms[(16 * w + r) * kMS + 16 * w + s], x[s], acc);
        x[r] = acc;
      }
      if (g == 0) {
#pragma unroll
        for (int r = 0; r < 16; ++r) Ds[w][r * 20 + i] = x[r];
      }
    }
    __syncthreads();
    // Column block w of the inverse: X_I = -D_I sum_{w <= S < I} M_IS X_S.
    f4 X[4];
#pragma unroll
    for (int I = 0; I < 4; ++I) {
      if (I < w) {
        X[I] = f4{0.0f, 0.0f, 0.0f, 0.0f};
      } else if (I == w) {
#pragma unroll
        for (int r = 0; r < 4; ++r) X[I][r] = Ds[I][(4 * g + r) * 20 + i];
      } else {
        f4 p = f4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int S = 0; S < I; ++S) {
          if (S < w) continue;
          const float4 m = *reinterpret_cast<const float4*>(&Ms[(16 * I + i) * kMS + 16 * S + 4 * g]);
          p = mfma4(m.x, X[S][0], p);
          p = mfma4(m.y, X[S][1], p);
          p = mfma4(m.z, X[S][2], p);
          p = mfma4(m.w, X[S][3], p);
        }
        const float4 d = *reinterpret_cast<const float4*>(&Ds[I][i * 20 + 4 * g]);
        f4 x = f4{0.0f, 0.0f, 0.0f, 0.0f};
        x = mfma4(d.x, p[0], x);
        x = mfma4(d.y, p[1], x);
        x = mfma4(d.z, p[2], x);
        x = mfma4(d.w, p[3], x);
        X[I] = -x;
      }
    }
    __syncthreads();  // M has been read: T takes its place
    const float beta = beta_s[16 * w + i];
#pragma unroll
    for (int I = 0; I < 4; ++I) {
      if (I < w) continue;
#pragma unroll
      for (int r = 0; r < 4; ++r) Ms[(16 * I + 4 * g + r) * kMS + 16 * w + i] = X[I][r] * beta;
    }
    __syncthreads();
    for (int b = w; b < 2 * kBlocks; b += 4) {
      const int bb = b < kBlocks ? b : b - kBlocks;
      const int I = bb < 1 ? 0 : bb < 3 ? 1 : bb < 6 ? 2 : 3;
      const int J = bb - I * (I + 1) / 2;
      const float* src = (b < kBlocks ? Ms : As) + (16 * I + i) * kMS + 16 * J + 4 * g;
      *reinterpret_cast<float4*>(rec + b * 256 + lane * 4) = *reinterpret_cast<const float4*>(src);
    }
  }
}

// ---- the walk over the chunks -------------------------------------------------------------------
// One wave per 16 columns of V, 4 waves a workgroup; the column groups of one head are spaced by
// the 8 XCDs' round-robin so that they share that XCD's L2.
template <typename Act, int K>
__global__ __launch_bounds__(kThreads) void walk_kernel(DeltaArgs a) {
  constexpr int NB = K / 16, KS = K + 4;
  __shared__ float Ks[kQ * KS];
  __shared__ float Qs[kQ * KS];
  const int xcd = blockIdx.x & 7, slot = blockIdx.x >> 3;
  const int64_t nh = int64_t(slot / a.col_groups) * 8 + xcd;
  if (nh >= int64_t(a.sequences) * a.hv) return;
  const int n = static_cast<int>(nh / a.hv), h = static_cast<int>(nh - int64_t(n) * a.hv);
  const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6, g = lane >> 4, i = lane & 15;
  const int col = ((slot % a.col_groups) * 4 + w) * 16 + i;  // of V
  const bool mine = col < a.value_dim;                       // wave-uniform: V is a multiple of 16
  int64_t begin, len, row0;
  if (a.starts) {
    begin = a.starts[n];
    len = a.starts[n + 1] - begin;
    row0 = a.block_starts[n];
    if (begin < 0 || begin > a.tokens || row0 < 0 || row0 > a.rows) begin = len = row0 = 0;
    if (len > a.tokens - begin) len = a.tokens - begin;
  } else {
    begin = n * a.seqlen, len = a.seqlen, row0 = int64_t(n) * a.chunks_per_seq;
  }
  int64_t chunks = len > 0 ? (len + kQ - 1) / kQ : 0;
  if (chunks > a.rows - row0) chunks = a.rows - row0;

  f4 S[NB];
  {
    const int64_t slot_in = a.in_slots ? a.in_slots[n] : n;
    const bool have = a.state_in && mine && slot_in >= 0 && slot_in < a.in_count;
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      S[b] = f4{0.0f, 0.0f, 0.0f, 0.0f};
      if (have) {
        const float4 v = load4(a.state_in + ((slot_in * a.hv + h) * a.value_dim + col) * K + 16 * b +
                               4 * g);
        S[b] = f4{v.x, v.y, v.z, v.w};
      }
    }
  }
  const int hk = h / a.ratio;
  for (int64_t c = 0; c < chunks; ++c) {
    const int64_t first = begin + c * kQ;
    const int count = len - c * kQ < kQ ? static_cast<int>(len - c * kQ) : kQ;
    const float* rec = a.records + ((row0 + c) * a.hv + h) * kRecord;
    {
      const Act* kp = static_cast<const Act*>(a.k) + first * a.k_stride + int64_t(hk) * K;
      const Act* qp = static_cast<const Act*>(a.q) + first * a.q_stride + int64_t(hk) * K;
      for (int e = tid; e < kQ * K / 4; e += kThreads) {
        const int t = e / (K / 4), kk = 4 * (e % (K / 4));
        const float4 kv = t < count ? load4(kp + t * a.k_stride + kk) : float4{};
        const float4 qv = t < count ? load4(qp + t * a.q_stride + kk) : float4{};
        *reinterpret_cast<float4*>(&Ks[t * KS + kk]) = kv;
        *reinterpret_cast<float4*>(&Qs[t * KS + kk]) = qv;
      }
    }
    __syncthreads();
    if (mine) {
      const Act* vp = static_cast<const Act*>(a.v) + first * a.v_stride + int64_t(h) * a.value_dim + col;
      f4 X[4], O[4];
#pragma unroll
      for (int tt = 0; tt < 4; ++tt) {
        f4 p = f4{0.0f, 0.0f, 0.0f, 0.0f}, o = p;
#pragma unroll
        for (int b = 0; b < NB; ++b) {
          const float4 kf = *reinterpret_cast<const float4*>(&Ks[(16 * tt + i) * KS + 16 * b + 4 * g]);
          const float4 qf = *reinterpret_cast<const float4*>(&Qs[(16 * tt + i) * KS + 16 * b + 4 * g]);
          p = mfma4(kf.x, S[b][0], p);
          o = mfma4(qf.x, S[b][0], o);
          p = mfma4(kf.y, S[b][1], p);
          o = mfma4(qf.y, S[b][1], o);
          p = mfma4(kf.z, S[b][2], p);
          o = mfma4(qf.z, S[b][2], o);
          p = mfma4(kf.w, S[b][3], p);
          o = mfma4(qf.w, S[b][3], o);
        }
        const float4 s1 = load4(rec + kOffRows + 16 * tt + 4 * g);
        const float4 s3 = load4(rec + kOffRows + 128 + 16 * tt + 4 * g);
        const float f1[4] = {s1.x, s1.y, s1.z, s1.w}, f3[4] = {s3.x, s3.y, s3.z, s3.w};
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int t = 16 * tt + 4 * g + r;
          const float v = t < count ? load_act(vp, t * a.v_stride) : 0.0f;
          X[tt][r] = fmaf(-f1[r], p[r], v);
          O[tt][r] = f3[r] * o[r];
        }
      }
      f4 D[4];
#pragma unroll
      for (int tt = 0; tt < 4; ++tt) {
        D[tt] = f4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int st = 0; st <= tt; ++st) {
          const float4 m = load4(rec + (tt * (tt + 1) / 2 + st) * 256 + lane * 4);
          D[tt] = mfma4(m.x, X[st][0], D[tt]);
          D[tt] = mfma4(m.y, X[st][1], D[tt]);
          D[tt] = mfma4(m.z, X[st][2], D[tt]);
          D[tt] = mfma4(m.w, X[st][3], D[tt]);
        }
      }
      Act* yp = static_cast<Act*>(a.y) + (first * a.hv + h) * a.value_dim + col;
#pragma unroll
      for (int tt = 0; tt < 4; ++tt) {
#pragma unroll
        for (int st = 0; st <= tt; ++st) {
          const float4 m = load4(rec + kOffA + (tt * (tt + 1) / 2 + st) * 256 + lane * 4);
          O[tt] = mfma4(m.x, D[st][0], O[tt]);
          O[tt] = mfma4(m.y, D[st][1], O[tt]);
          O[tt] = mfma4(m.z, D[st][2], O[tt]);
          O[tt] = mfma4(m.w, D[st][3], O[tt]);
        }
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int t = 16 * tt + 4 * g + r;
          if (t < count) store_act(yp, int64_t(t) * a.hv * a.value_dim, O[tt][r]);
        }
      }
      const float end = rec[kOffRows + 192];
#pragma unroll
      for (int b = 0; b < NB; ++b) S[b] *= end;
#pragma unroll
      for (int ts = 0; ts < 4; ++ts) {
        const float4 s2 = load4(rec + kOffRows + 64 + 16 * ts + 4 * g);
        const float d[4] = {D[ts][0] * s2.x, D[ts][1] * s2.y, D[ts][2] * s2.z, D[ts][3] * s2.w};
#pragma unroll
        for (int r = 0; r < 4; ++r) {
#pragma unroll
          for (int b = 0; b < NB; ++b)
            S[b] = mfma4(Ks[(16 * ts + 4 * g + r) * KS + 16 * b + i], d[r], S[b]);
        }
      }
    }
    __syncthreads();
  }
  const int64_t slot_out = a.out_slots ? a.out_slots[n] : n;
  if (a.state_out && mine && slot_out >= 0 && slot_out < a.out_count) {
#pragma unroll
    for (int b = 0; b < NB; ++b)
      *reinterpret_cast<float4*>(a.state_out + ((slot_out * a.hv + h) * a.value_dim + col) * K +
                                 16 * b + 4 * g) = make_float4(S[b][0], S[b][1], S[b][2], S[b][3]);
  }
}

// ---- one token a row ----------------------------------------------------------------------------
// Bound by reading and writing the states. K / 16 lanes hold a row of the state (16 values each, as
// four float4 spaced so that a load's lanes read whole 64 or 128 byte pieces); a wave passes over R
// times its 64 / lanes rows, all loaded before the first is used.
struct StepArgs {
  const void *q, *k, *v, *dt_raw, *beta_raw;
  const float *A_log, *dt_bias;
  float dt_min, dt_max, scale, eps;
  float* state;
  const int32_t* slots_of;
  void* y;
  int64_t q_stride, k_stride, v_stride, slots;
  int rows, hv, ratio, value_dim, waves_per_head;
};

template <typename Act, int K, int R>
__global__ __launch_bounds__(kThreads) void step_kernel(StepArgs a) {
  constexpr int LR = K / 16;      // lanes of a state row
  constexpr int RW = 64 / LR;     // state rows of a wave and pass
  const int lane = threadIdx.x & 63, l = lane % LR, rr = lane / LR;
  const int64_t wave = int64_t(blockIdx.x) * 4 + (threadIdx.x >> 6);
  const int64_t rh = wave / a.waves_per_head;
  const int part = static_cast<int>(wave - rh * a.waves_per_head);
  if (rh >= int64_t(a.rows) * a.hv) return;
  const int row = static_cast<int>(rh / a.hv), h = static_cast<int>(rh - int64_t(row) * a.hv);
  const int64_t slot = a.slots_of ? a.slots_of[row] : row;
  if (slot < 0 || slot >= a.slots) return;
  const int v0 = part * RW * R + rr;
  float* sp = a.state + ((slot * a.hv + h) * a.value_dim) * int64_t(K) + 4 * l;
  float4 s[R][4];
#pragma unroll
  for (int p = 0; p < R; ++p)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int v = v0 + p * RW;
      s[p][j] = v < a.value_dim ? load4(sp + int64_t(v) * K + 4 * LR * j) : float4{};
    }
  const int hk = h / a.ratio;
  float4 kv[4], qv[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    kv[j] = load4(static_cast<const Act*>(a.k) + row * a.k_stride + int64_t(hk) * K + 4 * l + 4 * LR * j);
    qv[j] = load4(static_cast<const Act*>(a.q) + row * a.q_stride + int64_t(hk) * K + 4 * l + 4 * LR * j);
  }
  const float dt = gate_step(load_act(static_cast<const Act*>(a.dt_raw), rh) + a.dt_bias[h], a.dt_min,
                             a.dt_max);
  const float decay = __builtin_amdgcn_exp2f(dt * decay_rate_log2(a.A_log[h]));
  const float beta = sigmoid(load_act(static_cast<const Act*>(a.beta_raw), rh));
  float sk = 0.0f, sq = 0.0f, kq = 0.0f;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    sk += kv[j].x * kv[j].x + kv[j].y * kv[j].y + kv[j].z * kv[j].z + kv[j].w * kv[j].w;
    sq += qv[j].x * qv[j].x + qv[j].y * qv[j].y + qv[j].z * qv[j].z + qv[j].w * qv[j].w;
    kq += kv[j].x * qv[j].x + kv[j].y * qv[j].y + kv[j].z * qv[j].z + kv[j].w * qv[j].w;
  }
#pragma unroll
  for (int d = 1; d < LR; d <<= 1) {
    sk += __shfl_xor(sk, d, 64);
    sq += __shfl_xor(sq, d, 64);
    kq += __shfl_xor(kq, d, 64);
  }
  const float rk = 1.0f / sqrtf(sk + a.eps), rq = a.scale / sqrtf(sq + a.eps);
#pragma unroll
  for (int p = 0; p < R; ++p) {
    const int v = v0 + p * RW;
    // With S' = a S: d = beta (v - S' k^), S = S' + d k^^T, y = S q^ = S' q^ + d (k^.q^).
    float pk = 0.0f, pq = 0.0f;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      pk += s[p][j].x * kv[j].x + s[p][j].y * kv[j].y + s[p][j].z * kv[j].z + s[p][j].w * kv[j].w;
      pq += s[p][j].x * qv[j].x + s[p][j].y * qv[j].y + s[p][j].z * qv[j].z + s[p][j].w * qv[j].w;
    }
#pragma unroll
    for (int d = 1; d < LR; d <<= 1) {
      pk += __shfl_xor(pk, d, 64);
      pq += __shfl_xor(pq, d, 64);
    }
    if (v < a.value_dim) {
      const float x = load_act(static_cast<const Act*>(a.v), row * a.v_stride + int64_t(h) * a.value_dim + v);
      const float d = beta * fmaf(-decay * rk, pk, x);
      const float dk = d * rk;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        float4 t = s[p][j];
        t.x = fmaf(dk, kv[j].x, decay * t.x);
        t.y = fmaf(dk, kv[j].y, decay * t.y);
        t.z = fmaf(dk, kv[j].z, decay * t.z);
        t.w = fmaf(dk, kv[j].w, decay * t.w);
        *reinterpret_cast<float4*>(sp + int64_t(v) * K + 4 * LR * j) = t;
      }
      if (l == 0)
        store_act(static_cast<Act*>(a.y), rh * a.value_dim + v,
                  rq * fmaf(dk, kq, decay * pq));
    }
  }
}

// ---- host side ----------------------------------------------------------------------------------
constexpr int64_t kMaxGrid = 65535;
constexpr int64_t kMaxElems = int64_t(1) << 40;

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }
bool product_ok(int64_t a, int64_t b, int64_t* out) {
  return !__builtin_mul_overflow(a, b, out) && *out <= kMaxElems;
}

axon_status check_shape(const axon_gated_delta_shape* s) {
  if (!s) return AXON_ERR_INVALID_ARGUMENT;
  if (s->sequences < 1 || s->tokens < 0 || s->key_heads < 1 || s->value_heads < 1 ||
      s->key_dim < 1 || s->value_dim < 1 || s->state_slots < 0 || s->out_slots < 0 || s->q_stride < 0 ||
      s->k_stride < 0 || s->v_stride < 0)
    return AXON_ERR_INVALID_ARGUMENT;
  if (s->sequences > kMaxGrid || s->value_heads > kMaxGrid || s->key_heads > kMaxGrid ||
      s->value_heads % s->key_heads || (s->key_dim != 64 && s->key_dim != 128) ||
      s->value_dim % 16 || s->value_dim > 256 || s->tokens >= (int64_t(1) << 29) ||
      s->sequences * s->value_heads >= (int64_t(1) << 20) ||
      (s->act_dtype != AXON_F32 && s->act_dtype != AXON_BF16))
    return AXON_ERR_UNSUPPORTED;
  const int64_t strides[] = {s->q_stride, s->k_stride, s->v_stride};
  const int64_t own[] = {s->key_heads * s->key_dim, s->key_heads * s->key_dim,
                         s->value_heads * s->value_dim};
  for (int j = 0; j < 3; ++j) {
    if (strides[j] && (strides[j] < own[j] || strides[j] % 8)) return AXON_ERR_INVALID_ARGUMENT;
    int64_t t;
    if (!product_ok(s->tokens, strides[j] ? strides[j] : own[j], &t)) return AXON_ERR_UNSUPPORTED;
  }
  int64_t t;
  const int64_t state = s->value_heads * s->value_dim * s->key_dim;
  if (!product_ok(s->state_slots, state, &t) || !product_ok(s->out_slots, state, &t))
    return AXON_ERR_UNSUPPORTED;
  return AXON_OK;
}

axon_status check_params(const axon_gated_delta_params* p) {
  if (!p) return AXON_ERR_INVALID_ARGUMENT;
  if (!p->A_log || !p->dt_bias || !aligned16(p->A_log) || !aligned16(p->dt_bias))
    return AXON_ERR_INVALID_ARGUMENT;
  if (!std::isfinite(p->dt_min) || !std::isfinite(p->dt_max) || p->dt_min < 0.0f ||
      p->dt_min > p->dt_max || !std::isfinite(p->scale) || !std::isfinite(p->eps) ||
      !(p->eps > 0.0f))
    return AXON_ERR_INVALID_ARGUMENT;
  return AXON_OK;
}

// Chunk rows for any lengths (axon_sequence_tables' rows for block 64).
int64_t rows_of(const axon_gated_delta_shape* s) { return s->tokens / kQ + s->sequences; }

size_t workspace_of(const axon_gated_delta_shape* s) {
  return s->tokens ? sizeof(float) * kRecord * size_t(rows_of(s)) * size_t(s->value_heads) : 0;
}

struct Strides {
  int64_t q, k, v;
};
Strides strides_of(const axon_gated_delta_shape* s) {
  const int64_t qk = s->key_heads * s->key_dim, v = s->value_heads * s->value_dim;
  return {s->q_stride ? s->q_stride : qk, s->k_stride ? s->k_stride : qk,
          s->v_stride ? s->v_stride : v};
}

// Byte ranges of q, k, v, dt_raw, beta_raw and the parameters.
void input_spans(const axon_gated_delta_shape* s, const axon_gated_delta_params* p, const void* q,
                 const void* k, const void* v, const void* dt_raw, const void* beta_raw,
                 Span out[7]) {
  const size_t es = s->act_dtype == AXON_BF16 ? 2 : 4;
  const Strides st = strides_of(s);
  const int64_t last = s->tokens - 1;
  out[0] = span(q, es * size_t(last * st.q + s->key_heads * s->key_dim));
  out[1] = span(k, es * size_t(last * st.k + s->key_heads * s->key_dim));
  out[2] = span(v, es * size_t(last * st.v + s->value_heads * s->value_dim));
  out[3] = span(dt_raw, es * size_t(s->tokens * s->value_heads));
  out[4] = span(beta_raw, es * size_t(s->tokens * s->value_heads));
  out[5] = span(p->A_log, 4 * size_t(s->value_heads));
  out[6] = span(p->dt_bias, 4 * size_t(s->value_heads));
}

template <typename Act, int K>
void launch_scan(const DeltaArgs& a, bool any, hipStream_t st) {
  if (any) {
    hipLaunchKernelGGL((prep_kernel<Act, K>), dim3(unsigned(a.rows), unsigned(a.hk)), dim3(kThreads),
                       0, st, a);
  }
  const int64_t heads8 = (int64_t(a.sequences) * a.hv + 7) / 8 * 8;
  hipLaunchKernelGGL((walk_kernel<Act, K>), dim3(unsigned(heads8 * a.col_groups)), dim3(kThreads), 0,
                     st, a);
}

template <typename Act, int K>
void launch_step(StepArgs a, hipStream_t st) {
  constexpr int RW = 64 / (K / 16);
  // Four passes a wave keep 16 KiB of state loads in flight; where that leaves fewer than two
  // waves a SIMD (1024 SIMDs), one pass spreads the rows over four times the waves.
  const int64_t heads = int64_t(a.rows) * a.hv;
  const int w4 = (a.value_dim + 4 * RW - 1) / (4 * RW);
  const bool wide = heads * w4 >= 2048;
  a.waves_per_head = wide ? w4 : (a.value_dim + RW - 1) / RW;
  const unsigned wgs = static_cast<unsigned>((heads * a.waves_per_head + 3) / 4);
  if (wide)
    hipLaunchKernelGGL((step_kernel<Act, K, 4>), dim3(wgs), dim3(kThreads), 0, st, a);
  else
    hipLaunchKernelGGL((step_kernel<Act, K, 1>), dim3(wgs), dim3(kThreads), 0, st, a);
}

}  // namespace
}  // namespace axon

extern "C" {

size_t axon_gated_delta_scan_workspace_bytes(const axon_gated_delta_shape* shape) {
  if (axon::check_shape(shape) != AXON_OK) return 0;
  return axon::workspace_of(shape);
}

axon_status axon_gated_delta_scan(const axon_gated_delta_shape* shape,
                                  const axon_gated_delta_params* params, const void* q,
                                  const void* k, const void* v, const void* dt_raw,
                                  const void* beta_raw, const int32_t* tables,
                                  const float* state_in, const int32_t* in_slots, void* y,
                                  float* state_out, const int32_t* out_slots, void* workspace,
                                  size_t workspace_bytes, void* stream) {
  using namespace axon;
  axon_status why = check_shape(shape);
  if (why != AXON_OK) return why;
  why = check_params(params);
  if (why != AXON_OK) return why;
  const axon_gated_delta_shape& s = *shape;
  if (!tables && s.tokens % s.sequences) return AXON_ERR_INVALID_ARGUMENT;
  if ((tables && !aligned4(tables)) || (in_slots && !aligned4(in_slots)) ||
      (out_slots && !aligned4(out_slots)) || (state_in && !aligned16(state_in)) ||
      (state_out && !aligned16(state_out)))
    return AXON_ERR_INVALID_ARGUMENT;
  // Without slots state n is sequence n's.
  if ((state_in && !in_slots && s.state_slots < s.sequences) ||
      (state_out && !out_slots && s.out_slots < s.sequences) ||
      (state_in && state_in == state_out && s.state_slots != s.out_slots))
    return AXON_ERR_INVALID_ARGUMENT;
  const bool any = s.tokens > 0;
  if (any) {
    const void* acts[] = {q, k, v, dt_raw, beta_raw, y};
    for (const void* p : acts)
      if (!p || !aligned16(p)) return AXON_ERR_INVALID_ARGUMENT;
  }
  const int64_t rows = rows_of(shape);
  const size_t need = workspace_of(shape);
  if (workspace_bytes < need) return AXON_ERR_WORKSPACE_TOO_SMALL;
  if (need && (!workspace || !aligned16(workspace))) return AXON_ERR_INVALID_ARGUMENT;

  const size_t es = s.act_dtype == AXON_BF16 ? 2 : 4;
  const size_t state4 = 4 * size_t(s.value_heads * s.value_dim * s.key_dim);
  const size_t seq4 = 4 * size_t(s.sequences);
  const Span in_state = span(state_in, state4 * size_t(s.state_slots));
  const Span out_state = span(state_out, state4 * size_t(s.out_slots));
  const Span out_y = any ? span(y, es * size_t(s.tokens * s.value_heads * s.value_dim)) : Span{};
  const Span ws = need ? span(workspace, need) : Span{};
  Span reads[10];
  if (any) input_spans(shape, params, q, k, v, dt_raw, beta_raw, reads);
  reads[7] = span(tables, 4 * (2 * (size_t(s.sequences) + 1) + 2 * size_t(rows)));
  reads[8] = span(in_slots, seq4);
  reads[9] = span(out_slots, seq4);
  for (const Span& r : reads)
    if (overlaps(out_y, r) || overlaps(out_state, r) || overlaps(ws, r))
      return AXON_ERR_INVALID_ARGUMENT;
  if (state_in != state_out && overlaps(in_state, out_state)) return AXON_ERR_INVALID_ARGUMENT;
  if (overlaps(out_y, in_state) || overlaps(out_y, out_state) || overlaps(out_y, ws) ||
      overlaps(ws, in_state) || overlaps(ws, out_state))
    return AXON_ERR_INVALID_ARGUMENT;

  DeltaArgs a{};
  a.q = q, a.k = k, a.v = v, a.dt_raw = dt_raw, a.beta_raw = beta_raw;
  a.A_log = params->A_log, a.dt_bias = params->dt_bias;
  a.dt_min = params->dt_min, a.dt_max = params->dt_max;
  a.scale = params->scale, a.eps = params->eps;
  if (tables) {
    a.starts = tables;
    a.block_starts = tables + (s.sequences + 1);
    a.block_seq = tables + 2 * (s.sequences + 1);
    a.block_first = a.block_seq + rows;
  }
  a.state_in = state_in, a.in_slots = in_slots, a.y = y, a.state_out = state_out;
  a.out_slots = out_slots, a.records = static_cast<float*>(workspace);
  const Strides st = strides_of(shape);
  a.tokens = s.tokens, a.q_stride = st.q, a.k_stride = st.k, a.v_stride = st.v;
  a.in_count = s.state_slots, a.out_count = s.out_slots;
  a.sequences = int(s.sequences), a.hk = int(s.key_heads), a.hv = int(s.value_heads);
  a.ratio = int(s.value_heads / s.key_heads), a.value_dim = int(s.value_dim);
  a.col_groups = int((s.value_dim + 63) / 64);
  a.seqlen = s.tokens / s.sequences;
  a.chunks_per_seq = int((a.seqlen + kQ - 1) / kQ);
  a.rows = int(tables ? rows : s.sequences * a.chunks_per_seq);
  const bool bf = s.act_dtype == AXON_BF16;
  hipStream_t stm = static_cast<hipStream_t>(stream);
  if (s.key_dim == 64)
    bf ? launch_scan<bf16_bits, 64>(a, any, stm) : launch_scan<float, 64>(a, any, stm);
  else
    bf ? launch_scan<bf16_bits, 128>(a, any, stm) : launch_scan<float, 128>(a, any, stm);
  return hipGetLastError() == hipSuccess ? AXON_OK : AXON_ERR_HIP;
}

axon_status axon_gated_delta_step(const axon_gated_delta_shape* shape,
                                  const axon_gated_delta_params* params, const void* q,
                                  const void* k, const void* v, const void* dt_raw,
                                  const void* beta_raw, float* state, const int32_t* slots,
                                  void* y, void* stream) {
  using namespace axon;
  axon_status why = check_shape(shape);
  if (why != AXON_OK) return why;
  why = check_params(params);
  if (why != AXON_OK) return why;
  const axon_gated_delta_shape& s = *shape;
  if (s.tokens != s.sequences) return AXON_ERR_INVALID_ARGUMENT;
  const void* ptrs[] = {q, k, v, dt_raw, beta_raw, state, y};
  for (const void* p : ptrs)
    if (!p || !aligned16(p)) return AXON_ERR_INVALID_ARGUMENT;
  if (slots ? !aligned4(slots) : s.state_slots < s.sequences) return AXON_ERR_INVALID_ARGUMENT;
  const size_t es = s.act_dtype == AXON_BF16 ? 2 : 4;
  const Span st = span(state, 4 * size_t(s.state_slots) *
                                  size_t(s.value_heads * s.value_dim * s.key_dim));
  const Span out_y = span(y, es * size_t(s.tokens * s.value_heads * s.value_dim));
  Span reads[8];
  input_spans(shape, params, q, k, v, dt_raw, beta_raw, reads);
  reads[7] = span(slots, 4 * size_t(s.sequences));
  for (const Span& r : reads)
    if (overlaps(out_y, r) || overlaps(st, r)) return AXON_ERR_INVALID_ARGUMENT;
  if (overlaps(out_y, st)) return AXON_ERR_INVALID_ARGUMENT;
  StepArgs a{};
  a.q = q, a.k = k, a.v = v, a.dt_raw = dt_raw, a.beta_raw = beta_raw;
  a.A_log = params->A_log, a.dt_bias = params->dt_bias;
  a.dt_min = params->dt_min, a.dt_max = params->dt_max;
  a.scale = params->scale, a.eps = params->eps;
  a.state = state, a.slots_of = slots, a.y = y;
  const Strides sr = strides_of(shape);
  a.q_stride = sr.q, a.k_stride = sr.k, a.v_stride = sr.v, a.slots = s.state_slots;
  a.rows = int(s.sequences), a.hv = int(s.value_heads);
  a.ratio = int(s.value_heads / s.key_heads), a.value_dim = int(s.value_dim);
  const bool bf = s.act_dtype == AXON_BF16;
  hipStream_t stm = static_cast<hipStream_t>(stream);
  if (s.key_dim == 64)
    bf ? launch_step<bf16_bits, 64>(a, stm) : launch_step<float, 64>(a, stm);
  else
    bf ? launch_step<bf16_bits, 128>(a, stm) : launch_step<float, 128>(a, stm);
  return hipGetLastError() == hipSuccess ? AXON_OK : AXON_ERR_HIP;
}

}  // extern "C"

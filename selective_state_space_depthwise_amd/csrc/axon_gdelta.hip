// The gated delta rule on gfx950: packed or uniform sequences in chunks of 64 tokens, and the
// single-token step (definitions in axonscan.h).
//
// Inside a chunk, with g_t the inclusive sum of dt A from the chunk's start and S0 (V x K) the
// entering state, the recurrence S_t = a_t S_{t-1} + D_t k^_t^T, D_t = beta_t (v_t - a_t S_{t-1} k^_t)
// unrolls, with D_t = beta_t E_t, to the unit lower triangular system
//   E_t + sum_{s<t} e^{g_t-g_s} (k^_t.k^_s) beta_s E_s = X_t = v_t - e^{g_t} S0 k^_t.
// The inverse T of its matrix I + M does not depend on the state, so it is computed for all chunks
// at once; the walk over the chunks is products only:
//   X = v - e^g (S0 k^),  E = T X,
//   y = scale (e^g S0 q^ + A E),  A[t,s] = e^{g_t-g_s} (q^_t.k^_s) beta_s (s <= t),
//   S <- e^{g_last} S0 + sum_t e^{g_last-g_t} beta_t E_t k^_t^T.
// Every exponent is <= 0; the sums are compensated (head and tail) because steps near dt_max push
// g to thousands, where the plain fp32 sum's ulp would be the error of later differences. The
// norms of q and k multiply rows of the products instead of the operands.
//
//   prep_kernel  per chunk and key head: the Gram products, then per value head T (16 x 16 diagonal
//                blocks by substitution, which stays accurate where keys are alike and powers of M
//                would cancel; the blocks below by matrix products), A and the row factors.
//   join_kernel  where there are few heads and long sequences, segments of a sequence are walked at
//                once: S behind a segment is S0 M + N (each row of S by itself), M (K x K) and N
//                being what a walk makes of the rows of the identity with v = 0 and of zeros with v.
//                A first walk finds M and N of all segments but the last, the join kernel the state
//                before each segment, a second walk the outputs: 2.6 times the work, spread over
//                the GPU. By the contraction of the delta rule a state shrinks at least as its decays
//                say; where those multiply to less than 2^-160 over a segment's last chunks (beyond
//                what an fp32 product of them holds) nothing before those chunks is left at its end:
//                the first walk begins there, and M is zero.
//   walk_kernel  per sequence, value head and slice of 16 or 32 columns of V one wave walks the
//                chunks with its slice of the state in registers. The state is held transposed
//                (S^T, K x 16): the result layout of a 16 x 16 product (lane (g, i), g = lane / 16,
//                i = lane % 16: rows 4 g + r, column i) is also the layout of the next product's
//                right operand when 32 contraction indices are dealt to (g, e) as 4 g + e for
//                e < 4 and 16 + 4 g + e - 4 above, so state, X and E go from product to product
//                without leaving their lanes.
//
// Precision. fp32 products would run at a sixteenth of the fp16 matrix rate, so the walk splits
// each fp32 operand into two fp16 pieces, x = hi + lo: off by 2^-23 of x at most, or by 2^-25 where x
// is below a quarter; of a product of pieces lo lo is left out (hi hi + hi lo + lo hi). If the largest
// operands of a sum lie near one, that is nearly what fp32 gives (2 x 2048 tokens against 64 bits: 4.2e-7
// in the mean, the plain form in fp32 2.7e-7), relative to the largest and not to each: T and A are at
// most 1; rows of k and q are scaled by a power of two that takes their largest
// entry to [1, 2) (bf16 entries are then exact in one piece); each column of S, with what the chunk
// makes of its v (X, E and the writes), is kept in a unit of its own, a power of two that takes the
// larger of S and v to about 2^5. By the contraction of the delta rule (0 <= beta <= 1) no entry of
// S, X or E exceeds 2^8 sqrt(K) + 64 2^8 < 2^15 before the next chunk looks at the unit again, so
// nothing leaves the range of fp16. The states, every accumulator and every factor are fp32. This
// holds for bf16 activations too, the operands that only y sees among them: y is what fp32 gives,
// rounded once. (With S, A and E of y's products in one piece, 2^-11, a value in twenty of y came out
// as another bf16 number; 16384 tokens took 406 us instead of 438 us, 32768 packed ones 487 us instead
// of 537 us.)
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <type_traits>

#include "axon_device.h"
#include "axon_internal.h"

namespace axon {
namespace {

constexpr int kQ = 64;  // tokens of a chunk
constexpr int kThreads = 256;

typedef float f4 __attribute__((ext_vector_type(4)));

// fp16 pieces of an activation (bf16: exact in one).
template <typename Act>
constexpr int kPieces = sizeof(Act) == 2 ? 1 : 2;

// What prep leaves for each (chunk, value head): T and A in two pieces, each as ten 16 x 16 blocks
// on and below the diagonal (at block_at), a block as 64 lanes x 4 fp16 in left-operand order (lane
// (g, i): row i, columns 4 g .. 4 g + 3); then the row
// factors of the 64 tokens, fp32, and e^{g_last} with its base-2 logarithm. What the walk keeps in
// LDS comes first.
constexpr int kBlocks = 10;
constexpr int kBlockBytes = 512;
enum Row { kRowX, kRowS, kRowY, kRowKQ, kRows = kRowKQ + 2 };
//   kRowX  e^g / |k| / 2^s                 of S0 k in X (2^s: the scale of k's row)
//   kRowS  beta e^{g_last-g} / |k| / 2^s   of E in the state's sum
//   kRowY  e^g / |q| / 2^s                 of S0 q in y
//   kRowKQ 2^s of k and of q, in pairs
// Pairs of blocks that make one operand (32 contraction indices) lie side by side, so that one
// instruction reads both; the two diagonal blocks without a partner come last.
__host__ __device__ constexpr int block_at(int I, int J) {
  return I == 0 ? 8 : I == 1 ? J : I == 3 ? 4 + J : J < 2 ? 2 + J : 9;
}
constexpr int kRowsAt = 4 * kBlocks * kBlockBytes;
constexpr int kRecordLds = kRowsAt + 4 * kQ * 4;
constexpr int kRecordBytes = kRowsAt + kRows * kQ * 4 + 64;

// Bytes of a segment's M: each row in units of its own, a power of two that takes its largest entry
// to [1, 2) (M shrinks with the decays of its segment, down to 2^-160, and pieces without a unit end at
// 2^-25), then the units as K floats.
constexpr int carry_bytes(int k) { return 4 * k * k + 4 * k; }

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
  char* records;
  int64_t tokens, seqlen, q_stride, k_stride, v_stride, in_count, out_count;
  int sequences, hk, hv, ratio, value_dim, col_groups;
  int rows;             // chunk rows of the workspace
  int chunks_per_seq;   // uniform batch
  int seg_chunks;       // chunks of a segment, 0: sequences are walked whole
  int segs;             // segments of a sequence at most
  char* seg_m;          // (segment, value head): M^T, two pieces of K x K fp16, and M's row factors
  int32_t* seg_flag;    // (segment, value head): whether M is not zero
  float* seg_s;         // (segment, value head): N, then the state before the segment, V x K
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

// softplus to the last bits: the step enters the exponent of the decay multiplied by the rate. NaN
// stays NaN (fminf and fmaxf would make a bound of it).
__device__ __forceinline__ float gate_step(float v, float lo, float hi) {
  const float dt = fmaxf(v, 0.0f) + log1pf(expf(-fabsf(v)));
  return dt < lo ? lo : dt > hi ? hi : dt;
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

// ---- fp16 pieces --------------------------------------------------------------------------------
typedef _Float16 h4 __attribute__((ext_vector_type(4)));
typedef _Float16 h8 __attribute__((ext_vector_type(8)));
typedef __bf16 b8 __attribute__((ext_vector_type(8)));
typedef uint16_t u2 __attribute__((ext_vector_type(2)));
typedef uint32_t w2 __attribute__((ext_vector_type(2)));
typedef uint32_t w4 __attribute__((ext_vector_type(4)));

__device__ __forceinline__ f4 mfma_h(h8 a, h8 b, f4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
}

// 2^s that takes m to [1, 2), and its inverse; m is held to [2^-97, 2^123], where both are normal
// numbers.
struct Scale {
  float up, down;
};
__device__ __forceinline__ Scale scale_of(float m) {
  int e = static_cast<int>(__float_as_uint(m) >> 23);
  e = e < 30 ? 30 : e > 250 ? 250 : e;
  return {__uint_as_float(static_cast<uint32_t>(254 - e) << 23),
          __uint_as_float(static_cast<uint32_t>(e) << 23)};
}

// Eight activations as loaded, and their fp16 pieces.
template <typename Act>
struct Eight;
template <>
struct Eight<bf16_bits> {
  w4 raw;
  __device__ __forceinline__ void load(rsrc_t r, uint32_t off) {
    raw = __builtin_bit_cast(w4, __builtin_amdgcn_raw_buffer_load_b128(r, off, 0, 0));
  }
  __device__ __forceinline__ void pieces(float up, w4* out) const {
    f4 a, b;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      a[2 * e] = __uint_as_float(raw[e] << 16) * up;
      a[2 * e + 1] = __uint_as_float(raw[e] & 0xFFFF0000u) * up;
      b[2 * e] = __uint_as_float(raw[e + 2] << 16) * up;
      b[2 * e + 1] = __uint_as_float(raw[e + 2] & 0xFFFF0000u) * up;
    }
    out[0] = __builtin_bit_cast(
        w4, __builtin_shufflevector(__builtin_convertvector(a, h4), __builtin_convertvector(b, h4), 0,
                                    1, 2, 3, 4, 5, 6, 7));
  }
};
template <>
struct Eight<float> {
  f4 lo, hi;
  __device__ __forceinline__ void load(rsrc_t r, uint32_t off) {
    lo = __builtin_bit_cast(f4, __builtin_amdgcn_raw_buffer_load_b128(r, off, 0, 0));
    hi = __builtin_bit_cast(f4, __builtin_amdgcn_raw_buffer_load_b128(r, off + 16, 0, 0));
  }
  __device__ __forceinline__ void pieces(float up, w4* out) const {
    const f4 a = lo * up, b = hi * up;
    const h4 ha = __builtin_convertvector(a, h4), hb = __builtin_convertvector(b, h4);
    const h4 la = __builtin_convertvector(a - __builtin_convertvector(ha, f4), h4);
    const h4 lb = __builtin_convertvector(b - __builtin_convertvector(hb, f4), h4);
    out[0] = __builtin_bit_cast(w4, __builtin_shufflevector(ha, hb, 0, 1, 2, 3, 4, 5, 6, 7));
    out[1] = __builtin_bit_cast(w4, __builtin_shufflevector(la, lb, 0, 1, 2, 3, 4, 5, 6, 7));
  }
};

// A lane's 16 values of a column of v, as loaded.
template <typename Act>
struct Column;
template <>
struct Column<bf16_bits> {
  uint32_t raw[8];
  __device__ __forceinline__ float largest() const {  // bf16 magnitudes are ordered as integers
    u2 m = __builtin_bit_cast(u2, raw[0] & 0x7FFF7FFFu);
#pragma unroll
    for (int e = 1; e < 8; ++e)
      m = __builtin_elementwise_max(m, __builtin_bit_cast(u2, raw[e] & 0x7FFF7FFFu));
    return __uint_as_float(static_cast<uint32_t>(m[0] > m[1] ? m[0] : m[1]) << 16);
  }
  __device__ __forceinline__ float value(int tt, int r) const {
    const uint32_t x = raw[2 * tt + (r >> 1)];
    return __uint_as_float(r & 1 ? x & 0xFFFF0000u : x << 16);
  }
};
template <>
struct Column<float> {
  float raw[16];
  __device__ __forceinline__ float largest() const {
    float m = 0.0f;
#pragma unroll
    for (int e = 0; e < 16; ++e) m = fmaxf(m, fabsf(raw[e]));
    return m;
  }
  __device__ __forceinline__ float value(int tt, int r) const { return raw[4 * tt + r]; }
};

// Two pieces of eight values (two accumulators of one column).
__device__ __forceinline__ h8 first_piece(f4 a, f4 b) {
  return __builtin_shufflevector(__builtin_convertvector(a, h4), __builtin_convertvector(b, h4), 0, 1,
                                 2, 3, 4, 5, 6, 7);
}
__device__ __forceinline__ void split8(f4 a, f4 b, h8* hi, h8* lo) {
  // One v_fma_mix_f32 takes a piece off its value; the compiler, if it knew the factor, would convert
  // the piece first.
  float minus = -1.0f;
  asm volatile("" : "+s"(minus));
  *hi = first_piece(a, b);
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    a[e] = fmaf(static_cast<float>((*hi)[e]), minus, a[e]);
    b[e] = fmaf(static_cast<float>((*hi)[e + 4]), minus, b[e]);
  }
  *lo = first_piece(a, b);
}

// 16 lanes read 4 rows x 16 fp16 (lane j: row j / 4, columns 4 (j % 4) ..) and lane j gets column j.
__device__ __forceinline__ h4 read_transposed(const char* p) {
  typedef short s4 __attribute__((ext_vector_type(4)));
  return __builtin_bit_cast(
      h4, __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s4*)p));
}

// The value, computed anew where it is used: sums with it are not kept in registers across a loop.
__device__ __forceinline__ uint32_t fresh(uint32_t v) {
  asm volatile("" : "+v"(v));
  return v;
}

// 16 bytes a lane from `base + off` to the wave's consecutive 1024 bytes at `to` in LDS. Written out
// because the compiler would wait for the copy before any read of LDS, also of another buffer; the
// caller waits for it (no register is written). m0, where the instruction takes the place in LDS from,
// is an operand, so that the compiler knows when it is in use.
__device__ __forceinline__ void load_to_lds(const char* base, uint32_t off, char* to) {
  const uint32_t m0 = __builtin_amdgcn_readfirstlane(
      static_cast<uint32_t>(reinterpret_cast<uintptr_t>((__attribute__((address_space(3))) char*)to)));
  asm volatile("s_nop 0\n\tglobal_load_lds_dwordx4 %1, %2"
               :
               : "{m0}"(m0), "v"(off), "s"(base)
               : "memory");
}

// The largest over the four lanes (g = 0 .. 3) that share a column.
__device__ __forceinline__ float column_max(float m) {
  const uint32_t u = __float_as_uint(m);
  const auto a = __builtin_amdgcn_permlane16_swap(u, u, false, false);
  const float x = fmaxf(__uint_as_float(a[0]), __uint_as_float(a[1]));
  const uint32_t v = __float_as_uint(x);
  const auto b = __builtin_amdgcn_permlane32_swap(v, v, false, false);
  return fmaxf(__uint_as_float(b[0]), __uint_as_float(b[1]));
}
__device__ __forceinline__ float max4(float m, f4 x) {
  m = fmaxf(fmaxf(m, fabsf(x[0])), fabsf(x[1]));
  return fmaxf(fmaxf(m, fabsf(x[2])), fabsf(x[3]));
}

// ---- T, A and the row factors of every chunk ----------------------------------------------------
// Grid (chunk rows, key heads), 4 waves; the value heads of the key head in pairs. Every 16 x 16
// block is computed transposed (rows: 4 columns of the block, column: its row i), which is at once
// the operand order of the record (a lane holds 4 consecutive entries of a row) and the layout in
// which one product's result is the next one's right operand, so only -M and the inverses of the
// diagonal blocks of I + M pass through LDS. Wave w owns rows 16 w .. of the Gram products (bf16:
// exact bf16 products; fp32 and the inverse: v_mfma_f32_16x16x4f32). The diagonal blocks of a head
// are inverted by one wave, block g by lane group g, a column a lane. From T (I + M) = I the blocks
// below follow row by row: T_IJ = (sum_{J < S <= I} T_IS (-M)_SJ) D_J with D_J the inverse of
// diagonal block J; one wave takes row block 3 of a head (9 products), another its rows 2 and 1 (7).
// 32768 tokens x 16 key and 32 value heads, bf16: 167 us for 0.53 GB read and written (3.2 TB/s); the
// phases of a workgroup wait for each other, four workgroups a CU fill most of that. (Five spill
// registers: the scan takes 5% longer. Records stored past the caches: no change.)
constexpr int kHeads = 2;      // value heads at a time
constexpr int kBlockRow = 20;  // floats between the rows of a block in LDS

template <typename Act, int K>
__global__ __launch_bounds__(kThreads, sizeof(Act) == 2 ? 4 : 3) void prep_kernel(DeltaArgs a) {
  constexpr int P = kPieces<Act>;
  __shared__ __align__(16) float Ms[kHeads][kBlocks][16 * kBlockRow];
  __shared__ __align__(16) float hi_s[kHeads][kQ], lo_s[kHeads][kQ], beta_s[kHeads][kQ];
  __shared__ __align__(16) float rk_s[kQ], rq_s[kQ], mk_s[kQ], mq_s[kQ];
  int64_t first;
  int count;
  if (!chunk_of(a, blockIdx.x, &first, &count)) return;
  const int hk = blockIdx.y;
  const int tid = threadIdx.x, lane = tid & 63, g = lane >> 4, i = lane & 15;
  const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
  // Rows behind the sequence lie outside the resources' ranges and read as zeros.
  constexpr uint32_t es = sizeof(Act);
  const uint32_t kst = static_cast<uint32_t>(a.k_stride) * es, qst = static_cast<uint32_t>(a.q_stride) * es;
  const rsrc_t kr = make_rsrc_bounded(
      const_cast<Act*>(static_cast<const Act*>(a.k) + first * a.k_stride + int64_t(hk) * K),
      (count - 1) * kst + K * es);
  const rsrc_t qr = make_rsrc_bounded(
      const_cast<Act*>(static_cast<const Act*>(a.q) + first * a.q_stride + int64_t(hk) * K),
      (count - 1) * qst + K * es);
  // Steps, decays and write strengths of one head: lane t is token t.
  auto gates = [&](int h, int at_head) {
    float dt = 0.0f, beta = 0.0f;
    if (lane < count) {
      const int64_t at = (first + lane) * a.hv + h;
      dt = gate_step(load_act(static_cast<const Act*>(a.dt_raw), at) + a.dt_bias[h], a.dt_min, a.dt_max);
      beta = sigmoid(load_act(static_cast<const Act*>(a.beta_raw), at));
    }
    // No decay below 2^-16384 differs from 0: the bound keeps the sums finite for any dt_max.
    float hi = dt * decay_rate_log2(a.A_log[h]), lo = 0.0f;
    if (hi < -16384.0f) hi = -16384.0f;
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
    hi_s[at_head][lane] = hi, lo_s[at_head][lane] = lo, beta_s[at_head][lane] = beta;
  };
  f4 gk[4], gq[4];
#pragma unroll
  for (int st = 0; st < 4; ++st) gk[st] = gq[st] = f4{0.0f, 0.0f, 0.0f, 0.0f};
  float rk, rq;  // of row 16 w + i
  {
    const int t = 16 * w + i;
    float sk = 0.0f, sq = 0.0f, mk = 0.0f, mq = 0.0f;
    if constexpr (P == 1) {
      constexpr int NB = K / 32;
      auto load = [&](rsrc_t r, uint32_t off, b8* to) {
#pragma unroll
        for (int b = 0; b < NB; ++b)
          to[b] = __builtin_bit_cast(b8, __builtin_amdgcn_raw_buffer_load_b128(r, off + 64 * b, 0, 0));
      };
      b8 krow[NB], qrow[NB], col[NB];
      load(kr, t * kst + 16 * g, krow);
      load(qr, t * qst + 16 * g, qrow);
      if (w < kHeads && w < a.ratio) gates(hk * a.ratio + w, w);  // while k and q are on their way
      f4 dk, dq = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int st = 0; st < 4; ++st) {
        if (st > w) continue;
        load(kr, (16 * st + i) * kst + 16 * g, col);
#pragma unroll
        for (int b = 0; b < NB; ++b) {
          gk[st] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(col[b], krow[b], gk[st], 0, 0, 0);
          gq[st] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(col[b], qrow[b], gq[st], 0, 0, 0);
        }
        dk = gk[st];  // of the last one, st = w
      }
      // The squared norms are the diagonals of the Gram products: row i's in lane (i / 4, i).
#pragma unroll
      for (int b = 0; b < NB; ++b) dq = __builtin_amdgcn_mfma_f32_16x16x32_bf16(qrow[b], qrow[b], dq, 0, 0, 0);
      if (g == i >> 2) {
        sk = i & 2 ? (i & 1 ? dk[3] : dk[2]) : (i & 1 ? dk[1] : dk[0]);
        sq = i & 2 ? (i & 1 ? dq[3] : dq[2]) : (i & 1 ? dq[1] : dq[0]);
      }
      auto largest = [](const b8* x) {  // bf16 magnitudes are ordered as integers
        u2 m = {0, 0};
#pragma unroll
        for (int b = 0; b < NB; ++b) {
          const w4 raw = __builtin_bit_cast(w4, x[b]);
#pragma unroll
          for (int e = 0; e < 4; ++e)
            m = __builtin_elementwise_max(m, __builtin_bit_cast(u2, raw[e] & 0x7FFF7FFFu));
        }
        return __uint_as_float(static_cast<uint32_t>(m[0] > m[1] ? m[0] : m[1]) << 16);
      };
      mk = largest(krow);
      mq = largest(qrow);
    } else {
      constexpr int NB = K / 16;
      auto load = [&](rsrc_t r, uint32_t off, f4* to) {
#pragma unroll
        for (int b = 0; b < NB; ++b)
          to[b] = __builtin_bit_cast(f4, __builtin_amdgcn_raw_buffer_load_b128(r, off + 64 * b, 0, 0));
      };
      auto sums = [](f4 x, float& s, float& m) {
        s += x[0] * x[0] + x[1] * x[1] + x[2] * x[2] + x[3] * x[3];
        m = max4(m, x);
      };
      f4 row[NB], col[NB];
      load(kr, t * kst + 16 * g, row);
      if (w < kHeads && w < a.ratio) gates(hk * a.ratio + w, w);
#pragma unroll
      for (int b = 0; b < NB; ++b) sums(row[b], sk, mk);
#pragma unroll
      for (int which = 0; which < 2; ++which) {
        if (which == 1) {
          load(qr, t * qst + 16 * g, row);
#pragma unroll
          for (int b = 0; b < NB; ++b) sums(row[b], sq, mq);
        }
#pragma unroll
        for (int st = 0; st < 4; ++st) {
          if (st > w) continue;
          load(kr, (16 * st + i) * kst + 16 * g, col);
#pragma unroll
          for (int b = 0; b < NB; ++b)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              f4& to = which ? gq[st] : gk[st];
              to = mfma4(col[b][e], row[b][e], to);
            }
        }
      }
    }
    sk += __shfl_xor(sk, 16, 64);
    sk += __shfl_xor(sk, 32, 64);
    sq += __shfl_xor(sq, 16, 64);
    sq += __shfl_xor(sq, 32, 64);
    mk = column_max(mk);
    mq = column_max(mq);
    rk = 1.0f / sqrtf(sk + a.eps);
    rq = 1.0f / sqrtf(sq + a.eps);
    if (g == 0) rk_s[t] = rk, rq_s[t] = rq, mk_s[t] = mk, mq_s[t] = mq;
  }
  for (int v0 = 0; v0 < a.ratio; v0 += kHeads) {
    const int heads = min(kHeads, a.ratio - v0);
    if (v0 > 0) {
      __syncthreads();  // every wave is done with the heads before
      if (w < heads) gates(hk * a.ratio + v0 + w, w);
    }
    __syncthreads();  // gates and norms are in
    if (v0 == 0) {
#pragma unroll
      for (int st = 0; st < 4; ++st) {
        if (st > w) continue;
        const f4 ks = *reinterpret_cast<const f4*>(&rk_s[16 * st + 4 * g]);
        gk[st] *= ks * -rk;
        gq[st] *= ks * rq;
      }
    }
    for (int hh = 0; hh < heads; ++hh) {
      char* rec = a.records + (int64_t(blockIdx.x) * a.hv + hk * a.ratio + v0 + hh) * kRecordBytes;
      const int t = 16 * w + i;
      const float ht = hi_s[hh][t], lt = lo_s[hh][t];
#pragma unroll
      for (int st = 0; st < 4; ++st) {
        if (st > w) continue;
        const int s = 16 * st + 4 * g, blk = w * (w + 1) / 2 + st;
        const f4 hs = *reinterpret_cast<const f4*>(&hi_s[hh][s]), ls = *reinterpret_cast<const f4*>(&lo_s[hh][s]);
        const f4 bs = *reinterpret_cast<const f4*>(&beta_s[hh][s]);
        f4 m, x;
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const float e = exp2_diff(ht, lt, hs[r], ls[r]) * bs[r];
          m[r] = e * gk[st][r];
          x[r] = e * gq[st][r];
        }
        if (st == w) {
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            m[r] = 4 * g + r < i ? m[r] : 0.0f;
            x[r] = 4 * g + r <= i ? x[r] : 0.0f;
          }
        }
        *reinterpret_cast<f4*>(&Ms[hh][blk][i * kBlockRow + 4 * g]) = m;
        const h4 hi = __builtin_convertvector(x, h4);
        char* dst = rec + (2 * kBlocks + block_at(w, st)) * kBlockBytes + lane * 8;
        *reinterpret_cast<h4*>(dst) = hi;
        *reinterpret_cast<h4*>(dst + kBlocks * kBlockBytes) =
            __builtin_convertvector(x - __builtin_convertvector(hi, f4), h4);
      }
      if (w == 2 + hh) {  // the row factors: lane t is token t
        const float hi = hi_s[hh][lane], lo = lo_s[hh][lane];
        const float e = __builtin_amdgcn_exp2f(hi + lo);
        const Scale k2 = scale_of(mk_s[lane]), q2 = scale_of(mq_s[lane]);
        float* row = reinterpret_cast<float*>(rec + kRowsAt) + lane;
        row[kRowX * kQ] = e * (rk_s[lane] * k2.down);
        row[kRowS * kQ] = beta_s[hh][lane] * exp2_diff(hi_s[hh][63], lo_s[hh][63], hi, lo) *
                          (rk_s[lane] * k2.down);
        row[kRowY * kQ] = e * (rq_s[lane] * q2.down);
        *reinterpret_cast<float2*>(row + kRowKQ * kQ + lane) = make_float2(k2.up, q2.up);
        if (lane == 63) *reinterpret_cast<float2*>(row + kRows * kQ - 63) = make_float2(e, hi + lo);
      }
    }
    __syncthreads();
    // Column i of the inverse of diagonal block g, in the block's place.
    if (w < heads) {
      float* m = Ms[w][g * (g + 1) / 2 + g];
      float x[16];
#pragma unroll
      for (int r = 0; r < 16; ++r) {
        float acc = r == i ? 1.0f : 0.0f;
#pragma unroll
        for (int s4 = 0; s4 < r; s4 += 4) {
          const f4 row = *reinterpret_cast<const f4*>(m + r * kBlockRow + s4);
#pragma unroll
          for (int s = 0; s < 4; ++s)
            if (s4 + s < r) acc = fmaf(row[s], x[s4 + s], acc);
        }
        x[r] = acc;
      }
      // One wave: its reads above are done before these writes are issued.
#pragma unroll
      for (int r = 0; r < 16; ++r) m[r * kBlockRow + i] = x[r];
    }
    __syncthreads();
    const int hh = w & 1;
    if (hh < heads) {
      char* rec = a.records + (int64_t(blockIdx.x) * a.hv + hk * a.ratio + v0 + hh) * kRecordBytes;
      const float(*m)[16 * kBlockRow] = Ms[hh];
      auto put = [&](int blk, f4 x) {
        const h4 hi = __builtin_convertvector(x, h4);
        char* dst = rec + blk * kBlockBytes + lane * 8;
        *reinterpret_cast<h4*>(dst) = hi;
        *reinterpret_cast<h4*>(dst + kBlocks * kBlockBytes) =
            __builtin_convertvector(x - __builtin_convertvector(hi, f4), h4);
      };
      // Row block I of T, from the diagonal leftwards.
      auto row_block = [&](auto index) {
        constexpr int I = decltype(index)::value;
        f4 T[I + 1];
        T[I] = *reinterpret_cast<const f4*>(m[I * (I + 1) / 2 + I] + i * kBlockRow + 4 * g);
        put(block_at(I, I), T[I]);
#pragma unroll
        for (int J = I - 1; J >= 0; --J) {
          f4 p = f4{0.0f, 0.0f, 0.0f, 0.0f}, x = p;
#pragma unroll
          for (int S = J + 1; S <= I; ++S)
#pragma unroll
            for (int r = 0; r < 4; ++r)
              p = mfma4(m[S * (S + 1) / 2 + J][(4 * g + r) * kBlockRow + i], T[S][r], p);
#pragma unroll
          for (int r = 0; r < 4; ++r) x = mfma4(m[J * (J + 1) / 2 + J][(4 * g + r) * kBlockRow + i], p[r], x);
          T[J] = x;
          put(block_at(I, J), T[J]);
        }
      };
      if (w < 2) {
        row_block(std::integral_constant<int, 3>{});
      } else {
        row_block(std::integral_constant<int, 2>{});
        row_block(std::integral_constant<int, 1>{});
        row_block(std::integral_constant<int, 0>{});
      }
    }
  }
}

// ---- the walk over the chunks -------------------------------------------------------------------
// Bound by a chunk's chain of dependent products and the LDS reads and conversions that feed them:
// 32768 packed tokens x 32 heads, bf16, K = V = 128: 371 us, of a CU's about 11700 clocks a chunk the
// matrix cores are busy for 4200, the vector units for 5400.
// W waves a workgroup, each with NC tiles of 16 columns of V of one head (two in the first walk over
// segments of bf16, which has no outputs to sum). Per chunk the workgroup brings k and q, converted to
// fp16 pieces on the way, as rows of K fp16 (read as left operand of S k^ and S q^, and k by
// transposing reads as left operand of the state's sum) and the chunk's record (two buffers). The next
// chunk's rows travel in registers while this one's are used.
//
// Row i of tile b of the transposed state is channel 32 (b / 2) + 8 (i / 4) + 4 (b % 2) + i % 4, so
// that a lane's eight values of two tiles are eight channels in a row of k or q. LDS holds a row's
// even and odd groups of four channels apart (two halves of 8-byte pieces, kHalf bytes from each
// other, read by one instruction), and piece c of token t lies at c ^ swizzle(t): any 16 lanes that
// LDS serves in one cycle (16 tokens of one piece; 4 tokens x 4 pieces of a transposing read; the
// pieces of a row as they are written) then differ in all banks.
template <int K>
__device__ __forceinline__ int swizzle(int t) {
  return K == 128 ? (t & 3) << 2 | ((t >> 2) & 3) : (t & 2) << 1 | ((t >> 2) & 3);
}

// The blocks of a lower triangular matrix as operands: row block, and pair of contraction blocks.
constexpr int kLowerRow[6] = {0, 1, 2, 3, 2, 3}, kLowerCol[6] = {0, 0, 0, 0, 1, 1};

// Packed sequences that are put in order at most. Every workgroup ranks them all, so the cost grows
// with the square of their number, and the gain is that of one long sequence left to run alone: 32
// heads, lengths skewed, in order and as they lie, 24 of 1300 tokens in the mean 546 and 564 us, 48 of
// 700 536 and 580 us, 64 of 500 531 and 548 us, 96 of 350 592 us both, 256 of 128 918 and 716 us; all of
// 32 tokens, 64 115 and 100 us, 1024 7.8 and 1.4 ms.
constexpr int kOrdered = 64;

// LOCAL: the first walk over segments: no outputs; columns V .. V + K - 1 are the identity's.
template <typename Act, int K, int W, int NC, bool LOCAL>
__global__ __launch_bounds__(64 * W, W == 4 && !LOCAL ? 1 : 2) void walk_kernel(DeltaArgs a) {
  constexpr int P = kPieces<Act>;
  constexpr int NB = K / 16, KB = K / 32;
  constexpr int kRow = K, kHalf = 16 * kRow;     // bytes of half a row, of one half of 16 rows
  constexpr int kMat = 8 * kHalf;                // of one piece (of an fp16 pair) of k or q of a chunk
  constexpr int kLoads = kRecordLds / 1024;
  constexpr int kThreadsW = 64 * W;
  constexpr int kBufs = P == 1 && (W == 8 || K == 64) ? 2 : 1;  // of k and q
  constexpr int kUnits = kQ * K / 8 / kThreadsW;     // 16-byte pieces of k (and q) a thread brings
  static_assert(kRecordLds % 1024 == 0, "whole wave loads");
  __shared__ __align__(16) char ks[kBufs][P * kMat];
  __shared__ __align__(16) char qs[kBufs][P * kMat];
  __shared__ __align__(16) char rs2[2][kRecordLds];
  __shared__ __align__(16) char vs[W][kQ * 16 * NC * sizeof(Act)];

  // The value heads of a key head, and the column groups of each, go to one XCD: k and q come to its
  // L2 once.
  const int xcd = blockIdx.x & 7;
  int slot = blockIdx.x >> 3;
  const int group = slot % a.col_groups;
  slot /= a.col_groups;
  const int vh = slot % a.ratio;
  slot /= a.ratio;
  const int seg = a.seg_chunks ? slot % a.segs : 0;
  if (a.seg_chunks) slot /= a.segs;
  const int64_t nk = int64_t(slot) * 8 + xcd;
  if (nk >= int64_t(a.sequences) * a.hk) return;
  int n = static_cast<int>(nk / a.hk);
  if (a.starts && a.sequences > 1 && a.sequences <= kOrdered) {
    // Packed sequences start in the order of their lengths, the longest first, so that no long one
    // is left to run alone at the end. The n-th longest is found here: each of the first threads
    // compares a sequence with all others.
    static_assert(kOrdered <= kThreadsW, "a thread a sequence");
    int* const lens = reinterpret_cast<int*>(rs2[0]);
    int* const found = lens + kOrdered;
    const int j = threadIdx.x;
    if (j < a.sequences) lens[j] = a.block_starts[j + 1] - a.block_starts[j];
    __syncthreads();
    if (j < a.sequences) {
      int before = 0;
      for (int o = 0; o < a.sequences; ++o) before += lens[o] > lens[j] || (lens[o] == lens[j] && o < j);
      if (before == n) *found = j;
    }
    __syncthreads();
    n = __builtin_amdgcn_readfirstlane(*found);
    __syncthreads();  // read before the records take the place
  }
  const int tid = threadIdx.x, lane = tid & 63, g = lane >> 4, i = lane & 15;
  const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int hk = static_cast<int>(nk % a.hk), h = hk * a.ratio + vh;
  const int col0 = (group * W + w) * 16 * NC;
  const int columns = LOCAL ? a.value_dim + K : a.value_dim;
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
  int64_t seg_row = 0;  // of this sequence's first segment: no two sequences share a row
  bool last = true;
  if (a.seg_chunks) {
    seg_row = row0 / a.seg_chunks + n;
    const int64_t before = int64_t(seg) * a.seg_chunks;
    if (seg > 0 && before >= chunks) return;
    last = before + a.seg_chunks >= chunks;
    if (LOCAL && last) return;
    begin += before * kQ, len -= before * kQ, row0 += before, chunks -= before;
    if (!last) chunks = a.seg_chunks, len = int64_t(a.seg_chunks) * kQ;
  }
  bool cut = false;
  if constexpr (LOCAL) {
    // Lane l: chunk l from the segment's end; the decays of it and of those behind it.
    const int64_t c = chunks - 1 - lane;
    float sum = 0.0f;
    if (c >= 0)
      sum = *reinterpret_cast<const float*>(a.records + ((row0 + c) * a.hv + h) * int64_t(kRecordBytes) + kRowsAt +
                                            (kRows * kQ + 1) * 4);
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const float o = __shfl_up(sum, d, 64);
      if (lane >= d) sum += o;
    }
    const uint64_t small = __ballot(c >= 0 && sum < -160.0f);
    cut = small != 0;
    if (group == 0 && tid == 0) a.seg_flag[(seg_row + seg) * a.hv + h] = !cut;
    if (cut) {
      if (group * W * 16 * NC >= a.value_dim) return;
      const int64_t skip = chunks - 1 - __builtin_ctzll(small);
      begin += skip * kQ, len -= skip * kQ, row0 += skip, chunks -= skip;
    }
  }

  // The state in units of its columns: S / unit.
  f4 S[NC][NB];
  float unit[NC], inverse[NC];
  // Element (z, b, r) is row 32 (b / 2) + 8 g + 4 (b % 2) + r of column col0 + 16 z + i.
  // Element (z, b, r) of the lane in a state, and the size of a state.
  const uint32_t state_lane = i * K + 8 * g;
  const int64_t state_head = (int64_t(h) * a.value_dim + col0) * K;
  const int64_t state_size = int64_t(a.hv) * a.value_dim * K;
  const float* from = nullptr;
  if (!LOCAL && a.seg_chunks) {
    from = a.seg_s + (seg_row + seg) * state_size;
  } else if (!LOCAL && a.state_in) {
    const int64_t slot_in = a.in_slots ? a.in_slots[n] : n;
    if (slot_in >= 0 && slot_in < a.in_count) from = a.state_in + slot_in * state_size;
  }
#pragma unroll
  for (int z = 0; z < NC; ++z) {
    unit[z] = inverse[z] = 1.0f;
    const int one = col0 + 16 * z + i - a.value_dim;  // LOCAL: the identity's row
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      S[z][b] = f4{0.0f, 0.0f, 0.0f, 0.0f};
      if (from && col0 + 16 * z < a.value_dim)
        S[z][b] = *reinterpret_cast<const f4*>(from + state_head + state_lane + 16 * z * K + 32 * (b >> 1) +
                                               4 * (b & 1));
      if (LOCAL) {
#pragma unroll
        for (int r = 0; r < 4; ++r)
          if (!cut && 32 * (b >> 1) + 8 * g + 4 * (b & 1) + r == one) S[z][b][r] = 1.0f;
      }
    }
  }

  constexpr uint32_t es = sizeof(Act);
  // This thread brings pieces tid, tid + 64 W, ... of the chunk's rows (K / 8 pieces a row).
  Eight<Act> pk[kUnits], pq[kUnits];
  float2 sh[kUnits];
  float end = 0.0f, end_next = 0.0f;
  // The record goes to LDS without passing through registers, 1 KiB a wave and instruction.
  // (Where the pieces are no multiple of the waves, the last one is brought more than once.)
  auto load_record = [&](int64_t c, int buf) {
    const char* rec = a.records + ((row0 + c) * a.hv + h) * int64_t(kRecordBytes);
    end_next = *reinterpret_cast<const float*>(rec + kRowsAt + kRows * kQ * 4);
#pragma unroll
    for (int u0 = 0; u0 < kLoads; u0 += W) {
      const int u = min(u0 + w, kLoads - 1);
      load_to_lds(rec + u * 1024, lane * 16, &rs2[buf][u * 1024]);
    }
  };
  // Rows behind the sequence lie outside the resource's range and read as zeros.
  auto load = [&](int64_t c) {
    const int64_t first = begin + c * kQ;
    const int count = len - c * kQ < kQ ? static_cast<int>(len - c * kQ) : kQ;
    const uint32_t koff = static_cast<uint32_t>(a.k_stride) * es, qoff = static_cast<uint32_t>(a.q_stride) * es;
    const rsrc_t kr = make_rsrc_bounded(
        const_cast<Act*>(static_cast<const Act*>(a.k) + first * a.k_stride + int64_t(hk) * K),
        (count - 1) * koff + K * es);
    const rsrc_t qr = make_rsrc_bounded(
        const_cast<Act*>(static_cast<const Act*>(a.q) + first * a.q_stride + int64_t(hk) * K),
        (count - 1) * qoff + K * es);
    const char* rec = a.records + ((row0 + c) * a.hv + h) * int64_t(kRecordBytes);
#pragma unroll
    for (int u = 0; u < kUnits; ++u) {
      const int at = tid + u * kThreadsW, t = at / (K / 8), piece = at % (K / 8);
      const uint32_t ko = fresh(t * koff + piece * 8 * es), qo = fresh(t * qoff + piece * 8 * es);
      sh[u] = *reinterpret_cast<const float2*>(rec + kRowsAt + kRowKQ * kQ * 4 + t * 8);
      pk[u].load(kr, ko);
      if (!LOCAL) pq[u].load(qr, qo);
    }
  };
  auto store = [&](int buf) {
#pragma unroll
    for (int u = 0; u < kUnits; ++u) {
      const int at = tid + u * kThreadsW, t = at / (K / 8), piece = at % (K / 8);
      const int to = (t >> 4) * 2 * kHalf + (t & 15) * kRow + (piece ^ swizzle<K>(t)) * 8;
      w4 out[P];
      pk[u].pieces(sh[u].x, out);
#pragma unroll
      for (int p = 0; p < P; ++p) {
        *reinterpret_cast<w2*>(&ks[buf][p * kMat + to]) = w2{out[p][0], out[p][1]};
        *reinterpret_cast<w2*>(&ks[buf][p * kMat + kHalf + to]) = w2{out[p][2], out[p][3]};
      }
      if (LOCAL) continue;
      pq[u].pieces(sh[u].y, out);
#pragma unroll
      for (int p = 0; p < P; ++p) {
        *reinterpret_cast<w2*>(&qs[buf][p * kMat + to]) = w2{out[p][0], out[p][1]};
        *reinterpret_cast<w2*>(&qs[buf][p * kMat + kHalf + to]) = w2{out[p][2], out[p][3]};
      }
    }
  };
  // This wave's columns of a chunk's v go to LDS as rows of 16 NC values (only this wave reads them):
  // 16-byte pieces, those of rows behind the sequence from its last row (their factors are zeros).
  // fp32 rows lie in the order that puts rows 4 g + r of one r in different banks.
  char* const vw = vs[w];
  auto load_v = [&](int64_t c) {
    const int64_t first = begin + c * kQ;
    const int count = len - c * kQ < kQ ? static_cast<int>(len - c * kQ) : kQ;
    const char* from = static_cast<const char*>(a.v) +
                       (first * a.v_stride + int64_t(h) * a.value_dim) * int64_t(es);
    constexpr int kPieces16 = NC * static_cast<int>(sizeof(Act));  // 16-byte pieces of a row
    constexpr int kRowsPer = 64 / kPieces16;
#pragma unroll
    for (int j = 0; j < kQ / kRowsPer; ++j) {
      const int at = lane / kPieces16;
      const int t = es == 2 ? j * kRowsPer + at : j * kRowsPer + 4 * (at & 3) + (at >> 2);
      const int colb = min((col0 * static_cast<int>(es)) + (lane % kPieces16) * 16, a.value_dim * static_cast<int>(es) - 16);
      load_to_lds(from, fresh(min(t, count - 1) * static_cast<uint32_t>(a.v_stride) * es + colb),
                  vw + j * 1024);
    }
  };
  // Rows 16 tt + 4 g .. + 3 of column 16 z + i.
  auto load4 = [&](Column<Act>& v, int z, int tt) {
    if constexpr (P == 1) {
      const w2 x = __builtin_bit_cast(
          w2, read_transposed(vw + (16 * tt + 4 * g + (i >> 2)) * 32 * NC + 32 * z + (i & 3) * 8));
      v.raw[2 * tt] = x[0], v.raw[2 * tt + 1] = x[1];
    } else {
#pragma unroll
      for (int r = 0; r < 4; ++r)
        v.raw[4 * tt + r] = *reinterpret_cast<const float*>(vw + (16 * tt + 4 * r + g) * 64 * NC + 64 * z + 4 * i);
    }
  };
  // y is computed transposed (rows: 4 columns 4 g + r, column: token i), so that a lane stores four
  // values in a row. Rows behind the sequence and columns behind V lie outside the range.
  const int64_t y_stride = int64_t(a.hv) * a.value_dim;
  uint32_t yoff = 0;  // computed where it is used
  auto store_y = [&](int64_t c, int z, int tt, f4 o) {
    const uint32_t off = col0 + 16 * z < a.value_dim ? yoff + 16 * z * es : kNoStore;
    const int64_t first = begin + c * kQ;
    const int left = (len - c * kQ < kQ ? static_cast<int>(len - c * kQ) : kQ) - 16 * tt;
    const rsrc_t yr = make_rsrc_bounded(
        static_cast<char*>(a.y) + ((first + 16 * tt) * y_stride + int64_t(h) * a.value_dim) * int64_t(es),
        left > 0 ? ((left - 1) * static_cast<uint32_t>(y_stride) + a.value_dim) * es : 0);
    if constexpr (P == 1) {
      typedef __bf16 b4 __attribute__((ext_vector_type(4)));
      __builtin_amdgcn_raw_buffer_store_b64(__builtin_bit_cast(w2, __builtin_convertvector(o, b4)), yr,
                                            off, 0, 0);
    } else {
      __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(w4, o), yr, off, 0, 0);
    }
  };
  // Left operand: rows 16 tt + i, channels 32 kb + 8 g .. + 7.
  const uint32_t rowop = i * kRow + (g ^ swizzle<K>(i)) * 8;
  uint32_t rowop_c = rowop, colop_c;  // of this chunk: the sums with them are not kept across chunks
  auto operand = [&](const char* m, int p, int tt, int kb) {
    const char* at = m + p * kMat + tt * 2 * kHalf + (rowop_c ^ (kb * 32));
    return __builtin_shufflevector(*reinterpret_cast<const h4*>(at),
                                   *reinterpret_cast<const h4*>(at + kHalf), 0, 1, 2, 3, 4, 5, 6, 7);
  };
  // Left operand: rows of state tile b, tokens 32 s + 4 g + e and 32 s + 16 + 4 g + e. The 16 lanes
  // of group g read 4 tokens x 16 channels, and each gets its own channel's 4 tokens.
  const uint32_t colop = (4 * g + (i >> 2)) * kRow + ((i & 3) ^ swizzle<K>(4 * g + (i >> 2))) * 8;
  auto transposed = [&](const char* m, int p, int b, int s) {
    const char* at = m + p * kMat + s * 4 * kHalf + (colop_c ^ ((b >> 1) * 32)) + (b & 1) * kHalf;
    const h4 x = read_transposed(at), y = read_transposed(at + 2 * kHalf);
    return __builtin_shufflevector(x, y, 0, 1, 2, 3, 4, 5, 6, 7);
  };
  const char* rs = rs2[0];
  // Row block tt, contraction blocks 2 ss and 2 ss + 1 of a lower triangular matrix.
  auto lower = [&](int mat, int tt, int ss) {
    const char* p = rs + (mat * kBlocks + block_at(tt, 2 * ss)) * kBlockBytes + lane * 8;
    const h4 x = *reinterpret_cast<const h4*>(p);
    h4 y = {};
    if (2 * ss + 1 <= tt) y = *reinterpret_cast<const h4*>(p + kBlockBytes);
    return __builtin_shufflevector(x, y, 0, 1, 2, 3, 4, 5, 6, 7);
  };
  auto row4 = [&](int row, int tt) {
    return *reinterpret_cast<const f4*>(rs + kRowsAt + (row * kQ + 16 * tt + 4 * g) * 4);
  };

  // No branch inside the loop but the loop itself, so that the waits for loads count exactly and
  // the next chunk's stay in flight: behind the last chunk it is loaded once more (and not used),
  // and waves without columns run on zeros.
  if (chunks > 0) {
    load_v(0);
    load_record(0, 0);
    load(0);
  }
  for (int64_t c = 0; c < chunks; ++c) {
    const int kb2 = kBufs == 2 ? c & 1 : 0;
    store(kb2);
    const char *kc = ks[kb2], *qc = qs[kb2];
    rs = rs2[c & 1];
    end = end_next;
    // This wave's parts of the record and v are in LDS: vector memory operations of a wave complete
    // in the order of their issue, and behind them and k and q only y's 4 stores were issued.
    static_assert(LOCAL || NC == 1, "stores counted");
    if (LOCAL)
      asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    else
      asm volatile("s_waitcnt vmcnt(4)" ::: "memory");
    // Behind this barrier chunk c is complete in LDS and every wave is done with chunk c - 1, whose
    // record buffer the next chunk takes.
    __syncthreads();
    const int64_t next = c + 1 < chunks ? c + 1 : c;
    rowop_c = fresh(rowop);
    colop_c = fresh(colop);
    load_record(next, (c + 1) & 1);
    // k and q have the whole chunk's time to arrive, where their registers fit.
    if (NC == 1 && P == 1) load(next);
    // A SIMD's waves serve a chunk together; the one that is behind goes first (its priority falls
    // from phase to phase), so that they reach the barrier together: 32768 packed tokens 535 -> 529 us,
    // 16384 of one sequence 455 -> 439 us.
    __builtin_amdgcn_s_setprio(3);
    f4 X[NC][4], O[NC][4];
#pragma unroll
    for (int z = 0; z < NC; ++z) {
      Column<Act> v;
#pragma unroll
      for (int tt = 0; tt < 4; ++tt) load4(v, z, tt);
      float m = 0.0f;
#pragma unroll
      for (int b = 0; b < NB; ++b) m = max4(m, S[z][b]);
      m = column_max(fmaxf(col0 + 16 * z < a.value_dim ? v.largest() : 0.0f, m * unit[z]));
      // The unit stays while the column's largest is between 2^2 and 2^8 of it.
      const float at = m * inverse[z];
      if (__any(m > 0.0f && !(at >= 0x1p2f && at <= 0x1p8f))) {
        // Columns of zeros keep theirs: from a large unit to the smallest the factor is infinite. Where
        // little is left of a state in a large unit it is as well, hence two steps.
        const Scale to = scale_of(m);
        const float up = m > 0.0f ? to.up * 0x1p5f : inverse[z], from = unit[z];
        inverse[z] = up;
        unit[z] = m > 0.0f ? to.down * 0x1p-5f : from;
#pragma unroll
        for (int b = 0; b < NB; ++b) S[z][b] = S[z][b] * from * up;
      }
    }
    // X and the state's part of y. Left operands are read ahead of their products (a read from LDS
    // takes as long as eight products); fences keep the compiler from moving the reads back, or all
    // of them ahead, which would not fit the registers.
    constexpr int kSets = P == 1 && NC == 1 ? 2 : 1;
    h8 kf[kSets][4][P], qf[kSets][4][P];
    auto fetch = [&](int kb) {
#pragma unroll
      for (int tt = 0; tt < 4; ++tt)
#pragma unroll
        for (int p = 0; p < P; ++p) {
          kf[kb % kSets][tt][p] = operand(kc, p, tt, kb);
          if (!LOCAL) qf[kb % kSets][tt][p] = operand(qc, p, tt, kb);
        }
    };
    if (kSets == 2) fetch(0);
#pragma unroll
    for (int kb = 0; kb < KB; ++kb) {
      if (kSets == 1) fetch(kb);
      if (kSets == 2 && kb + 1 < KB) fetch(kb + 1);
      h8 hi[NC], lo[NC];
#pragma unroll
      for (int z = 0; z < NC; ++z) split8(S[z][2 * kb], S[z][2 * kb + 1], &hi[z], &lo[z]);
      if (kSets == 2) __builtin_amdgcn_sched_barrier(0);
      const f4 zero = {0.0f, 0.0f, 0.0f, 0.0f};
      const auto& k = kf[kb % kSets];
      const auto& q = qf[kb % kSets];
#pragma unroll
      for (int tt = 0; tt < 4; ++tt)
#pragma unroll
        for (int z = 0; z < NC; ++z) X[z][tt] = mfma_h(k[tt][0], hi[z], kb ? X[z][tt] : zero);
#pragma unroll
      for (int tt = 0; tt < 4; ++tt)
#pragma unroll
        for (int z = 0; z < NC; ++z) X[z][tt] = mfma_h(k[tt][0], lo[z], X[z][tt]);
      if constexpr (!LOCAL) {
#pragma unroll
        for (int tt = 0; tt < 4; ++tt)
#pragma unroll
          for (int z = 0; z < NC; ++z) O[z][tt] = mfma_h(hi[z], q[tt][0], kb ? O[z][tt] : zero);
#pragma unroll
        for (int tt = 0; tt < 4; ++tt)
#pragma unroll
          for (int z = 0; z < NC; ++z) O[z][tt] = mfma_h(lo[z], q[tt][0], O[z][tt]);
      }
      if constexpr (P == 2) {
#pragma unroll
        for (int tt = 0; tt < 4; ++tt)
#pragma unroll
          for (int z = 0; z < NC; ++z) {
            X[z][tt] = mfma_h(k[tt][1], hi[z], X[z][tt]);
            if constexpr (!LOCAL) O[z][tt] = mfma_h(hi[z], q[tt][1], O[z][tt]);
          }
      }
      __builtin_amdgcn_sched_barrier(0);
    }
    __builtin_amdgcn_s_setprio(2);
    h8 xh[NC][2], xl[NC][2];
#pragma unroll
    for (int z = 0; z < NC; ++z) {
      Column<Act> v;  // read again: it would not fit the registers during the products
#pragma unroll
      for (int tt = 0; tt < 4; ++tt) load4(v, z, tt);
      const float up = !LOCAL || col0 + 16 * z < a.value_dim ? inverse[z] : 0.0f;
#pragma unroll
      for (int tt = 0; tt < 4; ++tt) {
        const f4 f = row4(kRowX, tt);
#pragma unroll
        for (int r = 0; r < 4; ++r)
          X[z][tt][r] = fmaf(-f[r], X[z][tt][r], v.value(tt, r) * up);
      }
#pragma unroll
      for (int s = 0; s < 2; ++s) split8(X[z][2 * s], X[z][2 * s + 1], &xh[z][s], &xl[z][s]);
    }
    // This wave has read its columns of v: the next chunk's may take their place.
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    load_v(next);
    __builtin_amdgcn_sched_barrier(0);
    __builtin_amdgcn_s_setprio(1);
    // E = T X.
    f4 E[NC][4];
#pragma unroll
    for (int e = 0; e < 6; ++e) {
      const int tt = kLowerRow[e], s = kLowerCol[e];
      const h8 t0 = lower(0, tt, s), t1 = lower(1, tt, s);
      const f4 zero = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int z = 0; z < NC; ++z) {
        E[z][tt] = mfma_h(t0, xh[z][s], s ? E[z][tt] : zero);
        E[z][tt] = mfma_h(t0, xl[z][s], E[z][tt]);
        E[z][tt] = mfma_h(t1, xh[z][s], E[z][tt]);
      }
    }
    if (NC > 1 || P > 1) load(next);
    __builtin_amdgcn_sched_barrier(0);
    // y, and the writes U.
    h8 uh[NC][2], ul[NC][2];
    {
      h8 eh[NC][2], el[NC][2];
#pragma unroll
      for (int z = 0; z < NC; ++z)
#pragma unroll
        for (int s = 0; s < 2; ++s) {
          if constexpr (!LOCAL)
            split8(E[z][2 * s], E[z][2 * s + 1], &eh[z][s], &el[z][s]);
          split8(E[z][2 * s] * row4(kRowS, 2 * s), E[z][2 * s + 1] * row4(kRowS, 2 * s + 1), &uh[z][s],
                 &ul[z][s]);
        }
      if constexpr (!LOCAL) {
#pragma unroll
        for (int tt = 0; tt < 4; ++tt) {
          const float f = *reinterpret_cast<const float*>(rs + kRowsAt + (kRowY * kQ + 16 * tt + i) * 4);
#pragma unroll
          for (int z = 0; z < NC; ++z) O[z][tt] *= f;
        }
#pragma unroll
        for (int e = 0; e < 6; ++e) {
          const int tt = kLowerRow[e], s = kLowerCol[e];
          const h8 a0 = lower(2, tt, s), a1 = lower(3, tt, s);
#pragma unroll
          for (int z = 0; z < NC; ++z) {
            O[z][tt] = mfma_h(eh[z][s], a0, O[z][tt]);
            O[z][tt] = mfma_h(el[z][s], a0, O[z][tt]);
            O[z][tt] = mfma_h(eh[z][s], a1, O[z][tt]);
          }
        }
      }
    }
    __builtin_amdgcn_sched_barrier(0);
    if constexpr (!LOCAL) {
      const uint32_t l = fresh(lane);
      yoff = ((l & 15) * static_cast<uint32_t>(y_stride) + col0 + 4 * (l >> 4)) * es;
#pragma unroll
      for (int z = 0; z < NC; ++z) {
        f4 out;  // of the columns 4 g + r
#pragma unroll
        for (int r = 0; r < 4; ++r) out[r] = a.scale * __shfl(unit[z], 4 * g + r, 16);
#pragma unroll
        for (int tt = 0; tt < 4; ++tt) store_y(c, z, tt, O[z][tt] * out);
      }
    }
    __builtin_amdgcn_s_setprio(0);
    // The state.
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      h8 k[2][P];
#pragma unroll
      for (int s = 0; s < 2; ++s)
#pragma unroll
        for (int p = 0; p < P; ++p) k[s][p] = transposed(kc, p, b, s);
#pragma unroll
      for (int z = 0; z < NC; ++z) S[z][b] *= end;
#pragma unroll
      for (int s = 0; s < 2; ++s)
#pragma unroll
        for (int z = 0; z < NC; ++z) {
          S[z][b] = mfma_h(k[s][0], uh[z][s], S[z][b]);
          S[z][b] = mfma_h(k[s][0], ul[z][s], S[z][b]);
          if constexpr (P == 2) S[z][b] = mfma_h(k[s][1], uh[z][s], S[z][b]);
        }
    }
    __builtin_amdgcn_sched_barrier(0);
    if (kBufs == 1) __syncthreads();  // every wave is done with k and q
  }
  if constexpr (LOCAL) {
    float* const to = a.seg_s + (seg_row + seg) * state_size + state_head + fresh(lane & 15) * K + 8 * g;
    char* const carry = a.seg_m + ((seg_row + seg) * a.hv + h) * int64_t(carry_bytes(K));
    _Float16* const mt = reinterpret_cast<_Float16*>(carry);
#pragma unroll
    for (int z = 0; z < NC; ++z) {
      if (col0 + 16 * z < a.value_dim) {
#pragma unroll
        for (int b = 0; b < NB; ++b)
          *reinterpret_cast<f4*>(to + 16 * z * K + 32 * (b >> 1) + 4 * (b & 1)) = S[z][b] * unit[z];
      } else if (!cut && col0 + 16 * z < columns) {
        const int row = col0 + 16 * z + i - a.value_dim;
        float m = 0.0f;
#pragma unroll
        for (int b = 0; b < NB; ++b) m = max4(m, S[z][b]);
        const Scale of_row = scale_of(column_max(m) * unit[z]);
        if (g == 0) reinterpret_cast<float*>(carry + 4 * K * K)[row] = of_row.down;
#pragma unroll
        for (int b = 0; b < NB; ++b) {
          const f4 x = S[z][b] * (unit[z] * of_row.up);
          const h4 hi = __builtin_convertvector(x, h4);
          const h4 lo = __builtin_convertvector(x - __builtin_convertvector(hi, f4), h4);
          // Operand (b, row / 32) of M^T: lane (row / 8 % 4, this row of the tile), entry row % 8.
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const int at = ((b * KB + (row >> 5)) * 64 + ((row >> 3) & 3) * 16 + 4 * g + r) * 8 + (row & 7);
            mt[at] = hi[r];
            mt[K * K + at] = lo[r];
          }
        }
      }
    }
    return;
  }
  const int64_t slot_out = a.out_slots ? a.out_slots[n] : n;
  if (a.state_out && last && slot_out >= 0 && slot_out < a.out_count) {
    const uint32_t l = fresh(lane);  // not kept through the loop
    float* const to = a.state_out + slot_out * state_size + state_head + (l & 15) * K + 8 * (l >> 4);
#pragma unroll
    for (int z = 0; z < NC; ++z)
#pragma unroll
      for (int b = 0; b < NB; ++b)
        if (col0 + 16 * z < a.value_dim)
          *reinterpret_cast<f4*>(to + 16 * z * K + 32 * (b >> 1) + 4 * (b & 1)) = S[z][b] * unit[z];
  }
}

// ---- the states before the segments -------------------------------------------------------------
// Grid (sequence and value head, groups of 128 columns of V), 4 waves of two column tiles: segment
// after segment S <- S M + N, transposed as in the walk, with M^T in LDS in operand order (the next
// segment's on its way meanwhile). N's place takes the state before the segment: the second walk
// reads no other, so that the last segment may write the state in place. Bound by the latency of a
// step (about 7 us: M and N arrive, 192 products a wave and its LDS reads); 48 us for 8 segments.
template <int K>
__global__ __launch_bounds__(kThreads) void join_kernel(DeltaArgs a) {
  constexpr int NB = K / 16, KB = K / 32, NC = 2;
  constexpr int kBytes = 4 * K * K, kLoads = kBytes / 1024;  // of M^T: two pieces
  __shared__ __align__(16) char ms[2][kBytes];
  const int lane = threadIdx.x & 63, g = lane >> 4, i = lane & 15;
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int n = blockIdx.x / a.hv, h = blockIdx.x - n * a.hv;
  const int col0 = (blockIdx.y * 4 + w) * 16 * NC;
  int64_t len, row0;
  if (a.starts) {
    const int64_t begin = a.starts[n];
    len = a.starts[n + 1] - begin;
    row0 = a.block_starts[n];
    if (begin < 0 || begin > a.tokens || row0 < 0 || row0 > a.rows) len = row0 = 0;
    if (len > a.tokens - begin) len = a.tokens - begin;
  } else {
    len = a.seqlen, row0 = int64_t(n) * a.chunks_per_seq;
  }
  int64_t chunks = len > 0 ? (len + kQ - 1) / kQ : 0;
  if (chunks > a.rows - row0) chunks = a.rows - row0;
  const int64_t seg_row = row0 / a.seg_chunks + n;
  const int64_t final = chunks > 0 ? (chunks - 1) / a.seg_chunks : 0;
  const int64_t state_size = int64_t(a.hv) * a.value_dim * K;
  // Tiles behind the columns work on the last one's and store nothing.
  // (State sizes are below 2^31 bytes here: a split scan has at most kSegmentUnits heads.)
  uint32_t state_at[NC], store_at[NC];
#pragma unroll
  for (int z = 0; z < NC; ++z) {
    const bool in = col0 + 16 * z < a.value_dim;
    const int col = in ? col0 + 16 * z + i : a.value_dim - 16 + i;
    state_at[z] = (static_cast<uint32_t>(h) * a.value_dim + col) * K + 8 * g;
    store_at[z] = in ? state_at[z] * 4 : kNoStore;
  }
  auto store = [&](rsrc_t to, int z, int b, f4 x) {
    __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(w4, x), to,
                                           store_at[z] + 128 * (b >> 1) + 16 * (b & 1), 0, 0);
  };
  auto nonzero = [&](int64_t seg) {
    return __builtin_amdgcn_readfirstlane(a.seg_flag[(seg_row + seg) * a.hv + h]) != 0;
  };
  f4 S[NC][NB], N[2][NC][NB], F[2][NB];  // F: M's row factors
  auto load = [&](int64_t seg, int buf) {
    const char* from = a.seg_m + ((seg_row + seg) * a.hv + h) * int64_t(carry_bytes(K));
#pragma unroll
    for (int u = 0; u < kLoads; u += 4)
      load_to_lds(from + (u + w) * 1024, lane * 16, &ms[buf][(u + w) * 1024]);
#pragma unroll
    for (int b = 0; b < NB; ++b)
      F[buf][b] = *reinterpret_cast<const f4*>(from + kBytes + (32 * (b >> 1) + 8 * g + 4 * (b & 1)) * 4);
  };
  auto load_n = [&](int64_t seg, int buf) {
    const float* from = a.seg_s + (seg_row + seg) * state_size;
#pragma unroll
    for (int z = 0; z < NC; ++z)
#pragma unroll
      for (int b = 0; b < NB; ++b)
        N[buf][z][b] = *reinterpret_cast<const f4*>(from + state_at[z] + 32 * (b >> 1) + 4 * (b & 1));
  };
  const int64_t slot_in = a.in_slots ? a.in_slots[n] : n;
  const bool have = a.state_in && slot_in >= 0 && slot_in < a.in_count;
#pragma unroll
  for (int z = 0; z < NC; ++z)
#pragma unroll
    for (int b = 0; b < NB; ++b)
      S[z][b] = have ? *reinterpret_cast<const f4*>(a.state_in + slot_in * state_size + state_at[z] +
                                                    32 * (b >> 1) + 4 * (b & 1))
                     : f4{0.0f, 0.0f, 0.0f, 0.0f};
  // One segment; m1: whether its M is not zero, m2: whether the next one's is.
  auto step = [&](int64_t seg, int buf, bool m1, bool m2) {
    const rsrc_t to = make_rsrc_bounded(a.seg_s + (seg_row + seg) * state_size,
                                        static_cast<uint32_t>(state_size * 4));
    // This wave's copies have arrived (behind them only the NC NB stores of the step before were
    // issued); behind the barrier all waves' have, and the other buffer is free.
    asm volatile("s_waitcnt vmcnt(%0)" ::"n"(NC * NB) : "memory");
    __syncthreads();
    const int64_t next = seg + 1 < final ? seg + 1 : seg;
    load_n(next, buf ^ 1);
    if (m2) load(next, buf ^ 1);
    if (!m1) {
#pragma unroll
      for (int z = 0; z < NC; ++z)
#pragma unroll
        for (int b = 0; b < NB; ++b) {
          store(to, z, b, S[z][b]);
          S[z][b] = N[buf][z][b];
        }
      return;
    }
    const char* m = ms[buf] + lane * 16;
    Scale unit[NC];
    h8 hi[NC][KB], lo[NC][KB];
#pragma unroll
    for (int z = 0; z < NC; ++z) {
      float big = 0.0f;
#pragma unroll
      for (int b = 0; b < NB; ++b) big = max4(big, S[z][b] * F[buf][b]);
      unit[z] = scale_of(column_max(big));
      const float up = unit[z].up * 0x1p5f;
#pragma unroll
      for (int kb = 0; kb < KB; ++kb)
        split8(S[z][2 * kb] * F[buf][2 * kb] * up, S[z][2 * kb + 1] * F[buf][2 * kb + 1] * up, &hi[z][kb],
               &lo[z][kb]);
    }
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      f4 x[NC];
#pragma unroll
      for (int z = 0; z < NC; ++z) x[z] = f4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int kb = 0; kb < KB; ++kb) {
        const h8 mh = *reinterpret_cast<const h8*>(m + (b * KB + kb) * 1024);
        const h8 ml = *reinterpret_cast<const h8*>(m + 2 * K * K + (b * KB + kb) * 1024);
#pragma unroll
        for (int z = 0; z < NC; ++z) {
          x[z] = mfma_h(mh, hi[z][kb], x[z]);
          x[z] = mfma_h(mh, lo[z][kb], x[z]);
          x[z] = mfma_h(ml, hi[z][kb], x[z]);
        }
      }
#pragma unroll
      for (int z = 0; z < NC; ++z) {
        store(to, z, b, S[z][b]);
        S[z][b] = x[z] * (unit[z].down * 0x1p-5f) + N[buf][z][b];
      }
    }
  };
  bool m1 = false, m2 = false;
  if (final > 0) {
    m1 = nonzero(0);
    load_n(0, 0);
    if (m1) load(0, 0);
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
  }
  // Two segments a turn: the buffers' indexes are constants.
  for (int64_t seg = 0; seg < final; seg += 2) {
    m2 = seg + 1 < final && nonzero(seg + 1);
    step(seg, 0, m1, m2);
    if (seg + 1 >= final) break;
    m1 = seg + 2 < final && nonzero(seg + 2);
    step(seg + 1, 1, m2, m1);
  }
  const rsrc_t to = make_rsrc_bounded(a.seg_s + (seg_row + final) * state_size,
                                      static_cast<uint32_t>(state_size * 4));
#pragma unroll
  for (int z = 0; z < NC; ++z)
#pragma unroll
    for (int b = 0; b < NB; ++b) store(to, z, b, S[z][b]);
}

// ---- one token a row ----------------------------------------------------------------------------
// Bound by reading and writing the states. K / 16 lanes hold a row of the state (16 values each, as
// four float4 spaced so that a load's lanes read whole 64 or 128 byte pieces); a wave passes over R
// times its 64 / lanes rows, all loaded before the first is used. 56 rows x 32 heads x 128 x 128 (and 8
// idle ones, which read and write nothing): 43 us, 5.5 TB/s; 448 rows (and 64): 326 us, 5.8 TB/s. A
// scaling of 512 MB in place reaches 6.1 TB/s.
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

// STREAM: states pass by the caches (no call finds them there again).
template <typename Act, int K, int R, bool STREAM>
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
  f4 s[R][4];
#pragma unroll
  for (int p = 0; p < R; ++p)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int v = v0 + p * RW;
      const f4* at = reinterpret_cast<const f4*>(sp + int64_t(v) * K + 4 * LR * j);
      s[p][j] = v >= a.value_dim ? f4{} : STREAM ? __builtin_nontemporal_load(at) : *at;
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
      pk += s[p][j][0] * kv[j].x + s[p][j][1] * kv[j].y + s[p][j][2] * kv[j].z + s[p][j][3] * kv[j].w;
      pq += s[p][j][0] * qv[j].x + s[p][j][1] * qv[j].y + s[p][j][2] * qv[j].z + s[p][j][3] * qv[j].w;
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
        const f4 k4 = {kv[j].x, kv[j].y, kv[j].z, kv[j].w};
        f4 t = s[p][j];
#pragma unroll
        for (int e = 0; e < 4; ++e) t[e] = fmaf(dk, k4[e], decay * t[e]);
        f4* at = reinterpret_cast<f4*>(sp + int64_t(v) * K + 4 * LR * j);
        if (STREAM)
          __builtin_nontemporal_store(t, at);
        else
          *at = t;
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

constexpr int64_t kMaxRow = int64_t(1) << 22;  // elements between two rows
constexpr int64_t kSegmentUnits = 64, kSegmentMin = 8;

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
  // The kernels address a chunk's 64 rows with 32-bit byte offsets below 2^31.
  if (own[0] > kMaxRow || own[2] > kMaxRow) return AXON_ERR_UNSUPPORTED;
  for (int j = 0; j < 3; ++j) {
    if (strides[j] > kMaxRow) return AXON_ERR_UNSUPPORTED;
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

struct ScanPlan {
  int64_t seg_chunks = 0;  // chunks of a segment, 0: none
  size_t off_m = 0, off_s = 0, off_flag = 0, bytes = 0;
};

// Workspace and segments from the shape alone. Sequences are split where their heads leave most of
// the 256 CUs idle (a workgroup a head) and they are long enough for it to pay: at 32 heads 16384
// tokens take 0.44 ms in 8 segments and 1.10 ms in one. Only the mean length is known here, so that a
// long sequence packed with short ones may be walked whole.
ScanPlan plan_scan(const axon_gated_delta_shape* s) {
  ScanPlan p;
  if (!s->tokens) return p;
  const size_t rows = size_t(rows_of(s)), hv = size_t(s->value_heads);
  p.bytes = kRecordBytes * rows * hv;
  const int64_t units = s->sequences * s->value_heads, chunks = s->tokens / kQ / s->sequences;
  if (units > kSegmentUnits || chunks < kSegmentMin * 4) return p;
  const int64_t segs = std::min<int64_t>(256 / units, chunks / kSegmentMin);
  p.seg_chunks = (chunks + segs - 1) / segs;
  const size_t count = (rows / size_t(p.seg_chunks) + size_t(s->sequences)) * hv;
  p.off_m = (p.bytes + 255) / 256 * 256;
  p.off_s = p.off_m + count * size_t(carry_bytes(int(s->key_dim)));
  p.off_flag = p.off_s + count * 4 * size_t(s->value_dim * s->key_dim);
  p.bytes = p.off_flag + (count * 4 + 255) / 256 * 256;
  return p;
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
void launch_scan(DeltaArgs a, bool any, hipStream_t st) {
  if (any) {
    hipLaunchKernelGGL((prep_kernel<Act, K>), dim3(unsigned(a.rows), unsigned(a.hk)), dim3(kThreads),
                       0, st, a);
  }
  const bool split = any && a.segs > 1;
  if (!split) a.seg_chunks = 0;
  auto go = [&](auto kernel, int waves, int tiles, int columns) {
    DeltaArgs b = a;
    b.col_groups = (columns + 16 * waves * tiles - 1) / (16 * waves * tiles);
    const int64_t keys = (int64_t(a.sequences) * a.hk + 7) / 8 * 8;
    const int64_t wgs = keys * a.ratio * b.col_groups * (split ? a.segs : 1);
    hipLaunchKernelGGL(kernel, dim3(unsigned(wgs)), dim3(64 * waves), 0, st, b);
  };
  if (split) {
    // (bf16 with eight waves of one tile: the scan takes 470 us against 439 us at 32 heads and 16384
    // tokens.)
    if constexpr (kPieces<Act> == 1)
      go(walk_kernel<Act, K, 4, 2, true>, 4, 2, a.value_dim + K);
    else
      go(walk_kernel<Act, K, 8, 1, true>, 8, 1, a.value_dim + K);
    hipLaunchKernelGGL(join_kernel<K>, dim3(unsigned(a.sequences * a.hv), unsigned((a.value_dim + 127) / 128)),
                       dim3(kThreads), 0, st, a);
  }
  // Four waves hold up to 64 columns (K = 128, V = 64, 16 x 2048 tokens x 32 heads: 445 us; eight
  // waves, half of them idle, 548 us). Eight waves of one tile beat four of two, which fill a CU's LDS
  // alone (V = 128: 491 us against 570 us).
  if (a.value_dim <= 64)
    go(walk_kernel<Act, K, 4, 1, false>, 4, 1, a.value_dim);
  else
    go(walk_kernel<Act, K, 8, 1, false>, 8, 1, a.value_dim);
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
  // A layer's states stream where those of a model's layers together pass the 256 MB cache (448 rows
  // x 32 heads: 327 us against 355 us; 56 rows, states of three calls in turn: 45 us against 48 us,
  // of one call again and again 43 us against 38 us).
  const bool stream = heads * a.value_dim * K * 4 > (int64_t(16) << 20);
  if (!wide)
    hipLaunchKernelGGL((step_kernel<Act, K, 1, false>), dim3(wgs), dim3(kThreads), 0, st, a);
  else if (stream)
    hipLaunchKernelGGL((step_kernel<Act, K, 4, true>), dim3(wgs), dim3(kThreads), 0, st, a);
  else
    hipLaunchKernelGGL((step_kernel<Act, K, 4, false>), dim3(wgs), dim3(kThreads), 0, st, a);
}

}  // namespace
}  // namespace axon

extern "C" {

size_t axon_gated_delta_scan_workspace_bytes(const axon_gated_delta_shape* shape) {
  if (axon::check_shape(shape) != AXON_OK) return 0;
  return axon::plan_scan(shape).bytes;
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
  const ScanPlan plan = plan_scan(shape);
  const size_t need = plan.bytes;
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
  a.out_slots = out_slots, a.records = static_cast<char*>(workspace);
  const Strides st = strides_of(shape);
  a.tokens = s.tokens, a.q_stride = st.q, a.k_stride = st.k, a.v_stride = st.v;
  a.in_count = s.state_slots, a.out_count = s.out_slots;
  a.sequences = int(s.sequences), a.hk = int(s.key_heads), a.hv = int(s.value_heads);
  a.ratio = int(s.value_heads / s.key_heads), a.value_dim = int(s.value_dim);
  a.seqlen = s.tokens / s.sequences;
  a.chunks_per_seq = int((a.seqlen + kQ - 1) / kQ);
  a.rows = int(tables ? rows : s.sequences * a.chunks_per_seq);
  if (plan.seg_chunks) {
    // The most chunks one sequence can have: all tokens in it.
    const int64_t most = tables ? (s.tokens + kQ - 1) / kQ : a.chunks_per_seq;
    a.seg_chunks = int(plan.seg_chunks);
    a.segs = int((most + plan.seg_chunks - 1) / plan.seg_chunks);
    a.seg_m = a.records + plan.off_m;
    a.seg_s = reinterpret_cast<float*>(a.records + plan.off_s);
    a.seg_flag = reinterpret_cast<int32_t*>(a.records + plan.off_flag);
  }
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

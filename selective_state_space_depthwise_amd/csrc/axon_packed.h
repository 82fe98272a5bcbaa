// Blocks of 64 tokens of packed or uniform sequences, as the kernels of the linear recurrence and of
// the convolution look them up (gfx950).
#pragma once

#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstdint>

#include "axon_internal.h"

namespace axon {

constexpr int kBlock = 64;  // tokens of a block

// A buffer of `tokens` rows: packed sequences with the tables of axon_sequence_tables (block 64), or,
// where starts is null, a uniform batch of `seqlen` tokens each.
struct Packed {
  const int32_t *starts, *block_seq, *block_first;
  int sequences, tokens, rows;   // rows: of the block tables, or of the batch's blocks
  int seqlen, blocks_per_seq;    // of a uniform batch
};

inline int64_t packed_rows(int64_t sequences, int64_t tokens, bool tables) {
  if (tables) return tokens / kBlock + sequences;
  return sequences * ((tokens / sequences + kBlock - 1) / kBlock);
}

inline Packed make_packed(int64_t sequences, int64_t tokens, const int32_t* tables) {
  Packed p{};
  p.sequences = static_cast<int>(sequences);
  p.tokens = static_cast<int>(tokens);
  p.rows = static_cast<int>(packed_rows(sequences, tokens, tables != nullptr));
  p.seqlen = static_cast<int>(tokens / sequences);
  p.blocks_per_seq = (p.seqlen + kBlock - 1) / kBlock;
  if (tables) {
    p.starts = tables;
    p.block_seq = tables + 2 * (sequences + 1);
    p.block_first = p.block_seq + p.rows;
  }
  return p;
}

// A table's entry at a wave-uniform place: through the constant address space, so that it comes by a
// scalar load, which waits for no vector load (no kernel that reads tables writes them).
__device__ __forceinline__ int table_at(const int32_t* p, int64_t i) {
  return ((const __attribute__((address_space(4))) int32_t*)p)[i];
}

// Where sequence n begins (n = sequences: where the last one ends). Entries are cut to the buffer, so
// that no contents of the tables lead outside it.
__device__ __forceinline__ int packed_start(const Packed& p, int n) {
  return p.starts ? min(max(table_at(p.starts, n), 0), p.tokens) : n * p.seqlen;
}

struct BlockAt {
  int seq;      // its sequence, -1: no block
  int first;    // its first row of the buffer
  int count;    // its tokens, 1 .. 64
  bool begins;  // the sequence's first block
  bool ends;    // its last
};

__device__ __forceinline__ BlockAt block_at(const Packed& p, int row) {
  BlockAt b{-1, 0, 0, false, false};
  if (row >= p.rows) return b;
  int s0, s1;
  if (p.starts) {
    const int seq = table_at(p.block_seq, row);
    if (seq < 0 || seq >= p.sequences) return b;
    s0 = packed_start(p, seq), s1 = packed_start(p, seq + 1);
    b.first = table_at(p.block_first, row);
    if (b.first < s0 || b.first >= s1 || (b.first - s0) % kBlock) return b;
    b.seq = seq;
  } else {
    b.seq = row / p.blocks_per_seq;
    s0 = b.seq * p.seqlen, s1 = s0 + p.seqlen;
    b.first = s0 + (row - b.seq * p.blocks_per_seq) * kBlock;
  }
  b.count = min(kBlock, s1 - b.first);
  b.begins = b.first == s0;
  b.ends = b.first + b.count == s1;
  return b;
}

// Checks that the recurrence and the convolution share. The limits are those of the header.
constexpr int64_t kMaxRowElems = int64_t(1) << 22;
constexpr int64_t kMaxTotal = int64_t(1) << 40;

inline bool aligned_to(const void* p, size_t a) {
  return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0;
}

inline axon_status check_packed(int64_t sequences, int64_t tokens, int64_t channels,
                                const int64_t* strides, int count, int64_t state, int64_t in_slots,
                                int64_t out_slots, int32_t act_dtype) {
  if (sequences < 1 || tokens < 0 || channels < 1 || in_slots < 0 || out_slots < 0)
    return AXON_ERR_INVALID_ARGUMENT;
  for (int j = 0; j < count; ++j)
    if (strides[j] < 0) return AXON_ERR_INVALID_ARGUMENT;
  if (sequences > 65535 || channels > kMaxRowElems || tokens >= (int64_t(1) << 29) ||
      (act_dtype != AXON_F32 && act_dtype != AXON_BF16))
    return AXON_ERR_UNSUPPORTED;
  if ((tokens / kBlock + sequences) * channels >= (int64_t(1) << 37)) return AXON_ERR_UNSUPPORTED;
  int64_t t;
  for (int j = 0; j < count; ++j) {
    if (strides[j] > kMaxRowElems) return AXON_ERR_UNSUPPORTED;
    if (strides[j] && strides[j] < channels) return AXON_ERR_INVALID_ARGUMENT;
    if (tokens * (strides[j] ? strides[j] : channels) > kMaxTotal) return AXON_ERR_UNSUPPORTED;
  }
  if (tokens * channels > kMaxTotal) return AXON_ERR_UNSUPPORTED;
  if (__builtin_mul_overflow(in_slots, state, &t) || t > kMaxTotal ||
      __builtin_mul_overflow(out_slots, state, &t) || t > kMaxTotal)
    return AXON_ERR_UNSUPPORTED;
  return AXON_OK;
}

// Outputs of at least twice the 32 MiB of L2 are stored past it: what is written last is not what is read
// next (convolution of 32768 x 7680 bf16 219 -> 214 us, its training pass 282 -> 269 us; head norm of 16384
// rows 80 -> 77 us).
inline bool past_caches(size_t bytes) { return bytes >= (size_t(64) << 20); }

// Bytes that the rows of a strided tensor span.
inline Span rows_span(const void* p, int64_t rows, int64_t stride, int64_t width, size_t es) {
  return span(p, rows > 0 ? es * size_t((rows - 1) * stride + width) : 0);
}

}  // namespace axon

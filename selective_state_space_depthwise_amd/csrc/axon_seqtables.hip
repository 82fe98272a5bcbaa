// Tables of packed sequences, built on the GPU from the request lengths (see axonscan.h).
//
// starts is a prefix sum of the lengths that saturates at the buffer's rows: with T the rows,
// a (+) b = min(a + b, T) is associative for a, b >= 0, so the scan may group its operands freely,
// and 32 bits hold every intermediate. block_starts is the prefix sum of ceil(length / block).
//
// One launch: every workgroup scans all lengths by itself (N <= 65535 int32 values, 256 KiB at
// most, from L2) in tiles of 4096 and writes a slice of its own of the block rows, each row found
// by a binary search among the tile's block starts in LDS. A scan split over workgroups would need
// a second launch or a wait between workgroups, which costs more than the repeated reads. Bound by
// the launch and the scan's chain of barriers: 7 sequences 2.6 us, 4096 sequences and 68111
// block rows 6.7 us.
#include <hip/hip_runtime.h>

#include <cstdint>

#include "axon_internal.h"

namespace axon {
namespace {

constexpr int kPer = 4;  // lengths a thread scans

struct TablesArgs {
  const int32_t* lengths;
  int32_t *starts, *block_starts, *block_seq, *block_first;
  uint32_t n, total, block, rows, rows_per_wg;
};

// Inclusive scan over the workgroup of one value a thread under `op` (associative).
template <int THREADS, typename Op>
__device__ __forceinline__ uint32_t scan_inclusive(uint32_t v, uint32_t* part, Op op) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const uint32_t o = __shfl_up(v, d, 64);
    if (lane >= d) v = op(v, o);
  }
  if (THREADS == 64) return v;
  if (lane == 63) part[wave] = v;
  __syncthreads();
  uint32_t before = 0;
  for (int w = 0; w < wave; ++w) before = op(before, part[w]);
  __syncthreads();
  return op(v, before);
}

template <int THREADS>
__global__ __launch_bounds__(THREADS) void sequence_tables_kernel(TablesArgs a) {
  constexpr uint32_t kTile = THREADS * kPer;
  __shared__ uint32_t st[kTile + 1], bl[kTile + 1], part[THREADS / 64];
  const uint32_t tid = threadIdx.x;
  const uint32_t row0 = blockIdx.x * a.rows_per_wg;
  const uint32_t row1 = min(a.rows, row0 + a.rows_per_wg);
  uint32_t carry_s = 0, carry_b = 0;
  const uint32_t total = a.total;
  auto sat = [total](uint32_t x, uint32_t y) { return min(x + y, total); };
  auto add = [](uint32_t x, uint32_t y) { return x + y; };
  for (uint32_t base = 0; base < a.n; base += kTile) {
    uint32_t s[kPer];
    uint32_t sum = 0;
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      const uint32_t at = base + tid * kPer + j;
      const int32_t len = at < a.n ? a.lengths[at] : 0;
      sum = sat(sum, min(static_cast<uint32_t>(max(len, 0)), total));
      s[j] = sum;
    }
    const uint32_t upto = scan_inclusive<THREADS>(sum, part, sat);
    // Exclusive part of this thread: the previous thread's inclusive value (saturating sums cannot
    // be taken back by a subtraction).
    st[tid + 1] = upto;
    if (tid == 0) st[0] = 0;
    __syncthreads();
    const uint32_t before = sat(carry_s, st[tid]);
    const uint32_t tile_s = sat(carry_s, st[THREADS]);
    __syncthreads();
    uint32_t b[kPer], prev = before, blocks = 0;
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      const uint32_t end = sat(before, s[j]);
      blocks += (end - prev) / a.block + ((end - prev) % a.block != 0);
      b[j] = blocks;
      s[j] = prev;  // where sequence j of this thread begins
      prev = end;
    }
    const uint32_t bupto = scan_inclusive<THREADS>(blocks, part, add);
    const uint32_t bbefore = carry_b + bupto - blocks;
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      st[tid * kPer + j] = s[j];
      bl[tid * kPer + j] = bbefore + (j ? b[j - 1] : 0);
    }
    if (tid == THREADS - 1) {
      st[kTile] = tile_s;
      bl[kTile] = bbefore + blocks;
    }
    __syncthreads();
    const uint32_t count = min(kTile, a.n - base);
    if (blockIdx.x == 0) {
      // the end of the last tile is entry n
      const uint32_t lim = count + (base + count == a.n);
      for (uint32_t j = tid; j < lim; j += THREADS) {
        a.starts[base + j] = static_cast<int32_t>(st[j]);
        a.block_starts[base + j] = static_cast<int32_t>(bl[j]);
      }
    }
    const uint32_t lo = max(row0, bl[0]), hi = min(row1, bl[kTile]);
    for (uint32_t r = lo + tid; r < hi; r += THREADS) {
      uint32_t i = 0, len = count;  // the last sequence with bl[i] <= r
      while (len > 1) {
        const uint32_t half = len >> 1;
        if (bl[i + half] <= r) i += half, len -= half;
        else len = half;
      }
      a.block_seq[r] = static_cast<int32_t>(base + i);
      a.block_first[r] = static_cast<int32_t>(st[i] + (r - bl[i]) * a.block);
    }
    carry_s = tile_s;
    carry_b = bl[kTile];
    __syncthreads();
  }
  for (uint32_t r = max(row0, carry_b) + tid; r < row1; r += THREADS) {
    a.block_seq[r] = -1;
    a.block_first[r] = -1;
  }
}

// Rows behind the last sequence. Mostly there are none, and a workgroup reads one number: 4.3 us of
// launch and of an empty grid behind a scan of 32768 tokens.
__global__ __launch_bounds__(256) void clear_behind_kernel(const int32_t* end, int64_t total,
                                                           int64_t units_a_row, uint4* rows) {
  const int64_t first = min(max(static_cast<int64_t>(*end), int64_t(0)), total) * units_a_row;
  const int64_t step = int64_t(gridDim.x) * 256;
  for (int64_t u = first + int64_t(blockIdx.x) * 256 + threadIdx.x; u < total * units_a_row; u += step)
    rows[u] = make_uint4(0, 0, 0, 0);
}

bool tables_rows(int64_t n, int64_t total, int64_t block, int64_t* rows, axon_status* why) {
  *why = AXON_ERR_INVALID_ARGUMENT;
  if (n < 1 || total < 0 || block < 1) return false;
  *why = AXON_ERR_UNSUPPORTED;
  if (n > 65535 || total >= (int64_t(1) << 31)) return false;
  *rows = total / block + n;
  if (*rows >= (int64_t(1) << 31)) return false;
  *why = AXON_OK;
  return true;
}

}  // namespace
}  // namespace axon

extern "C" {

size_t axon_sequence_tables_count(int64_t sequences, int64_t total_tokens, int64_t block) {
  int64_t rows;
  axon_status why;
  if (!axon::tables_rows(sequences, total_tokens, block, &rows, &why)) return 0;
  return 2 * (size_t(sequences) + 1) + 2 * size_t(rows);
}

axon_status axon_sequence_tables(int64_t sequences, int64_t total_tokens, int64_t block,
                                 const int32_t* lengths, int32_t* tables, void* stream) {
  using namespace axon;
  int64_t rows;
  axon_status why;
  if (!tables_rows(sequences, total_tokens, block, &rows, &why)) return why;
  if (!lengths || !tables || (reinterpret_cast<uintptr_t>(lengths) & 3) ||
      (reinterpret_cast<uintptr_t>(tables) & 3))
    return AXON_ERR_INVALID_ARGUMENT;
  const size_t n1 = size_t(sequences) + 1;
  if (overlaps(span(lengths, 4 * size_t(sequences)), span(tables, 4 * (2 * n1 + 2 * size_t(rows)))))
    return AXON_ERR_INVALID_ARGUMENT;
  TablesArgs a;
  a.lengths = lengths;
  a.starts = tables;
  a.block_starts = tables + n1;
  a.block_seq = tables + 2 * n1;
  a.block_first = tables + 2 * n1 + rows;
  a.n = static_cast<uint32_t>(sequences);
  a.total = static_cast<uint32_t>(total_tokens);
  // No block is longer than the buffer: a larger one only has to stay within 32 bits.
  a.block = static_cast<uint32_t>(block < (int64_t(1) << 31) ? block : (int64_t(1) << 31) - 1);
  a.rows = static_cast<uint32_t>(rows);
  hipStream_t st = static_cast<hipStream_t>(stream);
  // Rows a workgroup writes: enough workgroups that none writes more than a few rows a thread.
  a.rows_per_wg = sequences <= 256 ? 256 : 1024;
  int64_t wgs = (rows + a.rows_per_wg - 1) / a.rows_per_wg;
  if (wgs > 1024) {
    a.rows_per_wg = static_cast<uint32_t>((rows + 1023) / 1024);
    wgs = (rows + a.rows_per_wg - 1) / a.rows_per_wg;
  }
  const dim3 grid(static_cast<unsigned>(wgs));
  if (sequences <= 256)
    hipLaunchKernelGGL(sequence_tables_kernel<64>, grid, dim3(64), 0, st, a);
  else
    hipLaunchKernelGGL(sequence_tables_kernel<1024>, grid, dim3(1024), 0, st, a);
  return hipGetLastError() == hipSuccess ? AXON_OK : AXON_ERR_HIP;
}

axon_status axon_clear_behind_sequences(int64_t sequences, int64_t total_tokens, int64_t row_bytes,
                                        const int32_t* tables, void* rows, void* stream) {
  using namespace axon;
  if (sequences < 1 || total_tokens < 0 || row_bytes < 1 || row_bytes % 16) return AXON_ERR_INVALID_ARGUMENT;
  int64_t bytes;
  if (sequences > 65535 || total_tokens >= (int64_t(1) << 31) ||
      __builtin_mul_overflow(total_tokens, row_bytes, &bytes) || bytes > (int64_t(1) << 42))
    return AXON_ERR_UNSUPPORTED;
  if (total_tokens == 0) return AXON_OK;
  if (!tables || !rows || (reinterpret_cast<uintptr_t>(tables) & 3) ||
      (reinterpret_cast<uintptr_t>(rows) & 15) ||
      overlaps(span(tables, 4 * (size_t(sequences) + 1)), span(rows, size_t(bytes))))
    return AXON_ERR_INVALID_ARGUMENT;
  const int64_t wgs = (bytes / 16 + 1023) / 1024;  // four stores a thread, or more
  hipLaunchKernelGGL(clear_behind_kernel, dim3(static_cast<unsigned>(wgs < 512 ? wgs : 512)), dim3(256), 0,
                     static_cast<hipStream_t>(stream), tables + sequences, total_tokens, row_bytes / 16,
                     static_cast<uint4*>(rows));
  return hipGetLastError() == hipSuccess ? AXON_OK : AXON_ERR_HIP;
}

}  // extern "C"

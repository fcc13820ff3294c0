// Device helpers of the paged 8-bit cache: addressing, and the conversions
// between e4m3 codes and wider types.
//
// The cache holds keys and values as e4m3 codes in pages of `page` tokens,
// each page with one scale per KV head for its keys and one for its values,
// a power of two 2^e: a row's value is code * 2^e. With a power of two the
// product is exact in fp16, bf16 and fp32, a code moved to a larger scale
// keeps its value unless it becomes subnormal, and a scale acts on a score
// (base-2 logarithm) as an addition of e.
#pragma once

#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "common.cuh"
#include "kernels.h"

namespace quoka {
namespace cache {

// Two e4m3 codes (low byte first) to two halves; every code is exact in fp16.
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint16_t c) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(c));
  return r;
}

// Two floats to e4m3 codes (lo in the low byte), to nearest even; beyond
// +-448 (infinities too) saturates, NaN stays NaN.
__device__ __forceinline__ uint16_t f32x2_to_e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

__device__ __forceinline__ void e4m3x4_to_f32(uint32_t c, float* v) {
  const uint32_t a = e4m3x2_to_f16x2((uint16_t)c), b = e4m3x2_to_f16x2((uint16_t)(c >> 16));
  const float2 x = __half22float2(*reinterpret_cast<const __half2*>(&a));
  const float2 y = __half22float2(*reinterpret_cast<const __half2*>(&b));
  v[0] = x.x;
  v[1] = x.y;
  v[2] = y.x;
  v[3] = y.y;
}

// 2^e, -126 <= e <= 127.
__device__ __forceinline__ float exp2i(int e) { return __int_as_float((e + 127) << 23); }

// The exponent of a stored scale. Only the exponent field is used, kept to
// the range of scales; anything that is not a power of two in that range sets
// *bad.
__device__ __forceinline__ int scale_exp(float s, bool* bad) {
  const int u = __float_as_int(s);
  const int e = (u >> 23) - 127;  // (a sign bit makes it negative, out of range)
  const int k = min(max(e, kCacheMinExp), kCacheMaxExp);
  *bad |= k != e || (u & 0x7FFFFF) != 0;
  return k;
}

// The smallest e with amax <= 448 * 2^e (448 = 1.75 * 2^8), in the range of
// scales; amax is finite and >= 0.
__device__ __forceinline__ int scale_exp_for(float amax) {
  const uint32_t u = __float_as_uint(amax);
  const int k = (int)(u >> 23) - 127;  // amax = m * 2^k, 1 <= m < 2 (subnormals lie below every scale)
  const int e = k - 8 + ((u & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  return min(max(e, kCacheMinExp), kCacheMaxExp);
}

// c (16 x 8, fp32) += a (16 x 16, fp16) * b (16 x 8, fp16)
__device__ __forceinline__ void mma_f16(float* c, const uint32_t* a, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Byte of chunk c (16 bytes) of row r of code rows in shared memory: the
// layout of a tiled TMA load swizzled by 128 (d = 128) or 64 bytes (d = 64).
template <int D>
__device__ __forceinline__ int at_chunk(int r, int c) {
  return r * D + ((D == 128 ? c ^ (r & 7) : c ^ ((r >> 1) & 3)) << 4);
}

// ---- Ranges: the keys of all rows (sequence, KV head) cut into runs of near
// equal length, one CTA each. Lengths are known on the device only, so the
// grid is an upper bound and every CTA finds its own range.

struct Range {
  int row, k0, k1;   // keys [k0, k1) of row; row < 0: none
  int first, parts;  // the row's first range and their number
};

// Beyond this many rows each takes one CTA: they fill the GPU several times over,
// and a look at all lengths would cost each CTA more than it evens out.
constexpr int kRangeRows = 1024;

// Ranges asked for (before rounding up row by row; ctas >= 2), and the grid that
// holds them: sum over rows of max(1, ceil(n / most)) <= target + rows with
// most >= total / target, and <= rows * ceil(N / least).
__host__ __device__ __forceinline__ int64_t range_target(int64_t rows, int ctas) {
  return ctas - rows / 2 > ctas / 2 ? ctas - rows / 2 : ctas / 2;
}
__host__ __forceinline__ int64_t range_grid(int64_t rows, int N, int ctas, int least) {
  if (rows > kRangeRows) return rows;
  const int64_t a = range_target(rows, ctas) + rows, b = rows * (N > least ? (N + least - 1) / least : 1);
  return a < b ? a : b;
}

// Range `cta`, or, for -1 - row, the first range of that row (called by one warp;
// written to *out). keys(row): a row's keys, at most 2^30. Rows are cut into equal
// runs of at most max(least, total / target) keys, rounded up to `step`. held:
// shared memory for a length per row.
template <typename Keys>
__device__ __forceinline__ void find_range(int rows, int target, int least, int step, int cta, int lane, Keys&& keys,
                                           int* held, Range* out) {
  if (rows > kRangeRows) {
    const int row = cta < 0 ? -1 - cta : cta;
    if (lane == 0) *out = Range{row, 0, keys(row), row, 1};
    return;
  }
  int64_t total = 0;
#pragma unroll 4
  for (int i = lane; i < rows; i += 32) {
    const int n = keys(i);
    total += n;
    held[i] = n;  // (read again by this lane only)
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
  const int64_t even = total < 0x7FFFFFFF - target ? (int64_t)((unsigned)(total + target - 1) / (unsigned)target)
                                                   : (total + target - 1) / target;
  const int most = (int)min(max((int64_t)least, even), (int64_t)1 << 30);
  if (lane == 0) out->row = -1;
  __syncwarp();
  int before = 0;  // ranges of the rows before
#pragma unroll 1
  for (int i0 = 0; i0 < rows; i0 += 32) {
    const int i = i0 + lane, n = i < rows ? held[i] : 0;
    const int parts = i < rows ? max(1, (n + most - 1) / most) : 0;
    const int all = __reduce_add_sync(0xffffffffu, parts);
    if (cta < 0 ? -1 - cta < i0 + 32 : cta < before + all) {  // among these 32 rows
      int incl = parts;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int x = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += x;
      }
      const int first = before + incl - parts, at = cta < 0 ? first : cta;
      if (cta < 0 ? i == -1 - cta : cta >= first && cta < first + parts) {
        const int per = ((n + parts - 1) / parts + step - 1) & ~(step - 1);
        const int k0 = (int)min((int64_t)n, (int64_t)(at - first) * per);
        *out = Range{i, k0, min(n, k0 + per), first, parts};
      }
      return;
    }
    before += all;
  }
}

// Keys of sequence bi that a selection scores: none without a query.
__device__ __forceinline__ int scored_keys(const CacheScoreArgs& a, int bi) {
  const int n = min(max(__ldcg(a.c.seq_len + bi), 0), a.max_len);
  return a.new_len != nullptr && __ldcg(a.new_len + bi) <= 0 ? 0 : n;
}

// Latches lengths and counts of a sequence that are out of range (of a selection).
__device__ __forceinline__ void check_scored(const CacheScoreArgs& a, int bi) {
  const int want = __ldcg(a.c.seq_len + bi), live = a.new_len != nullptr ? __ldcg(a.new_len + bi) : 0;
  if (want < 0 || want > a.max_len || live < 0 || live > a.BCP) latch_status(a.status, 6 /* QUOKA_ERR_BOUNDS */);
}

// Rows of a box of the pools' tensor maps: a run of keys that starts on a
// multiple of 64 splits into boxes of one page each.
__host__ __device__ __forceinline__ int box_log2(const CacheView& c) { return c.page_log2 < 6 ? c.page_log2 : 6; }

}  // namespace cache
}  // namespace quoka

// Key scoring over the paged 8-bit cache.
//
// [QUOKA §2.2] cosine score, [QUOKA §2.3] S = Q_group . K_norm^T reduced by a
// max over the NQ chosen queries:
//   S_agg[b, j, tau] = max_i (Q_group[b, j, i] . k) / |k|,  k = code row * 2^e.
// The page's scale cancels: the score reads the codes alone.
//
// Precision. Codes are exact in fp16; the fp32 group means (|q| <= 1) are
// scaled by 2^12 and split into two halves (22 bits of each element), both
// multiplied on the tensor core with fp32 accumulation; |k|^2 is summed in
// fp32 from the same codes.
//
// Work split: one CTA of 4 warps per 128 keys of a (sequence, KV head); a warp
// holds the code rows of 32 keys in registers, loaded in the operand layout of
// mma.sync (the columns of a k-step may be any 16 as long as Q_group is
// permuted alike, so a lane reads whole 16-byte chunks), and multiplies them
// with the group means in 16-row tiles from shared memory, at most 4 tiles
// at a time.
#include "cache.cuh"

namespace quoka {

namespace {

using namespace cache;

constexpr int kThreads = 128;
constexpr int kKeys = 128;   // keys of one CTA
constexpr int kTiles = 4;    // 16-row tiles of group means in shared memory at a time
constexpr float kQScale = 4096.f;

__device__ __forceinline__ void mma_f16(float* c, const uint32_t* a, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// acc + x^2 of a half, in fp32
__device__ __forceinline__ float sq_add(float acc, uint32_t h2) {
  const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h2));
  return fmaf(f.y, f.y, fmaf(f.x, f.x, acc));
}

// grid (ceil(max_len / 128), nkv, b)
template <int D>
__global__ void __launch_bounds__(kThreads) cache_score_kernel(const CacheScoreArgs a) {
  constexpr int KS = D / 16;
  __shared__ uint4 qs[kTiles][2][KS][32];  // fragments of the group means: halves hi, lo
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t4 = lane & 3;
  const int j = blockIdx.y, bi = blockIdx.z;
  const int64_t row = (int64_t)bi * a.c.nkv + j;
  pdl_trigger();
  pdl_wait();
  const int len = cache_len(a.c, bi, a.max_len, a.status);
  const int key0 = blockIdx.x * kKeys;
  if (key0 >= len) return;
  const int base = key0 + warp * 32;
  const int plog = a.c.page_log2, pmask = (1 << plog) - 1;

  // this warp's keys: n-tile nt holds keys base + 8 nt + g
  uint32_t kw[4][KS];
  {
    int64_t off = -1;  // lane i answers for key i
    if (base + lane < len) {
      const int p = cache_page(a.c, bi, (base + lane) >> plog, a.status);
      if (p >= 0) off = p * a.c.sp + j * a.c.sh + (int64_t)((base + lane) & pmask) * a.c.sr;
    }
#pragma unroll
    for (int nt = 0; nt < 4; ++nt) {
      const int64_t ro = __shfl_sync(0xffffffffu, off, 8 * nt + g);
#pragma unroll
      for (int w = 0; w < KS; ++w) kw[nt][w] = 0u;
      if (ro >= 0) {
#pragma unroll
        for (int h = 0; h < D / 64; ++h) {
          const uint4 v = *reinterpret_cast<const uint4*>(a.c.k + ro + 16 * t4 + 64 * h);
          kw[nt][4 * h] = v.x;
          kw[nt][4 * h + 1] = v.y;
          kw[nt][4 * h + 2] = v.z;
          kw[nt][4 * h + 3] = v.w;
        }
      }
    }
  }

  float best[4][2];  // per n-tile: keys 2 t, 2 t + 1, over the lane's rows
  float ss[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int nt = 0; nt < 4; ++nt) best[nt][0] = best[nt][1] = -INFINITY;
  const float* qg = a.Qg + row * a.NQ * D;
  for (int i0 = 0; i0 < a.NQ; i0 += 16 * kTiles) {
    const int tiles = min(kTiles, (a.NQ - i0 + 15) / 16);
    if (i0 > 0) __syncthreads();
    // column d of row i belongs to lane t = (d / 16) % 4, k-step 4 (d / 64) + (d % 16) / 4
    for (int e = tid; e < tiles * 16 * (D / 2); e += kThreads) {
      const int i = e / (D / 2), d = 2 * (e % (D / 2));
      float2 x = make_float2(0.f, 0.f);
      if (i0 + i < a.NQ) x = __ldcg(reinterpret_cast<const float2*>(qg + (int64_t)(i0 + i) * D + d));
      x.x *= kQScale;
      x.y *= kQScale;
      const __half2 hi = __floats2half2_rn(x.x, x.y);
      const float2 f = __half22float2(hi);
      const __half2 lo = __floats2half2_rn(x.x - f.x, x.y - f.y);
      const int ch = d >> 4, ks = 4 * (ch >> 2) + ((d & 15) >> 2), r = i & 15;
      const int reg = ((d >> 1) & 1) * 2 + (r >> 3), ln = (r & 7) * 4 + (ch & 3);
      reinterpret_cast<__half2*>(&qs[i >> 4][0][ks][ln])[reg] = hi;
      reinterpret_cast<__half2*>(&qs[i >> 4][1][ks][ln])[reg] = lo;
    }
    __syncthreads();
    float c[kTiles][4][4];
#pragma unroll
    for (int m = 0; m < kTiles; ++m)
#pragma unroll
      for (int nt = 0; nt < 4; ++nt) c[m][nt][0] = c[m][nt][1] = c[m][nt][2] = c[m][nt][3] = 0.f;
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) {
      uint32_t b0[4], b1[4];
#pragma unroll
      for (int nt = 0; nt < 4; ++nt) {
        b0[nt] = e4m3x2_to_f16x2((uint16_t)kw[nt][ks]);
        b1[nt] = e4m3x2_to_f16x2((uint16_t)(kw[nt][ks] >> 16));
        if (i0 == 0) ss[nt] = sq_add(sq_add(ss[nt], b0[nt]), b1[nt]);
      }
#pragma unroll
      for (int m = 0; m < kTiles; ++m) {
        if (m < tiles) {
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            const uint4 q = qs[m][half][ks][lane];
            const uint32_t qa[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
            for (int nt = 0; nt < 4; ++nt) mma_f16(c[m][nt], qa, b0[nt], b1[nt]);
          }
        }
      }
    }
#pragma unroll
    for (int m = 0; m < kTiles; ++m) {
      const bool r0 = i0 + 16 * m + g < a.NQ, r1 = i0 + 16 * m + g + 8 < a.NQ;
#pragma unroll
      for (int nt = 0; nt < 4; ++nt)
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          if (r0) best[nt][u] = fmaxf(best[nt][u], c[m][nt][u]);
          if (r1) best[nt][u] = fmaxf(best[nt][u], c[m][nt][2 + u]);
        }
    }
  }
#pragma unroll
  for (int nt = 0; nt < 4; ++nt) {
    // |k|^2 of key g over the quad; then the norms of keys 2 t, 2 t + 1
    ss[nt] += __shfl_xor_sync(0xffffffffu, ss[nt], 1);
    ss[nt] += __shfl_xor_sync(0xffffffffu, ss[nt], 2);
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      float x = best[nt][u];
      x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 4));
      x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 8));
      x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 16));
      const float k2 = __shfl_sync(0xffffffffu, ss[nt], 4 * (2 * t4 + u));
      const int key = base + 8 * nt + 2 * t4 + u;
      if (g == 0 && key < len)
        a.S_agg[row * a.max_len + key] = x * (1.f / kQScale) / fmaxf(sqrtf(k2), 1e-12f);
    }
  }
}

}  // namespace

cudaError_t launch_cache_score(int d, const CacheScoreArgs& a, cudaStream_t stream) {
  if (a.NQ < 1 || a.max_len < 1) return cudaErrorInvalidValue;
  if (d != 64 && d != 128) return cudaErrorNotSupported;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((a.max_len + kKeys - 1) / kKeys, a.c.nkv, a.b);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;  // waits for the group means inside
  return cudaLaunchKernelEx(&cfg, d == 128 ? cache_score_kernel<128> : cache_score_kernel<64>, a);
}

}  // namespace quoka

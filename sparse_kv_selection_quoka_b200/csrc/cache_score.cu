// Key scoring over the paged 8-bit cache with up to four group means (more:
// cache_score_tc.cu).
//
// [QUOKA §2.2] cosine score, [QUOKA §2.3] S = Q_group . K_norm^T reduced by a
// max over the NQ chosen queries:
//   S_agg[b, j, tau] = max_i (Q_group[b, j, i] . k) / |k|,  k = code row * 2^e.
// The page's scale cancels: the score reads the codes alone.
//
// Precision. Codes are exact in fp16; the fp32 group means (|q| <= 1) are
// scaled by 2^12 and split into two halves hi + lo (22 bits of each element),
// both multiplied on the tensor core with fp32 accumulation. |k|^2 is the
// diagonal of K K^T, whose operands are the registers already there: its
// products are exact too.
//
// Work split. The keys of every (sequence, KV head) are cut into ranges of near
// equal length, one CTA each (cache.cuh): a loader warp copies 128 code rows at a
// time into a ring of stages (TMA, boxes of up to 64 rows of one page; the page
// table is read two stages ahead), four warps take 32 of them each. Keys are the
// rows of the product, hi and lo of the group means its 8 columns, kept in
// registers: a 16 x 16 step costs three products. The operand reads are those of
// cache_attn.cu (any 16 columns make a k-step; chunk c of row r lies at c ^ (r &
// 7)). The scores' value-bucket histogram (the top-k's first digit) is made on
// the way: counts in shared memory, added to the row's at the end.
// Bound by issue and the legacy tensor pipe together (3 products a 16 x 16 step),
// 1.7 times the codes' bytes at HBM's rate: 16 ragged sequences of up to 8191
// keys, 8 heads, d = 128, one group mean: 22.5 us for 85.3 MB, 3.8 TB/s; 32768 keys
// and 4 group means 13.1 us for 33.6 MB. cp.async rows instead of TMA boxes took
// 40.2 us on the first, 4 CTAs an SM with 2 stages the same as 3 with 3, the
// histogram straight in global memory 2 us more, |k|^2 with e4m3 products
// (m16n8k32) or by fp32 pairs on the CUDA cores 2 us more.
#include "cache.cuh"
#include "sm100.cuh"
#include "tmap.cuh"

namespace quoka {

namespace {

using namespace cache;

constexpr int kThreads = 160;     // four computing warps and the loader
constexpr int kStage = 128;       // keys of a stage
constexpr int kStages = 3;
constexpr int kMost = 4;          // group means: hi and lo fill one tile
constexpr float kQScale = 4096.f;
// One round of CTAs at three an SM, a range being at least 256 keys.
constexpr int kSplitCTAs = 444, kSplitKeys = 256;

struct Shared {
  uint64_t full[kStages], empty[kStages];
  int abort;
  Range range;
  alignas(16) uint32_t hist[TOPK_HIST_BINS];
};

// Dynamic shared memory: the ring, then the group means' fragments [k-step][lane]
// of two words.
template <int D>
constexpr size_t smem_bytes() {
  return (size_t)kStages * kStage * D + (size_t)(D / 16) * 256 + 1024;
}

// The loader warp: code rows [k0, k1) of the (sequence, head) by boxes of one page
// each (rows behind k1 come along, and are not used).
template <int D>
__device__ __forceinline__ void load_rows(const CacheScoreArgs& a, const CUtensorMap& map, Shared& sh, uint8_t* ring,
                                          int lane, int bi, int j, int k0, int k1) {
  const int plog = a.c.page_log2, pmask = (1 << plog) - 1, blog = box_log2(a.c);
  const int32_t* table = a.c.page_table + (int64_t)bi * a.c.table_stride;
  const int total = (k1 - k0 + kStage - 1) / kStage;
  bool bad = false;
  // this lane's box of the it-th stage: its first key, whether there is one, its page
  auto key_of = [&](int it) { return k0 + it * kStage + (lane << blog); };
  auto here = [&](int it) { return it < total && (lane << blog) < kStage && key_of(it) < k1; };
  auto page_of = [&](int it) { return here(it) ? __ldcg(table + (key_of(it) >> plog)) : -1; };
  int p0 = page_of(0), p1 = page_of(1), it = 0;
  for (; it < total; ++it) {
    const int p2 = page_of(it + 2), st = it % kStages;
    if (it >= kStages && !__all_sync(0xffffffffu, sm100::mbar_wait(&sh.empty[st], (it / kStages - 1) & 1, &sh.abort, a.wait_ns))) {
      if (lane == 0) {
        sh.abort = 1;
        latch_status(a.status, 5 /* QUOKA_ERR_TIMEOUT */);
        latch_where(a.status, 63);
      }
      break;
    }
    if (here(it)) {
      const bool held = p0 >= 0 && p0 < a.c.npages;
      bad |= !held;  // (a page that is not there lies out of bounds: zeros)
      sm100::mbar_arrive_expect_tx(&sh.full[st], (uint32_t)D << blog);
      sm100::tma_load_4d(sm100::smem_u32(ring + st * kStage * D) + (lane << blog) * D, &map, &sh.full[st], 0,
                         key_of(it) & pmask, j, held ? p0 : a.c.npages);
    } else {
      sm100::mbar_arrive(&sh.full[st]);
    }
    p0 = p1;
    p1 = p2;
  }
  // no copy may be in flight when the CTA ends, even if a wait gave up
  for (int i = max(0, it - kStages); i < it; ++i) sm100::mbar_drain(&sh.full[i % kStages], (i / kStages) & 1, a.wait_ns);
  if (bad) latch_status(a.status, 6 /* QUOKA_ERR_BOUNDS */);
}

// One CTA per range.
template <int D>
__global__ void __launch_bounds__(kThreads, 3)
cache_score_kernel(const __grid_constant__ CUtensorMap map, const CacheScoreArgs a) {
  constexpr int KS = D / 16;
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ Shared sh;
  uint8_t* ring = sm100::align_smem_1024(smem);
  uint2* qs = reinterpret_cast<uint2*>(ring + kStages * kStage * D);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t4 = lane & 3;
  pdl_trigger();
  // (the cache, its table and lengths are inputs of the call: only the group
  // means, the histogram and the status words are waited for)
  if (tid == 0) {
    for (int i = 0; i < kStages; ++i) {
      sm100::mbar_init(&sh.full[i], 32);
      sm100::mbar_init(&sh.empty[i], a.inject && i == 0 ? 5 : 4);  // (the hook: an arrival that never comes)
    }
    sh.abort = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  for (int i = tid; i < TOPK_HIST_BINS / 4; i += kThreads) reinterpret_cast<uint4*>(sh.hist)[i] = make_uint4(0u, 0u, 0u, 0u);
  if (warp == 4)
    find_range(a.b * a.c.nkv, a.target, kSplitKeys, kStage, blockIdx.x, lane,
               [&](int i) { return scored_keys(a, i / a.c.nkv); },
               reinterpret_cast<int*>(ring), &sh.range);
  if (warp == 4) sm100::fence_proxy_async_smem();  // (the ring's copies come behind the lengths)
  __syncthreads();
  const int k0 = sh.range.k0, k1 = sh.range.k1;
  if (sh.range.row < 0) {
    pdl_wait();
    return;
  }
  const int64_t row = sh.range.row;
  const int bi = sh.range.row / a.c.nkv, j = sh.range.row % a.c.nkv;
  if (tid == 0) check_scored(a, bi);
  if (k0 >= k1) {
    pdl_wait();
    return;
  }
  if (warp == 4) {
    load_rows<D>(a, map, sh, ring, lane, bi, j, k0, k1);
  } else {
    pdl_wait();
    const float* qg = a.Qg + row * a.NQ * D;
    const int nst = (k1 - k0 + kStage - 1) / kStage;
    const int gk = g ^ ((g & 1) << 2);  // operand row g (and g + 8) of a step is key gk (and gk + 8)
    // column d of group mean i: k-step ks of lane 4 i + t, with chunk d / 16 = t + 4 (ks / 4) and word
    // (d % 16) / 4 = ks % 4; columns 0 .. 3 of the tile are hi, 4 .. 7 lo
    for (int e = tid; e < kMost * (D / 2); e += 128) {
      const int i = e / (D / 2), d = 2 * (e % (D / 2));
      float2 x = make_float2(0.f, 0.f);
      if (i < a.NQ) x = __ldcg(reinterpret_cast<const float2*>(qg + (int64_t)i * D + d));
      x.x *= kQScale;
      x.y *= kQScale;
      const __half2 hi = __floats2half2_rn(x.x, x.y);
      const float2 f = __half22float2(hi);
      const __half2 lo = __floats2half2_rn(x.x - f.x, x.y - f.y);
      const int ch = d >> 4, ks = 4 * (ch >> 2) + ((d & 15) >> 2), reg = (d >> 1) & 1;
      uint2* q = qs + ks * 32 + (ch & 3);
      reinterpret_cast<__half2*>(q + 4 * i)[reg] = hi;
      reinterpret_cast<__half2*>(q + 4 * (i + 4))[reg] = lo;
    }
    sm100::named_barrier_sync(1, 128);
    uint2 qb[KS];
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) qb[ks] = qs[ks * 32 + lane];
    for (int s = 0; s < nst; ++s) {
      const int st = s % kStages;
      if (!__all_sync(0xffffffffu, sm100::mbar_wait(&sh.full[st], (s / kStages) & 1, &sh.abort, a.wait_ns))) {
        if (lane == 0) {
          sh.abort = 1;
          latch_status(a.status, 5 /* QUOKA_ERR_TIMEOUT */);
          latch_where(a.status, 64);
        }
        break;
      }
      const uint8_t* stage = ring + st * kStage * D;
      const int r0 = warp * 32;
      float x[2][2];   // the best of keys gk, gk + 8 of both 16-key tiles over the lane's columns
      float k2[2][2];  // |k|^2 of the keys whose diagonal element this lane holds
      // both tiles side by side: six independent chains of products
      {
        float n0[2][4], n1[2][4], c[2][4];
#pragma unroll
        for (int m = 0; m < 2; ++m)
#pragma unroll
          for (int u = 0; u < 4; ++u) n0[m][u] = n1[m][u] = c[m][u] = 0.f;
#pragma unroll
        for (int h = 0; h < D / 64; ++h) {
          uint4 kw[2][2];
#pragma unroll
          for (int m = 0; m < 2; ++m)
#pragma unroll
            for (int u = 0; u < 2; ++u)
              kw[m][u] = *reinterpret_cast<const uint4*>(stage + at_chunk<D>(r0 + 16 * m + gk + 8 * u, t4 + 4 * h));
#pragma unroll
          for (int w = 0; w < 4; ++w) {
            const int ks = 4 * h + w;
#pragma unroll
            for (int m = 0; m < 2; ++m) {
              const uint32_t w0 = reinterpret_cast<const uint32_t*>(&kw[m][0])[w];
              const uint32_t w1 = reinterpret_cast<const uint32_t*>(&kw[m][1])[w];
              const uint32_t ka[4] = {e4m3x2_to_f16x2((uint16_t)w0), e4m3x2_to_f16x2((uint16_t)w1),
                                      e4m3x2_to_f16x2((uint16_t)(w0 >> 16)), e4m3x2_to_f16x2((uint16_t)(w1 >> 16))};
              mma_f16(c[m], ka, qb[ks].x, qb[ks].y);
              mma_f16(n0[m], ka, ka[0], ka[2]);
              mma_f16(n1[m], ka, ka[1], ka[3]);
            }
          }
        }
#pragma unroll
        for (int m = 0; m < 2; ++m) {
#pragma unroll
          for (int u = 0; u < 4; ++u) c[m][u] += __shfl_xor_sync(0xffffffffu, c[m][u], 2);
#pragma unroll
          for (int v = 0; v < 2; ++v) {
            const bool one = 2 * (t4 & 1) < a.NQ, two = 2 * (t4 & 1) + 1 < a.NQ;
            x[m][v] = fmaxf(one ? c[m][2 * v] : -INFINITY, two ? c[m][2 * v + 1] : -INFINITY);
          }
          k2[m][0] = g & 1 ? n0[m][1] : n0[m][0];
          k2[m][1] = g & 1 ? n1[m][3] : n1[m][2];
        }
      }
#pragma unroll
      for (int m = 0; m < 2; ++m)
#pragma unroll
        for (int v = 0; v < 2; ++v) x[m][v] = fmaxf(x[m][v], __shfl_xor_sync(0xffffffffu, x[m][v], 1));
      // lane l takes key l of the 32: from the lane of its quad that holds the
      // diagonal's element
      {
        const int lg = (lane & 7) ^ ((lane & 1) << 2), src = 4 * lg + (lg >> 1);
        float best = 0.f, n = 0.f;
#pragma unroll
        for (int m = 0; m < 2; ++m)
#pragma unroll
          for (int v = 0; v < 2; ++v) {
            const float x_ = __shfl_sync(0xffffffffu, x[m][v], src), n_ = __shfl_sync(0xffffffffu, k2[m][v], src);
            if ((lane >> 3) == 2 * m + v) {
              best = x_;
              n = n_;
            }
          }
        const int key = k0 + s * kStage + r0 + lane;
        if (key < k1) {
          // (rsqrt is within 2^-22; a key of zeros scores 0, one with a NaN -inf)
          const float y = n > 0.f ? best * (1.f / kQScale) * rsqrtf(n) : n == 0.f ? 0.f : -INFINITY;
          a.S_agg[row * a.max_len + key] = y;
          atomicAdd(&sh.hist[score_bin(y)], 1u);
        }
      }
      __syncwarp();
      if (lane == 0) sm100::mbar_arrive(&sh.empty[st]);
    }
  }
  __syncthreads();
  pdl_wait();  // (the loader's threads: the histogram's zeros)
  uint32_t* hist = a.hist + row * TOPK_HIST_BINS;
  for (int i = tid; i < TOPK_HIST_BINS / 4; i += kThreads) {
    const uint4 n = reinterpret_cast<const uint4*>(sh.hist)[i];
    if ((n.x | n.y | n.z | n.w) == 0u) continue;
    if (n.x != 0u) atomicAdd(hist + 4 * i, n.x);
    if (n.y != 0u) atomicAdd(hist + 4 * i + 1, n.y);
    if (n.z != 0u) atomicAdd(hist + 4 * i + 2, n.z);
    if (n.w != 0u) atomicAdd(hist + 4 * i + 3, n.w);
  }
}

template <int D>
cudaError_t launch_typed(const CacheScoreArgs& args, cudaStream_t stream) {
  CacheScoreArgs a = args;
  const int64_t rows = (int64_t)a.b * a.c.nkv, ranges = range_grid(rows, a.max_len, kSplitCTAs, kSplitKeys);
  if (ranges > 0x7FFFFFFF) return cudaErrorNotSupported;
  a.target = (int)range_target(rows, kSplitCTAs);
  auto* kern = cache_score_kernel<D>;
  const size_t smem = smem_bytes<D>();
  const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  CUtensorMap map;
  if (!encode_codes_4d(&map, a.c.k, D, 1 << a.c.page_log2, a.c.nkv, a.c.npages, a.c.sr, a.c.sh, a.c.sp, 1 << box_log2(a.c)))
    return cudaErrorNotSupported;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)ranges);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;  // waits for the group means inside
  return cudaLaunchKernelEx(&cfg, kern, map, a);
}

}  // namespace

cudaError_t launch_cache_score(int d, const CacheScoreArgs& args, cudaStream_t stream) {
  CacheScoreArgs a = args;
  const WaitHooks hooks = wait_hooks();
  a.wait_ns = hooks.wait_ns;
  a.inject = hooks.inject == INJECT_CACHE_SCORE ? 1 : 0;
  if (a.NQ < 1 || a.max_len < 1) return cudaErrorInvalidValue;
  if (d != 64 && d != 128) return cudaErrorNotSupported;
  if (a.NQ > kMost) return launch_cache_score_tc(d, a, stream);
  return d == 128 ? launch_typed<128>(a, stream) : launch_typed<64>(a, stream);
}

}  // namespace quoka

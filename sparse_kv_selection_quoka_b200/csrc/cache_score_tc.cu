// Key scoring over the paged 8-bit cache on the tcgen05 tensor cores, for more
// group means than cache_score.cu keeps in registers.
//
// [QUOKA §2.2] cosine score, [QUOKA §2.3] S = Q_group . K_norm^T reduced by a
// max over the NQ chosen queries:
//   S_agg[b, j, tau] = max_i (Q_group[b, j, i] . k) / |k|,  k = code row * 2^e.
// The page's scale cancels: the score reads the codes alone, and the codes are
// the operand: a tile of 128 code rows, as TMA lays it into shared memory, is A
// of both products of the tile,
//   D_q = K Qp^T   (128 x N)    the scores, against pieces of the group means,
//   D_k = K K^T    (128 x 128)  whose diagonal is |k|^2.
//
// Precision. A group mean's element q (|q| <= 1) is split into P e4m3 pieces,
//   q = sum_p 2^-(8 + 4 p) piece_p + r,  piece_p = e4m3(2^(8 + 4 p) rest_p),
// A piece of four significant bits leaves at most 2^-4 of its leading power of two,
// exactly that only where the next piece ends it, else less, so that the next one's
// leading power is half as large: |r| <= 2^-(5P - 1) |q| (of elements below 2^-14: of
// 2^-14). P = 5 (2^-24, all of an fp32 number) for up to 24 group means a pass, else
// 4 (2^-19), 32 a pass. Code products are exact and accumulate in fp32; the pieces'
// columns are added in fp32.
//
// Work split. The keys of every (sequence, KV head) are cut into ranges of near
// equal length, one CTA each (cache.cuh), two CTAs an SM. Warp 4 loads: boxes of
// up to 64 rows of one page, the page table read two stages ahead. Warp 5 issues
// both products of a tile as soon as it has landed and the accumulators
// (128 + N TMEM columns) are free. Warps 0-3 take a key a thread: the diagonal
// element is one of the warp's 32 columns of D_k, then the pieces' columns, 32 at
// a time (6 group means of 5 pieces and 2 idle rows, or 8 of 4; idle slots repeat
// the first group mean). The scores' value-bucket histogram (the top-k's first
// digit) is counted in shared memory and added to the row's at the end.
// Bound by its latency chain a tile (product, accumulator load, release) and the
// fixed costs of a range (pieces, TMEM, histogram). Measured: 32768 keys, 8 heads,
// d = 128: selection with 5 group means 24.7 us, 8 26.5, 32 28.9 (mma.sync products
// took 14 us more), 64 43.0, 128 61.8; 4 24.7 against 22.8 with mma.sync, so that few
// stay there. 444 ranges instead of 296: 3 us more.
// Every wait is bounded; one that gives up records QUOKA_ERR_TIMEOUT and the CTA
// unwinds (copies and products drained, TMEM freed).
#include "cache.cuh"
#include "sm100.cuh"
#include "tmap.cuh"

namespace quoka {

namespace {

using namespace cache;

constexpr int kThreads = 192;
constexpr int kLoadWarp = 4, kMmaWarp = 5;
constexpr int kStage = 128;          // keys of a tile
constexpr int kRingBytes = 65536;    // the ring (with the rest: two CTAs an SM, whose TMEM fits)
constexpr int kMaxGroups = 4;        // groups of 32 piece columns of a pass
constexpr uint32_t kTmemCols = 256;  // D_k: columns 0 .. 127, D_q: 128 ..
// One round of CTAs at two an SM, a range being at least 256 keys.
constexpr int kSplitCTAs = 296, kSplitKeys = 256;

template <int D>
struct Ring {
  static constexpr int kBytes = kStage * D;  // a tile
  static constexpr int kStages = kRingBytes / kBytes;
};

template <int D>
struct Shared {
  uint64_t full[Ring<D>::kStages], empty[Ring<D>::kStages];
  uint64_t acc_full, acc_empty, b_ready, done;
  uint32_t tmem;
  int abort;
  Range range;
  alignas(16) uint32_t hist[TOPK_HIST_BINS];
};

// Group means of a pass: per group of 32 columns, and how many groups.
template <int P>
struct Pass {
  static constexpr int kPer = 32 / P;
  static constexpr int kMost = kMaxGroups * kPer;
};

template <typename Sh>
__device__ __forceinline__ void give_up(Sh& sh, int* status, int where) {
  sh.abort = 1;
  latch_status(status, 5 /* QUOKA_ERR_TIMEOUT */);
  latch_where(status, where);
}

// The loader warp: code rows [k0, k1) of the (sequence, head), `passes` times, by
// boxes of one page each (rows behind k1 come along, and are not used).
template <int D>
__device__ __forceinline__ void load_rows(const CacheScoreArgs& a, const CUtensorMap& map, Shared<D>& sh, uint8_t* ring,
                                          int lane, int bi, int j, int k0, int k1, int passes) {
  constexpr int kStages = Ring<D>::kStages;
  const int plog = a.c.page_log2, pmask = (1 << plog) - 1, blog = box_log2(a.c);
  const int32_t* table = a.c.page_table + (int64_t)bi * a.c.table_stride;
  const int nst = (k1 - k0 + kStage - 1) / kStage, total = nst * passes;
  bool bad = false;
  // this lane's box of the it-th tile: its first key, whether there is one, its page
  auto key_of = [&](int it) { return k0 + it % nst * kStage + (lane << blog); };
  auto here = [&](int it) { return it < total && (lane << blog) < kStage && key_of(it) < k1; };
  auto page_of = [&](int it) { return here(it) ? __ldcg(table + (key_of(it) >> plog)) : -1; };
  int p0 = page_of(0), p1 = page_of(1), it = 0;
  for (; it < total; ++it) {
    const int p2 = page_of(it + 2), st = it % kStages;
    if (it >= kStages && !sm100::mbar_wait_warp(&sh.empty[st], (it / kStages - 1) & 1, &sh.abort, a.wait_ns)) {
      if (lane == 0) give_up(sh, a.status, 63);
      break;
    }
    if (here(it)) {
      const bool held = p0 >= 0 && p0 < a.c.npages;
      bad |= !held;  // (a page that is not there lies out of bounds: zeros)
      sm100::mbar_arrive_expect_tx(&sh.full[st], (uint32_t)D << blog);
      sm100::tma_load_4d(sm100::smem_u32(ring + st * Ring<D>::kBytes) + (lane << blog) * D, &map, &sh.full[st], 0,
                         key_of(it) & pmask, j, held ? p0 : a.c.npages);
    } else {
      sm100::mbar_arrive(&sh.full[st]);
    }
    __syncwarp();
    p0 = p1;
    p1 = p2;
  }
  // no copy may be in flight when the CTA ends, even if a wait gave up
  for (int i = max(0, it - kStages); i < it; ++i) sm100::mbar_drain(&sh.full[i % kStages], (i / kStages) & 1, a.wait_ns);
  if (bad) latch_status(a.status, 6 /* QUOKA_ERR_BOUNDS */);
}

// Group means [i0, i0 + n) as pieces: row 32 g + P s + p of the operand is piece p
// of slot s of group g (the idle rows and slots are finite and change nothing).
template <int D, int P>
__device__ __forceinline__ void stage_pieces(const float* qg, uint8_t* qs, int n, int groups, int tid) {
  constexpr int CPR = D / 16, kPer = Pass<P>::kPer;
#pragma unroll 1
  for (int e = tid; e < groups * kPer * (D / 8); e += 128) {  // 8 columns of a slot
    const int slot = e / (D / 8), c = e % (D / 8);
    const float* src = qg + (int64_t)(slot < n ? slot : 0) * D + 8 * c;
    float x[8];
#pragma unroll
    for (int u = 0; u < 8; u += 4) {
      const float4 v = __ldcg(reinterpret_cast<const float4*>(src + u));
      x[u] = v.x * 256.f;
      x[u + 1] = v.y * 256.f;
      x[u + 2] = v.z * 256.f;
      x[u + 3] = v.w * 256.f;
    }
    const int row = 32 * (slot / kPer) + P * (slot % kPer);
#pragma unroll
    for (int p = 0; p < P; ++p) {
      uint32_t w[2];
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        w[u] = f32x2_to_e4m3x2(x[4 * u], x[4 * u + 1]) | (uint32_t)f32x2_to_e4m3x2(x[4 * u + 2], x[4 * u + 3]) << 16;
        float t[4];
        e4m3x4_to_f32(w[u], t);
#pragma unroll
        for (int i = 0; i < 4; ++i) x[4 * u + i] = (x[4 * u + i] - t[i]) * 16.f;  // (exact)
      }
      *reinterpret_cast<uint2*>(qs + at_chunk<D>(row + p, c >> 1) + 8 * (c & 1)) = make_uint2(w[0], w[1]);
    }
  }
  if constexpr (32 % P != 0) {
    for (int e = tid; e < groups * (32 % P) * CPR; e += 128) {
      const int r = e / CPR;
      *reinterpret_cast<uint4*>(qs + at_chunk<D>(32 * (r / (32 % P)) + P * kPer + r % (32 % P), e % CPR)) =
          make_uint4(0u, 0u, 0u, 0u);
    }
  }
}

// One CTA per range.
template <int D, int P>
__global__ void __launch_bounds__(kThreads, 2) cache_score_tc_kernel(const __grid_constant__ CUtensorMap map,
                                                                  const CacheScoreArgs a) {
  constexpr int kStages = Ring<D>::kStages, kPer = Pass<P>::kPer, kMost = Pass<P>::kMost;
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ Shared<D> sh;
  uint8_t* ring = sm100::align_smem_1024(smem);
  uint8_t* qs = ring + kRingBytes;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  pdl_trigger();
  // (the cache, its table and lengths are inputs of the call: only the group
  // means, the histogram and the status words are waited for)
  const int passes = (a.NQ + kMost - 1) / kMost;
  const int groups = ((passes > 1 ? kMost : a.NQ) + kPer - 1) / kPer;
  if (tid == 0) {
    for (int i = 0; i < kStages; ++i) {
      sm100::mbar_init(&sh.full[i], 32);
      sm100::mbar_init(&sh.empty[i], 1);
    }
    sm100::mbar_init(&sh.acc_full, 1);
    sm100::mbar_init(&sh.acc_empty, a.inject ? 5 : 4);  // (the hook: an arrival that never comes)
    sm100::mbar_init(&sh.b_ready, 4);
    sm100::mbar_init(&sh.done, 1);
    sh.abort = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  for (int i = tid; i < TOPK_HIST_BINS / 4; i += kThreads) reinterpret_cast<uint4*>(sh.hist)[i] = make_uint4(0u, 0u, 0u, 0u);
  if (warp == kLoadWarp)
    find_range(a.b * a.c.nkv, a.target, kSplitKeys, kStage, blockIdx.x, lane,
               [&](int i) { return scored_keys(a, i / a.c.nkv); },
               reinterpret_cast<int*>(ring), &sh.range);
  if (warp == kLoadWarp) sm100::fence_proxy_async_smem();  // (the ring's copies come behind the lengths)
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
  if (warp == kMmaWarp) {
    sm100::tmem_alloc(&sh.tmem, kTmemCols);
    sm100::tmem_relinquish();
  }
  sm100::tc_fence_before();
  __syncthreads();
  sm100::tc_fence_after();
  const uint32_t tmem = sh.tmem;
  const int nst = (k1 - k0 + kStage - 1) / kStage, total = nst * passes;

  if (warp == kLoadWarp) {
    load_rows<D>(a, map, sh, ring, lane, bi, j, k0, k1, passes);
  } else if (warp == kMmaWarp) {
    // the whole warp in step; one elected lane issues
    const uint32_t idesc_k = sm100::idesc_e4m3_f32(128, 128), idesc_q = sm100::idesc_e4m3_f32(128, 32 * groups);
    auto desc = [](uint32_t s) { return D == 128 ? sm100::sw128_desc(s, 16, 1024) : sm100::sw64_desc(s, 16, 512); };
    const uint32_t q0 = sm100::smem_u32(qs);
    bool alive = true;
    for (int it = 0; it < total && alive; ++it) {
      const int st = it % kStages;
      if (it % nst == 0) alive = sm100::mbar_wait_warp(&sh.b_ready, (it / nst) & 1, &sh.abort, a.wait_ns);
      if (alive) alive = sm100::mbar_wait_warp(&sh.full[st], (it / kStages) & 1, &sh.abort, a.wait_ns);
      if (alive && it > 0) alive = sm100::mbar_wait_warp(&sh.acc_empty, (it - 1) & 1, &sh.abort, a.wait_ns);
      if (!alive) break;
      sm100::tc_fence_after();
      const uint32_t k = sm100::smem_u32(ring + st * Ring<D>::kBytes);
#pragma unroll
      for (int kk = 0; kk < D / 32; ++kk) {
        sm100::umma_f8_ss_warp(tmem + 128u, desc(k + 32 * kk), desc(q0 + 32 * kk), idesc_q, kk > 0);
        sm100::umma_f8_ss_warp(tmem, desc(k + 32 * kk), desc(k + 32 * kk), idesc_k, kk > 0);
      }
      sm100::umma_commit_warp(&sh.empty[st]);
      sm100::umma_commit_warp(&sh.acc_full);
    }
    if (!alive && lane == 0) give_up(sh, a.status, 64);
    sm100::umma_commit_warp(&sh.done);
    if (!__all_sync(0xffffffffu, sm100::mbar_drain(&sh.done, 0, a.wait_ns)) && lane == 0) give_up(sh, a.status, 65);
    __syncwarp();
  } else {
    pdl_wait();
    const uint32_t acc = tmem + ((uint32_t)(warp * 32) << 16);
    for (int pass = 0, it = 0; pass < passes; ++pass) {
      // (every product of the pass before is done: its last accumulator was waited for)
      const int i0 = pass * kMost, nq = min(kMost, a.NQ - i0);
      stage_pieces<D, P>(a.Qg + (row * a.NQ + i0) * D, qs, nq, groups, tid);
      sm100::fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) sm100::mbar_arrive(&sh.b_ready);
      bool alive = true;
      for (int s = 0; s < nst; ++s, ++it) {
        alive = sm100::mbar_wait_warp(&sh.acc_full, it & 1, &sh.abort, a.wait_ns);
        if (!alive) {
          if (lane == 0) give_up(sh, a.status, 66);
          break;
        }
        sm100::tc_fence_after();
        float v[32];
        sm100::tmem_ld32(acc + 32 * warp, v);  // D_k of keys 32 warp .. of this warp's own
        sm100::tmem_wait_ld();
        // |k|^2: column `lane`
#pragma unroll
        for (int w = 16; w > 0; w >>= 1)
#pragma unroll
          for (int u = 0; u < w; ++u) v[u] = lane & w ? v[u + w] : v[u];
        const float n = v[0];
        float best = -INFINITY;
        for (int g = 0; g < groups; ++g) {
          sm100::tmem_ld32(acc + 128 + 32 * g, v);
          sm100::tmem_wait_ld();
#pragma unroll
          for (int i = 0; i < kPer; ++i) {
            float x = v[P * i + P - 1];
#pragma unroll
            for (int p = P - 2; p >= 0; --p) x = fmaf(x, 0.0625f, v[P * i + p]);
            best = fmaxf(best, x);
          }
        }
        sm100::tc_fence_before();
        __syncwarp();
        if (lane == 0) sm100::mbar_arrive(&sh.acc_empty);
        const int key = k0 + s * kStage + tid;
        if (key < k1) {
          // (rsqrt is within 2^-22; a key of zeros scores 0, one with a NaN -inf)
          float y = n > 0.f ? best * (1.f / 256.f) * rsqrtf(n) : n == 0.f ? 0.f : -INFINITY;
          float* S = a.S_agg + row * a.max_len + key;
          if (pass > 0) y = fmaxf(y, *S);  // (this thread's own score of the passes before)
          *S = y;
          if (pass == passes - 1) atomicAdd(&sh.hist[score_bin(y)], 1u);
        }
      }
      if (!alive) break;
    }
  }
  sm100::tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    sm100::tc_fence_after();
    sm100::tmem_dealloc(tmem, kTmemCols);
  }
  pdl_wait();  // (the loader's and the issuer's threads: the histogram's zeros)
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

template <int D, int P>
cudaError_t launch_typed(const CacheScoreArgs& args, cudaStream_t stream) {
  CacheScoreArgs a = args;
  const int64_t rows = (int64_t)a.b * a.c.nkv, ranges = range_grid(rows, a.max_len, kSplitCTAs, kSplitKeys);
  if (ranges > 0x7FFFFFFF) return cudaErrorNotSupported;
  a.target = (int)range_target(rows, kSplitCTAs);
  auto* kern = cache_score_tc_kernel<D, P>;
  const int groups = ((a.NQ < Pass<P>::kMost ? a.NQ : Pass<P>::kMost) + Pass<P>::kPer - 1) / Pass<P>::kPer;
  const size_t smem = (size_t)kRingBytes + (size_t)32 * groups * D + 1024;
  // (the same bound in every call: another thread's launch may come in between)
  const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             kRingBytes + 32 * kMaxGroups * D + 1024);
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

cudaError_t launch_cache_score_tc(int d, const CacheScoreArgs& a, cudaStream_t stream) {
  if (a.NQ <= Pass<5>::kMost) return d == 128 ? launch_typed<128, 5>(a, stream) : launch_typed<64, 5>(a, stream);
  return d == 128 ? launch_typed<128, 4>(a, stream) : launch_typed<64, 4>(a, stream);
}

}  // namespace quoka

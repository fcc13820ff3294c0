// GQA attention over the paged 8-bit cache straight from its codes: decode steps
// and short blocks (G * BCP <= 32 query rows per KV head), and all fp32 queries.
//
// [QUOKA §4.2, problem 3] the attention of the other paths,
//   O[b,h,t] = sum_k softmax_k(scale * q . k) v,  j = floor(h / G),
// over the cached keys of the sequence (all of them, or those of an index
// list) and the chunk's own keys Kc[b, j, s], s <= t.
//
// Mathematics. With key codes c_k in a page of scale 2^ek, value codes u_k in
// one of 2^ev, and s_k = scale * log2(e) * 2^ek (q . c_k):
//   O = sum_k 2^(s_k) 2^ev u_k / sum_k 2^(s_k)
//     = sum_k w_k u_k / sum_k w_k 2^-ev,   w_k = 2^(s_k + ev - M),
// M a running reference near the maximum of s_k + ev over the row. One pass,
// one exponential a key; the value scales only shift exponents, and no weight
// that meets the tensor core exceeds 2^kLazy whatever the scales are. The
// denominator is summed in fp32, where 2^-ev cannot overflow (|e| <= 50).
//
// Precision. e4m3 codes are exact in fp16. A query row is scaled by a power of
// two so that its largest element lies in [2^13, 2^14): a bf16 row is then
// exact in fp16 down to 2^-28 of its largest element and within 2^-39 of it
// below. fp32 rows are split into two halves (22 bits), and so are their
// weights; with bf16 rows a weight is rounded to fp16 once (2^-11 of it, finer
// than the bf16 output). Products accumulate in fp32.
//
// Work split. The keys of every (sequence, KV head) are cut into ranges of
// near equal length, so many in all as CTAs are resident at once, one CTA
// each: every CTA reads all lengths and finds its own range. A loader warp
// looks the rows up (list entry, page, scales: each a stage ahead of the next,
// so that no lookup is waited for) and copies 128 keys at a time into a ring of
// stages: listed rows with cp.async, runs of keys by boxes of up to 64 with
// TMA; a row that is not there reads as zeros. Four warps compute (and copy the
// first stage of listed rows: a CTA may have no other). They
// share the query tiles (8 rows, or 16 where there are more) and take a
// stage's 32-key steps in turn.
// Keys are the rows of the first product S^T = K Q^T, columns of the head those
// of the second, O^T = V^T P^T, so that few query rows fill its 8 columns.
// Codes go from shared memory straight into the operand layouts of mma.sync:
// for K Q^T the columns of a k-step may be any 16 as long as Q is permuted
// alike, so lane (g, t) reads the 16-byte chunks t and t + 4 of a key's row;
// V^T needs 4 keys of a lane and any columns, so lane (g, t) reads the columns
// [16 g, 16 g + 16) of four keys; P is transposed between the two by
// movmatrix. Chunk c of row r lies at c ^ (r & 7), and operand row n of a step
// stands for key n ^ 4 (n & 1), so that neither read has a bank conflict
// (d = 128; d = 64 keeps a two-way one on V). A second kernel joins the ranges
// of every query row and adds the chunk's own keys in fp32.
// Bound by the cache's bytes, each read once per 64 query rows. Measured: a
// decode step of 32 ragged sequences of up to 8192 keys, 32 query and 8 KV heads,
// d = 128: 61.5 us for 337.9 MB, 5.5 TB/s, and 6 us for the join (187 us when every
// warp loaded its own fragments from global memory, 76.6 with a cp.async ring);
// the products left out of that kernel, it took 66 us. One sequence of 4096
// listed keys: 8.4 us a call, a chain of count, list, table, rows (9.7 when the
// loader alone fetched the first stage and a warp took a query row at a time).
#include <algorithm>

#include "cache.cuh"
#include "sm100.cuh"
#include "tmap.cuh"

namespace quoka {

namespace {

using namespace cache;

constexpr int kThreads = 160;      // four computing warps and the loader
constexpr int kStep = 32;          // keys of one step of a warp: two operand tiles
constexpr int kStage = 128;        // keys of a stage of the ring
constexpr int kStages = 2;
// M is set kHead below the row maximum and may lag it by kLazy: weights then
// stay below 2^15 (fp16 holds 65504), and one that fp16 holds as a subnormal
// is off by at most 2^-25, 2^-32 of the row's largest.
constexpr float kHead = 7.f, kLazy = 15.f;
constexpr int kSplitKeys = 128;    // a range has at least this many keys
constexpr int kBlockRows = 64;     // query rows of a CTA
constexpr int kMaxParts = 444;     // ranges of a row: at most the ranges asked for
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

__device__ __forceinline__ uint32_t pack_h2(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
// what fp16 left of (lo, hi), again in fp16
__device__ __forceinline__ uint32_t rest_h2(float lo, float hi, uint32_t h) {
  const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
  return pack_h2(lo - f.x, hi - f.y);
}

// 8 x 8 halves, a row's pairs over four lanes: transposed.
__device__ __forceinline__ uint32_t transpose_8x8(uint32_t x) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}

// Shared memory: the query fragments [8-row tiles][D / 16][32 lanes] of two
// words (four for fp32 rows: hi, lo) and the rows' factors, behind the stages of
// codes (keys, then values; aligned to 1024 bytes). After the loop the warps'
// outputs [4][8 RT][D] fp32 and their (M, l) [4][8 RT][2] lie over the stages.
template <int D>
struct Ring {
  static constexpr int kBytes = kStage * D;   // codes of a stage's keys (or values)
  static constexpr int kPitch = 2 * kBytes;   // a stage
  static constexpr int kTotal = kStages * kPitch;
  static_assert(kTotal >= 4 * 16 * D * 4 + 4 * 16 * 2 * 4, "the join's scratch lies over the ring");
};
template <int D, int SPLIT>
constexpr size_t smem_bytes(int tiles8) {
  return (size_t)tiles8 * (D / 16) * 32 * 8 * SPLIT + (size_t)tiles8 * 32 + Ring<D>::kTotal + 1024;
}

struct Shared {
  uint64_t full[kStages], empty[kStages];
  uint32_t ex[kStages][kStage];  // scale exponents: ek + 64 in the low half, ev + 64 in the high
  int abort, fault, site;
  Range range;  // this CTA's
};

// Keys of row `row` = sequence * nkv + head.
template <bool IDX>
__device__ __forceinline__ int row_keys(const CacheAttnArgs& a, int row) {
  if (IDX) return min(max(__ldcg(a.kv_count + row), 0), a.N);
  return min(max(__ldcg(a.c.seq_len + row / a.c.nkv), 0), a.max_len);
}

struct Maps {
  CUtensorMap k, v;  // the pools (only read without an index list)
};

// The loader warp: rows [k0, k1) of the (sequence, head), 128 at a time.
// Listed rows are copied one by one with cp.async; without a list a run of keys
// is copied by boxes of one page each with TMA (rows behind k1 then come along).
template <int D, bool IDX>
__device__ __forceinline__ void load_rows(const CacheAttnArgs& a, const Maps& maps, Shared& sh, uint8_t* ring, int lane,
                                          int bi, int j, int len, int k0, int k1) {
  using R = Ring<D>;
  constexpr int CPR = D / 16;           // 16-byte chunks of a row
  constexpr int RPI = 32 / CPR;         // rows a warp-wide copy covers
  constexpr int NU = IDX ? 4 : 1;       // keys (or boxes) a lane looks up
  const int64_t kvrow = (int64_t)bi * a.c.nkv + j;
  const int plog = a.c.page_log2, pmask = (1 << plog) - 1, blog = box_log2(a.c);
  const int32_t* table = a.c.page_table + (int64_t)bi * a.c.table_stride;
  const int nst = (k1 - k0 + kStage - 1) / kStage;
  bool bad = false;
  // this lane's slot u of stage s: key lane + 32 u of a list; without a list,
  // the first key of box `lane`. -1: absent.
  auto key_of = [&](int s, int u) { return k0 + s * kStage + (IDX ? lane + 32 * u : lane << blog); };
  auto here = [&](int s, int u) { return key_of(s, u) < k1 && (IDX || (lane << blog) < kStage); };
  auto tau_of = [&](int s, int u) {
    if (!here(s, u)) return -1;
    if constexpr (IDX) return __ldcg(a.kv_idx + kvrow * a.N + key_of(s, u));
    return key_of(s, u);
  };
  auto page_of = [&](int tau) {
    if (tau < 0 || tau >= len) return -1;
    return __ldcg(table + (tau >> plog));
  };
  auto held = [&](int p) { return p >= 0 && p < a.c.npages; };
  int s = IDX ? 1 : 0;  // (listed rows: the computing warps load stage 0)
  int tau[3][NU], pg[2][NU];
  float ks[NU], vs[NU];
#pragma unroll
  for (int u = 0; u < NU; ++u) {
    ks[u] = vs[u] = 1.f;
#pragma unroll
    for (int i = 0; i < 3; ++i) tau[i][u] = tau_of(s + i, u);
    pg[0][u] = page_of(tau[0][u]);
    pg[1][u] = page_of(tau[1][u]);
    if (held(pg[0][u])) {
      ks[u] = __ldcg(a.c.k_scale + (int64_t)pg[0][u] * a.c.nkv + j);
      vs[u] = __ldcg(a.c.v_scale + (int64_t)pg[0][u] * a.c.nkv + j);
    }
  }
  for (; s < nst; ++s) {
    // the lookups of the stages to come
    int tau3[NU], pg2[NU];
    float ks1[NU], vs1[NU];
#pragma unroll
    for (int u = 0; u < NU; ++u) {
      ks1[u] = vs1[u] = 1.f;
      tau3[u] = tau_of(s + 3, u);
      pg2[u] = page_of(tau[2][u]);
      if (held(pg[1][u])) {
        ks1[u] = __ldcg(a.c.k_scale + (int64_t)pg[1][u] * a.c.nkv + j);
        vs1[u] = __ldcg(a.c.v_scale + (int64_t)pg[1][u] * a.c.nkv + j);
      }
    }
    const int st = s % kStages;
    if (s >= kStages && !__all_sync(0xffffffffu, sm100::mbar_wait(&sh.empty[st], (s / kStages - 1) & 1, &sh.abort, a.wait_ns))) {
      if (lane == 0) {
        sh.abort = 1;
        sh.fault = 5;  // QUOKA_ERR_TIMEOUT
        sh.site = 61;
      }
      break;
    }
    const uint32_t dst = sm100::smem_u32(ring + st * R::kPitch);
    // the copies first: the scales may still be on their way
    if constexpr (IDX) {
      int64_t off[NU];
#pragma unroll
      for (int u = 0; u < NU; ++u)
        off[u] = held(pg[0][u]) ? pg[0][u] * a.c.sp + (int64_t)(tau[0][u] & pmask) * a.c.sr : -1;
      const int c = lane % CPR, r0 = lane / CPR;
      const uint8_t* kb = a.c.k + j * a.c.sh + 16 * c;
      const uint8_t* vb = a.c.v + j * a.c.sh + 16 * c;
#pragma unroll
      for (int i = 0; i < kStage / RPI; ++i) {
        const int r = i * RPI + r0;
        const int64_t o = __shfl_sync(0xffffffffu, off[i * RPI / 32], r & 31);
        const int64_t so = o >= 0 ? o : 0;
        const uint32_t n = o >= 0 ? 16u : 0u, at = at_chunk<D>(r, c);
        sm100::cp_async_16(dst + at, kb + so, n);
        sm100::cp_async_16(dst + R::kBytes + at, vb + so, n);
      }
      sm100::cp_async_arrive_noinc(&sh.full[st]);
    } else if (here(s, 0)) {
      const uint32_t at = dst + ((lane << blog) * D);
      // (a page that is not there lies out of bounds: zeros)
      const int p = held(pg[0][0]) ? pg[0][0] : a.c.npages, r = tau[0][0] & pmask;
      sm100::mbar_expect_tx(&sh.full[st], 2u * D << blog);
      sm100::tma_load_4d(at, &maps.k, &sh.full[st], 0, r, j, p);
      sm100::tma_load_4d(at + R::kBytes, &maps.v, &sh.full[st], 0, r, j, p);
    }
    __syncwarp();
    uint32_t* ex = sh.ex[st];
    uint32_t e[NU];
#pragma unroll
    for (int u = 0; u < NU; ++u) {
      int ek = 0, ev = 0;
      if (held(pg[0][u])) {
        ek = scale_exp(ks[u], &bad);
        ev = scale_exp(vs[u], &bad);
      } else {
        bad |= here(s, u);  // reads as zeros
      }
      e[u] = (uint32_t)(ek + 64) | (uint32_t)(ev + 64) << 16;
    }
#pragma unroll
    for (int i = 0; i < kStage / 32; ++i)
      ex[lane + 32 * i] = IDX ? e[i % NU] : __shfl_sync(0xffffffffu, e[0], (lane + 32 * i) >> blog);
    sm100::mbar_arrive(&sh.full[st]);  // (releases the exponents)
#pragma unroll
    for (int u = 0; u < NU; ++u) {
      tau[0][u] = tau[1][u];
      tau[1][u] = tau[2][u];
      tau[2][u] = tau3[u];
      pg[0][u] = pg[1][u];
      pg[1][u] = pg2[u];
      ks[u] = ks1[u];
      vs[u] = vs1[u];
    }
  }
  if constexpr (IDX) {
    sm100::cp_async_commit();
    sm100::cp_async_wait<0>();
  } else {  // no copy may be in flight when the CTA goes on, even if a wait gave up
    for (int i = max(0, s - kStages); i < s; ++i) sm100::mbar_drain(&sh.full[i % kStages], (i / kStages) & 1, a.wait_ns);
  }
  if (__any_sync(0xffffffffu, bad) && lane == 0 && sh.fault == 0) sh.fault = 6;  // QUOKA_ERR_BOUNDS
}

// Stage 0 of listed rows, by the four computing warps, 32 rows each: their chain
// index -> page -> row is the longest of a CTA with few keys, and one warp would
// take as long again to issue the copies. Returns the stages there are (the
// caller waits for its copies, and at a barrier for those of the others).
template <int D>
__device__ __forceinline__ int load_first(const CacheAttnArgs& a, Shared& sh, uint8_t* ring, int warp, int lane, int bi,
                                          int j, int k0, int k1) {
  using R = Ring<D>;
  constexpr int CPR = D / 16, RPI = 32 / CPR;
  if (k0 >= k1) return 0;
  const int key = k0 + 32 * warp + lane;
  const bool here = key < k1;
  int tau = -1, p = -1;
  if (here) tau = __ldcg(a.kv_idx + ((int64_t)bi * a.c.nkv + j) * a.N + key);
  const int len = min(max(__ldcg(a.c.seq_len + bi), 0), a.max_len);
  if (tau >= 0 && tau < len) p = __ldcg(a.c.page_table + (int64_t)bi * a.c.table_stride + (tau >> a.c.page_log2));
  const bool held = p >= 0 && p < a.c.npages;
  int64_t off = -1;
  float ks = 1.f, vs = 1.f;
  if (held) {
    ks = __ldcg(a.c.k_scale + (int64_t)p * a.c.nkv + j);
    vs = __ldcg(a.c.v_scale + (int64_t)p * a.c.nkv + j);
    off = p * a.c.sp + (int64_t)(tau & ((1 << a.c.page_log2) - 1)) * a.c.sr;
  }
  const int c = lane % CPR, r0 = lane / CPR;
  const uint8_t* kb = a.c.k + j * a.c.sh + 16 * c;
  const uint8_t* vb = a.c.v + j * a.c.sh + 16 * c;
  const uint32_t dst = sm100::smem_u32(ring);
#pragma unroll
  for (int i = 0; i < 32 / RPI; ++i) {
    const int r = i * RPI + r0;
    const int64_t o = __shfl_sync(0xffffffffu, off, r);
    const int64_t so = o >= 0 ? o : 0;
    const uint32_t n = o >= 0 ? 16u : 0u, at = at_chunk<D>(32 * warp + r, c);
    sm100::cp_async_16(dst + at, kb + so, n);
    sm100::cp_async_16(dst + R::kBytes + at, vb + so, n);
  }
  bool bad = here && !held;  // (reads as zeros)
  const int ek = held ? scale_exp(ks, &bad) : 0, ev = held ? scale_exp(vs, &bad) : 0;
  sh.ex[0][32 * warp + lane] = (uint32_t)(ek + 64) | (uint32_t)(ev + 64) << 16;
  if (__any_sync(0xffffffffu, bad) && lane == 0) sh.fault = 6;  // QUOKA_ERR_BOUNDS
  return (k1 - k0 + kStage - 1) / kStage;
}

// 16 elements of a query row.
__device__ __forceinline__ void load_row16(const bf16* q, float (&x)[16]) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint4 w = __ldg(reinterpret_cast<const uint4*>(q) + i);
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      x[8 * i + 2 * k] = __uint_as_float(u[k] << 16);
      x[8 * i + 2 * k + 1] = __uint_as_float(u[k] & 0xFFFF0000u);
    }
  }
}
__device__ __forceinline__ void load_row16(const float* q, float (&x)[16]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float4 w = __ldg(reinterpret_cast<const float4*>(q) + i);
    x[4 * i] = w.x;
    x[4 * i + 1] = w.y;
    x[4 * i + 2] = w.z;
    x[4 * i + 3] = w.w;
  }
}

// One CTA per range and block of 64 query rows. RT: 8-row query tiles of a warp.
template <typename T, int D, bool IDX, int RT>
__global__ void __launch_bounds__(kThreads, RT == 1 ? 3 : 2)
cache_slice_kernel(const __grid_constant__ Maps maps, const CacheAttnArgs a) {
  constexpr int SPLIT = sizeof(T) == 2 ? 1 : 2;
  constexpr int KS = D / 16;  // k-steps of K Q^T, and row tiles of O^T
  using Rg = Ring<D>;
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ Shared sh;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t4 = lane & 3;
  const int G = a.nq / a.c.nkv, R = G * a.BCP;
  const int blocks = (R + kBlockRows - 1) / kBlockRows, range = blockIdx.x / blocks;
  const int rb = (int)blockIdx.x % blocks * kBlockRows, Rb = min(R - rb, kBlockRows);  // this block's rows
  const int tiles = RT == 1 || R <= 16 ? 1 : R <= 32 ? 2 : 4;  // (a third tile alone would leave a warp idle as well)
  uint8_t* ring = sm100::align_smem_1024(smem);
  uint32_t* qs = reinterpret_cast<uint32_t*>(ring + Rg::kTotal);
  float* rowf = reinterpret_cast<float*>(ring + Rg::kTotal + (size_t)tiles * RT * KS * 32 * 8 * SPLIT);
  pdl_trigger();
  clear_status(a.status);  // (the faults of this kernel are latched by the next)
  if (tid == 0) {
    for (int i = 0; i < kStages; ++i) {
      sm100::mbar_init(&sh.full[i], IDX ? 64 : 32);
      sm100::mbar_init(&sh.empty[i], a.inject && i == 0 ? 5 : 4);  // (the hook: an arrival that never comes)
    }
    sh.abort = sh.fault = sh.site = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 4)
    find_range(a.b * a.c.nkv, a.target, kSplitKeys, 64, range, lane, [&](int row) { return row_keys<IDX>(a, row); },
               reinterpret_cast<int*>(ring), &sh.range);
  if (warp == 4) sm100::fence_proxy_async_smem();  // (the ring's copies come behind the lengths)
  __syncthreads();
  const int row = sh.range.row, k0 = sh.range.k0, k1 = sh.range.k1;
  if (row < 0) return;
  if (tid == 0 && rb == 0 && range == sh.range.first)
    a.row_parts[row] = make_int2(sh.range.first, sh.range.parts);
  const int bi = row / a.c.nkv, j = row % a.c.nkv;

  float o[RT][KS][4];
#pragma unroll
  for (int rt = 0; rt < RT; ++rt)
#pragma unroll
    for (int i = 0; i < KS; ++i) o[rt][i][0] = o[rt][i][1] = o[rt][i][2] = o[rt][i][3] = 0.f;
  float m[RT][2], l[RT][2];  // query rows 2 t, 2 t + 1 of each tile
#pragma unroll
  for (int rt = 0; rt < RT; ++rt) {
    m[rt][0] = m[rt][1] = -INFINITY;
    l[rt][0] = l[rt][1] = 0.f;
  }
  const int kgroups = 4 / tiles, tile = warp % tiles, kg = warp / tiles;  // (computing warps)

  if (warp == 4) {
    const int want = __ldcg(a.c.seq_len + bi), len = min(max(want, 0), a.max_len);
    if (want != len && lane == 0) sh.fault = 6;  // QUOKA_ERR_BOUNDS
    load_rows<D, IDX>(a, maps, sh, ring, lane, bi, j, len, k0, k1);
  } else {
    const int nst0 = IDX ? load_first<D>(a, sh, ring, warp, lane, bi, j, k0, k1) : 0;
    // ---- query rows: row r is head j G + (rb + r) / BCP, chunk position (rb + r) % BCP. A
    // lane takes a 16-column chunk of a row, a warp RPW rows at a time.
    constexpr int CPR = D / 16, RPW = 32 / CPR;
    const int ch = lane % CPR;
    for (int r = RPW * warp + lane / CPR; r < tiles * RT * 8; r += 4 * RPW) {
      float x[16];
      if (r < Rb) {
        const int h = (rb + r) / a.BCP, t = rb + r - h * a.BCP;
        const T* q = static_cast<const T*>(a.Q.data) + bi * a.Q.sb + (int64_t)(j * G + h) * a.Q.sh + (int64_t)t * a.Q.st;
        load_row16(q + 16 * ch, x);
      } else {
#pragma unroll
        for (int i = 0; i < 16; ++i) x[i] = 0.f;
      }
      float top = 0.f;
#pragma unroll
      for (int i = 0; i < 16; ++i) top = fmaxf(top, fabsf(x[i]));
#pragma unroll
      for (int o_ = CPR / 2; o_ > 0; o_ >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o_));
      int e = (int)(__float_as_uint(top) >> 23) - 127 - 13;  // top * 2^-e lies in [2^13, 2^14)
      e = min(max(e, -100), 114);                            // (zero and tiny rows, infinities)
      const float f = exp2i(-e);
      if (ch == 0) rowf[r] = exp2i(e) * a.scale * kLog2e;
      // word w of chunk ch belongs to k-step 4 (ch / 4) + w and lane 4 (r % 8) + ch % 4
      uint32_t* dst = qs + (((r >> 3) * KS + 4 * (ch >> 2)) * 32 + (r & 7) * 4 + (ch & 3)) * (2 * SPLIT);
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        const float y0 = x[4 * w] * f, y1 = x[4 * w + 1] * f, y2 = x[4 * w + 2] * f, y3 = x[4 * w + 3] * f;
        const uint32_t h0 = pack_h2(y0, y1), h1 = pack_h2(y2, y3);
        if constexpr (SPLIT == 2)
          *reinterpret_cast<uint4*>(dst + w * 32 * 4) = make_uint4(h0, h1, rest_h2(y0, y1, h0), rest_h2(y2, y3, h1));
        else
          *reinterpret_cast<uint2*>(dst + w * 32 * 2) = make_uint2(h0, h1);
      }
    }
    if (nst0 > 0) {  // the first stage's copies, which this warp issued
      sm100::cp_async_commit();
      sm100::cp_async_wait<0>();
    }
    sm100::named_barrier_sync(1, 128);
    float f[RT][2];
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
      f[rt][0] = rowf[(tile * RT + rt) * 8 + 2 * t4];
      f[rt][1] = rowf[(tile * RT + rt) * 8 + 2 * t4 + 1];
    }
    const uint32_t* qt = qs + ((size_t)tile * RT * KS * 32 + lane) * (2 * SPLIT);
    const int gk = g ^ ((g & 1) << 2);             // this lane's key of an operand tile (and gk + 8)
    const int v0 = 2 * t4, v1 = (2 * t4 + 1) ^ 4;  // its keys of V^T P^T: v0, v1, v0 + 8, v1 + 8

    auto compute = [&](const uint8_t* stage, const uint32_t* exs, int row0, int left) {
      const uint8_t* kr = stage + row0 * D;
      const uint8_t* vr = kr + Rg::kBytes;
      const uint32_t* ex = exs + row0;
      // ---- S^T: c[y][rt]: keys gk, gk + 8 of tile y by rows 2 t, 2 t + 1
      float c[2][RT][4];
#pragma unroll
      for (int y = 0; y < 2; ++y)
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) c[y][rt][0] = c[y][rt][1] = c[y][rt][2] = c[y][rt][3] = 0.f;
#pragma unroll
      for (int h = 0; h < D / 64; ++h) {
        uint4 kw[2][2];
#pragma unroll
        for (int y = 0; y < 2; ++y)
#pragma unroll
          for (int u = 0; u < 2; ++u)
            kw[y][u] = *reinterpret_cast<const uint4*>(kr + at_chunk<D>(16 * y + gk + 8 * u, t4 + 4 * h));
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          uint32_t qb[RT][2 * SPLIT];
#pragma unroll
          for (int rt = 0; rt < RT; ++rt) {
            const uint32_t* q = qt + (rt * KS + 4 * h + w) * 32 * (2 * SPLIT);
            if constexpr (SPLIT == 2) {
              const uint4 x = *reinterpret_cast<const uint4*>(q);
              qb[rt][0] = x.x; qb[rt][1] = x.y; qb[rt][2] = x.z; qb[rt][3] = x.w;
            } else {
              const uint2 x = *reinterpret_cast<const uint2*>(q);
              qb[rt][0] = x.x; qb[rt][1] = x.y;
            }
          }
#pragma unroll
          for (int y = 0; y < 2; ++y) {
            const uint32_t w0 = reinterpret_cast<const uint32_t*>(&kw[y][0])[w];
            const uint32_t w1 = reinterpret_cast<const uint32_t*>(&kw[y][1])[w];
            const uint32_t ka[4] = {e4m3x2_to_f16x2((uint16_t)w0), e4m3x2_to_f16x2((uint16_t)w1),
                                    e4m3x2_to_f16x2((uint16_t)(w0 >> 16)), e4m3x2_to_f16x2((uint16_t)(w1 >> 16))};
#pragma unroll
            for (int rt = 0; rt < RT; ++rt) {
              mma_f16(c[y][rt], ka, qb[rt][0], qb[rt][1]);
              if constexpr (SPLIT == 2) mma_f16(c[y][rt], ka, qb[rt][2], qb[rt][3]);
            }
          }
        }
      }
      // ---- scores in log2 units, with the value scale's exponent added
      float x[RT][2], inv[2][2];  // row maxima; 2^-ev of the lane's keys
#pragma unroll
      for (int rt = 0; rt < RT; ++rt) x[rt][0] = x[rt][1] = -INFINITY;
#pragma unroll
      for (int y = 0; y < 2; ++y)
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const int key = 16 * y + gk + 8 * u;
          const uint32_t e = ex[key];
          const float ks = exp2i((int)(e & 0xFFFFu) - 64);
          const int ev = (int)(e >> 16) - 64;
          inv[y][u] = exp2i(-ev);
          const bool there = key < left;
#pragma unroll
          for (int rt = 0; rt < RT; ++rt)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              float& s_ = c[y][rt][2 * u + i];
              s_ = there ? fmaf(s_ * f[rt][i], ks, (float)ev) : -INFINITY;
              x[rt][i] = fmaxf(x[rt][i], s_);
            }
        }
      bool rise = false;
#pragma unroll
      for (int rt = 0; rt < RT; ++rt)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
#pragma unroll
          for (int d = 4; d < 32; d <<= 1) x[rt][i] = fmaxf(x[rt][i], __shfl_xor_sync(0xffffffffu, x[rt][i], d));
          rise = rise || x[rt][i] > m[rt][i] + kLazy;
        }
      if (__any_sync(0xffffffffu, rise)) {
#pragma unroll
        for (int rt = 0; rt < RT; ++rt)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const float n = fmaxf(m[rt][i], x[rt][i] - kHead);
            const float r = m[rt][i] == -INFINITY ? 0.f : exp2f(m[rt][i] - n);
            m[rt][i] = n;
            l[rt][i] *= r;
#pragma unroll
            for (int k = 0; k < KS; ++k) {
              o[rt][k][i] *= r;
              o[rt][k][2 + i] *= r;
            }
          }
      }
      // ---- P^T as the second product's operand
      uint32_t pb[2][RT][2 * SPLIT];
#pragma unroll
      for (int rt = 0; rt < RT; ++rt) {
        const float b0 = m[rt][0] == -INFINITY ? 0.f : m[rt][0], b1 = m[rt][1] == -INFINITY ? 0.f : m[rt][1];
#pragma unroll
        for (int y = 0; y < 2; ++y)
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            const float p0 = sm100::ex2(c[y][rt][2 * u] - b0), p1 = sm100::ex2(c[y][rt][2 * u + 1] - b1);
            l[rt][0] = fmaf(p0, inv[y][u], l[rt][0]);
            l[rt][1] = fmaf(p1, inv[y][u], l[rt][1]);
            const uint32_t hi = pack_h2(p0, p1);
            pb[y][rt][u] = transpose_8x8(hi);
            if constexpr (SPLIT == 2) pb[y][rt][2 + u] = transpose_8x8(rest_h2(p0, p1, hi));
          }
      }
      // ---- O^T += V^T P^T: row tile i holds columns 2 i, 2 i + 1 of every lane's chunk
#pragma unroll
      for (int y = 0; y < 2; ++y) {
        uint32_t vw[4][D / 32];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int r = 16 * y + (i & 1 ? v1 : v0) + 8 * (i >> 1);
          if constexpr (D == 128) {
            const uint4 w = *reinterpret_cast<const uint4*>(vr + at_chunk<D>(r, g));
            vw[i][0] = w.x;
            vw[i][1] = w.y;
            vw[i][2] = w.z;
            vw[i][3] = w.w;
          } else {
            const uint2 w = *reinterpret_cast<const uint2*>(vr + at_chunk<D>(r, g >> 1) + 8 * (g & 1));
            vw[i][0] = w.x;
            vw[i][1] = w.y;
          }
          if (!IDX && left < kStep && r >= left) {  // (a row behind the range may hold a NaN)
#pragma unroll
            for (int w = 0; w < D / 32; ++w) vw[i][w] = 0u;
          }
        }
#pragma unroll
        for (int k = 0; k < KS; ++k) {
          const uint32_t sel = k & 1 ? 0x7362 : 0x5140;  // bytes 2 (k % 2), 2 (k % 2) + 1 of both keys
          const uint32_t lo = __byte_perm(vw[0][k >> 1], vw[1][k >> 1], sel);
          const uint32_t hi = __byte_perm(vw[2][k >> 1], vw[3][k >> 1], sel);
          const uint32_t va[4] = {e4m3x2_to_f16x2((uint16_t)lo), e4m3x2_to_f16x2((uint16_t)(lo >> 16)),
                                  e4m3x2_to_f16x2((uint16_t)hi), e4m3x2_to_f16x2((uint16_t)(hi >> 16))};
#pragma unroll
          for (int rt = 0; rt < RT; ++rt) {
            mma_f16(o[rt][k], va, pb[y][rt][0], pb[y][rt][1]);
            if constexpr (SPLIT == 2) mma_f16(o[rt][k], va, pb[y][rt][2], pb[y][rt][3]);
          }
        }
      }
    };

    const int nst = (k1 - k0 + kStage - 1) / kStage;
    for (int i = 0; i < nst; ++i) {
      const int st = i % kStages;
      // (of listed rows stage 0 is there: slot 0 is filled by the loader one time less)
      const uint32_t parity = (i / kStages - (IDX && st == 0 ? 1 : 0)) & 1;
      if ((!IDX || i > 0) && !__all_sync(0xffffffffu, sm100::mbar_wait(&sh.full[st], parity, &sh.abort, a.wait_ns))) {
        if (lane == 0) {
          sh.abort = 1;
          sh.fault = 5;  // QUOKA_ERR_TIMEOUT
          sh.site = 62;
        }
        break;
      }
      const int left = k1 - k0 - i * kStage;
      for (int r = kg * kStep; r < min(left, kStage); r += kgroups * kStep)
        compute(ring + st * Rg::kPitch, sh.ex[st], r, left - r);
      __syncwarp();
      if (lane == 0) sm100::mbar_arrive(&sh.empty[st]);
    }
  }

  // ---- join the warps of each query tile
  __syncthreads();  // the ring is no longer read, and no copy into it is in flight
  constexpr int TR = 8 * RT;                   // rows of a warp's tile
  float* os = reinterpret_cast<float*>(ring);  // [4 warps][TR][D]
  float* ml = os + 4 * TR * D;                 // [4][TR][2]
  if (warp < 4) {
#pragma unroll
    for (int rt = 0; rt < RT; ++rt)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
#pragma unroll
        for (int d = 4; d < 32; d <<= 1) l[rt][i] += __shfl_xor_sync(0xffffffffu, l[rt][i], d);
        const int r = 8 * rt + 2 * t4 + i;
        if (g == 0) {
          ml[(warp * TR + r) * 2] = m[rt][i];
          ml[(warp * TR + r) * 2 + 1] = l[rt][i];
        }
        if (tile * TR + r < Rb) {  // columns [D / 8 * g, + D / 8)
          float4* dst = reinterpret_cast<float4*>(os + (warp * TR + r) * D + D / 8 * g);
#pragma unroll
          for (int k = 0; k < KS; k += 2)
            dst[k / 2] = make_float4(o[rt][k][i], o[rt][k][2 + i], o[rt][k + 1][i], o[rt][k + 1][2 + i]);
        }
      }
  }
  __syncthreads();
  for (int e = tid; e < Rb * (D / 4); e += kThreads) {
    const int r = e / (D / 4), c4 = e % (D / 4);
    const int tl = r / TR, rr = r % TR;
    // (all four groups' loads together; a group that is not there repeats the last one's)
    float mk[4], lk[4], M = -INFINITY;
    float4 y[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int w = (min(k, kgroups - 1) * tiles + tl) * TR + rr;
      mk[k] = ml[w * 2];
      lk[k] = k < kgroups ? ml[w * 2 + 1] : 0.f;
      y[k] = *reinterpret_cast<const float4*>(os + w * D + 4 * c4);
      M = fmaxf(M, mk[k]);
    }
    float L = 0.f;
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if (lk[k] == 0.f) continue;  // the warp saw no key (not so for NaN scores: they come through)
      const float fw = exp2f(mk[k] - M);
      L = fmaf(fw, lk[k], L);
      x.x = fmaf(fw, y[k].x, x.x);
      x.y = fmaf(fw, y[k].y, x.y);
      x.z = fmaf(fw, y[k].z, x.z);
      x.w = fmaf(fw, y[k].w, x.w);
    }
    const float inv = L != 0.f ? 1.f / L : 0.f;
    const int64_t at = (int64_t)range * R + rb + r;
    *reinterpret_cast<float4*>(a.O_parts + at * D + 4 * c4) = make_float4(x.x * inv, x.y * inv, x.z * inv, x.w * inv);
    // log2 of the range's partition function (-inf: no key)
    if (c4 == 0) a.lse_parts[at] = L != 0.f ? M + log2f(L) : -INFINITY;
  }
  if (tid == 0) a.faults[blockIdx.x] = sh.fault | sh.site << 8;
}

// Joins the ranges of one query row, adds the chunk's own keys s <= t, and
// writes the row: O = sum_i 2^(x_i - X) O_i, X = log2 sum_i 2^(x_i). One CTA
// per row: a thread owns four columns of every kGroups-th range and chunk
// key. The first ranges' outputs are fetched together with all sums, so that
// a row usually costs one round of loads.
__device__ __forceinline__ float4 ld4(const float* p) { return __ldg(reinterpret_cast<const float4*>(p)); }
__device__ __forceinline__ float4 ld4(const bf16* p) {
  const uint2 w = __ldg(reinterpret_cast<const uint2*>(p));
  return make_float4(__uint_as_float(w.x << 16), __uint_as_float(w.x & 0xFFFF0000u), __uint_as_float(w.y << 16),
                     __uint_as_float(w.y & 0xFFFF0000u));
}
__device__ __forceinline__ void st4(float* p, float4 v) { *reinterpret_cast<float4*>(p) = v; }
__device__ __forceinline__ void st4(bf16* p, float4 v) {
  uint2 o;
  __nv_bfloat162* h = reinterpret_cast<__nv_bfloat162*>(&o);
  h[0] = __floats2bfloat162_rn(v.x, v.y);
  h[1] = __floats2bfloat162_rn(v.z, v.w);
  *reinterpret_cast<uint2*>(p) = o;
}

// MT threads.
template <typename T, int D, int MT>
__global__ void __launch_bounds__(MT) cache_merge_kernel(const CacheAttnArgs a) {
  constexpr int C4 = D / 4, kGroups = MT / C4, kWarps = MT / 32;
  constexpr int kOwn = MT == 512 ? 4 : 8;  // ranges a group fetches ahead
  __shared__ float4 acc[kGroups][C4];
  __shared__ float sw[kMaxParts];
  __shared__ float red[2][kWarps];
  __shared__ Range found;
  __shared__ int lens[32];
  extern __shared__ float sc[];  // the chunk's keys: scores, then weights
  const int64_t row = blockIdx.x;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, c4 = tid % C4, grp = tid / C4;
  const int t = (int)(row % a.BCP), h = (int)(row / a.BCP % a.nq), bi = (int)(row / a.BCP / a.nq);
  const int G = a.nq / a.c.nkv, j = h / G, R = G * a.BCP;
  const int nc = a.chunk ? t + 1 : 0;
  const T* vc = static_cast<const T*>(a.Vc.data) + bi * a.Vc.sb + j * a.Vc.sh + 4 * c4;
  float4 v0 = make_float4(0.f, 0.f, 0.f, 0.f);
  if (nc > 0) {  // (inputs of the call: read before the partials are waited for)
    if (grp < nc) v0 = ld4(vc + grp * a.Vc.st);
    // scores of the chunk's keys in log2 units: eight lanes a key
    constexpr int W = D / 8;
    const int part = lane & 7;
    const T* kc = static_cast<const T*>(a.Kc.data) + bi * a.Kc.sb + j * a.Kc.sh + W * part;
    const T* q = static_cast<const T*>(a.Q.data) + bi * a.Q.sb + h * a.Q.sh + t * a.Q.st + W * part;
    float4 qv[W / 4];
#pragma unroll
    for (int i = 0; i < W / 4; ++i) qv[i] = ld4(q + 4 * i);
    for (int k = warp * 4 + (lane >> 3); k < (nc + 3) / 4 * 4; k += MT / 8) {
      float x = 0.f;
      if (k < nc) {
#pragma unroll
        for (int i = 0; i < W / 4; ++i) {
          const float4 kv = ld4(kc + k * a.Kc.st + 4 * i);
          x = fmaf(qv[i].x, kv.x, x);
          x = fmaf(qv[i].y, kv.y, x);
          x = fmaf(qv[i].z, kv.z, x);
          x = fmaf(qv[i].w, kv.w, x);
        }
      }
#pragma unroll
      for (int o = 1; o < 8; o <<= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
      if (part == 0 && k < nc) sc[k] = x * (a.scale * kLog2e);
    }
    __syncthreads();
  }
  // the row's first range and their number: found again while the ranges are
  // still at work when that is cheap, else read behind them
  int2 parts;
  const int nrows = a.b * a.c.nkv, row_of = bi * a.c.nkv + j;
  if (nrows <= 32) {
    if (tid < 32)
      find_range(nrows, a.target, kSplitKeys, 64, -1 - row_of, lane,
                 [&](int i) { return a.kv_idx != nullptr ? row_keys<true>(a, i) : row_keys<false>(a, i); }, lens, &found);
    __syncthreads();
    parts = make_int2(found.first, found.parts);
    pdl_wait();
  } else {
    pdl_wait();
    parts = __ldcg(a.row_parts + row_of);
  }
  parts.y = min(parts.y, kMaxParts);
  const int64_t at = (int64_t)parts.x * R + (h - j * G) * a.BCP + t;
  const float* lp = a.lse_parts + at;
  const float4* op = reinterpret_cast<const float4*>(a.O_parts + at * D) + c4;
  const int64_t pitch = (int64_t)R * C4;  // from range to range
  float4 own[kOwn];
#pragma unroll
  for (int i = 0; i < kOwn; ++i) {
    const int s = i * kGroups + grp;
    own[i] = make_float4(0.f, 0.f, 0.f, 0.f);
    if (s < parts.y) own[i] = __ldcg(op + s * pitch);
  }
  float M = -INFINITY;
  for (int s = tid; s < parts.y; s += MT) M = fmaxf(M, sw[s] = __ldcg(lp + (int64_t)s * R));
  for (int k = tid; k < nc; k += MT) M = fmaxf(M, sc[k]);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
  if (lane == 0) red[0][warp] = M;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kWarps; ++w) M = fmaxf(M, red[0][w]);
  const float ref = M == -INFINITY ? 0.f : M;  // (no key, or scores that are NaN)
  float L = 0.f;
  // (a range without keys has a weight of 0 and a zero output)
  for (int s = tid; s < parts.y; s += MT) L += sw[s] = exp2f(sw[s] - ref);
  for (int k = tid; k < nc; k += MT) L += sc[k] = exp2f(sc[k] - ref);
  L = warp_sum(L);
  if (lane == 0) red[1][warp] = L;
  __syncthreads();
  L = 0.f;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) L += red[1][w];
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
  auto add = [&](float w, float4 x) {
    o.x = fmaf(w, x.x, o.x);
    o.y = fmaf(w, x.y, o.y);
    o.z = fmaf(w, x.z, o.z);
    o.w = fmaf(w, x.w, o.w);
  };
#pragma unroll
  for (int i = 0; i < kOwn; ++i)
    if (i * kGroups + grp < parts.y) add(sw[i * kGroups + grp], own[i]);
#pragma unroll 4
  for (int s = kOwn * kGroups + grp; s < parts.y; s += kGroups) add(sw[s], __ldcg(op + s * pitch));
  if (grp < nc) add(sc[grp], v0);
#pragma unroll 4
  for (int k = grp + kGroups; k < nc; k += kGroups) add(sc[k], ld4(vc + k * a.Vc.st));
  acc[grp][c4] = o;
  __syncthreads();
  if (grp == 0) {
#pragma unroll
    for (int i = 1; i < kGroups; ++i) add(1.f, acc[i][c4]);
    const float inv = L != 0.f ? 1.f / L : 0.f;
    st4(static_cast<T*>(a.O) + row * D + 4 * c4, make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv));
    if (a.lse != nullptr && tid == 0) a.lse[row] = L != 0.f ? (M + log2f(L)) * kLn2 : -INFINITY;
  }
  if (warp == 1) {
    const int blocks = (R + kBlockRows - 1) / kBlockRows;
    for (int s = lane; s < parts.y; s += 32) {
      const int x = __ldcg(a.faults + (int64_t)(parts.x + s) * blocks + ((h - j * G) * a.BCP + t) / kBlockRows);
      if (x != 0) {
        latch_status(a.status, x & 255);
        if (x >> 8) latch_where(a.status, x >> 8);
      }
    }
  }
}

// A row takes 512 threads while every row has an SM for itself (its keys are then
// cut into many ranges), else 128.
constexpr int kManyRows = 149;
constexpr int kMostChunk = 16384;  // the longest chunk the C ABI takes

template <typename T, int D, int MT>
cudaError_t launch_merge(const CacheAttnArgs& a, cudaStream_t stream) {
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t mc = {};
  mc.gridDim = dim3((unsigned)((int64_t)a.b * a.nq * a.BCP));
  mc.blockDim = dim3(MT);
  mc.dynamicSmemBytes = a.chunk ? a.BCP * sizeof(float) : 0;
  mc.stream = stream;
  mc.attrs = attr;
  mc.numAttrs = 1;  // waits for the ranges inside
  auto* kern = cache_merge_kernel<T, D, MT>;
  if (mc.dynamicSmemBytes > 16 * 1024) {
    const cudaError_t e =
        cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kMostChunk * (int)sizeof(float));
    if (e != cudaSuccess) return e;
  }
  return cudaLaunchKernelEx(&mc, kern, a);
}

template <typename T, int D, int RT>
cudaError_t launch_typed(const CacheAttnArgs& a, cudaStream_t stream) {
  const int R = (a.nq / a.c.nkv) * a.BCP;
  const int tiles8 = RT == 1 ? 1 : R <= 16 ? 2 : R <= 32 ? 4 : 8;
  const size_t smem = smem_bytes<D, sizeof(T) == 2 ? 1 : 2>(tiles8);
  auto* kern = a.kv_idx != nullptr ? cache_slice_kernel<T, D, true, RT> : cache_slice_kernel<T, D, false, RT>;
  // (the same bound in every call: another thread's launch may come in between)
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       (int)smem_bytes<D, sizeof(T) == 2 ? 1 : 2>(RT == 1 ? 1 : 8));
  if (e != cudaSuccess) return e;
  Maps maps = {};
  const int page = 1 << a.c.page_log2, box = 1 << box_log2(a.c);
  if (a.kv_idx == nullptr && (!encode_codes_4d(&maps.k, a.c.k, D, page, a.c.nkv, a.c.npages, a.c.sr, a.c.sh, a.c.sp, box) ||
                              !encode_codes_4d(&maps.v, a.c.v, D, page, a.c.nkv, a.c.npages, a.c.sr, a.c.sh, a.c.sp, box)))
    return cudaErrorNotSupported;
  cudaLaunchConfig_t cfg = {};  // (clears the status words: behind everything before)
  cfg.gridDim = dim3((unsigned)((int64_t)a.ranges * ((R + kBlockRows - 1) / kBlockRows)));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  e = cudaLaunchKernelEx(&cfg, kern, maps, a);
  if (e != cudaSuccess) return e;
  return (int64_t)a.b * a.nq * a.BCP >= kManyRows ? launch_merge<T, D, 128>(a, stream) : launch_merge<T, D, 512>(a, stream);
}

// CTAs of a launch: one round of those resident at once (R <= 8 query rows:
// three an SM, else two), over the blocks of query rows.
int split_ctas(int64_t R) {
  const int64_t blocks = (R + kBlockRows - 1) / kBlockRows;
  static_assert(148 * 3 <= kMaxParts, "a row's ranges fit the join's table");
  return (int)std::max<int64_t>(2, 148 * (R <= 8 ? 3 : 2) / blocks);
}

}  // namespace

int64_t cache_attn_ranges(int64_t rows, int64_t R, int N) { return range_grid(rows, N, split_ctas(R), kSplitKeys); }

cudaError_t launch_cache_attn(bool is_bf16, int d, const CacheAttnArgs& args, cudaStream_t stream) {
  CacheAttnArgs a = args;
  const int R = (a.nq / a.c.nkv) * a.BCP;
  const int64_t rows = (int64_t)a.b * a.c.nkv, ranges = cache_attn_ranges(rows, R, a.N);
  if (R < 1 || a.BCP > kMostChunk) return cudaErrorInvalidValue;
  if (ranges * ((R + kBlockRows - 1) / kBlockRows) > 0x7FFFFFFF || (int64_t)a.b * a.nq * a.BCP > 0x7FFFFFFF) return cudaErrorNotSupported;
  a.target = (int)range_target(rows, split_ctas(R));
  a.ranges = (int)ranges;
  const WaitHooks hooks = wait_hooks();
  a.wait_ns = hooks.wait_ns;
  a.inject = hooks.inject == INJECT_CACHE_ATTN ? 1 : 0;
  if (d != 64 && d != 128) return cudaErrorNotSupported;
  if (R <= 8) {
    if (d == 128) return is_bf16 ? launch_typed<bf16, 128, 1>(a, stream) : launch_typed<float, 128, 1>(a, stream);
    return is_bf16 ? launch_typed<bf16, 64, 1>(a, stream) : launch_typed<float, 64, 1>(a, stream);
  }
  if (d == 128) return is_bf16 ? launch_typed<bf16, 128, 2>(a, stream) : launch_typed<float, 128, 2>(a, stream);
  return is_bf16 ? launch_typed<bf16, 64, 2>(a, stream) : launch_typed<float, 64, 2>(a, stream);
}

}  // namespace quoka

// GQA attention of a few query rows over the paged 8-bit cache: decode steps
// and short blocks (G * BCP <= 64 query rows per KV head).
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
// Work split. The keys of a (sequence, KV head) are cut into nsplit contiguous
// ranges, one CTA each: a loader warp and four that compute. The loader looks
// the rows up (list entry, page, scales: each one stage ahead of the next, so
// that no lookup is waited for) and copies 64 keys at a time into a ring of
// stages with cp.async, zeros in place of rows that are absent; rows of any
// stride, whole pages and listed rows go the same way. The computing warps
// share the 16-row query tiles and take a stage's four 16-key steps in turn.
// Codes go from shared memory straight into the operand layouts of mma.sync:
// for Q K^T the columns of a k-step may be any 16 as long as Q is permuted
// alike, so lane (g, t) reads the 16-byte chunks t and t + 4 of a key's row;
// for P V a lane needs the 4 keys of its P fragment and may own any column per
// n-tile, so lane (g, t) reads the columns [16 g, 16 g + 16) of four keys.
// Chunk c of row r lies at c ^ (r & 7), and operand row n of a step stands for
// key n ^ 4 (n & 1), so that neither read has a bank conflict (d = 128; d = 64
// keeps a two-way one on V). A second kernel joins the ranges of every query
// row and adds the chunk's own keys (at most 64) in fp32.
// Bound by the cache's bytes, each read once per 64 query rows.
#include "cache.cuh"
#include "sm100.cuh"

namespace quoka {

namespace {

using namespace cache;

constexpr int kThreads = 160;      // four computing warps and the loader
constexpr int kStep = 16;          // keys of one step of a warp
constexpr int kStage = 64;         // keys of a stage of the ring
constexpr int kStages = 4;
// M is set kHead below the row maximum and may lag it by kLazy: weights then
// stay below 2^15 (fp16 holds 65504), and one that fp16 holds as a subnormal
// is off by at most 2^-25, 2^-32 of the row's largest.
constexpr float kHead = 7.f, kLazy = 15.f;
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

// c (16 x 8, fp32) += a (16 x 16, fp16) * b (16 x 8, fp16)
__device__ __forceinline__ void mma_f16(float* c, const uint32_t* a, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t pack_h2(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
// what fp16 left of (lo, hi), again in fp16
__device__ __forceinline__ uint32_t rest_h2(float lo, float hi, uint32_t h) {
  const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
  return pack_h2(lo - f.x, hi - f.y);
}

// Shared memory: the query fragments [tiles][SPLIT][D / 16][32 lanes] of 16
// bytes and the rows' factors [tiles * 16]; the stages of codes (keys, then
// values, then the 64 keys' scale exponents). After the loop the warps'
// outputs [4][16][D] fp32 and their (M, l) [4][16][2] lie over the stages.
template <int D>
struct Ring {
  static constexpr int kBytes = kStage * D;                  // codes of a stage's keys (or values)
  static constexpr int kPitch = 2 * kBytes + kStage * 4;     // a stage
  static constexpr int kTotal = kStages * kPitch;
  static_assert(kTotal >= 4 * 16 * D * 4 + 4 * 16 * 2 * 4, "the join's scratch lies over the ring");
};
template <int D, int SPLIT>
constexpr size_t smem_bytes(int tiles) {
  return (size_t)tiles * SPLIT * (D / 16) * 512 + (size_t)tiles * 16 * 4 + Ring<D>::kTotal;
}

// Byte of chunk c (16 bytes) of row r of a stage.
template <int D>
__device__ __forceinline__ int at_chunk(int r, int c) {
  return r * D + ((D == 128 ? c ^ (r & 7) : c ^ ((r >> 1) & 3)) << 4);
}

struct Shared {
  uint64_t full[kStages], empty[kStages];
  int abort, fault, site;
};

// The loader warp: rows [k0, k1) of the (sequence, head), 64 at a time.
template <int D, bool IDX>
__device__ __forceinline__ void load_rows(const CacheAttnArgs& a, Shared& sh, uint8_t* ring, int lane, int bi, int j,
                                          int len, int k0, int k1) {
  using R = Ring<D>;
  constexpr int CPR = D / 16;       // 16-byte chunks of a row
  constexpr int RPI = 32 / CPR;     // rows a warp-wide copy covers
  const int64_t kvrow = (int64_t)bi * a.c.nkv + j;
  const int plog = a.c.page_log2, pmask = (1 << plog) - 1;
  const int32_t* table = a.c.page_table + (int64_t)bi * a.c.table_stride;
  const int nst = (k1 - k0 + kStage - 1) / kStage;
  bool bad = false;
  // key (-1: absent) of this lane's slot u (lane + 32 u) of stage s
  auto tau_of = [&](int s, int u) {
    const int key = k0 + s * kStage + lane + 32 * u;
    if (key >= k1) return -1;
    if constexpr (IDX) return __ldcg(a.kv_idx + kvrow * a.N + key);
    return key;
  };
  auto page_of = [&](int tau) {
    if (tau < 0 || tau >= len) return -1;
    return __ldcg(table + (tau >> plog));
  };
  auto held = [&](int p) { return p >= 0 && p < a.c.npages; };
  int tau[3][2], pg[2][2];
  float ks[2] = {1.f, 1.f}, vs[2] = {1.f, 1.f};
#pragma unroll
  for (int u = 0; u < 2; ++u) {
#pragma unroll
    for (int i = 0; i < 3; ++i) tau[i][u] = tau_of(i, u);
    pg[0][u] = page_of(tau[0][u]);
    pg[1][u] = page_of(tau[1][u]);
    if (held(pg[0][u])) {
      ks[u] = __ldcg(a.c.k_scale + (int64_t)pg[0][u] * a.c.nkv + j);
      vs[u] = __ldcg(a.c.v_scale + (int64_t)pg[0][u] * a.c.nkv + j);
    }
  }
  for (int s = 0; s < nst; ++s) {
    // the lookups of the stages to come
    int tau3[2], pg2[2];
    float ks1[2] = {1.f, 1.f}, vs1[2] = {1.f, 1.f};
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      tau3[u] = tau_of(s + 3, u);
      pg2[u] = page_of(tau[2][u]);
      if (held(pg[1][u])) {
        ks1[u] = __ldcg(a.c.k_scale + (int64_t)pg[1][u] * a.c.nkv + j);
        vs1[u] = __ldcg(a.c.v_scale + (int64_t)pg[1][u] * a.c.nkv + j);
      }
    }
    const int st = s % kStages;
    if (s >= kStages && !__all_sync(0xffffffffu, sm100::mbar_wait(&sh.empty[st], (s / kStages - 1) & 1, &sh.abort))) {
      if (lane == 0) {
        sh.abort = 1;
        sh.fault = 5;  // QUOKA_ERR_TIMEOUT
        sh.site = 61;
      }
      break;
    }
    uint8_t* stage = ring + st * R::kPitch;
    int64_t off[2];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int key = k0 + s * kStage + lane + 32 * u;
      off[u] = -1;
      int ek = 0, ev = 0;
      if (key < k1) {
        if (held(pg[0][u])) {
          off[u] = pg[0][u] * a.c.sp + (int64_t)(tau[0][u] & pmask) * a.c.sr;
          ek = scale_exp(ks[u], &bad);
          ev = scale_exp(vs[u], &bad);
        } else {
          bad = true;  // reads as zeros
        }
      }
      reinterpret_cast<uint32_t*>(stage + 2 * R::kBytes)[lane + 32 * u] = (uint32_t)(ek + 64) | (uint32_t)(ev + 64) << 16;
    }
    const uint32_t dst = sm100::smem_u32(stage);
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
    sm100::mbar_arrive(&sh.full[st]);  // (releases the exponents)
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      tau[0][u] = tau[1][u];
      tau[1][u] = tau[2][u];
      tau[2][u] = tau3[u];
      pg[0][u] = pg[1][u];
      pg[1][u] = pg2[u];
      ks[u] = ks1[u];
      vs[u] = vs1[u];
    }
  }
  sm100::cp_async_commit();
  sm100::cp_async_wait<0>();
  if (__any_sync(0xffffffffu, bad) && lane == 0 && sh.fault == 0) sh.fault = 6;  // QUOKA_ERR_BOUNDS
}

// grid (nsplit, nkv, b)
template <typename T, int D, bool IDX>
__global__ void __launch_bounds__(kThreads, 3) cache_slice_kernel(const CacheAttnArgs a) {
  constexpr int SPLIT = sizeof(T) == 2 ? 1 : 2;
  constexpr int KS = D / 16;  // k-steps of Q K^T
  constexpr int NT = D / 8;   // n-tiles of P V
  using Rg = Ring<D>;
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ Shared sh;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t4 = lane & 3;
  const int s = blockIdx.x, j = blockIdx.y, bi = blockIdx.z;
  const int G = a.nq / a.c.nkv, R = G * a.BCP;
  const int tiles = R <= 16 ? 1 : R <= 32 ? 2 : 4;  // (a third tile alone would leave a warp idle as well)
  uint4* qs = reinterpret_cast<uint4*>(smem);
  float* rowf = reinterpret_cast<float*>(smem + (size_t)tiles * SPLIT * KS * 512);
  uint8_t* ring = smem + (size_t)tiles * SPLIT * KS * 512 + (size_t)tiles * 16 * 4;
  pdl_trigger();
  clear_status(a.status);  // (the faults of this kernel are latched by the next)

  const int64_t kvrow = (int64_t)bi * a.c.nkv + j;
  const int want = __ldcg(a.c.seq_len + bi), len = min(max(want, 0), a.max_len);
  const int n = IDX ? min(max(__ldcg(a.kv_count + kvrow), 0), a.N) : len;
  const int per = ((n + a.nsplit * kStep - 1) / (a.nsplit * kStep)) * kStep;  // keys of a range
  const int k0 = min(n, s * per), k1 = min(n, k0 + per);
  if (tid == 0) {
    for (int i = 0; i < kStages; ++i) {
      sm100::mbar_init(&sh.full[i], 64);
      sm100::mbar_init(&sh.empty[i], 4);
    }
    sh.abort = 0;
    sh.fault = want != len ? 6 : 0;  // QUOKA_ERR_BOUNDS
    sh.site = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  __syncthreads();

  float o[NT][4];
#pragma unroll
  for (int i = 0; i < NT; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
  float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.f, l1 = 0.f;
  const int kgroups = 4 / tiles, tile = warp % tiles, kg = warp / tiles;  // (computing warps)

  if (warp == 4) {
    load_rows<D, IDX>(a, sh, ring, lane, bi, j, len, k0, k1);
  } else {
    // ---- query rows: row r is head j G + r / BCP, chunk position r % BCP; a
    // warp takes a row at a time
    for (int r = warp; r < tiles * 16; r += 4) {
      float x[D / 32];
      float top = 0.f;
      const T* q = static_cast<const T*>(a.Q.data) + bi * a.Q.sb + (int64_t)(j * G + r / a.BCP) * a.Q.sh +
                   (int64_t)(r % a.BCP) * a.Q.st;
      // lane: columns [D / 32 * lane, + D / 32)
#pragma unroll
      for (int i = 0; i < D / 32; ++i) {
        x[i] = r < R ? to_f32(q[D / 32 * lane + i]) : 0.f;
        top = fmaxf(top, fabsf(x[i]));
      }
#pragma unroll
      for (int o_ = 16; o_ > 0; o_ >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o_));
      int e = (int)(__float_as_uint(top) >> 23) - 127 - 13;  // top * 2^-e lies in [2^13, 2^14)
      e = min(max(e, -100), 100);                            // (zero, tiny, infinite rows)
      const float f = exp2i(-e);
      if (lane == 0) rowf[r] = exp2i(e) * a.scale * kLog2e;
#pragma unroll
      for (int i = 0; i < D / 32; i += 2) {
        const int d = D / 32 * lane + i;
        // column d belongs to chunk d / 16 = t + 4 * (ks / 4), word (d % 16) / 4 = ks % 4 of it
        const int ch = d >> 4, ks = 4 * (ch >> 2) + ((d & 15) >> 2);
        const int reg = ((d >> 1) & 1) * 2 + ((r & 15) >> 3);
        uint32_t* dst =
            reinterpret_cast<uint32_t*>(qs + (((r >> 4) * SPLIT) * KS + ks) * 32 + (r & 7) * 4 + (ch & 3)) + reg;
        const uint32_t hi = pack_h2(x[i] * f, x[i + 1] * f);
        *dst = hi;
        if constexpr (SPLIT == 2) dst[KS * 32 * 4] = rest_h2(x[i] * f, x[i + 1] * f, hi);
      }
    }
    sm100::named_barrier_sync(1, 128);
    const float f0 = rowf[tile * 16 + g], f1 = rowf[tile * 16 + g + 8];
    const uint4* qt = qs + (size_t)tile * SPLIT * KS * 32 + lane;
    const int gk = g ^ ((g & 1) << 2);               // this lane's key of a step (and gk + 8)
    const int v0 = 2 * t4, v1 = (2 * t4 + 1) ^ 4;    // its keys of P V: v0, v1, v0 + 8, v1 + 8

    auto compute = [&](const uint8_t* stage, int row, int left) {
      const uint8_t* kr = stage + row * D;
      const uint8_t* vr = kr + Rg::kBytes;
      const uint32_t* ex = reinterpret_cast<const uint32_t*>(stage + 2 * Rg::kBytes) + row;
      float c[2][4];
#pragma unroll
      for (int nt = 0; nt < 2; ++nt) c[nt][0] = c[nt][1] = c[nt][2] = c[nt][3] = 0.f;
      uint32_t kw[2][KS];
#pragma unroll
      for (int nt = 0; nt < 2; ++nt)
#pragma unroll
        for (int h = 0; h < D / 64; ++h) {
          const uint4 w = *reinterpret_cast<const uint4*>(kr + at_chunk<D>(gk + 8 * nt, t4 + 4 * h));
          kw[nt][4 * h] = w.x;
          kw[nt][4 * h + 1] = w.y;
          kw[nt][4 * h + 2] = w.z;
          kw[nt][4 * h + 3] = w.w;
        }
      uint32_t vw[4][D / 32];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int r = (i & 1 ? v1 : v0) + 8 * (i >> 1);
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
      }
#pragma unroll
      for (int ks = 0; ks < KS; ++ks) {
        const uint4 q0 = qt[ks * 32];
        const uint32_t qa[4] = {q0.x, q0.y, q0.z, q0.w};
        uint32_t qb[4];
        if constexpr (SPLIT == 2) {
          const uint4 q1 = qt[(KS + ks) * 32];
          qb[0] = q1.x; qb[1] = q1.y; qb[2] = q1.z; qb[3] = q1.w;
        }
#pragma unroll
        for (int nt = 0; nt < 2; ++nt) {
          const uint32_t w = kw[nt][ks];
          const uint32_t b0 = e4m3x2_to_f16x2((uint16_t)w), b1 = e4m3x2_to_f16x2((uint16_t)(w >> 16));
          mma_f16(c[nt], qa, b0, b1);
          if constexpr (SPLIT == 2) mma_f16(c[nt], qb, b0, b1);
        }
      }
      // scores in log2 units, with the value scale's exponent added
      float x0 = -INFINITY, x1 = -INFINITY;
      float inv[4];  // 2^-ev of the lane's four keys
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int key = (i & 1 ? v1 : v0) + 8 * (i >> 1);
        const uint32_t e = ex[key];
        const float ks = exp2i((int)(e & 0xFFFFu) - 64);
        const int ev = (int)(e >> 16) - 64;
        inv[i] = exp2i(-ev);
        const bool there = key < left;
        float& a0 = c[i >> 1][i & 1];
        float& a1 = c[i >> 1][2 + (i & 1)];
        a0 = there ? fmaf(a0, f0 * ks, (float)ev) : -INFINITY;
        a1 = there ? fmaf(a1, f1 * ks, (float)ev) : -INFINITY;
        x0 = fmaxf(x0, a0);
        x1 = fmaxf(x1, a1);
      }
      x0 = fmaxf(x0, __shfl_xor_sync(0xffffffffu, x0, 1));
      x1 = fmaxf(x1, __shfl_xor_sync(0xffffffffu, x1, 1));
      x0 = fmaxf(x0, __shfl_xor_sync(0xffffffffu, x0, 2));
      x1 = fmaxf(x1, __shfl_xor_sync(0xffffffffu, x1, 2));
      if (__any_sync(0xffffffffu, x0 > m0 + kLazy || x1 > m1 + kLazy)) {
        const float n0 = fmaxf(m0, x0 - kHead), n1 = fmaxf(m1, x1 - kHead);
        const float r0 = m0 == -INFINITY ? 0.f : exp2f(m0 - n0), r1 = m1 == -INFINITY ? 0.f : exp2f(m1 - n1);
        m0 = n0;
        m1 = n1;
        l0 *= r0;
        l1 *= r1;
#pragma unroll
        for (int i = 0; i < NT; ++i) {
          o[i][0] *= r0;
          o[i][1] *= r0;
          o[i][2] *= r1;
          o[i][3] *= r1;
        }
      }
      const float b0 = m0 == -INFINITY ? 0.f : m0, b1 = m1 == -INFINITY ? 0.f : m1;
      float p[2][4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float p0 = sm100::ex2(c[i >> 1][i & 1] - b0), p1 = sm100::ex2(c[i >> 1][2 + (i & 1)] - b1);
        l0 = fmaf(p0, inv[i], l0);
        l1 = fmaf(p1, inv[i], l1);
        p[i >> 1][i & 1] = p0;
        p[i >> 1][2 + (i & 1)] = p1;
      }
      uint32_t pa[4], pb[4];
      pa[0] = pack_h2(p[0][0], p[0][1]);
      pa[1] = pack_h2(p[0][2], p[0][3]);
      pa[2] = pack_h2(p[1][0], p[1][1]);
      pa[3] = pack_h2(p[1][2], p[1][3]);
      if constexpr (SPLIT == 2) {
        pb[0] = rest_h2(p[0][0], p[0][1], pa[0]);
        pb[1] = rest_h2(p[0][2], p[0][3], pa[1]);
        pb[2] = rest_h2(p[1][0], p[1][1], pa[2]);
        pb[3] = rest_h2(p[1][2], p[1][3], pa[3]);
      }
      // O += P V: n-tile 4 w + u multiplies byte u of every lane's word w
#pragma unroll
      for (int w = 0; w < D / 32; ++w) {
        uint32_t lo[2], hi[2];
        lo[0] = __byte_perm(vw[0][w], vw[1][w], 0x5140);
        lo[1] = __byte_perm(vw[0][w], vw[1][w], 0x7362);
        hi[0] = __byte_perm(vw[2][w], vw[3][w], 0x5140);
        hi[1] = __byte_perm(vw[2][w], vw[3][w], 0x7362);
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const uint32_t b0_ = e4m3x2_to_f16x2((uint16_t)(lo[u >> 1] >> (16 * (u & 1))));
          const uint32_t b1_ = e4m3x2_to_f16x2((uint16_t)(hi[u >> 1] >> (16 * (u & 1))));
          mma_f16(o[4 * w + u], pa, b0_, b1_);
          if constexpr (SPLIT == 2) mma_f16(o[4 * w + u], pb, b0_, b1_);
        }
      }
    };

    const int nst = (k1 - k0 + kStage - 1) / kStage;
    for (int i = 0; i < nst; ++i) {
      const int st = i % kStages;
      if (!__all_sync(0xffffffffu, sm100::mbar_wait(&sh.full[st], (i / kStages) & 1, &sh.abort))) {
        if (lane == 0) {
          sh.abort = 1;
          sh.fault = 5;  // QUOKA_ERR_TIMEOUT
          sh.site = 62;
        }
        break;
      }
      const int left = k1 - k0 - i * kStage;
      for (int row = kg * kStep; row < min(left, kStage); row += kgroups * kStep)
        compute(ring + st * Rg::kPitch, row, left - row);
      __syncwarp();
      if (lane == 0) sm100::mbar_arrive(&sh.empty[st]);
    }
  }

  // ---- join the warps of each query tile
  l0 += __shfl_xor_sync(0xffffffffu, l0, 1);
  l1 += __shfl_xor_sync(0xffffffffu, l1, 1);
  l0 += __shfl_xor_sync(0xffffffffu, l0, 2);
  l1 += __shfl_xor_sync(0xffffffffu, l1, 2);
  __syncthreads();  // the ring is no longer read, and no copy into it is in flight
  float* os = reinterpret_cast<float*>(ring);  // [4 warps][16][D]
  float* ml = os + 4 * 16 * D;                 // [4][16][2]
  if (warp < 4) {
#pragma unroll
    for (int hf = 0; hf < 2; ++hf) {
      const int r = g + 8 * hf;
      if (t4 == 0) {
        ml[(warp * 16 + r) * 2] = hf ? m1 : m0;
        ml[(warp * 16 + r) * 2 + 1] = hf ? l1 : l0;
      }
      if (tile * 16 + r < R) {
        // n-tile i of lane (g, t): columns D/8 * 2t + i and D/8 * (2t + 1) + i
        float4* row = reinterpret_cast<float4*>(os + (warp * 16 + r) * D + D / 4 * t4);
#pragma unroll
        for (int i = 0; i < NT; i += 4) {
          row[i / 4] = make_float4(o[i][2 * hf], o[i + 1][2 * hf], o[i + 2][2 * hf], o[i + 3][2 * hf]);
          row[D / 32 + i / 4] =
              make_float4(o[i][2 * hf + 1], o[i + 1][2 * hf + 1], o[i + 2][2 * hf + 1], o[i + 3][2 * hf + 1]);
        }
      }
    }
  }
  __syncthreads();
  const int64_t rows = (int64_t)a.b * a.nq * a.BCP;
  for (int e = tid; e < R * (D / 4); e += kThreads) {
    const int r = e / (D / 4), c4 = e % (D / 4);
    const int tl = r >> 4, rr = r & 15;
    float M = -INFINITY;
    for (int k = 0; k < kgroups; ++k) M = fmaxf(M, ml[((k * tiles + tl) * 16 + rr) * 2]);
    float L = 0.f;
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int k = 0; k < kgroups; ++k) {
      const int w = k * tiles + tl;
      const float lw = ml[(w * 16 + rr) * 2 + 1];
      if (lw == 0.f) continue;  // the warp saw no key (not so for NaN scores: they come through)
      const float f = exp2f(ml[(w * 16 + rr) * 2] - M);
      const float4 y = *reinterpret_cast<const float4*>(os + (w * 16 + rr) * D + 4 * c4);
      L = fmaf(f, lw, L);
      x.x = fmaf(f, y.x, x.x);
      x.y = fmaf(f, y.y, x.y);
      x.z = fmaf(f, y.z, x.z);
      x.w = fmaf(f, y.w, x.w);
    }
    const float inv = L != 0.f ? 1.f / L : 0.f;
    const int h = j * G + r / a.BCP, t = r % a.BCP;
    const int64_t row = ((int64_t)bi * a.nq + h) * a.BCP + t;
    *reinterpret_cast<float4*>(a.O_parts + ((int64_t)s * rows + row) * D + 4 * c4) =
        make_float4(x.x * inv, x.y * inv, x.z * inv, x.w * inv);
    // log2 of the range's partition function (-inf: no key)
    if (c4 == 0) a.lse_parts[(int64_t)s * rows + row] = L != 0.f ? M + log2f(L) : -INFINITY;
  }
  if (tid == 0) a.faults[kvrow * a.nsplit + s] = sh.fault | sh.site << 8;
}

// Joins the ranges of one query row, adds the chunk's own keys s <= t, and
// writes the row: O = sum_i 2^(x_i - X) O_i, X = log2 sum_i 2^(x_i). One CTA
// per row: a thread owns four columns of every kGroups-th range and chunk
// key, so that a row's partials are fetched in one or two rounds of loads.
constexpr int kMergeThreads = 128;

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

template <typename T, int D>
__global__ void __launch_bounds__(kMergeThreads) cache_merge_kernel(const CacheAttnArgs a) {
  constexpr int C4 = D / 4, kGroups = kMergeThreads / C4;
  __shared__ float4 acc[kGroups][C4];
  __shared__ float sc[kCacheMaxRows];
  const int64_t row = blockIdx.x, rows = (int64_t)a.b * a.nq * a.BCP;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, c4 = tid % C4, grp = tid / C4;
  const int t = (int)(row % a.BCP), h = (int)(row / a.BCP % a.nq), bi = (int)(row / a.BCP / a.nq);
  const int j = h / (a.nq / a.c.nkv);
  const int nc = a.chunk ? t + 1 : 0;
  const T* vc = static_cast<const T*>(a.Vc.data) + bi * a.Vc.sb + j * a.Vc.sh;
  if (nc > 0) {  // (inputs of the call: read before the partials are waited for)
    // scores of the chunk's keys in log2 units: eight lanes a key
    constexpr int W = D / 8;
    const int part = lane & 7;
    const T* kc = static_cast<const T*>(a.Kc.data) + bi * a.Kc.sb + j * a.Kc.sh + W * part;
    const T* q = static_cast<const T*>(a.Q.data) + bi * a.Q.sb + h * a.Q.sh + t * a.Q.st + W * part;
    float4 qv[W / 4];
#pragma unroll
    for (int i = 0; i < W / 4; ++i) qv[i] = ld4(q + 4 * i);
    for (int k = warp * 4 + (lane >> 3); k < (nc + 3) / 4 * 4; k += kMergeThreads / 8) {
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
  pdl_wait();
  const float* lp = a.lse_parts + row;
  float M = -INFINITY;
  for (int s = lane; s < a.nsplit; s += 32) M = fmaxf(M, __ldcg(lp + (int64_t)s * rows));
  for (int k = lane; k < nc; k += 32) M = fmaxf(M, sc[k]);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
  const float ref = M == -INFINITY ? 0.f : M;  // (no key, or scores that are NaN)
  float L = 0.f;
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
  auto add = [&](float w, float4 x) {
    o.x = fmaf(w, x.x, o.x);
    o.y = fmaf(w, x.y, o.y);
    o.z = fmaf(w, x.z, o.z);
    o.w = fmaf(w, x.w, o.w);
  };
  for (int s0 = 0; s0 < a.nsplit; s0 += 32) {
    // (a range without keys has a weight of 0 and a zero output)
    const float w = s0 + lane < a.nsplit ? exp2f(__ldcg(lp + (int64_t)(s0 + lane) * rows) - ref) : 0.f;
    L += w;
#pragma unroll
    for (int i = 0; i < 32 / kGroups; ++i) {
      const int s = i * kGroups + grp;
      const float ws = __shfl_sync(0xffffffffu, w, s);
      if (s0 + s < a.nsplit)
        add(ws, __ldcg(reinterpret_cast<const float4*>(a.O_parts + ((int64_t)(s0 + s) * rows + row) * D) + c4));
    }
  }
  for (int k = lane; k < nc; k += 32) L += exp2f(sc[k] - ref);
  L = warp_sum(L);
  for (int k = grp; k < nc; k += kGroups) add(exp2f(sc[k] - ref), ld4(vc + k * a.Vc.st + 4 * c4));
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
    const int* f = a.faults + ((int64_t)bi * a.c.nkv + j) * a.nsplit;
    for (int s = lane; s < a.nsplit; s += 32) {
      const int x = __ldcg(f + s);
      if (x != 0) {
        latch_status(a.status, x & 255);
        if (x >> 8) latch_where(a.status, x >> 8);
      }
    }
  }
}

template <typename T, int D>
cudaError_t launch_typed(const CacheAttnArgs& a, cudaStream_t stream) {
  const int R = (a.nq / a.c.nkv) * a.BCP;
  const int tiles = R <= 16 ? 1 : R <= 32 ? 2 : 4;
  const size_t smem = smem_bytes<D, sizeof(T) == 2 ? 1 : 2>(tiles);
  auto* kern = a.kv_idx != nullptr ? cache_slice_kernel<T, D, true> : cache_slice_kernel<T, D, false>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(a.nsplit, a.c.nkv, a.b);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 0;  // (clears the status words: behind everything before)
  e = cudaLaunchKernelEx(&cfg, kern, a);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t mc = {};
  mc.gridDim = dim3((unsigned)((int64_t)a.b * a.nq * a.BCP));
  mc.blockDim = dim3(kMergeThreads);
  mc.stream = stream;
  mc.attrs = attr;
  mc.numAttrs = 1;  // waits for the slices inside
  return cudaLaunchKernelEx(&mc, cache_merge_kernel<T, D>, a);
}

// One round of CTAs at three an SM, a range being at least 128 keys. (Decode
// steps of 32 sequences of up to 8192 keys, d = 128: 79.9 us with 296 or 444
// CTAs, 81.9 with 888, 86.0 with 1776; one sequence of 4096 listed keys the
// same with 128 and 256 keys at least, blocks of 1500 keys 2 us slower with 256.)
constexpr int kSplitCTAs = 444, kSplitKeys = 128;

}  // namespace

int cache_attn_splits(int64_t heads, int N) {
  const int64_t want = (kSplitCTAs + heads - 1) / heads, most = (N + kSplitKeys - 1) / kSplitKeys;
  return (int)(want < 1 ? 1 : want < most ? want : most < 1 ? 1 : most);
}

cudaError_t launch_cache_attn(bool is_bf16, int d, const CacheAttnArgs& a, cudaStream_t stream) {
  const int R = (a.nq / a.c.nkv) * a.BCP;
  if (R < 1 || R > kCacheMaxRows || a.nsplit < 1) return cudaErrorInvalidValue;
  if (d == 128) return is_bf16 ? launch_typed<bf16, 128>(a, stream) : launch_typed<float, 128>(a, stream);
  if (d == 64) return is_bf16 ? launch_typed<bf16, 64>(a, stream) : launch_typed<float, 64>(a, stream);
  return cudaErrorNotSupported;
}

}  // namespace quoka

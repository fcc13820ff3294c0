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
// ranges, one CTA of 4 warps each; the warps share the 16-row query tiles and
// take the range's 16-key steps in turn. A warp works alone on registers: the
// operand layouts of mma.sync let a lane use 16-byte loads straight from the
// cache rows. For Q K^T the columns of a k-step may be any 16 as long as Q is
// permuted alike, so lane (g, t) reads chunks t and t + 4 of key g's row; for
// P V a lane needs the 4 keys of its P fragment and may own any column per
// n-tile, so lane (g, t) reads columns [16 g, 16 g + 16) of keys 2t, 2t + 1,
// 2t + 8, 2t + 9. No shared memory, no barrier and no transposition stands
// between the load and the product; the next step's rows are loaded while the
// present one is multiplied. A second kernel joins the ranges of every query
// row and adds the chunk's own keys (at most 64) in fp32.
// Bound by the cache's bytes, each read once per 16 query rows.
#include "cache.cuh"
#include "sm100.cuh"

namespace quoka {

namespace {

using namespace cache;

constexpr int kThreads = 128;
constexpr int kStep = 16;          // keys of one step of a warp
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

// The words of codes a lane holds of a 16-key step. D = 128: 2 chunks of 16
// bytes per key row and one per value row; D = 64: 1 and a half.
template <int D>
struct Step {
  uint32_t k[2][D / 16];  // keys g and g + 8
  uint32_t v[4][D / 32];  // keys 2t, 2t + 1, 2t + 8, 2t + 9
};

template <int N>
__device__ __forceinline__ void ld_words(const uint8_t* p, uint32_t* w) {
  if constexpr (N == 4)
    asm volatile("ld.global.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]) : "l"(p));
  else
    asm volatile("ld.global.v2.u32 {%0, %1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "l"(p));
}

// Shared memory: the query fragments [tiles][SPLIT][D / 16][32 lanes] of 16
// bytes, the rows' factors [tiles * 16]; after the loop the warps' outputs
// [4][16][D] fp32 and their (M, l) [4][16][2] take the same space.
template <int D, int SPLIT>
constexpr size_t smem_bytes(int tiles) {
  const size_t q = (size_t)tiles * SPLIT * (D / 16) * 512 + (size_t)tiles * 16 * 4;
  const size_t o = (size_t)4 * 16 * D * 4 + 4 * 16 * 2 * 4;
  return q > o ? q : o;
}

// grid (nsplit, nkv, b)
template <typename T, int D, bool IDX>
__global__ void __launch_bounds__(kThreads) cache_slice_kernel(const CacheAttnArgs a) {
  constexpr int SPLIT = sizeof(T) == 2 ? 1 : 2;
  constexpr int KS = D / 16;  // k-steps of Q K^T
  constexpr int NT = D / 8;   // n-tiles of P V
  extern __shared__ __align__(16) uint8_t smem[];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t4 = lane & 3;
  const int s = blockIdx.x, j = blockIdx.y, bi = blockIdx.z;
  const int G = a.nq / a.c.nkv, R = G * a.BCP;
  const int tiles = R <= 16 ? 1 : R <= 32 ? 2 : 4;  // (a third tile alone would leave a warp idle as well)
  uint4* qs = reinterpret_cast<uint4*>(smem);
  float* rowf = reinterpret_cast<float*>(smem + (size_t)tiles * SPLIT * KS * 512);
  pdl_trigger();

  // ---- query rows (inputs of the call): row r is head j G + r / BCP, chunk
  // position r % BCP; a warp takes a row at a time
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
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
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
      uint32_t* dst = reinterpret_cast<uint32_t*>(qs + (((r >> 4) * SPLIT) * KS + ks) * 32 + (r & 7) * 4 + (ch & 3)) + reg;
      const uint32_t hi = pack_h2(x[i] * f, x[i + 1] * f);
      *dst = hi;
      if constexpr (SPLIT == 2) dst[KS * 32 * 4] = rest_h2(x[i] * f, x[i + 1] * f, hi);
    }
  }
  pdl_wait();  // lengths, tables, lists and the status word may come from earlier kernels

  const int64_t kvrow = (int64_t)bi * a.c.nkv + j;
  const int len = cache_len(a.c, bi, a.max_len, a.status);
  const int n = IDX ? min(max(__ldcg(a.kv_count + kvrow), 0), a.N) : len;
  const int per = ((n + a.nsplit * kStep - 1) / (a.nsplit * kStep)) * kStep;  // keys of a range
  const int k0 = min(n, s * per), k1 = min(n, k0 + per);
  const int kgroups = 4 / tiles, tile = warp % tiles, kg = warp / tiles;
  __syncthreads();
  const float f0 = rowf[tile * 16 + g], f1 = rowf[tile * 16 + g + 8];
  const uint4* qt = qs + (size_t)tile * SPLIT * KS * 32 + lane;
  const int plog = a.c.page_log2, pmask = (1 << plog) - 1;
  const uint8_t* kb = a.c.k + j * a.c.sh;
  const uint8_t* vb = a.c.v + j * a.c.sh;

  float o[NT][4];
#pragma unroll
  for (int i = 0; i < NT; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
  float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.f, l1 = 0.f;

  // Where a step's rows are: lane i (and i + 16) answers for key i of the
  // step: its row's byte offset (or -1: absent, or on no page), and the
  // exponents of its page's scales, ek + 64 in the low and ev + 64 in the
  // high half.
  auto locate = [&](int base, int64_t* off, uint32_t* ee) {
    const int key = base + (lane & 15);
    *off = -1;
    *ee = 64u | 64u << 16;
    if (key >= k1) return;
    int tau = key;
    if constexpr (IDX) {
      tau = __ldcg(a.kv_idx + kvrow * a.N + key);
      if (tau < 0 || tau >= len) {
        if (a.status != nullptr) latch_status(a.status, 6 /* QUOKA_ERR_BOUNDS */);
        return;  // reads as zeros
      }
    }
    const int p = cache_page(a.c, bi, tau >> plog, a.status);
    if (p < 0) return;
    *off = p * a.c.sp + (int64_t)(tau & pmask) * a.c.sr;
    const int ek = scale_exp(__ldg(a.c.k_scale + (int64_t)p * a.c.nkv + j), a.status);
    const int ev = scale_exp(__ldg(a.c.v_scale + (int64_t)p * a.c.nkv + j), a.status);
    *ee = (uint32_t)(ek + 64) | (uint32_t)(ev + 64) << 16;
  };
  auto load = [&](int64_t off, Step<D>& st) {
#pragma unroll
    for (int nt = 0; nt < 2; ++nt) {
      const int64_t ro = __shfl_sync(0xffffffffu, off, 8 * nt + g);
#pragma unroll
      for (int w = 0; w < D / 16; ++w) st.k[nt][w] = 0u;
      if (ro >= 0) {
#pragma unroll
        for (int h = 0; h < D / 64; ++h) ld_words<4>(kb + ro + 16 * t4 + 64 * h, st.k[nt] + 4 * h);
      }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int64_t ro = __shfl_sync(0xffffffffu, off, 2 * t4 + (i & 1) + 8 * (i >> 1));
#pragma unroll
      for (int w = 0; w < D / 32; ++w) st.v[i][w] = 0u;
      if (ro >= 0) ld_words<D / 32>(vb + ro + D / 8 * g, st.v[i]);
    }
  };
  auto compute = [&](int base, const Step<D>& st, uint32_t ee) {
    float c[2][4];
#pragma unroll
    for (int nt = 0; nt < 2; ++nt) c[nt][0] = c[nt][1] = c[nt][2] = c[nt][3] = 0.f;
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
        const uint32_t w = st.k[nt][ks];
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
      const int key = 2 * t4 + (i & 1) + 8 * (i >> 1);
      const uint32_t e = __shfl_sync(0xffffffffu, ee, key);
      const float ks = exp2i((int)(e & 0xFFFFu) - 64);
      const int ev = (int)(e >> 16) - 64;
      inv[i] = exp2i(-ev);
      const bool there = base + key < k1;
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
      lo[0] = __byte_perm(st.v[0][w], st.v[1][w], 0x5140);
      lo[1] = __byte_perm(st.v[0][w], st.v[1][w], 0x7362);
      hi[0] = __byte_perm(st.v[2][w], st.v[3][w], 0x5140);
      hi[1] = __byte_perm(st.v[2][w], st.v[3][w], 0x7362);
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const uint32_t b0_ = e4m3x2_to_f16x2((uint16_t)(lo[u >> 1] >> (16 * (u & 1))));
        const uint32_t b1_ = e4m3x2_to_f16x2((uint16_t)(hi[u >> 1] >> (16 * (u & 1))));
        mma_f16(o[4 * w + u], pa, b0_, b1_);
        if constexpr (SPLIT == 2) mma_f16(o[4 * w + u], pb, b0_, b1_);
      }
    }
  };

  {
    const int stride = kStep * kgroups;
    int base = k0 + kg * kStep;
    if (base < k1) {
      Step<D> cur, nxt;
      int64_t off;
      uint32_t ee, ee_n;
      locate(base, &off, &ee);
      load(off, cur);
      for (;;) {
        const int next = base + stride;
        const bool more = next < k1;
        if (more) {
          locate(next, &off, &ee_n);
          load(off, nxt);
        }
        compute(base, cur, ee);
        if (!more) break;
        cur = nxt;
        ee = ee_n;
        base = next;
      }
    }
  }

  // ---- join the warps of each query tile
  l0 += __shfl_xor_sync(0xffffffffu, l0, 1);
  l1 += __shfl_xor_sync(0xffffffffu, l1, 1);
  l0 += __shfl_xor_sync(0xffffffffu, l0, 2);
  l1 += __shfl_xor_sync(0xffffffffu, l1, 2);
  __syncthreads();  // the query fragments are no longer read
  float* os = reinterpret_cast<float*>(smem);  // [4 warps][16][D]
  float* ml = os + 4 * 16 * D;                 // [4][16][2]
#pragma unroll
  for (int hf = 0; hf < 2; ++hf) {
    const int r = g + 8 * hf;
    if (t4 == 0) {
      ml[(warp * 16 + r) * 2] = hf ? m1 : m0;
      ml[(warp * 16 + r) * 2 + 1] = hf ? l1 : l0;
    }
    // n-tile i of lane (g, t): columns D/8 * 2t + i and D/8 * (2t + 1) + i
    float* row = os + (warp * 16 + r) * D + D / 4 * t4;
#pragma unroll
    for (int i = 0; i < NT; ++i) {
      row[i] = o[i][2 * hf];
      row[D / 8 + i] = o[i][2 * hf + 1];
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
}

// Joins the ranges of one query row, adds the chunk's own keys s <= t, and
// writes the row: O = sum_i 2^(x_i - X) O_i, X = log2 sum_i 2^(x_i). One CTA
// of D threads per row, a thread per column.
template <typename T, int D>
__global__ void __launch_bounds__(D) cache_merge_kernel(const CacheAttnArgs a) {
  __shared__ float qrow[D];
  __shared__ float sc[kCacheMaxRows];
  const int64_t row = blockIdx.x, rows = (int64_t)a.b * a.nq * a.BCP;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int t = (int)(row % a.BCP), h = (int)(row / a.BCP % a.nq), bi = (int)(row / a.BCP / a.nq);
  const int j = h / (a.nq / a.c.nkv);
  const int nc = a.chunk ? t + 1 : 0;
  const T* kc = static_cast<const T*>(a.Kc.data) + bi * a.Kc.sb + j * a.Kc.sh;
  const T* vc = static_cast<const T*>(a.Vc.data) + bi * a.Vc.sb + j * a.Vc.sh;
  if (nc > 0) {  // (inputs of the call: read before the partials are waited for)
    qrow[tid] = to_f32(static_cast<const T*>(a.Q.data)[bi * a.Q.sb + h * a.Q.sh + t * a.Q.st + tid]) * (a.scale * kLog2e);
    __syncthreads();
    for (int k = warp; k < nc; k += D / 32) {
      float x = 0.f;
#pragma unroll
      for (int i = 0; i < D / 32; ++i) x = fmaf(qrow[lane + 32 * i], to_f32(kc[k * a.Kc.st + lane + 32 * i]), x);
      x = warp_sum(x);
      if (lane == 0) sc[k] = x;
    }
    __syncthreads();
  }
  pdl_wait();
  float M = -INFINITY;
  for (int s = 0; s < a.nsplit; ++s) M = fmaxf(M, __ldcg(a.lse_parts + (int64_t)s * rows + row));
  for (int k = 0; k < nc; ++k) M = fmaxf(M, sc[k]);
  const float ref = M == -INFINITY ? 0.f : M;  // (no key, or scores that are NaN)
  float L = 0.f, o = 0.f;
  for (int s = 0; s < a.nsplit; ++s) {
    const float x = __ldcg(a.lse_parts + (int64_t)s * rows + row);
    if (x == -INFINITY) continue;  // (its partial output is zero)
    const float w = exp2f(x - ref);
    L += w;
    o = fmaf(w, __ldcg(a.O_parts + ((int64_t)s * rows + row) * D + tid), o);
  }
  for (int k = 0; k < nc; ++k) {
    const float w = exp2f(sc[k] - ref);
    L += w;
    o = fmaf(w, to_f32(vc[k * a.Vc.st + tid]), o);
  }
  static_cast<T*>(a.O)[row * D + tid] = from_f32<T>(L != 0.f ? o / L : 0.f);
  if (a.lse != nullptr && tid == 0) a.lse[row] = L != 0.f ? (M + log2f(L)) * kLn2 : -INFINITY;
}

template <typename T, int D>
cudaError_t launch_typed(const CacheAttnArgs& a, bool pdl, cudaStream_t stream) {
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
  cfg.numAttrs = pdl ? 1 : 0;
  e = cudaLaunchKernelEx(&cfg, kern, a);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t mc = {};
  mc.gridDim = dim3((unsigned)((int64_t)a.b * a.nq * a.BCP));
  mc.blockDim = dim3(D);
  mc.stream = stream;
  mc.attrs = attr;
  mc.numAttrs = 1;  // waits for the slices inside
  return cudaLaunchKernelEx(&mc, cache_merge_kernel<T, D>, a);
}

}  // namespace

int cache_attn_splits(int64_t heads, int N) {
  // enough CTAs to fill the GPU twice over with three resident per SM, each
  // with at least one step per warp
  const int64_t want = (888 + heads - 1) / heads, most = (N + 63) / 64;
  return (int)(want < 1 ? 1 : want < most ? want : most < 1 ? 1 : most);
}

cudaError_t launch_cache_attn(bool is_bf16, int d, const CacheAttnArgs& a, bool pdl, cudaStream_t stream) {
  const int R = (a.nq / a.c.nkv) * a.BCP;
  if (R < 1 || R > kCacheMaxRows || a.nsplit < 1) return cudaErrorInvalidValue;
  if (d == 128) return is_bf16 ? launch_typed<bf16, 128>(a, pdl, stream) : launch_typed<float, 128>(a, pdl, stream);
  if (d == 64) return is_bf16 ? launch_typed<bf16, 64>(a, pdl, stream) : launch_typed<float, 64>(a, pdl, stream);
  return cudaErrorNotSupported;
}

}  // namespace quoka

// Appending a chunk's keys and values to the paged 8-bit cache, with the
// position rotation applied on the way.
//
// Token t of sequence s takes position p = seq_len[s] + t. Its key (and, when
// asked for, its query) is rotated by p: with c = cos[p, i], s = sin[p, i]
// and (x1, x2) the i-th pair of columns,
//   x1' = x1 c - x2 s,   x2' = x2 c + x1 s,
// each product and sum rounded to fp32 by itself, so that the result is the
// one elementary fp32 operations give, bit for bit. The keys and values of a
// page that the chunk touches are then quantised together:
//   a = max |finite x| over the page's new tokens and the head's d columns,
//   e = the smallest exponent with a <= 448 * 2^e,
//   code = e4m3(x * 2^-e), to nearest even, saturating.
// A page that already holds earlier tokens keeps a scale at least as large as
// the one it has; when it grows, the codes it holds are brought to the new
// one. (The quantisation takes the fp32 rotation, not its rounded copy Kr.)
//
// Work split: one CTA per (sequence, touched page, KV head, keys or values),
// whose rows stay in registers between the maximum and the quantisation; a
// page has one writer, so nothing is atomic and the result does not depend on
// the order of the CTAs. The queries are rotated by further CTAs of the same
// launch, each over a few heads of the same tokens, so that a token's cosines
// are read once for several heads. A thread owns two 8-column chunks of a row,
// the two halves of its pairs, and issues all its loads before it computes.
// Bound by bytes: every row is read once and written once as codes (and once
// rotated); a chunk of few tokens by the chain length, page, scale, and takes
// small CTAs so that all of them are resident at once. Measured (32 query and 8
// KV heads, d = 128, bf16): 4 x 2048 tokens 37.7 us for 205.5 MB, 5.4 TB/s; one
// token of 64 sequences 5.8 us with CTAs of 64 threads, 11.3 with 256 (which are
// then not all resident) and each element's partner loaded a second time.
#include "cache.cuh"

namespace quoka {

namespace {

using namespace cache;

constexpr int kQHeads = 4;  // query heads of one rotating CTA

struct RotArgs {
  const float* cos;
  const float* sin;  // (npos, rot / 2)
  int rot, interleaved;
};

// 8 elements as they lie in memory.
template <typename T>
struct Raw8 {
  uint4 w[sizeof(T) / 2];
};
template <typename T>
__device__ __forceinline__ void load_raw(const T* p, Raw8<T>& r) {
#pragma unroll
  for (int i = 0; i < (int)sizeof(T) / 2; ++i) r.w[i] = __ldg(reinterpret_cast<const uint4*>(p) + i);
}
__device__ __forceinline__ void to_floats(const Raw8<bf16>& r, float (&v)[8]) {
  const __nv_bfloat162* h = reinterpret_cast<const __nv_bfloat162*>(&r);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = __bfloat1622float2(h[i]);
    v[2 * i] = f.x;
    v[2 * i + 1] = f.y;
  }
}
__device__ __forceinline__ void to_floats(const Raw8<float>& r, float (&v)[8]) {
  const float* f = reinterpret_cast<const float*>(&r);
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = f[i];
}

__device__ __forceinline__ void store8(bf16* p, const float (&v)[8]) {
  uint4 o;
  __nv_bfloat162* h = reinterpret_cast<__nv_bfloat162*>(&o);
#pragma unroll
  for (int i = 0; i < 4; ++i) h[i] = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
  *reinterpret_cast<uint4*>(p) = o;
}
__device__ __forceinline__ void store8(float* p, const float (&v)[8]) {
  reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
  reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
}
__device__ __forceinline__ uint2 quantise8(const float (&v)[8], float f) {
  uint2 o;
  o.x = f32x2_to_e4m3x2(v[0] * f, v[1] * f) | (uint32_t)f32x2_to_e4m3x2(v[2] * f, v[3] * f) << 16;
  o.y = f32x2_to_e4m3x2(v[4] * f, v[5] * f) | (uint32_t)f32x2_to_e4m3x2(v[6] * f, v[7] * f) << 16;
  return o;
}

// The two chunks of thread i (of D / 16) of a row: with pairs (c, c + rot / 2)
// the halves of 8 pairs, else two neighbouring chunks.
__device__ __forceinline__ void chunks_of(const RotArgs& r, int i, int* c0, int* c1) {
  const bool split = !r.interleaved && 16 * i < r.rot;
  *c0 = split ? i : 2 * i;
  *c1 = split ? i + (r.rot >> 4) : 2 * i + 1;
}

// Rotates the two chunks x, y of thread i by the angles of a position, cs and
// sn being the 8 cosines and sines from 8 i of its row of the tables.
__device__ __forceinline__ void rotate(const RotArgs& r, const float (&cs)[8], const float (&sn)[8], float (&x)[8],
                                       float (&y)[8]) {
  if (r.interleaved) {
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const float a = x[2 * u], z = x[2 * u + 1];
      x[2 * u] = __fsub_rn(__fmul_rn(a, cs[u]), __fmul_rn(z, sn[u]));
      x[2 * u + 1] = __fadd_rn(__fmul_rn(z, cs[u]), __fmul_rn(a, sn[u]));
      const float b = y[2 * u], w = y[2 * u + 1];
      y[2 * u] = __fsub_rn(__fmul_rn(b, cs[4 + u]), __fmul_rn(w, sn[4 + u]));
      y[2 * u + 1] = __fadd_rn(__fmul_rn(w, cs[4 + u]), __fmul_rn(b, sn[4 + u]));
    }
  } else {
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      const float a = x[u], z = y[u];
      x[u] = __fsub_rn(__fmul_rn(a, cs[u]), __fmul_rn(z, sn[u]));
      y[u] = __fadd_rn(__fmul_rn(z, cs[u]), __fmul_rn(a, sn[u]));
    }
  }
}

// New tokens of sequence bi: positions [start, end), end <= start + BCP. Negative lengths, counts
// out of range, and tokens past the cache or the angle table, are latched and
// left out.
__device__ __forceinline__ void new_range(const CacheAppendArgs& a, int bi, int* start, int* end) {
  const int len = __ldcg(a.c.seq_len + bi);
  const int want = a.new_len != nullptr ? __ldcg(a.new_len + bi) : a.BCP;
  const int n = min(max(want, 0), a.BCP);
  bool bad = n != want;
  if (len < 0 || len > a.limit) {
    *start = *end = 0;
    bad = bad || len < 0 || n > 0;  // (no tokens: the angles need not reach the length)
  } else {
    *start = len;
    *end = (int)min((int64_t)len + n, (int64_t)a.limit);
    bad = bad || *end - *start < n;
  }
  if (bad && a.status != nullptr) latch_status(a.status, 6 /* QUOKA_ERR_BOUNDS */);
}

// Grid: nkvu key / value CTAs, then the query CTAs. NT threads; NP passes of
// NT * 16 / D rows that cover the new tokens of a page.
template <typename T, int D, int NT, int NP>
__global__ void __launch_bounds__(NT) cache_append_kernel(const CacheAppendArgs a, int npt, int nkvu) {
  constexpr int TPR = D / 16;    // threads of a row
  constexpr int RPP = NT / TPR;  // rows of a pass
  const int tid = threadIdx.x, i = tid % TPR, rr = tid / TPR;
  const RotArgs rot{a.cos, a.sin, a.rot, a.interleaved};
  const int half = a.rot >> 1;
  pdl_wait();

  if ((int)blockIdx.x >= nkvu) {
    // ---------------------------------------------------------- queries
    const int hgroups = (a.nq + kQHeads - 1) / kQHeads;
    const int u = blockIdx.x - nkvu;
    const int64_t g = (int64_t)(u / hgroups) * RPP + rr;  // token over the batch
    const int h0 = (u % hgroups) * kQHeads;
    if (g >= (int64_t)a.b * a.BCP) return;
    const int bi = (int)(g / a.BCP), t = (int)(g % a.BCP);
    int c0, c1;
    chunks_of(rot, i, &c0, &c1);
    const T* q = static_cast<const T*>(a.Q.data) + bi * a.Q.sb + (int64_t)t * a.Q.st;
    Raw8<T> rx[kQHeads], ry[kQHeads];
#pragma unroll
    for (int k = 0; k < kQHeads; ++k)
      if (h0 + k < a.nq) {
        load_raw(q + (h0 + k) * a.Q.sh + 8 * c0, rx[k]);
        load_raw(q + (h0 + k) * a.Q.sh + 8 * c1, ry[k]);
      }
    int start, end;
    new_range(a, bi, &start, &end);
    T* o = static_cast<T*>(a.Qr) + ((int64_t)bi * a.nq * a.BCP + t) * D;
    if (start + t >= end) {
      if (a.zero_rest != 0) {
        const float z[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
        for (int h = h0; h < min(h0 + kQHeads, a.nq); ++h) {
          store8(o + (int64_t)h * a.BCP * D + 8 * c0, z);
          store8(o + (int64_t)h * a.BCP * D + 8 * c1, z);
        }
      }
      return;
    }
    const bool turn = 16 * i < a.rot;
    float cs[8], sn[8];
    if (turn) {
      load8(a.cos + (int64_t)(start + t) * half + 8 * i, cs);
      load8(a.sin + (int64_t)(start + t) * half + 8 * i, sn);
    }
#pragma unroll
    for (int k = 0; k < kQHeads; ++k)
      if (h0 + k < a.nq) {
        float x[8], y[8];
        to_floats(rx[k], x);
        to_floats(ry[k], y);
        if (turn) rotate(rot, cs, sn, x, y);
        store8(o + (int64_t)(h0 + k) * a.BCP * D + 8 * c0, x);
        store8(o + (int64_t)(h0 + k) * a.BCP * D + 8 * c1, y);
      }
    return;
  }

  // ------------------------------------------------------------ keys, values
  __shared__ uint32_t wmax[NT / 32];
  const int nkv = a.c.nkv;
  const bool is_v = blockIdx.x & 1;
  const int j = (blockIdx.x >> 1) % nkv;
  const int pt = (int)(blockIdx.x >> 1) / nkv % npt;
  const int bi = (int)(blockIdx.x >> 1) / nkv / npt;
  int start, end;
  new_range(a, bi, &start, &end);
  const int col = (start >> a.c.page_log2) + pt;
  const int p0 = col << a.c.page_log2;
  const int t0 = max(start, p0), t1 = min(end, p0 + (1 << a.c.page_log2));
  if (a.zero_rest != 0 && !is_v && a.Kr != nullptr) {  // rows of tokens at this page's positions that are left out
    const float z[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    const int z1 = min(start + a.BCP, p0 + (1 << a.c.page_log2));
    for (int t = max(end, p0) + rr; t < z1; t += RPP) {
      T* o = static_cast<T*>(a.Kr) + (((int64_t)bi * nkv + j) * a.BCP + (t - start)) * D + 16 * i;
      store8(o, z);
      store8(o + 8, z);
    }
  }
  if (t0 >= t1) return;  // (the same for the whole CTA)
  const int pid = __ldcg(a.c.page_table + (int64_t)bi * a.c.table_stride + col);
  const Strided X = is_v ? a.V : a.K;
  const T* x0 = static_cast<const T*>(X.data) + bi * X.sb + j * X.sh;
  int c0 = 2 * i, c1 = 2 * i + 1;
  const bool turn = !is_v && 16 * i < a.rot;
  if (turn) chunks_of(rot, i, &c0, &c1);

  float x[NP][8], y[NP][8];
  uint32_t top = 0u;  // bits of the largest finite magnitude
  Raw8<T> rx[NP], ry[NP];
#pragma unroll
  for (int k = 0; k < NP; ++k) {
    const int t = t0 + k * RPP + rr;
    if (t < t1) {
      load_raw(x0 + (int64_t)(t - start) * X.st + 8 * c0, rx[k]);
      load_raw(x0 + (int64_t)(t - start) * X.st + 8 * c1, ry[k]);
    }
  }
  float cs[8], sn[8];  // angles: the first pass's are fetched with the rows
  auto angles = [&](int t) {
    load8(a.cos + (int64_t)t * half + 8 * i, cs);
    load8(a.sin + (int64_t)t * half + 8 * i, sn);
  };
  if (turn && t0 + rr < t1) angles(t0 + rr);
  float* scale = (is_v ? a.c.v_scale : a.c.k_scale) + (int64_t)pid * nkv + j;
  float old = 0.f;  // (fetched while the rows arrive)
  if (t0 > p0 && pid >= 0 && pid < a.c.npages) old = __ldcg(scale);
#pragma unroll
  for (int k = 0; k < NP; ++k) {
    const int t = t0 + k * RPP + rr;
    if (t >= t1) continue;
    to_floats(rx[k], x[k]);
    to_floats(ry[k], y[k]);
    if (turn) {
      if (k > 0) angles(t);
      rotate(rot, cs, sn, x[k], y[k]);
    }
    if (!is_v && a.Kr != nullptr) {
      T* o = static_cast<T*>(a.Kr) + (((int64_t)bi * nkv + j) * a.BCP + (t - start)) * D;
      store8(o + 8 * c0, x[k]);
      store8(o + 8 * c1, y[k]);
    }
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      const uint32_t mx = __float_as_uint(x[k][u]) & 0x7FFFFFFFu, my = __float_as_uint(y[k][u]) & 0x7FFFFFFFu;
      if (mx < 0x7F800000u) top = max(top, mx);
      if (my < 0x7F800000u) top = max(top, my);
    }
  }
  const bool held = pid >= 0 && pid < a.c.npages;
  if (!held) {  // (the same for the whole CTA)
    if (tid == 0 && a.status != nullptr) latch_status(a.status, 6 /* QUOKA_ERR_BOUNDS */);
    return;
  }
  top = __reduce_max_sync(0xffffffffu, top);
  if ((tid & 31) == 0) wmax[tid >> 5] = top;
  __syncthreads();  // (the old scale is read by all before it is replaced below)
#pragma unroll
  for (int w = 0; w < NT / 32; ++w) top = max(top, wmax[w]);
  int e = scale_exp_for(__uint_as_float(top));
  uint8_t* dst = (is_v ? a.c.v : a.c.k) + pid * a.c.sp + j * a.c.sh;
  if (t0 > p0) {  // the page holds earlier tokens
    bool bad = false;
    const int eo = scale_exp(old, &bad);
    if (bad && tid == 0 && a.status != nullptr) latch_status(a.status, 6 /* QUOKA_ERR_BOUNDS */);
    if (e > eo) {
      const float f = exp2i(eo - e);
      for (int r = rr; r < t0 - p0; r += RPP) {
        uint4* p = reinterpret_cast<uint4*>(dst + r * a.c.sr + 16 * i);
        const uint4 w = *p;
        float v[8], z[8];
        e4m3x4_to_f32(w.x, v);
        e4m3x4_to_f32(w.y, v + 4);
        e4m3x4_to_f32(w.z, z);
        e4m3x4_to_f32(w.w, z + 4);
        const uint2 lo = quantise8(v, f), hi = quantise8(z, f);
        *p = make_uint4(lo.x, lo.y, hi.x, hi.y);
      }
    } else {
      e = eo;
    }
  }
  const float f = exp2i(-e);
#pragma unroll
  for (int k = 0; k < NP; ++k) {
    const int t = t0 + k * RPP + rr;
    if (t < t1) {
      uint8_t* o = dst + (int64_t)(t - p0) * a.c.sr;
      *reinterpret_cast<uint2*>(o + 8 * c0) = quantise8(x[k], f);
      *reinterpret_cast<uint2*>(o + 8 * c1) = quantise8(y[k], f);
    }
  }
  if (tid == 0) *scale = exp2i(e);
}

template <typename T, int D, int NT, int NP>
cudaError_t launch_grid(const CacheAppendArgs& a, bool pdl, cudaStream_t stream) {
  constexpr int RPP = NT * 16 / D;
  const int page = 1 << a.c.page_log2;
  const int npt = (a.BCP + 2 * page - 2) / page;  // pages a run of BCP tokens can touch
  const int64_t nkvu = (int64_t)a.b * npt * a.c.nkv * 2;
  const int64_t nqu = a.Qr != nullptr ? ((int64_t)a.b * a.BCP + RPP - 1) / RPP * ((a.nq + kQHeads - 1) / kQHeads) : 0;
  if (nkvu + nqu > 0x7FFFFFFF) return cudaErrorNotSupported;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(nkvu + nqu));
  cfg.blockDim = dim3(NT);
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = pdl ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, cache_append_kernel<T, D, NT, NP>, a, npt, (int)nkvu);
}

// CTAs of 64 threads while one pass of theirs covers the new tokens of a page,
// else of 256.
template <typename T, int D>
cudaError_t launch_typed(const CacheAppendArgs& a, bool pdl, cudaStream_t stream) {
  const int page = 1 << a.c.page_log2, rows = a.BCP < page ? a.BCP : page;
  if (rows <= 1024 / D) return launch_grid<T, D, 64, 1>(a, pdl, stream);
  const int np = (rows + 4096 / D - 1) / (4096 / D);
  if (np <= 1) return launch_grid<T, D, 256, 1>(a, pdl, stream);
  if (np <= 2) return launch_grid<T, D, 256, 2>(a, pdl, stream);
  return launch_grid<T, D, 256, 4>(a, pdl, stream);  // (pages have at most 128 rows)
}

}  // namespace

cudaError_t launch_cache_append(bool is_bf16, int d, const CacheAppendArgs& a, bool pdl, cudaStream_t stream) {
  if (a.b < 1 || a.BCP < 1) return cudaErrorInvalidValue;
  if (d == 128) return is_bf16 ? launch_typed<bf16, 128>(a, pdl, stream) : launch_typed<float, 128>(a, pdl, stream);
  if (d == 64) return is_bf16 ? launch_typed<bf16, 64>(a, pdl, stream) : launch_typed<float, 64>(a, pdl, stream);
  return cudaErrorNotSupported;
}

}  // namespace quoka

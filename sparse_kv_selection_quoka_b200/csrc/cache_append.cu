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
// launch, each over a few heads of 256 * 8 / d tokens, so that a token's
// cosines are read once for several heads.
// Bound by bytes: every row is read once and written once as codes (and once
// rotated).
#include "cache.cuh"

namespace quoka {

namespace {

using namespace cache;

constexpr int kThreads = 256;
constexpr int kQHeads = 4;  // query heads of one rotating CTA

struct RotArgs {
  const float* cos;
  const float* sin;  // (npos, rot / 2)
  int rot, interleaved;
};

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

// cos / sin of the 8 columns from 8 * c of a row at position `pos`, ready for
// out[u] = x[u] * cs[u] + y[u] * sn[u] with y the partner columns (sn carries
// the sign). Columns past `rot` are left alone by the caller.
__device__ __forceinline__ void load_angles(const RotArgs& r, int pos, int c, float (&cs)[8], float (&sn)[8]) {
  const int half = r.rot >> 1;
  if (r.interleaved) {  // pairs (2i, 2i + 1): this chunk holds pairs 4c .. 4c + 3
    const float4 a = __ldg(reinterpret_cast<const float4*>(r.cos + (int64_t)pos * half + 4 * c));
    const float4 b = __ldg(reinterpret_cast<const float4*>(r.sin + (int64_t)pos * half + 4 * c));
    cs[0] = cs[1] = a.x; cs[2] = cs[3] = a.y; cs[4] = cs[5] = a.z; cs[6] = cs[7] = a.w;
    sn[1] = b.x; sn[3] = b.y; sn[5] = b.z; sn[7] = b.w;
    sn[0] = -b.x; sn[2] = -b.y; sn[4] = -b.z; sn[6] = -b.w;
  } else {  // pairs (i, i + rot / 2)
    const bool second = 8 * c >= half;
    const int i = 8 * c - (second ? half : 0);
    load8(r.cos + (int64_t)pos * half + i, cs);
    load8(r.sin + (int64_t)pos * half + i, sn);
    if (!second) {
#pragma unroll
      for (int u = 0; u < 8; ++u) sn[u] = -sn[u];
    }
  }
}

// The rotated 8 columns from 8 * c of the row at `p`. (x * c + y * (-s) and
// x * c - y * s round alike.)
template <typename T>
__device__ __forceinline__ void load_rotated(const T* p, const RotArgs& r, int c, const float (&cs)[8],
                                             const float (&sn)[8], float (&x)[8]) {
  load8(p + 8 * c, x);
  if (8 * c >= r.rot) return;
  float y[8];
  if (r.interleaved) {
#pragma unroll
    for (int u = 0; u < 8; ++u) y[u] = x[u ^ 1];
  } else {
    const int half = r.rot >> 1;
    load8(p + 8 * c + (8 * c < half ? half : -half), y);
  }
#pragma unroll
  for (int u = 0; u < 8; ++u) x[u] = __fadd_rn(__fmul_rn(x[u], cs[u]), __fmul_rn(y[u], sn[u]));
}

// New tokens of sequence bi: positions [start, end). Lengths and counts out
// of range, and tokens past the cache or the angle table, are latched and
// left out.
__device__ __forceinline__ void new_range(const CacheAppendArgs& a, int bi, int* start, int* end) {
  const int len = __ldcg(a.c.seq_len + bi);
  const int want = a.new_len != nullptr ? __ldcg(a.new_len + bi) : a.BCP;
  const int n = min(max(want, 0), a.BCP);
  bool bad = n != want;
  if (len < 0 || len > a.limit) {
    *start = *end = 0;
    bad = true;
  } else {
    *start = len;
    *end = (int)min((int64_t)len + n, (int64_t)a.limit);
    bad = bad || *end - *start < n;
  }
  if (bad && a.status != nullptr) latch_status(a.status, 6 /* QUOKA_ERR_BOUNDS */);
}

// Grid: nkvu key / value CTAs, then the query CTAs. NP: passes of
// 256 * 8 / D rows that cover a page.
template <typename T, int D, int NP>
__global__ void __launch_bounds__(kThreads) cache_append_kernel(const CacheAppendArgs a, int npt, int nkvu) {
  constexpr int CPR = D / 8;           // 8-column chunks per row
  constexpr int RPP = kThreads / CPR;  // rows per pass
  const int tid = threadIdx.x, c = tid % CPR, rr = tid / CPR;
  const RotArgs rot{a.cos, a.sin, a.rot, a.interleaved};
  pdl_wait();

  if ((int)blockIdx.x >= nkvu) {
    // ---------------------------------------------------------- queries
    const int hgroups = (a.nq + kQHeads - 1) / kQHeads;
    const int u = blockIdx.x - nkvu;
    const int64_t g = (int64_t)(u / hgroups) * RPP + rr;  // token over the batch
    const int h0 = (u % hgroups) * kQHeads;
    if (g >= (int64_t)a.b * a.BCP) return;
    const int bi = (int)(g / a.BCP), t = (int)(g % a.BCP);
    int start, end;
    new_range(a, bi, &start, &end);
    if (start + t >= end) return;
    float cs[8], sn[8];
    if (8 * c < a.rot) load_angles(rot, start + t, c, cs, sn);
    const T* q = static_cast<const T*>(a.Q.data) + bi * a.Q.sb + t * a.Q.st;
    T* o = static_cast<T*>(a.Qr) + ((int64_t)bi * a.nq * a.BCP + t) * D + 8 * c;
#pragma unroll
    for (int i = 0; i < kQHeads; ++i) {
      const int h = h0 + i;
      if (h < a.nq) {
        float x[8];
        load_rotated(q + h * a.Q.sh, rot, c, cs, sn, x);
        store8(o + (int64_t)h * a.BCP * D, x);
      }
    }
    return;
  }

  // ------------------------------------------------------------ keys, values
  __shared__ uint32_t wmax[kThreads / 32];
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
  if (t0 >= t1) return;  // (the same for the whole CTA)
  const Strided X = is_v ? a.V : a.K;
  const T* x0 = static_cast<const T*>(X.data) + bi * X.sb + j * X.sh;
  const int page = cache_page(a.c, bi, col, a.status);

  float x[NP][8];
  uint32_t top = 0u;  // bits of the largest finite magnitude
#pragma unroll
  for (int i = 0; i < NP; ++i) {
    const int t = t0 + i * RPP + rr;
    if (t < t1) {
      const T* row = x0 + (int64_t)(t - start) * X.st;
      if (is_v) {
        load8(row + 8 * c, x[i]);
      } else {
        float cs[8], sn[8];
        if (8 * c < a.rot) load_angles(rot, t, c, cs, sn);
        load_rotated(row, rot, c, cs, sn, x[i]);
        if (a.Kr != nullptr)
          store8(static_cast<T*>(a.Kr) + (((int64_t)bi * nkv + j) * a.BCP + (t - start)) * D + 8 * c, x[i]);
      }
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        const uint32_t m = __float_as_uint(x[i][u]) & 0x7FFFFFFFu;
        if (m < 0x7F800000u) top = max(top, m);
      }
    }
  }
  top = __reduce_max_sync(0xffffffffu, top);
  if ((tid & 31) == 0) wmax[tid >> 5] = top;
  float* scale = (is_v ? a.c.v_scale : a.c.k_scale) + (int64_t)max(page, 0) * nkv + j;
  const float old = page >= 0 && t0 > p0 ? __ldcg(scale) : 0.f;
  __syncthreads();  // (the old scale is read by all before it is replaced below)
  if (page < 0) return;
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) top = max(top, wmax[w]);
  int e = scale_exp_for(__uint_as_float(top));
  uint8_t* dst = (is_v ? a.c.v : a.c.k) + page * a.c.sp + j * a.c.sh;
  if (t0 > p0) {  // the page holds earlier tokens
    bool bad = false;
    const int eo = scale_exp(old, &bad);
    if (bad && tid == 0 && a.status != nullptr) latch_status(a.status, 6 /* QUOKA_ERR_BOUNDS */);
    if (e > eo) {
      const float f = exp2i(eo - e);
      for (int r = rr; r < t0 - p0; r += RPP) {
        uint2* p = reinterpret_cast<uint2*>(dst + r * a.c.sr + 8 * c);
        const uint2 w = *p;
        float v[8];
        e4m3x4_to_f32(w.x, v);
        e4m3x4_to_f32(w.y, v + 4);
        uint2 o;
        o.x = f32x2_to_e4m3x2(v[0] * f, v[1] * f) | (uint32_t)f32x2_to_e4m3x2(v[2] * f, v[3] * f) << 16;
        o.y = f32x2_to_e4m3x2(v[4] * f, v[5] * f) | (uint32_t)f32x2_to_e4m3x2(v[6] * f, v[7] * f) << 16;
        *p = o;
      }
    } else {
      e = eo;
    }
  }
  const float f = exp2i(-e);
#pragma unroll
  for (int i = 0; i < NP; ++i) {
    const int t = t0 + i * RPP + rr;
    if (t < t1) {
      uint2 o;
      o.x = f32x2_to_e4m3x2(x[i][0] * f, x[i][1] * f) | (uint32_t)f32x2_to_e4m3x2(x[i][2] * f, x[i][3] * f) << 16;
      o.y = f32x2_to_e4m3x2(x[i][4] * f, x[i][5] * f) | (uint32_t)f32x2_to_e4m3x2(x[i][6] * f, x[i][7] * f) << 16;
      *reinterpret_cast<uint2*>(dst + (int64_t)(t - p0) * a.c.sr + 8 * c) = o;
    }
  }
  if (tid == 0) *scale = exp2i(e);
}

template <typename T, int D>
cudaError_t launch_typed(const CacheAppendArgs& a, bool pdl, cudaStream_t stream) {
  constexpr int RPP = kThreads * 8 / D;
  const int page = 1 << a.c.page_log2;
  const int npt = (a.BCP + 2 * page - 2) / page;  // pages a run of BCP tokens can touch
  const int64_t nkvu = (int64_t)a.b * npt * a.c.nkv * 2;
  const int64_t nqu = a.Qr != nullptr ? ((int64_t)a.b * a.BCP + RPP - 1) / RPP * ((a.nq + kQHeads - 1) / kQHeads) : 0;
  if (nkvu + nqu > 0x7FFFFFFF) return cudaErrorNotSupported;
  const int np = (page + RPP - 1) / RPP;
  auto* kern = np <= 1   ? cache_append_kernel<T, D, 1>
               : np <= 2 ? cache_append_kernel<T, D, 2>
               : np <= 4 ? cache_append_kernel<T, D, 4>
                         : cache_append_kernel<T, D, 8>;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(nkvu + nqu));
  cfg.blockDim = dim3(kThreads);
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = pdl ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kern, a, npt, (int)nkvu);
}

}  // namespace

cudaError_t launch_cache_append(bool is_bf16, int d, const CacheAppendArgs& a, bool pdl, cudaStream_t stream) {
  if (a.b < 1 || a.BCP < 1) return cudaErrorInvalidValue;
  if (d == 128) return is_bf16 ? launch_typed<bf16, 128>(a, pdl, stream) : launch_typed<float, 128>(a, pdl, stream);
  if (d == 64) return is_bf16 ? launch_typed<bf16, 64>(a, pdl, stream) : launch_typed<float, 64>(a, pdl, stream);
  return cudaErrorNotSupported;
}

}  // namespace quoka

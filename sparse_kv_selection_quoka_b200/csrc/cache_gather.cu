// Rows of the paged 8-bit cache as contiguous wider rows.
//
// [QUOKA §4.2, problem 3] the selected KV becomes the attention's input KV:
//   Ksel[b, j, n] = K[b, j, kv_idx[b, j, n]] for n < kv_count[b, j],
// with K read through the page table and multiplied by its page's scale
// (exact: a code has 4 significant bits and the scale is a power of two).
// Without an index list row n is key n, n < seq_len[b]. Rows past the count
// are zeros, so that the copy can be handed to the attention as it is.
//
// Bound by bytes: a row of d codes is read, one of d bf16 or fp32 written.
// Each thread converts kItems chunks of 8 codes of K and of V, all their
// loads in flight together; consecutive threads take consecutive chunks.
#include "cache.cuh"

namespace quoka {

namespace {

using namespace cache;

constexpr int kThreads = 256;
constexpr int kItems = 4;

__device__ __forceinline__ uint2 ld_codes(const uint8_t* p) {
  uint2 v;
  asm volatile("ld.global.L1::no_allocate.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "l"(p));
  return v;
}

__device__ __forceinline__ void store8(bf16* p, uint2 w, float f) {
  float v[8];
  e4m3x4_to_f32(w.x, v);
  e4m3x4_to_f32(w.y, v + 4);
  uint4 o;
  __nv_bfloat162* h = reinterpret_cast<__nv_bfloat162*>(&o);
#pragma unroll
  for (int i = 0; i < 4; ++i) h[i] = __floats2bfloat162_rn(v[2 * i] * f, v[2 * i + 1] * f);
  *reinterpret_cast<uint4*>(p) = o;
}
__device__ __forceinline__ void store8(float* p, uint2 w, float f) {
  float v[8];
  e4m3x4_to_f32(w.x, v);
  e4m3x4_to_f32(w.y, v + 4);
  reinterpret_cast<float4*>(p)[0] = make_float4(v[0] * f, v[1] * f, v[2] * f, v[3] * f);
  reinterpret_cast<float4*>(p)[1] = make_float4(v[4] * f, v[5] * f, v[6] * f, v[7] * f);
}

// grid (ceil(N * D / 8 / (kThreads * kItems)), nkv, b)
template <typename T, int D>
__global__ void __launch_bounds__(kThreads) cache_gather_kernel(const CacheGatherArgs a) {
  constexpr int CPR = D / 8;
  const int j = blockIdx.y, bi = blockIdx.z;
  const int64_t row = (int64_t)bi * a.c.nkv + j;
  pdl_trigger();
  pdl_wait();
  const int len = cache_len(a.c, bi, a.max_len, a.status);
  const int cnt = a.kv_idx != nullptr ? min(max(__ldcg(a.kv_count + row), 0), a.N) : len;
  if (a.count_out != nullptr && blockIdx.x == 0 && threadIdx.x == 0) a.count_out[row] = cnt;
  const int64_t nitems = (int64_t)a.N * CPR;
  const int64_t i0 = (int64_t)blockIdx.x * (kThreads * kItems) + threadIdx.x;
  uint2 kw[kItems], vw[kItems];
  float kf[kItems], vf[kItems];
  bool bad = false;
#pragma unroll
  for (int u = 0; u < kItems; ++u) {
    const int64_t i = i0 + u * kThreads;
    const int n = (int)(i / CPR), c = (int)(i % CPR);
    kw[u] = vw[u] = make_uint2(0u, 0u);
    kf[u] = vf[u] = 1.f;
    if (i >= nitems || n >= cnt) continue;
    const int tau = a.kv_idx != nullptr ? __ldcg(a.kv_idx + row * a.N + n) : n;
    if (tau < 0 || tau >= len) {
      bad = true;  // not read; written as zeros
      continue;
    }
    const int p = cache_page(a.c, bi, tau >> a.c.page_log2, a.status);
    if (p < 0) continue;
    const int64_t off = p * a.c.sp + j * a.c.sh + (tau & ((1 << a.c.page_log2) - 1)) * a.c.sr + 8 * c;
    kw[u] = ld_codes(a.c.k + off);
    vw[u] = ld_codes(a.c.v + off);
    kf[u] = exp2i(scale_exp(__ldcg(a.c.k_scale + (int64_t)p * a.c.nkv + j), &bad));
    vf[u] = exp2i(scale_exp(__ldcg(a.c.v_scale + (int64_t)p * a.c.nkv + j), &bad));
  }
#pragma unroll
  for (int u = 0; u < kItems; ++u) {
    const int64_t i = i0 + u * kThreads;
    if (i < nitems) {
      store8(static_cast<T*>(a.Ksel) + row * a.N * D + 8 * i, kw[u], kf[u]);
      store8(static_cast<T*>(a.Vsel) + row * a.N * D + 8 * i, vw[u], vf[u]);
    }
  }
  if (bad && a.status != nullptr) latch_status(a.status, 6 /* QUOKA_ERR_BOUNDS */);
}

}  // namespace

cudaError_t launch_cache_gather(bool is_bf16, int d, const CacheGatherArgs& a, bool pdl, cudaStream_t stream) {
  if (a.N < 1) return cudaErrorInvalidValue;
  if (d != 64 && d != 128) return cudaErrorNotSupported;
  const int64_t nitems = (int64_t)a.N * (d / 8), per_block = (int64_t)kThreads * kItems;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((nitems + per_block - 1) / per_block), a.c.nkv, a.b);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = pdl ? 1 : 0;
  auto* kern = d == 128 ? (is_bf16 ? cache_gather_kernel<bf16, 128> : cache_gather_kernel<float, 128>)
                        : (is_bf16 ? cache_gather_kernel<bf16, 64> : cache_gather_kernel<float, 64>);
  return cudaLaunchKernelEx(&cfg, kern, a);
}

}  // namespace quoka

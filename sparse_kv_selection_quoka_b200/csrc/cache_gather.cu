// Rows of the paged 8-bit cache as contiguous wider rows.
//
// [QUOKA §4.2, problem 3] the selected KV becomes the attention's input KV:
//   Ksel[b, j, n] = K[b, j, kv_idx[b, j, n]] for n < kv_count[b, j],
// with K read through the page table and multiplied by its page's scale
// (exact: a code has 4 significant bits and the scale is a power of two).
// Without an index list row n is key n, n < seq_len[b]. Rows past the count
// are zeros, so that the copy can be handed to the attention as it is.
//
// Bound by bytes: a row of d codes is read, one of d bf16 or fp32 written. A
// warp takes 16 rows: each is looked up by one lane, then all their code loads
// (K and V) are issued together and converted as they arrive, 16 bytes of
// output a lane, consecutive lanes writing consecutive bytes. Measured: 4096 of
// 32768 rows of 8 heads, d = 128, bf16 7.6 us for 25.2 MB (10.9 with every lane
// looking up its own 8 codes); 5 ragged sequences of up to 2999 rows, d = 64,
// fp32 8.1 us for 35.5 MB (15.1).
#include "cache.cuh"

namespace quoka {

namespace {

using namespace cache;

constexpr int kThreads = 128;
constexpr int kRows = 16;  // rows of a warp

template <int N>
struct Codes {  // N codes
  uint32_t w[N / 4];
};
__device__ __forceinline__ Codes<8> ld_codes(const uint8_t* p, Codes<8>*) {
  Codes<8> c;
  asm volatile("ld.global.L1::no_allocate.v2.u32 {%0, %1}, [%2];" : "=r"(c.w[0]), "=r"(c.w[1]) : "l"(p));
  return c;
}
__device__ __forceinline__ Codes<4> ld_codes(const uint8_t* p, Codes<4>*) {
  Codes<4> c;
  asm volatile("ld.global.L1::no_allocate.u32 %0, [%1];" : "=r"(c.w[0]) : "l"(p));
  return c;
}

__device__ __forceinline__ void st_row(bf16* p, const Codes<8>& c, float f) {
  float v[8];
  e4m3x4_to_f32(c.w[0], v);
  e4m3x4_to_f32(c.w[1], v + 4);
  uint4 o;
  __nv_bfloat162* h = reinterpret_cast<__nv_bfloat162*>(&o);
#pragma unroll
  for (int i = 0; i < 4; ++i) h[i] = __floats2bfloat162_rn(v[2 * i] * f, v[2 * i + 1] * f);
  *reinterpret_cast<uint4*>(p) = o;
}
__device__ __forceinline__ void st_row(float* p, const Codes<4>& c, float f) {
  float v[4];
  e4m3x4_to_f32(c.w[0], v);
  *reinterpret_cast<float4*>(p) = make_float4(v[0] * f, v[1] * f, v[2] * f, v[3] * f);
}

// grid (ceil(N / (kRows * warps)), nkv, b)
template <typename T, int D>
__global__ void __launch_bounds__(kThreads) cache_gather_kernel(const CacheGatherArgs a) {
  constexpr int VE = 16 / sizeof(T);  // codes of a lane
  constexpr int LPR = D / VE, RPI = 32 / LPR, ITER = kRows / RPI;
  const int j = blockIdx.y, bi = blockIdx.z, lane = threadIdx.x & 31;
  const int64_t row = (int64_t)bi * a.c.nkv + j;
  pdl_trigger();
  pdl_wait();
  const int n0 = ((int)blockIdx.x * (kThreads / 32) + ((int)threadIdx.x >> 5)) * kRows;
  const int n = n0 + (lane & (kRows - 1));  // the row this lane looks up
  // (an entry past the count is read, not used: the load need not wait for the count)
  int tau = n;
  if (a.kv_idx != nullptr && n < a.N) tau = __ldcg(a.kv_idx + row * a.N + n);
  const int want = __ldcg(a.c.seq_len + bi), len = min(max(want, 0), a.max_len);
  const int cnt = a.kv_idx != nullptr ? min(max(__ldcg(a.kv_count + row), 0), a.N) : len;
  if (a.count_out != nullptr && blockIdx.x == 0 && threadIdx.x == 0) a.count_out[row] = cnt;
  bool bad = want != len;
  int64_t off = -1;
  float kf = 1.f, vf = 1.f;
  if (n < cnt) {
    int p = -1;
    if (tau >= 0 && tau < len) p = __ldcg(a.c.page_table + (int64_t)bi * a.c.table_stride + (tau >> a.c.page_log2));
    if (p >= 0 && p < a.c.npages) {
      off = p * a.c.sp + j * a.c.sh + (int64_t)(tau & ((1 << a.c.page_log2) - 1)) * a.c.sr;
      kf = exp2i(scale_exp(__ldcg(a.c.k_scale + (int64_t)p * a.c.nkv + j), &bad));
      vf = exp2i(scale_exp(__ldcg(a.c.v_scale + (int64_t)p * a.c.nkv + j), &bad));
    } else {
      bad = true;  // not read; written as zeros
    }
  }
  const int r0 = lane / LPR, c = lane % LPR;
  Codes<VE> kc[ITER], vc[ITER];
#pragma unroll
  for (int i = 0; i < ITER; ++i) {
    const int64_t o = __shfl_sync(0xffffffffu, off, i * RPI + r0);
#pragma unroll
    for (int w = 0; w < VE / 4; ++w) kc[i].w[w] = vc[i].w[w] = 0u;
    if (o >= 0) {
      kc[i] = ld_codes(a.c.k + o + VE * c, static_cast<Codes<VE>*>(nullptr));
      vc[i] = ld_codes(a.c.v + o + VE * c, static_cast<Codes<VE>*>(nullptr));
    }
  }
  const int64_t at = (row * a.N + n0) * D + VE * lane;
  T* ko = static_cast<T*>(a.Ksel) + at;
  T* vo = static_cast<T*>(a.Vsel) + at;
#pragma unroll
  for (int i = 0; i < ITER; ++i) {
    const float fk = __shfl_sync(0xffffffffu, kf, i * RPI + r0), fv = __shfl_sync(0xffffffffu, vf, i * RPI + r0);
    if (n0 + i * RPI + r0 < a.N) {
      st_row(ko + i * RPI * D, kc[i], fk);
      st_row(vo + i * RPI * D, vc[i], fv);
    }
  }
  if (bad && a.status != nullptr) latch_status(a.status, 6 /* QUOKA_ERR_BOUNDS */);
}

}  // namespace

cudaError_t launch_cache_gather(bool is_bf16, int d, const CacheGatherArgs& a, bool pdl, cudaStream_t stream) {
  if (a.N < 1) return cudaErrorInvalidValue;
  if (d != 64 && d != 128) return cudaErrorNotSupported;
  const int64_t per_block = (int64_t)kRows * (kThreads / 32);
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((a.N + per_block - 1) / per_block), a.c.nkv, a.b);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = pdl ? 1 : 0;
  auto* kern = d == 128 ? (is_bf16 ? cache_gather_kernel<bf16, 128> : cache_gather_kernel<float, 128>)
                        : (is_bf16 ? cache_gather_kernel<bf16, 64> : cache_gather_kernel<float, 64>);
  return cudaLaunchKernelEx(&cfg, kern, a);
}

}  // namespace quoka

// C ABI of libquoka.so: argument validation, workspace carving and the launch
// sequence of the QUOKA step. See include/quoka.h for the contract of every
// entry point.
#include <cuda_runtime.h>
#include <stdint.h>
#include <string.h>

#include <algorithm>
#include <atomic>

#include "common.cuh"
#include "nvtx_range.h"
#include "kernels.h"
#include "quoka.h"

namespace quoka {

namespace {
// Test hooks of quoka_debug_set_wait_hooks (process-wide).
std::atomic<uint64_t> g_wait_ns{0};
std::atomic<uint32_t> g_inject{INJECT_NONE};
}  // namespace

WaitHooks wait_hooks() {
  const uint64_t ns = g_wait_ns.load(std::memory_order_relaxed);
  return WaitHooks{ns == 0 ? 2000000000ull : ns, g_inject.load(std::memory_order_relaxed)};
}

// Device address of quoka_select_static's fixed scratch (select_static.cu).
quoka_status static_scratch_address(void** out);

namespace {

// The status words of a call whose first kernel can itself latch a fault
// are cleared by this one-thread kernel. It lets the call's next kernel
// (launched with programmatic stream serialisation) start at once; that
// kernel's latches wait for this grid to complete first (latch_status).
__global__ void clear_status_kernel(int* status) {
  pdl_trigger();
  status[0] = 0;
  status[1] = 0;
}

}  // namespace

cudaError_t clear_status_async(int* status, cudaStream_t stream) {
  clear_status_kernel<<<1, 1, 0, stream>>>(status);
  return cudaGetLastError();
}

}  // namespace quoka

namespace {

using quoka::Strided;

constexpr size_t kAlign = 256;

size_t align_up(size_t x) { return (x + kAlign - 1) / kAlign * kAlign; }

// Workspace layout. Every region starts on a 256-byte boundary.
struct WsLayout {
  size_t status = 0;    // int32 device status word
  size_t qhat = 0;      // (b, nq, NQ, d) fp32: normalised chosen queries
  size_t qgroup = 0;    // (b, nkv, NQ, d) fp32: group means
  size_t qhilo = 0;     // (b, nkv, 2*NQ, d) bf16: hi / lo split of the group means
  size_t qidx = 0;      // (b, nq, NQ) int32
  size_t sagg = 0;      // (b, nkv, T) fp32
  size_t kvidx = 0;     // (b, nkv, BSA_eff) int32
  size_t kvcount = 0;   // (b, nkv) int32
  size_t hist = 0;      // (b, nkv, 4096) uint32: first-digit histogram of the score keys
  size_t select_total = 0;  // end of what quoka_select needs
  size_t ksel = 0;      // (b, nkv, BSA_eff, d) bf16: gathered selected K (tensor-core attention)
  size_t vsel = 0;      // (b, nkv, BSA_eff, d) bf16: gathered selected V
  size_t aparts = 0;    // split key ranges of the tensor-core attention: partials
  size_t aparts_bytes = 0;
  size_t dparts = 0;    // short chunks: (nsplit, b, nq, BCP, d) fp32 partial outputs
  size_t dlse = 0;      // short chunks: (nsplit, b, nq, BCP) fp32 partial log-sum-exps
  size_t total = 0;
};

// Key-range splits of the tensor-core attention over the gathered rows
// (bf16, d = 128) for a chunk of b * nq * ceil(BCP / 128) query tiles and
// BSA_eff selected keys (with the chunk's own keys unless no_chunk).
int attn_nsplit(int64_t b, int64_t nq, int64_t BCP, int64_t d, int64_t bsa_eff, bool bf16, bool no_chunk) {
  if (!bf16 || d != 128) return 1;
  const int64_t tiles = b * nq * ((BCP + 127) / 128);
  const int64_t nt = (bsa_eff + 127) / 128 + (no_chunk ? 0 : 1);
  return quoka::attn_splits(tiles, (int)std::min<int64_t>(nt, 1 << 20));
}

// Bytes of the partials of `nsplit` key ranges: (nsplit * b, nq, BCP, d)
// bf16 outputs, then (nsplit, b, nq, BCP) fp32 log-sum-exps.
size_t attn_parts_bytes(int64_t b, int64_t nq, int64_t BCP, int64_t d, int nsplit) {
  if (nsplit <= 1) return 0;
  const int64_t rows = (int64_t)nsplit * b * nq * BCP;
  return align_up((size_t)(rows * d) * 2) + align_up((size_t)rows * 4);
}

// Chunks whose G * BCP query rows per KV head fit one CTA of the decode
// attention take it (its fp32 partials live in the workspace).
bool short_chunk(int64_t nq, int64_t nkv, int64_t BCP, int64_t d) {
  return nkv > 0 && nq % nkv == 0 && (nq / nkv) * BCP <= quoka::kDecodeMaxRows && (d == 64 || d == 128);
}

// The tensor-core attention (bf16, d = 128) streams the selected rows from a
// contiguous gathered copy when the workspace holds one.
bool uses_gather_buffers(quoka_dtype dtype, int64_t d, int64_t bsa_eff) {
  return dtype == QUOKA_BF16 && d == 128 && bsa_eff > 0;
}

WsLayout ws_layout(int64_t b, int64_t nq, int64_t nkv, int64_t d, int64_t T, int64_t NQ,
                   int64_t bsa_eff, bool gather_buffers, int64_t BCP = 0, bool decode = false) {
  // (gather_buffers implies bf16, d = 128)
  WsLayout L;
  size_t off = 0;
  auto take = [&](size_t bytes) {
    const size_t at = off;
    off += align_up(bytes);
    return at;
  };
  L.status = take(kAlign);
  L.qhat = take((size_t)(b * nq * NQ * d) * 4);
  L.qgroup = take((size_t)(b * nkv * NQ * d) * 4);
  L.qhilo = take((size_t)(b * nkv * 2 * NQ * d) * 2);
  L.qidx = take((size_t)(b * nq * NQ) * 4);
  L.sagg = take((size_t)(b * nkv * T) * 4);
  L.kvidx = take((size_t)(b * nkv * bsa_eff) * 4);
  L.kvcount = take((size_t)(b * nkv) * 4);
  L.hist = take((size_t)(b * nkv) * quoka::TOPK_HIST_BINS * 4);
  L.select_total = off;
  if (gather_buffers) {
    L.ksel = take((size_t)(b * nkv * bsa_eff * d) * 2);
    L.vsel = take((size_t)(b * nkv * bsa_eff * d) * 2);
    if (BCP > 0) {
      L.aparts_bytes = attn_parts_bytes(b, nq, BCP, d, attn_nsplit(b, nq, BCP, d, bsa_eff, true, false));
      if (L.aparts_bytes > 0) L.aparts = take(L.aparts_bytes);
    }
  }
  if (decode) {
    const int64_t rows = (int64_t)quoka::decode_splits((int)bsa_eff, (int)BCP) * b * nq * BCP;
    L.dparts = take((size_t)(rows * d) * 4);
    L.dlse = take((size_t)rows * 4);
  }
  L.total = off;
  return L;
}

// Workspace of quoka_decode_attn: the status words, then the partials.
size_t decode_ws_bytes(int64_t b, int64_t nq, int64_t d, int64_t BCP, int64_t bsa_eff) {
  const int64_t rows = (int64_t)quoka::decode_splits((int)bsa_eff, (int)BCP) * b * nq * BCP;
  return kAlign + align_up((size_t)(rows * d) * 4) + align_up((size_t)rows * 4);
}

// Workspace of quoka_sparse_gqa_attn alone: the status words, then (when
// used) the gathered selected K and V.
size_t attn_ws_bytes(int64_t b, int64_t nkv, int64_t d, int64_t bsa_eff, bool gather_buffers) {
  size_t n = kAlign;
  if (gather_buffers) n += 2 * align_up((size_t)(b * nkv * bsa_eff * d) * 2);
  return n;
}

size_t elt_size(quoka_dtype t) { return t == QUOKA_BF16 ? 2 : 4; }

bool aligned16(const void* p) { return ((uintptr_t)p & 15u) == 0; }

// Checks a tensor's dtype, shape and strides. Extents equal to -1 in `want`
// are free and returned through `want`.
bool check_tensor(const quoka_tensor* t, quoka_dtype dtype, int64_t want[4]) {
  if (t == nullptr) return false;
  if (t->dtype != dtype) return false;
  for (int i = 0; i < 4; ++i) {
    if (t->shape[i] < 0) return false;
    if (want[i] >= 0 && t->shape[i] != want[i]) return false;
    want[i] = t->shape[i];
  }
  int64_t n = 1;
  for (int i = 0; i < 4; ++i) n *= t->shape[i];
  if (n == 0) return true;  // nothing is read: pointer and strides are irrelevant
  if (t->stride[3] != 1) return false;
  const int64_t es = (int64_t)elt_size(dtype);
  for (int i = 0; i < 3; ++i) {
    if (t->stride[i] < 0) return false;
    if ((t->stride[i] * es) % 16 != 0) return false;
  }
  if (t->data == nullptr || !aligned16(t->data)) return false;
  return true;
}

Strided strided(const quoka_tensor* t) {
  return Strided{t->data, t->stride[0], t->stride[1], t->stride[2]};
}

bool supported_d(int64_t d) { return d == 64 || d == 128; }

constexpr int64_t kMaxBCP = 16384;
constexpr int64_t kMaxHeads = 65535;

quoka_status cuda_status(cudaError_t e) {
  if (e == cudaSuccess) return QUOKA_OK;
  if (e == cudaErrorNotSupported) return QUOKA_ERR_UNSUPPORTED;
  return QUOKA_ERR_CUDA;
}

struct SelectShapes {
  int64_t b, nq, nkv, d, T, BCP;
};

quoka_status validate_select(const quoka_tensor* Q, const quoka_tensor* K, int NQ, int BSA,
                             SelectShapes* s) {
  if (Q == nullptr || K == nullptr) return QUOKA_ERR_INVALID_ARG;
  int64_t qs[4] = {-1, -1, -1, -1};
  if (!check_tensor(Q, Q->dtype, qs)) return QUOKA_ERR_INVALID_ARG;
  if (Q->dtype != QUOKA_F32 && Q->dtype != QUOKA_BF16) return QUOKA_ERR_INVALID_ARG;
  int64_t ks[4] = {qs[0], -1, -1, qs[3]};
  if (!check_tensor(K, Q->dtype, ks)) return QUOKA_ERR_INVALID_ARG;
  s->b = qs[0];
  s->nq = qs[1];
  s->BCP = qs[2];
  s->d = qs[3];
  s->nkv = ks[1];
  s->T = ks[2];
  if (s->b < 1 || s->nq < 1 || s->nkv < 1 || s->BCP < 1) return QUOKA_ERR_INVALID_ARG;
  if (s->nq % s->nkv != 0) return QUOKA_ERR_INVALID_ARG;
  if (NQ < 1 || NQ > s->BCP || BSA < 0) return QUOKA_ERR_INVALID_ARG;
  if (!supported_d(s->d)) return QUOKA_ERR_UNSUPPORTED;
  if (s->BCP > kMaxBCP || s->nq > kMaxHeads || s->nkv > kMaxHeads || s->b > kMaxHeads)
    return QUOKA_ERR_UNSUPPORTED;
  if (s->T > quoka::topk_max_T()) return QUOKA_ERR_UNSUPPORTED;
  return QUOKA_OK;
}

quoka_status check_ws(void* ws, size_t ws_bytes, size_t need) {
  if (ws == nullptr || ((uintptr_t)ws % kAlign) != 0 || ws_bytes < need) return QUOKA_ERR_WORKSPACE;
  return QUOKA_OK;
}

template <typename P>
P* at(void* ws, size_t off) {
  return reinterpret_cast<P*>(static_cast<char*>(ws) + off);
}

// Steps (a)-(e) after validation. kv_idx / kv_count / q_idx / s_agg are the
// final destinations (workspace regions when the caller passed none).
// `flags`: QUOKA_SCORE_DOT_PRODUCT selects the plain dot-product score (no
// L2 normalisation of the chosen queries or of the keys).
quoka_status run_select(const quoka_tensor* Q, const quoka_tensor* K, const SelectShapes& s, int NQ,
                        int bsa_eff, int32_t* kv_idx, int32_t* kv_count, int32_t* q_idx,
                        float* s_agg, void* ws, const WsLayout& L, cudaStream_t stream, uint32_t flags = 0u) {
  const bool cosine = (flags & QUOKA_SCORE_DOT_PRODUCT) == 0u;
  const bool bf = Q->dtype == QUOKA_BF16;
  const int b = (int)s.b, nq = (int)s.nq, nkv = (int)s.nkv, d = (int)s.d, BCP = (int)s.BCP;
  float* qhat = at<float>(ws, L.qhat);
  float* qg = at<float>(ws, L.qgroup);
  uint16_t* qhilo = at<uint16_t>(ws, L.qhilo);
  int32_t* qidx = q_idx != nullptr ? q_idx : at<int32_t>(ws, L.qidx);
  float* sagg = s_agg != nullptr ? s_agg : at<float>(ws, L.sagg);
  int* status = at<int>(ws, L.status);
  uint32_t* hist = at<uint32_t>(ws, L.hist);

  cudaError_t e = cudaErrorNotSupported;
  if (bf && d == 128)
    e = quoka::launch_qsel_group_fast(strided(Q), b, nq, nkv, BCP, NQ, qidx, qg, qhilo, hist, status, cosine,
                                      stream);
  if (e == cudaErrorNotSupported) {
    e = quoka::launch_qsel(bf, d, strided(Q), b, nq, BCP, NQ, qhat, qidx, cosine, stream);
    if (e != cudaSuccess) return cuda_status(e);
    e = quoka::launch_qgroup(d, qhat, b, nq, nkv, NQ, qg, bf ? qhilo : nullptr, bf ? hist : nullptr, status,
                             stream);
  }
  if (e != cudaSuccess) return cuda_status(e);
  bool hist_made = false;
  if (s.T > 0) {
    e = cudaErrorNotSupported;
    if (bf) {
      e = quoka::launch_score_tc(d, strided(K), b, nkv, s.T, qhilo, NQ, sagg, hist, status, true, cosine,
                                 stream);
      // the value-bucket histogram spans the cosine range [-1, 1]
      hist_made = e == cudaSuccess && cosine;
    }
    if (e == cudaErrorNotSupported)
      e = quoka::launch_score_simt(bf, d, strided(K), b, nkv, s.T, qg, NQ, sagg, cosine, stream);
    if (e != cudaSuccess) return cuda_status(e);
  }
  if (bsa_eff > 0) {
    e = quoka::launch_topk(sagg, b, nkv, s.T, bsa_eff, hist_made ? hist : nullptr, kv_idx, kv_count, status,
                           true, stream);
    if (e != cudaSuccess) return cuda_status(e);
  } else {
    e = cudaMemsetAsync(kv_count, 0, sizeof(int32_t) * b * nkv, stream);
    if (e != cudaSuccess) return QUOKA_ERR_CUDA;
  }
  return QUOKA_OK;
}

struct AttnShapes {
  int64_t b, nq, nkv, d, T, BCP;
};

quoka_status validate_attn(const quoka_tensor* Q, const quoka_tensor* K, const quoka_tensor* V,
                           const quoka_tensor* Kc, const quoka_tensor* Vc, AttnShapes* s) {
  if (Q == nullptr || K == nullptr || V == nullptr || Kc == nullptr || Vc == nullptr)
    return QUOKA_ERR_INVALID_ARG;
  int64_t qs[4] = {-1, -1, -1, -1};
  if (!check_tensor(Q, Q->dtype, qs)) return QUOKA_ERR_INVALID_ARG;
  if (Q->dtype != QUOKA_F32 && Q->dtype != QUOKA_BF16) return QUOKA_ERR_INVALID_ARG;
  int64_t ks[4] = {qs[0], -1, -1, qs[3]};
  if (!check_tensor(K, Q->dtype, ks)) return QUOKA_ERR_INVALID_ARG;
  int64_t vs[4] = {ks[0], ks[1], ks[2], ks[3]};
  if (!check_tensor(V, Q->dtype, vs)) return QUOKA_ERR_INVALID_ARG;
  int64_t kcs[4] = {qs[0], ks[1], qs[2], qs[3]};
  if (!check_tensor(Kc, Q->dtype, kcs)) return QUOKA_ERR_INVALID_ARG;
  int64_t vcs[4] = {qs[0], ks[1], qs[2], qs[3]};
  if (!check_tensor(Vc, Q->dtype, vcs)) return QUOKA_ERR_INVALID_ARG;
  s->b = qs[0];
  s->nq = qs[1];
  s->BCP = qs[2];
  s->d = qs[3];
  s->nkv = ks[1];
  s->T = ks[2];
  if (s->b < 1 || s->nq < 1 || s->nkv < 1 || s->BCP < 1) return QUOKA_ERR_INVALID_ARG;
  if (s->nq % s->nkv != 0) return QUOKA_ERR_INVALID_ARG;
  if (!supported_d(s->d)) return QUOKA_ERR_UNSUPPORTED;
  if (s->BCP > kMaxBCP || s->nq > kMaxHeads || s->nkv > kMaxHeads || s->b > kMaxHeads)
    return QUOKA_ERR_UNSUPPORTED;
  if (s->T > (int64_t)INT32_MAX) return QUOKA_ERR_UNSUPPORTED;
  return QUOKA_OK;
}

// Step (g) (with step (f) fused into the loads when kv_idx is given; with
// kv_idx null, K / V are the gathered selected rows and T their row count).
quoka_status run_attn(const quoka_tensor* Q, Strided K, Strided V, const quoka_tensor* Kc,
                      const quoka_tensor* Vc, const AttnShapes& s, int64_t T, const int32_t* kv_idx,
                      const int32_t* kv_count, int bsa_eff, float scale, void* O, float* lse,
                      int* status, cudaStream_t stream, bool pdl = false, bool no_chunk = false,
                      void* parts = nullptr, size_t parts_bytes = 0) {
  quoka::AttnArgs a;
  a.no_chunk = no_chunk ? 1 : 0;
  a.Q = strided(Q);
  a.K = K;
  a.V = V;
  a.Kc = strided(Kc);
  a.Vc = strided(Vc);
  a.b = (int)s.b;
  a.nq = (int)s.nq;
  a.nkv = (int)s.nkv;
  a.d = (int)s.d;
  a.BCP = (int)s.BCP;
  a.T = T;
  a.kv_idx = kv_idx;
  a.kv_count = kv_count;
  a.bsa = bsa_eff;
  a.scale = scale;
  a.O = O;
  a.lse = lse;
  a.status = status;
  if (kv_idx == nullptr && parts != nullptr) {
    // split key ranges when the query tiles leave most SMs idle and the
    // workspace holds the partials
    const int ns = attn_nsplit(s.b, s.nq, s.BCP, s.d, bsa_eff, Q->dtype == QUOKA_BF16, no_chunk);
    if (ns > 1 && parts_bytes >= attn_parts_bytes(s.b, s.nq, s.BCP, s.d, ns)) {
      const int64_t rows = (int64_t)ns * s.b * s.nq * s.BCP;
      a.nsplit = ns;
      a.O_parts = parts;
      a.lse_parts = reinterpret_cast<float*>(static_cast<char*>(parts) + align_up((size_t)(rows * s.d) * 2));
    }
  }
  cudaError_t e = cudaErrorNotSupported;
  if (Q->dtype == QUOKA_BF16) e = quoka::launch_attn_tc(a, pdl, stream);
  if (e == cudaErrorNotSupported) e = quoka::launch_attn_simt(Q->dtype == QUOKA_BF16, a, stream);
  return cuda_status(e);
}

// Steps (f)+(g) on the full cache K / V: when `gathered` (the workspace's
// Ksel / Vsel buffers) is given, step (f) runs as its own kernel into it and
// the attention streams the copy; otherwise the attention gathers in place.
quoka_status gather_then_attn(const quoka_tensor* Q, const quoka_tensor* K, const quoka_tensor* V,
                              const quoka_tensor* Kc, const quoka_tensor* Vc, const AttnShapes& s,
                              const int32_t* kv_idx, const int32_t* kv_count, int bsa_eff, float scale,
                              void* O, float* lse, void* ksel, void* vsel, int* status,
                              cudaStream_t stream, bool no_chunk = false, void* parts = nullptr,
                              size_t parts_bytes = 0) {
  if (ksel == nullptr || vsel == nullptr || bsa_eff == 0)
    return run_attn(Q, strided(K), strided(V), Kc, Vc, s, s.T, kv_idx, kv_count, bsa_eff, scale, O, lse,
                    status, stream, false, no_chunk);
  cudaError_t e = quoka::launch_gather(Q->dtype == QUOKA_BF16, (int)s.d, strided(K), strided(V), (int)s.b,
                                       (int)s.nkv, s.T, kv_idx, kv_count, bsa_eff, ksel, vsel, status, true,
                                       stream);
  if (e != cudaSuccess) return cuda_status(e);
  const int64_t sh = (int64_t)bsa_eff * s.d, sb = s.nkv * sh;
  // the attention may launch while the gather finishes (it waits for it)
  return run_attn(Q, Strided{ksel, sb, sh, s.d}, Strided{vsel, sb, sh, s.d}, Kc, Vc, s, bsa_eff, nullptr,
                  kv_count, bsa_eff, scale, O, lse, status, stream, true, no_chunk, parts, parts_bytes);
}

// Steps (f)+(g) for a short chunk (short_chunk()): the slice kernel reads the
// selected rows by index from the cache, then the merge kernel.
quoka_status run_decode(const quoka_tensor* Q, const quoka_tensor* K, const quoka_tensor* V,
                        const quoka_tensor* Kc, const quoka_tensor* Vc, const AttnShapes& s,
                        const int32_t* kv_idx, const int32_t* kv_count, int bsa_eff, float scale, void* O,
                        float* lse, float* O_parts, float* lse_parts, int* status, cudaStream_t stream,
                        bool pdl) {
  quoka::DecodeArgs a;
  a.Q = strided(Q);
  a.K = strided(K);
  a.V = strided(V);
  a.Kc = strided(Kc);
  a.Vc = strided(Vc);
  a.b = (int)s.b;
  a.nq = (int)s.nq;
  a.nkv = (int)s.nkv;
  a.d = (int)s.d;
  a.BCP = (int)s.BCP;
  a.T = s.T;
  a.kv_idx = kv_idx;
  a.kv_count = kv_count;
  a.bsa = bsa_eff;
  a.scale = scale;
  a.O_parts = O_parts;
  a.lse_parts = lse_parts;
  a.nsplit = quoka::decode_splits(bsa_eff, (int)s.BCP);
  a.O = O;
  a.lse = lse;
  a.status = status;
  return cuda_status(quoka::launch_decode_attn(Q->dtype == QUOKA_BF16, a, pdl, stream));
}

// ---- the paged 8-bit cache

bool cache_page_ok(int page) { return page == 16 || page == 32 || page == 64 || page == 128; }

// Checks the description of a cache and turns it into the kernels' view.
quoka_status validate_cache(const quoka_cache* c, quoka::CacheView* v) {
  if (c == nullptr || c->k == nullptr || c->v == nullptr || c->k_scale == nullptr || c->v_scale == nullptr ||
      c->page_table == nullptr || c->seq_len == nullptr)
    return QUOKA_ERR_INVALID_ARG;
  if (!aligned16(c->k) || !aligned16(c->v)) return QUOKA_ERR_INVALID_ARG;
  if (c->npages < 1 || c->nkv < 1 || c->b < 1 || c->max_pages < 1 || c->table_stride < c->max_pages)
    return QUOKA_ERR_INVALID_ARG;
  const int64_t st[3] = {c->page_stride, c->head_stride, c->row_stride};
  const int64_t n[3] = {c->npages, c->nkv, c->page};
  for (int i = 0; i < 3; ++i)
    if (st[i] < 0 || st[i] % 16 != 0 || (n[i] > 1 && st[i] < c->d)) return QUOKA_ERR_INVALID_ARG;
  if (!supported_d(c->d) || !cache_page_ok(c->page)) return QUOKA_ERR_UNSUPPORTED;
  // (what a tensor map takes; refused here, before a call's first kernels are enqueued)
  for (int i = 0; i < 3; ++i)
    if (n[i] > 1 && st[i] >= (int64_t)1 << 40) return QUOKA_ERR_UNSUPPORTED;
  if (c->b > kMaxHeads || c->nkv > kMaxHeads || c->npages > (int64_t)INT32_MAX) return QUOKA_ERR_UNSUPPORTED;
  v->k = static_cast<uint8_t*>(c->k);
  v->v = static_cast<uint8_t*>(c->v);
  v->k_scale = c->k_scale;
  v->v_scale = c->v_scale;
  v->sp = st[0];
  v->sh = st[1];
  v->sr = st[2];
  v->npages = (int)c->npages;
  v->nkv = c->nkv;
  v->page_log2 = c->page == 16 ? 4 : c->page == 32 ? 5 : c->page == 64 ? 6 : 7;
  v->page_table = c->page_table;
  v->table_stride = c->table_stride;
  v->seq_len = c->seq_len;
  return QUOKA_OK;
}

// Positions that the page table's columns cover (kept clear of the end of int32).
int cache_room(const quoka_cache* c) {
  return (int)std::min<int64_t>((int64_t)c->max_pages * c->page, (int64_t)1 << 30);
}

// The optional workspace of the calls that only need the status words there:
// clears them and returns their address.
quoka_status optional_status(void* ws, size_t ws_bytes, cudaStream_t stream, int** status) {
  *status = nullptr;
  if (ws == nullptr) return QUOKA_OK;
  if (((uintptr_t)ws % kAlign) != 0 || ws_bytes < 2 * sizeof(int)) return QUOKA_ERR_WORKSPACE;
  *status = static_cast<int*>(ws);
  return quoka::clear_status_async(*status, stream) == cudaSuccess ? QUOKA_OK : QUOKA_ERR_CUDA;
}

// Whether [a, a + na) and the bytes that t spans overlap.
bool overlaps(const void* a, size_t na, const quoka_tensor* t) {
  int64_t last = 0;
  for (int i = 0; i < 4; ++i) {
    if (t->shape[i] == 0) return false;
    last += (t->shape[i] - 1) * t->stride[i];
  }
  const uintptr_t a0 = (uintptr_t)a, t0 = (uintptr_t)t->data;
  const uintptr_t t1 = t0 + (size_t)(last + 1) * elt_size(t->dtype);
  return a0 < t1 && t0 < a0 + na;
}

// The attention of many bf16 query rows over dequantised rows: whether a tile
// takes rows of several heads (fewer tiles then), and into how many ranges the
// keys are cut.
bool cache_attn_packs(int64_t nq, int64_t nkv, int64_t BCP) {
  return nkv * ((nq / nkv * BCP + 127) / 128) < nq * ((BCP + 127) / 128);
}
int cache_attn_nsplit(int64_t b, int64_t nq, int64_t nkv, int64_t BCP, int64_t N, bool no_chunk, bool pack) {
  const int64_t tiles = pack ? b * nkv * ((nq / nkv * BCP + 127) / 128) : b * nq * ((BCP + 127) / 128);
  const int64_t nt = (N + 127) / 128 + (no_chunk ? 0 : (BCP + 127) / 128);
  return quoka::attn_splits(tiles, (int)std::min<int64_t>(nt, 1 << 20), quoka::kAttnMaxSplits);
}

// Workspace of quoka_cache_attn: the status words, then either the partials
// of the key ranges (few query rows, or fp32) or the dequantised keys and values
// with their counts and the partials of the tensor-core attention.
struct CacheAttnWs {
  bool few;
  size_t o_parts, lse_parts, row_parts, faults, ksel, vsel, count, aparts, aparts_bytes, total;
};

CacheAttnWs cache_attn_ws(int64_t b, int64_t nq, int64_t nkv, int64_t d, int64_t BCP, int64_t N, quoka_dtype dtype,
                          bool no_chunk) {
  CacheAttnWs w = {};
  size_t off = kAlign;
  auto take = [&](size_t bytes) {
    const size_t p = off;
    off += align_up(bytes);
    return p;
  };
  const int64_t R = (nq / nkv) * BCP;
  w.few = dtype == QUOKA_F32 || R <= quoka::kCacheMaxRows;
  if (w.few) {
    const int64_t ranges = quoka::cache_attn_ranges(b * nkv, R, (int)N), rows = ranges * R;
    w.o_parts = take((size_t)(rows * d) * 4);
    w.lse_parts = take((size_t)rows * 4);
    w.row_parts = take((size_t)(b * nkv) * 8);
    w.faults = take((size_t)(ranges * ((R + 63) / 64)) * 4);
  } else {
    w.ksel = take((size_t)(b * nkv * N * d) * elt_size(dtype));
    w.vsel = take((size_t)(b * nkv * N * d) * elt_size(dtype));
    w.count = take((size_t)(b * nkv) * 4);
    // (whether rows can be packed depends on Q's strides: room for either)
    const int n = std::max(cache_attn_nsplit(b, nq, nkv, BCP, N, no_chunk, false),
                           cache_attn_packs(nq, nkv, BCP) ? cache_attn_nsplit(b, nq, nkv, BCP, N, no_chunk, true) : 1);
    w.aparts_bytes = attn_parts_bytes(b, nq, BCP, d, n);
    w.aparts = take(w.aparts_bytes);
  }
  w.total = off;
  return w;
}

// Steps (a)-(e) over the cache; new_len: null, or the queries of a padded chunk.
quoka_status run_cache_select(const quoka_tensor* Q, const int32_t* new_len, const quoka_cache* cache, int max_len,
                              int NQ, int BSA, int32_t* kv_idx, int32_t* kv_count, int32_t* q_idx, float* s_agg,
                              void* ws, size_t ws_bytes, void* stream) {
  quoka::CacheScoreArgs a = {};
  quoka_status st = validate_cache(cache, &a.c);
  if (st != QUOKA_OK) return st;
  if (Q == nullptr || (Q->dtype != QUOKA_F32 && Q->dtype != QUOKA_BF16)) return QUOKA_ERR_INVALID_ARG;
  int64_t qs[4] = {cache->b, -1, -1, cache->d};
  if (!check_tensor(Q, Q->dtype, qs)) return QUOKA_ERR_INVALID_ARG;
  const int b = cache->b, nkv = cache->nkv, d = cache->d;
  if (qs[1] < 1 || qs[2] < 1 || qs[1] % nkv != 0 || NQ < 1 || NQ > qs[2] || BSA < 0) return QUOKA_ERR_INVALID_ARG;
  if (max_len < 0 || max_len > cache_room(cache) || kv_count == nullptr) return QUOKA_ERR_INVALID_ARG;
  if (qs[1] > kMaxHeads || qs[2] > kMaxBCP || max_len > quoka::topk_max_T()) return QUOKA_ERR_UNSUPPORTED;
  const int nq = (int)qs[1], BCP = (int)qs[2], bsa_eff = std::min(BSA, max_len);
  if (bsa_eff > 0 && kv_idx == nullptr) return QUOKA_ERR_INVALID_ARG;
  const WsLayout L = ws_layout(b, nq, nkv, d, max_len, NQ, bsa_eff, false);
  st = check_ws(ws, ws_bytes, L.select_total);
  if (st != QUOKA_OK) return st;
  cudaStream_t cs = static_cast<cudaStream_t>(stream);
  const bool bf = Q->dtype == QUOKA_BF16;
  float* qg = at<float>(ws, L.qgroup);
  int32_t* qidx = q_idx != nullptr ? q_idx : at<int32_t>(ws, L.qidx);
  a.status = at<int>(ws, L.status);
  a.hist = at<uint32_t>(ws, L.hist);
  // (the status words and the histogram are cleared by the kernel that makes the group means)
  cudaError_t e = cudaErrorNotSupported;
  // The fused query select takes an SM per query head for any chunk length: with
  // more heads than one round holds, short chunks are faster through the
  // general kernels (whole call, 1000 keys, 16 sequences x 32 heads: 16 tokens 33.2
  // us against 41.9 fused, 64 38.4 and 42.1, 128 47.0 and 41.9; 1 x 32 heads: 14.6
  // both at 16, 19.5 and 14.7 at 128).
  const bool fused = BCP == 1 || BCP > 64 || (int64_t)b * nq <= 128;
  if (bf && d == 128 && fused)
    e = quoka::launch_qsel_group_fast(strided(Q), b, nq, nkv, BCP, NQ, qidx, qg, nullptr, a.hist, a.status, true, cs,
                                      new_len);
  if (e == cudaErrorNotSupported) {
    e = quoka::launch_qsel(bf, d, strided(Q), b, nq, BCP, NQ, at<float>(ws, L.qhat), qidx, true, cs, new_len);
    if (e != cudaSuccess) return cuda_status(e);
    e = quoka::launch_qgroup(d, at<float>(ws, L.qhat), b, nq, nkv, NQ, qg, nullptr, a.hist, a.status, cs);
  }
  if (e != cudaSuccess) return cuda_status(e);
  a.b = b;
  a.max_len = max_len;
  a.Qg = qg;
  a.NQ = NQ;
  a.new_len = new_len;
  a.BCP = BCP;
  a.S_agg = s_agg != nullptr ? s_agg : at<float>(ws, L.sagg);
  if (max_len > 0) {
    e = quoka::launch_cache_score(d, a, cs);
    if (e != cudaSuccess) return cuda_status(e);
  }
  if (bsa_eff > 0)
    return cuda_status(quoka::launch_topk(a.S_agg, b, nkv, max_len, bsa_eff, a.hist, kv_idx, kv_count, a.status, true,
                                          cs, cache->seq_len, new_len));
  return cudaMemsetAsync(kv_count, 0, sizeof(int32_t) * b * nkv, cs) == cudaSuccess ? QUOKA_OK : QUOKA_ERR_CUDA;
}

}  // namespace

extern "C" {

size_t quoka_workspace_size(int b, int nq, int nkv, int d, int64_t T, int BCP, int NQ, int BSA,
                            quoka_dtype dtype) {
  if (b < 1 || nq < 1 || nkv < 1 || d < 1 || T < 0 || BCP < 1 || NQ < 1 || BSA < 0) return 0;
  if (nq % nkv != 0 || (dtype != QUOKA_F32 && dtype != QUOKA_BF16)) return 0;
  const int64_t bsa_eff = std::min<int64_t>(BSA, T);
  const bool dec = short_chunk(nq, nkv, BCP, d);
  // (a short chunk's layout keeps the gather buffers too: the same workspace
  // then also gives quoka_sparse_gqa_attn its fastest path)
  return ws_layout(b, nq, nkv, d, T, NQ, bsa_eff, uses_gather_buffers(dtype, d, bsa_eff), BCP, dec).total;
}

size_t quoka_select_workspace_size(int b, int nq, int nkv, int d, int64_t T, int BCP, int NQ, int BSA,
                                   quoka_dtype dtype) {
  if (quoka_workspace_size(b, nq, nkv, d, T, BCP, NQ, BSA, dtype) == 0) return 0;
  const int64_t bsa_eff = std::min<int64_t>(BSA, T);
  return ws_layout(b, nq, nkv, d, T, NQ, bsa_eff, false).select_total;
}

size_t quoka_attn_workspace_size(int b, int nkv, int d, int BSA_eff, quoka_dtype dtype) {
  if (b < 1 || nkv < 1 || d < 1 || BSA_eff < 0) return 0;
  if (dtype != QUOKA_F32 && dtype != QUOKA_BF16) return 0;
  return attn_ws_bytes(b, nkv, d, BSA_eff, uses_gather_buffers(dtype, d, BSA_eff));
}

quoka_status quoka_select(const quoka_tensor* Q, const quoka_tensor* K, int NQ, int BSA,
                          int32_t* kv_idx, int32_t* kv_count, int32_t* q_idx, float* s_agg,
                          void* ws, size_t ws_bytes, void* stream) {
  quoka::NvtxRange nvtx_range("quoka_select");
  return quoka_select_ex(Q, K, NQ, BSA, kv_idx, kv_count, q_idx, s_agg, 0u, ws, ws_bytes, stream);
}

quoka_status quoka_select_ex(const quoka_tensor* Q, const quoka_tensor* K, int NQ, int BSA,
                             int32_t* kv_idx, int32_t* kv_count, int32_t* q_idx, float* s_agg,
                             uint32_t flags, void* ws, size_t ws_bytes, void* stream) {
  quoka::NvtxRange nvtx_range("quoka_select_ex");
  if ((flags & ~QUOKA_SCORE_DOT_PRODUCT) != 0u) return QUOKA_ERR_INVALID_ARG;
  SelectShapes s;
  quoka_status st = validate_select(Q, K, NQ, BSA, &s);
  if (st != QUOKA_OK) return st;
  const int64_t bsa_eff = std::min<int64_t>(BSA, s.T);
  if (kv_count == nullptr || (bsa_eff > 0 && kv_idx == nullptr)) return QUOKA_ERR_INVALID_ARG;
  const WsLayout L = ws_layout(s.b, s.nq, s.nkv, s.d, s.T, NQ, bsa_eff, false);
  st = check_ws(ws, ws_bytes, L.select_total);
  if (st != QUOKA_OK) return st;
  cudaStream_t cs = static_cast<cudaStream_t>(stream);
  // (the status words are cleared by the first kernel)
  return run_select(Q, K, s, NQ, (int)bsa_eff, kv_idx, kv_count, q_idx, s_agg, ws, L, cs, flags);
}

quoka_status quoka_gather_kv(const quoka_tensor* K, const quoka_tensor* V, const int32_t* kv_idx,
                             const int32_t* kv_count, int BSA_eff, void* Ksel, void* Vsel,
                             void* ws, size_t ws_bytes, void* stream) {
  quoka::NvtxRange nvtx_range("quoka_gather_kv");
  if (K == nullptr || V == nullptr || kv_count == nullptr || BSA_eff < 0) return QUOKA_ERR_INVALID_ARG;
  int64_t ks[4] = {-1, -1, -1, -1};
  if (!check_tensor(K, K->dtype, ks)) return QUOKA_ERR_INVALID_ARG;
  if (K->dtype != QUOKA_F32 && K->dtype != QUOKA_BF16) return QUOKA_ERR_INVALID_ARG;
  int64_t vs[4] = {ks[0], ks[1], ks[2], ks[3]};
  if (!check_tensor(V, K->dtype, vs)) return QUOKA_ERR_INVALID_ARG;
  if (!supported_d(ks[3])) return QUOKA_ERR_UNSUPPORTED;
  if (ks[0] < 1 || ks[1] < 1 || ks[0] > kMaxHeads || ks[1] > kMaxHeads) return QUOKA_ERR_INVALID_ARG;
  if (BSA_eff > 0 && (kv_idx == nullptr || Ksel == nullptr || Vsel == nullptr || !aligned16(Ksel) ||
                      !aligned16(Vsel)))
    return QUOKA_ERR_INVALID_ARG;
  cudaStream_t cs = static_cast<cudaStream_t>(stream);
  int* status = nullptr;
  if (ws != nullptr) {
    if (((uintptr_t)ws % kAlign) != 0 || ws_bytes < 2 * sizeof(int)) return QUOKA_ERR_WORKSPACE;
    status = static_cast<int*>(ws);
    if (quoka::clear_status_async(status, cs) != cudaSuccess) return QUOKA_ERR_CUDA;
  }
  cudaError_t e = quoka::launch_gather(K->dtype == QUOKA_BF16, (int)ks[3], strided(K), strided(V),
                                       (int)ks[0], (int)ks[1], ks[2], kv_idx, kv_count, BSA_eff, Ksel,
                                       Vsel, status, true, cs);
  return cuda_status(e);
}

quoka_status quoka_sparse_gqa_attn(const quoka_tensor* Q, const quoka_tensor* K,
                                   const quoka_tensor* V, const int32_t* kv_idx,
                                   const int32_t* kv_count, int BSA_eff, const quoka_tensor* Kc,
                                   const quoka_tensor* Vc, float scale, void* O, float* lse,
                                   void* ws, size_t ws_bytes, void* stream) {
  quoka::NvtxRange nvtx_range("quoka_sparse_gqa_attn");
  return quoka_sparse_gqa_attn_ex(Q, K, V, kv_idx, kv_count, BSA_eff, Kc, Vc, scale, O, lse, 0u, ws, ws_bytes,
                                  stream);
}

quoka_status quoka_sparse_gqa_attn_ex(const quoka_tensor* Q, const quoka_tensor* K,
                                      const quoka_tensor* V, const int32_t* kv_idx,
                                      const int32_t* kv_count, int BSA_eff, const quoka_tensor* Kc,
                                      const quoka_tensor* Vc, float scale, void* O, float* lse,
                                      uint32_t flags, void* ws, size_t ws_bytes, void* stream) {
  quoka::NvtxRange nvtx_range("quoka_sparse_gqa_attn_ex");
  if ((flags & ~QUOKA_ATTN_NO_CHUNK_KEYS) != 0u) return QUOKA_ERR_INVALID_ARG;
  const bool no_chunk = (flags & QUOKA_ATTN_NO_CHUNK_KEYS) != 0u;
  AttnShapes s;
  quoka_status st = validate_attn(Q, K, V, Kc, Vc, &s);
  if (st != QUOKA_OK) return st;
  if (BSA_eff < 0 || kv_count == nullptr || (BSA_eff > 0 && kv_idx == nullptr)) return QUOKA_ERR_INVALID_ARG;
  if (O == nullptr || !aligned16(O)) return QUOKA_ERR_INVALID_ARG;
  if (!(scale > 0.f) || scale != scale) return QUOKA_ERR_INVALID_ARG;
  if (ws == nullptr || ((uintptr_t)ws % kAlign) != 0 || ws_bytes < kAlign) return QUOKA_ERR_WORKSPACE;
  cudaStream_t cs = static_cast<cudaStream_t>(stream);
  int* status = static_cast<int*>(ws);
  // (a memset here: launched early behind a clear kernel, the attention measured ~2 us slower)
  if (cudaMemsetAsync(status, 0, 2 * sizeof(int), cs) != cudaSuccess) return QUOKA_ERR_CUDA;
  // with room for the gathered copy, the selected rows are gathered first
  void* ksel = nullptr;
  void* vsel = nullptr;
  void* parts = nullptr;
  size_t parts_bytes = 0;
  const bool gb = uses_gather_buffers(Q->dtype, s.d, BSA_eff);
  const size_t gb_end = attn_ws_bytes(s.b, s.nkv, s.d, BSA_eff, true);
  if (gb && ws_bytes >= gb_end) {
    ksel = static_cast<char*>(ws) + kAlign;
    vsel = static_cast<char*>(ksel) + align_up((size_t)(s.b * s.nkv * BSA_eff * s.d) * 2);
    // (room past the gathered copy takes the split ranges' partials)
    parts = static_cast<char*>(ws) + gb_end;
    parts_bytes = ws_bytes - gb_end;
  }
  return gather_then_attn(Q, K, V, Kc, Vc, s, kv_idx, kv_count, BSA_eff, scale, O, lse, ksel, vsel, status,
                          cs, no_chunk, parts, parts_bytes);
}

quoka_status quoka_sparse_gqa_attn_gathered(const quoka_tensor* Q, const quoka_tensor* Ksel,
                                            const quoka_tensor* Vsel, const int32_t* kv_count,
                                            const quoka_tensor* Kc, const quoka_tensor* Vc, float scale,
                                            void* O, float* lse, void* ws, size_t ws_bytes,
                                            void* stream) {
  quoka::NvtxRange nvtx_range("quoka_sparse_gqa_attn_gathered");
  AttnShapes s;
  quoka_status st = validate_attn(Q, Ksel, Vsel, Kc, Vc, &s);
  if (st != QUOKA_OK) return st;
  if (kv_count == nullptr) return QUOKA_ERR_INVALID_ARG;
  if (O == nullptr || !aligned16(O)) return QUOKA_ERR_INVALID_ARG;
  if (!(scale > 0.f) || scale != scale) return QUOKA_ERR_INVALID_ARG;
  if (ws == nullptr || ((uintptr_t)ws % kAlign) != 0 || ws_bytes < kAlign) return QUOKA_ERR_WORKSPACE;
  cudaStream_t cs = static_cast<cudaStream_t>(stream);
  int* status = static_cast<int*>(ws);
  // (a memset here: launched early behind a clear kernel, the attention measured ~2 us slower)
  if (cudaMemsetAsync(status, 0, 2 * sizeof(int), cs) != cudaSuccess) return QUOKA_ERR_CUDA;
  // the rows of Ksel / Vsel are the selected keys in list order: BSA_eff = T
  // (room past the status words takes the split ranges' partials)
  return run_attn(Q, strided(Ksel), strided(Vsel), Kc, Vc, s, s.T, nullptr, kv_count, (int)s.T, scale, O,
                  lse, status, cs, true, false, static_cast<char*>(ws) + kAlign, ws_bytes - kAlign);
}

size_t quoka_decode_workspace_size(int b, int nq, int nkv, int d, int BCP, int BSA_eff, quoka_dtype dtype) {
  if (b < 1 || nq < 1 || nkv < 1 || BCP < 1 || BSA_eff < 0) return 0;
  if (dtype != QUOKA_F32 && dtype != QUOKA_BF16) return 0;
  if (!short_chunk(nq, nkv, BCP, d)) return 0;
  return decode_ws_bytes(b, nq, d, BCP, BSA_eff);
}

quoka_status quoka_decode_attn(const quoka_tensor* Q, const quoka_tensor* K, const quoka_tensor* V,
                               const int32_t* kv_idx, const int32_t* kv_count, int BSA_eff,
                               const quoka_tensor* Kc, const quoka_tensor* Vc, float scale, void* O,
                               float* lse, void* ws, size_t ws_bytes, void* stream) {
  quoka::NvtxRange nvtx_range("quoka_decode_attn");
  AttnShapes s;
  quoka_status st = validate_attn(Q, K, V, Kc, Vc, &s);
  if (st != QUOKA_OK) return st;
  if (!short_chunk(s.nq, s.nkv, s.BCP, s.d)) return QUOKA_ERR_UNSUPPORTED;
  if (BSA_eff < 0 || kv_count == nullptr || (BSA_eff > 0 && kv_idx == nullptr)) return QUOKA_ERR_INVALID_ARG;
  if (O == nullptr || !aligned16(O)) return QUOKA_ERR_INVALID_ARG;
  if (!(scale > 0.f) || scale != scale) return QUOKA_ERR_INVALID_ARG;
  const size_t need = decode_ws_bytes(s.b, s.nq, s.d, s.BCP, BSA_eff);
  if (ws == nullptr || ((uintptr_t)ws % kAlign) != 0 || ws_bytes < need) return QUOKA_ERR_WORKSPACE;
  cudaStream_t cs = static_cast<cudaStream_t>(stream);
  int* status = static_cast<int*>(ws);
  if (quoka::clear_status_async(status, cs) != cudaSuccess) return QUOKA_ERR_CUDA;
  const int64_t rows = (int64_t)quoka::decode_splits(BSA_eff, (int)s.BCP) * s.b * s.nq * s.BCP;
  float* O_parts = reinterpret_cast<float*>(static_cast<char*>(ws) + kAlign);
  float* lse_parts = reinterpret_cast<float*>(reinterpret_cast<char*>(O_parts) + align_up((size_t)(rows * s.d) * 4));
  return run_decode(Q, K, V, Kc, Vc, s, kv_idx, kv_count, BSA_eff, scale, O, lse, O_parts, lse_parts, status, cs,
                    true);
}

quoka_status quoka_prefill_chunk(const quoka_tensor* Q, const quoka_tensor* K,
                                 const quoka_tensor* V, const quoka_tensor* Kc,
                                 const quoka_tensor* Vc, int NQ, int BSA, float scale, void* O,
                                 float* lse, int32_t* kv_idx_out, void* ws, size_t ws_bytes,
                                 void* stream) {
  quoka::NvtxRange nvtx_range("quoka_prefill_chunk");
  AttnShapes as;
  quoka_status st = validate_attn(Q, K, V, Kc, Vc, &as);
  if (st != QUOKA_OK) return st;
  SelectShapes s;
  st = validate_select(Q, K, NQ, BSA, &s);
  if (st != QUOKA_OK) return st;
  if (O == nullptr || !aligned16(O)) return QUOKA_ERR_INVALID_ARG;
  if (!(scale > 0.f) || scale != scale) return QUOKA_ERR_INVALID_ARG;
  const int64_t bsa_eff = std::min<int64_t>(BSA, s.T);
  const bool dec = short_chunk(s.nq, s.nkv, s.BCP, s.d);
  const bool gb = uses_gather_buffers(Q->dtype, s.d, bsa_eff);
  const WsLayout L = ws_layout(s.b, s.nq, s.nkv, s.d, s.T, NQ, bsa_eff, gb, s.BCP, dec);
  st = check_ws(ws, ws_bytes, L.total);
  if (st != QUOKA_OK) return st;
  cudaStream_t cs = static_cast<cudaStream_t>(stream);
  int* status = at<int>(ws, L.status);  // cleared by the selection's first kernel
  int32_t* kv_idx = kv_idx_out != nullptr ? kv_idx_out : at<int32_t>(ws, L.kvidx);
  int32_t* kv_count = at<int32_t>(ws, L.kvcount);
  st = run_select(Q, K, s, NQ, (int)bsa_eff, kv_idx, kv_count, nullptr, nullptr, ws, L, cs);
  if (st != QUOKA_OK) return st;
  if (dec)  // a short chunk: the decode attention (waits for the selection's last kernel)
    return run_decode(Q, K, V, Kc, Vc, as, kv_idx, kv_count, (int)bsa_eff, scale, O, lse, at<float>(ws, L.dparts),
                      at<float>(ws, L.dlse), status, cs, true);
  return gather_then_attn(Q, K, V, Kc, Vc, as, kv_idx, kv_count, (int)bsa_eff, scale, O, lse,
                          gb ? at<void>(ws, L.ksel) : nullptr, gb ? at<void>(ws, L.vsel) : nullptr, status, cs,
                          false, L.aparts_bytes > 0 ? at<void>(ws, L.aparts) : nullptr, L.aparts_bytes);
}

quoka_status quoka_cache_append(const quoka_cache* cache, const quoka_tensor* K, const quoka_tensor* V,
                                const quoka_tensor* Q, const float* cos, const float* sin, int64_t npos, int rot,
                                uint32_t flags, const int32_t* new_len, void* Kr, void* Qr, void* ws,
                                size_t ws_bytes, void* stream) {
  quoka::NvtxRange nvtx_range("quoka_cache_append");
  quoka::CacheAppendArgs a = {};
  quoka_status st = validate_cache(cache, &a.c);
  if (st != QUOKA_OK) return st;
  if ((flags & ~(QUOKA_ROTATE_NEIGHBOURS | QUOKA_ZERO_REST)) != 0u || K == nullptr || V == nullptr) return QUOKA_ERR_INVALID_ARG;
  if (K->dtype != QUOKA_F32 && K->dtype != QUOKA_BF16) return QUOKA_ERR_INVALID_ARG;
  int64_t ks[4] = {cache->b, cache->nkv, -1, cache->d};
  if (!check_tensor(K, K->dtype, ks) || !check_tensor(V, K->dtype, ks)) return QUOKA_ERR_INVALID_ARG;
  const int64_t BCP = ks[2];
  int64_t nq = 0;
  // (a chunk of no tokens has nothing to write: its outputs may be null, as an empty tensor's address is)
  if (Q == nullptr ? Qr != nullptr : Qr == nullptr && BCP > 0) return QUOKA_ERR_INVALID_ARG;
  if (Q != nullptr) {
    int64_t qs[4] = {cache->b, -1, BCP, cache->d};
    if (!check_tensor(Q, K->dtype, qs) || qs[1] < 1) return QUOKA_ERR_INVALID_ARG;
    nq = qs[1];
    if (!aligned16(Qr)) return QUOKA_ERR_INVALID_ARG;
  }
  if (rot < 0 || rot > cache->d || rot % 16 != 0) return QUOKA_ERR_INVALID_ARG;
  if (rot > 0 && (cos == nullptr || sin == nullptr || !aligned16(cos) || !aligned16(sin) || npos < 1))
    return QUOKA_ERR_INVALID_ARG;
  if (Kr != nullptr && !aligned16(Kr)) return QUOKA_ERR_INVALID_ARG;
  if (BCP > kMaxBCP || nq > kMaxHeads) return QUOKA_ERR_UNSUPPORTED;
  // the rotation reads both columns of a pair: it cannot run in place
  const size_t es = elt_size(K->dtype), kb = (size_t)cache->b * cache->nkv * BCP * cache->d * es;
  const size_t qb = (size_t)cache->b * nq * BCP * cache->d * es;
  const quoka_tensor* ins[3] = {K, V, Q};
  for (const quoka_tensor* t : ins) {
    if (t == nullptr) continue;
    if (Kr != nullptr && overlaps(Kr, kb, t)) return QUOKA_ERR_INVALID_ARG;
    if (Qr != nullptr && overlaps(Qr, qb, t)) return QUOKA_ERR_INVALID_ARG;
  }
  cudaStream_t cs = static_cast<cudaStream_t>(stream);
  st = optional_status(ws, ws_bytes, cs, &a.status);
  if (st != QUOKA_OK || BCP == 0) return st;
  a.K = strided(K);
  a.V = strided(V);
  if (Q != nullptr) a.Q = strided(Q);
  a.b = cache->b;
  a.nq = (int)nq;
  a.BCP = (int)BCP;
  a.cos = cos;
  a.sin = sin;
  a.rot = rot;
  a.interleaved = (flags & QUOKA_ROTATE_NEIGHBOURS) != 0u ? 1 : 0;
  a.new_len = new_len;
  a.limit = rot > 0 ? (int)std::min<int64_t>(cache_room(cache), npos) : cache_room(cache);
  a.Kr = Kr;
  a.Qr = Qr;
  a.zero_rest = (flags & QUOKA_ZERO_REST) != 0u ? 1 : 0;
  return cuda_status(quoka::launch_cache_append(K->dtype == QUOKA_BF16, cache->d, a, a.status != nullptr, cs));
}

quoka_status quoka_cache_select(const quoka_tensor* Q, const quoka_cache* cache, int max_len, int NQ, int BSA,
                                int32_t* kv_idx, int32_t* kv_count, int32_t* q_idx, float* s_agg, void* ws,
                                size_t ws_bytes, void* stream) {
  quoka::NvtxRange nvtx_range("quoka_cache_select");
  return run_cache_select(Q, nullptr, cache, max_len, NQ, BSA, kv_idx, kv_count, q_idx, s_agg, ws, ws_bytes, stream);
}

quoka_status quoka_cache_select_padded(const quoka_tensor* Q, const int32_t* new_len, const quoka_cache* cache,
                                       int max_len, int NQ, int BSA, int32_t* kv_idx, int32_t* kv_count,
                                       int32_t* q_idx, float* s_agg, void* ws, size_t ws_bytes, void* stream) {
  quoka::NvtxRange nvtx_range("quoka_cache_select_padded");
  if (new_len == nullptr) return QUOKA_ERR_INVALID_ARG;
  return run_cache_select(Q, new_len, cache, max_len, NQ, BSA, kv_idx, kv_count, q_idx, s_agg, ws, ws_bytes, stream);
}

quoka_status quoka_cache_gather(const quoka_cache* cache, int max_len, const int32_t* kv_idx,
                                const int32_t* kv_count, int N, quoka_dtype dtype, void* Ksel, void* Vsel, void* ws,
                                size_t ws_bytes, void* stream) {
  quoka::NvtxRange nvtx_range("quoka_cache_gather");
  quoka::CacheGatherArgs a = {};
  quoka_status st = validate_cache(cache, &a.c);
  if (st != QUOKA_OK) return st;
  if (dtype != QUOKA_F32 && dtype != QUOKA_BF16) return QUOKA_ERR_INVALID_ARG;
  if (max_len < 0 || max_len > cache_room(cache) || N < 0 || (kv_idx == nullptr) != (kv_count == nullptr))
    return QUOKA_ERR_INVALID_ARG;
  if (kv_idx == nullptr && N != max_len) return QUOKA_ERR_INVALID_ARG;
  if (N > 0 && (Ksel == nullptr || Vsel == nullptr || !aligned16(Ksel) || !aligned16(Vsel)))
    return QUOKA_ERR_INVALID_ARG;
  cudaStream_t cs = static_cast<cudaStream_t>(stream);
  st = optional_status(ws, ws_bytes, cs, &a.status);
  if (st != QUOKA_OK || N == 0) return st;
  a.b = cache->b;
  a.max_len = max_len;
  a.kv_idx = kv_idx;
  a.kv_count = kv_count;
  a.N = N;
  a.Ksel = Ksel;
  a.Vsel = Vsel;
  return cuda_status(quoka::launch_cache_gather(dtype == QUOKA_BF16, cache->d, a, a.status != nullptr, cs));
}

size_t quoka_cache_attn_workspace_size(int b, int nq, int nkv, int d, int BCP, int N, quoka_dtype dtype) {
  if (b < 1 || nq < 1 || nkv < 1 || BCP < 1 || N < 0 || N > (1 << 30) || nq % nkv != 0 || !supported_d(d)) return 0;
  if (dtype != QUOKA_F32 && dtype != QUOKA_BF16) return 0;
  return std::max(cache_attn_ws(b, nq, nkv, d, BCP, N, dtype, false).total,
                  cache_attn_ws(b, nq, nkv, d, BCP, N, dtype, true).total);
}

quoka_status quoka_cache_attn(const quoka_tensor* Q, const quoka_cache* cache, int max_len, const int32_t* kv_idx,
                              const int32_t* kv_count, int N, const quoka_tensor* Kc, const quoka_tensor* Vc,
                              float scale, void* O, float* lse, void* ws, size_t ws_bytes, void* stream) {
  quoka::NvtxRange nvtx_range("quoka_cache_attn");
  quoka::CacheAttnArgs a = {};
  quoka_status st = validate_cache(cache, &a.c);
  if (st != QUOKA_OK) return st;
  if (Q == nullptr || (Q->dtype != QUOKA_F32 && Q->dtype != QUOKA_BF16)) return QUOKA_ERR_INVALID_ARG;
  int64_t qs[4] = {cache->b, -1, -1, cache->d};
  if (!check_tensor(Q, Q->dtype, qs)) return QUOKA_ERR_INVALID_ARG;
  const int64_t b = cache->b, nkv = cache->nkv, d = cache->d, nq = qs[1], BCP = qs[2];
  if (nq < 1 || BCP < 1 || nq % nkv != 0) return QUOKA_ERR_INVALID_ARG;
  if ((Kc == nullptr) != (Vc == nullptr)) return QUOKA_ERR_INVALID_ARG;
  int64_t cs4[4] = {b, nkv, BCP, d};
  if (Kc != nullptr && (!check_tensor(Kc, Q->dtype, cs4) || !check_tensor(Vc, Q->dtype, cs4)))
    return QUOKA_ERR_INVALID_ARG;
  if (max_len < 0 || max_len > cache_room(cache) || N < 0 || (kv_idx == nullptr) != (kv_count == nullptr))
    return QUOKA_ERR_INVALID_ARG;
  if (kv_idx == nullptr && N != max_len) return QUOKA_ERR_INVALID_ARG;
  if (O == nullptr || !aligned16(O) || !(scale > 0.f)) return QUOKA_ERR_INVALID_ARG;
  if (nq > kMaxHeads || BCP > kMaxBCP || N > (1 << 30)) return QUOKA_ERR_UNSUPPORTED;
  const bool no_chunk = Kc == nullptr, bf = Q->dtype == QUOKA_BF16;
  const CacheAttnWs w = cache_attn_ws(b, nq, nkv, d, BCP, N, Q->dtype, no_chunk);
  st = check_ws(ws, ws_bytes, w.total);
  if (st != QUOKA_OK) return st;
  cudaStream_t cs = static_cast<cudaStream_t>(stream);
  int* status = static_cast<int*>(ws);
  if (w.few) {
    a.Q = strided(Q);
    if (!no_chunk) {
      a.Kc = strided(Kc);
      a.Vc = strided(Vc);
    }
    a.b = (int)b;
    a.nq = (int)nq;
    a.BCP = (int)BCP;
    a.max_len = max_len;
    a.kv_idx = kv_idx;
    a.kv_count = kv_count;
    a.N = N;
    a.chunk = no_chunk ? 0 : 1;
    a.scale = scale;
    a.O_parts = at<float>(ws, w.o_parts);
    a.lse_parts = at<float>(ws, w.lse_parts);
    a.O = O;
    a.lse = lse;
    a.status = status;
    a.row_parts = at<int2>(ws, w.row_parts);
    a.faults = at<int>(ws, w.faults);
    return cuda_status(quoka::launch_cache_attn(bf, (int)d, a, cs));
  }
  if (quoka::clear_status_async(status, cs) != cudaSuccess) return QUOKA_ERR_CUDA;
  // many query rows: the rows dequantised once, then the attention over dense rows
  if (N > 0) {
    quoka::CacheGatherArgs g = {};
    g.c = a.c;
    g.b = (int)b;
    g.max_len = max_len;
    g.kv_idx = kv_idx;
    g.kv_count = kv_count;
    g.N = N;
    g.Ksel = at<void>(ws, w.ksel);
    g.Vsel = at<void>(ws, w.vsel);
    g.count_out = at<int32_t>(ws, w.count);
    g.status = status;
    const cudaError_t e = quoka::launch_cache_gather(bf, (int)d, g, true, cs);
    if (e != cudaSuccess) return cuda_status(e);
  }
  const int64_t sh = (int64_t)N * d, sb = nkv * sh;
  quoka::AttnArgs t;
  t.Q = strided(Q);
  t.K = Strided{at<void>(ws, w.ksel), sb, sh, d};
  t.V = Strided{at<void>(ws, w.vsel), sb, sh, d};
  t.Kc = no_chunk ? t.Q : strided(Kc);  // (without chunk keys: any valid rows, not read)
  t.Vc = no_chunk ? t.Q : strided(Vc);
  t.b = (int)b;
  t.nq = (int)nq;
  t.nkv = (int)nkv;
  t.d = (int)d;
  t.BCP = (int)BCP;
  t.T = N;
  t.kv_idx = nullptr;
  t.kv_count = at<int32_t>(ws, w.count);
  t.bsa = N;
  t.scale = scale;
  t.O = O;
  t.lse = lse;
  t.status = status;
  t.no_chunk = no_chunk ? 1 : 0;
  t.tc_d64 = 1;
  if (BCP == 1) t.Q.st = t.Q.sh;  // (the only row: any stride)
  t.pack = cache_attn_packs(nq, nkv, BCP) && t.Q.sh == BCP * t.Q.st ? 1 : 0;
  t.nsplit = cache_attn_nsplit(b, nq, nkv, BCP, N, no_chunk, t.pack != 0);
  if (t.nsplit > 1) {
    t.O_parts = at<void>(ws, w.aparts);
    t.lse_parts = reinterpret_cast<float*>(at<char>(ws, w.aparts) + align_up((size_t)(t.nsplit * b * nq * BCP * d) * 2));
  }
  // (an error here is an error: there is no other path)
  return cuda_status(quoka::launch_attn_tc(t, true, cs));
}

quoka_status quoka_get_device_status(const void* ws, void* stream, int32_t* device_status) {
  quoka::NvtxRange nvtx_range("quoka_get_device_status");
  if (device_status == nullptr) return QUOKA_ERR_INVALID_ARG;
  if (ws == nullptr) {  // the fixed scratch of quoka_select_static
    void* p = nullptr;
    const quoka_status st = quoka::static_scratch_address(&p);
    if (st != QUOKA_OK) return st;
    ws = p;
  }
  cudaStream_t cs = static_cast<cudaStream_t>(stream);
  int32_t v = 0;
  if (cudaMemcpyAsync(&v, ws, sizeof(int32_t), cudaMemcpyDeviceToHost, cs) != cudaSuccess)
    return QUOKA_ERR_CUDA;
  if (cudaStreamSynchronize(cs) != cudaSuccess) return QUOKA_ERR_CUDA;
  *device_status = v;
  return QUOKA_OK;
}

quoka_status quoka_get_device_fault_site(const void* ws, void* stream, int32_t* site) {
  quoka::NvtxRange nvtx_range("quoka_get_device_fault_site");
  if (site == nullptr) return QUOKA_ERR_INVALID_ARG;
  if (ws == nullptr) {  // the fixed scratch of quoka_select_static
    void* p = nullptr;
    const quoka_status st = quoka::static_scratch_address(&p);
    if (st != QUOKA_OK) return st;
    ws = p;
  }
  cudaStream_t cs = static_cast<cudaStream_t>(stream);
  int32_t v = 0;
  if (cudaMemcpyAsync(&v, static_cast<const int32_t*>(ws) + 1, sizeof(int32_t), cudaMemcpyDeviceToHost, cs) !=
      cudaSuccess)
    return QUOKA_ERR_CUDA;
  if (cudaStreamSynchronize(cs) != cudaSuccess) return QUOKA_ERR_CUDA;
  *site = v;
  return QUOKA_OK;
}

quoka_status quoka_debug_set_wait_hooks(uint64_t wait_limit_ns, uint32_t inject) {
  if (inject > QUOKA_DEBUG_INJECT_CACHE_ATTN) return QUOKA_ERR_INVALID_ARG;
  quoka::g_wait_ns.store(wait_limit_ns, std::memory_order_relaxed);
  quoka::g_inject.store(inject, std::memory_order_relaxed);
  return QUOKA_OK;
}

const char* quoka_status_string(quoka_status status) {
  switch (status) {
    case QUOKA_OK: return "QUOKA_OK";
    case QUOKA_ERR_INVALID_ARG: return "QUOKA_ERR_INVALID_ARG";
    case QUOKA_ERR_UNSUPPORTED: return "QUOKA_ERR_UNSUPPORTED";
    case QUOKA_ERR_WORKSPACE: return "QUOKA_ERR_WORKSPACE";
    case QUOKA_ERR_CUDA: return "QUOKA_ERR_CUDA";
    case QUOKA_ERR_TIMEOUT: return "QUOKA_ERR_TIMEOUT";
    case QUOKA_ERR_BOUNDS: return "QUOKA_ERR_BOUNDS";
  }
  return "QUOKA_ERR_UNKNOWN";
}

}  // extern "C"

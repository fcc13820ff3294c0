// Host helper: the driver's tensor-map encoder, fetched through the runtime (no
// link-time dependency on libcuda) at the first call that finds it, whichever
// thread makes it; a lookup that fails is made again by the next call.
#pragma once

#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_runtime.h>

#include <atomic>

namespace quoka {

inline PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder() {
  static std::atomic<PFN_cuTensorMapEncodeTiled_v12000> known{nullptr};
  PFN_cuTensorMapEncodeTiled_v12000 fn = known.load(std::memory_order_acquire);
  if (fn == nullptr) {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess) {
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
      known.store(fn, std::memory_order_release);
    }
  }
  return fn;
}

// 4-D bf16 map (d, rows, heads, batch) with a box of 64 columns x `box_rows`
// rows, 128-byte swizzle, zero fill out of bounds. Strides in elements.
inline bool encode_bf16_4d(CUtensorMap* m, const void* base, uint64_t d, uint64_t rows, uint64_t heads,
                           uint64_t batch, int64_t s_row, int64_t s_head, int64_t s_batch, uint32_t box_rows) {
  auto enc = tensor_map_encoder();
  if (enc == nullptr) return false;
  const cuuint64_t dims[4] = {d, rows, heads, batch};
  const cuuint64_t strides[3] = {(cuuint64_t)s_row * 2, (cuuint64_t)s_head * 2, (cuuint64_t)s_batch * 2};
  const cuuint32_t box[4] = {64, box_rows, 1, 1};
  const cuuint32_t estr[4] = {1, 1, 1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(base), dims, strides, box, estr,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// 4-D map of a pool of 1-byte codes (d, rows, heads, pages) with a box of d
// columns x `box_rows` rows, swizzled by its row length (128 or 64 bytes), zero
// fill out of bounds. Strides in bytes; that of a dimension of extent 1 is
// not used.
inline bool encode_codes_4d(CUtensorMap* m, const void* base, uint64_t d, uint64_t rows, uint64_t heads,
                            uint64_t pages, int64_t s_row, int64_t s_head, int64_t s_page, uint32_t box_rows) {
  auto enc = tensor_map_encoder();
  if (enc == nullptr) return false;
  const cuuint64_t dims[4] = {d, rows, heads, pages};
  const cuuint64_t strides[3] = {(cuuint64_t)s_row, heads > 1 ? (cuuint64_t)s_head : d,
                                 pages > 1 ? (cuuint64_t)s_page : d};
  const cuuint32_t box[4] = {(cuuint32_t)d, box_rows, 1, 1};
  const cuuint32_t estr[4] = {1, 1, 1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, const_cast<void*>(base), dims, strides, box, estr,
             CU_TENSOR_MAP_INTERLEAVE_NONE, d == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace quoka

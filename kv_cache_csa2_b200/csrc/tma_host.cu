// Host side of TMA: encoding tensor maps through the driver entry point
// (resolved once through the runtime, so the library needs no -lcuda).
#include <cuda.h>
#include <cudaTypedefs.h>

#include <mutex>

#include "common.cuh"
#include "sm100.cuh"

namespace csa2 {

static PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
  static std::once_flag once;
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  std::call_once(once, [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q = cudaDriverEntryPointSymbolNotFound;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
    else
      cudaGetLastError();
  });
  return fn;
}

csa2_status make_tensor_map_bf16_2d(CUtensorMap* map, const void* base, uint64_t rows,
                                    uint64_t cols, uint64_t row_pitch_bytes, uint32_t box_cols,
                                    uint32_t box_rows) {
  auto fn = encode_fn();
  if (!fn) return fail(CSA2_ERR_CUDA, "cuTensorMapEncodeTiled unavailable");
  if ((reinterpret_cast<uintptr_t>(base) & 15u) || (row_pitch_bytes & 15u) || box_cols * 2 > 128 ||
      box_rows > 256 || (box_cols * 2) % 16)
    return fail(CSA2_ERR_INVALID, "tensor map: base, pitch or box not valid for a 128-byte swizzle");
  const cuuint64_t dims[2] = {cols, rows};
  const cuuint64_t strides[1] = {row_pitch_bytes};
  const cuuint32_t box[2] = {box_cols, box_rows};
  const cuuint32_t estr[2] = {1, 1};
  const CUresult r = fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(base), dims,
                        strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                        CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                        CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) return fail(CSA2_ERR_CUDA, "cuTensorMapEncodeTiled failed (%d)", int(r));
  return CSA2_OK;
}

csa2_status make_tensor_map_paged(CUtensorMap* map, const void* base, int dim, int heads, int64_t head_stride,
                                  int page_size, int64_t token_stride, int64_t n_pages, int64_t page_stride,
                                  int box_rows) {
  auto fn = encode_fn();
  if (!fn) return fail(CSA2_ERR_CUDA, "cuTensorMapEncodeTiled unavailable");
  // a dimension of one element may carry any stride; give it a valid one
  const cuuint64_t row = static_cast<cuuint64_t>(dim) * 2;
  const cuuint64_t dims[4] = {static_cast<cuuint64_t>(dim), static_cast<cuuint64_t>(heads),
                              static_cast<cuuint64_t>(page_size), static_cast<cuuint64_t>(n_pages)};
  const cuuint64_t strides[3] = {heads > 1 ? static_cast<cuuint64_t>(head_stride) * 2 : row,
                                 page_size > 1 ? static_cast<cuuint64_t>(token_stride) * 2 : row,
                                 n_pages > 1 ? static_cast<cuuint64_t>(page_stride) * 2 : row};
  const cuuint32_t box[4] = {64, 1, static_cast<cuuint32_t>(box_rows), 1};
  const cuuint32_t estr[4] = {1, 1, 1, 1};
  const CUresult r = fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(base), dims, strides, box, estr,
                        CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                        CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) return fail(CSA2_ERR_CUDA, "cuTensorMapEncodeTiled failed (%d)", int(r));
  return CSA2_OK;
}

csa2_status make_tensor_map_heads(CUtensorMap* map, const void* base, int dim, int heads, int64_t head_stride,
                                  int64_t tokens, int64_t token_stride, int box_heads, int box_tokens) {
  auto fn = encode_fn();
  if (!fn) return fail(CSA2_ERR_CUDA, "cuTensorMapEncodeTiled unavailable");
  const cuuint64_t row = static_cast<cuuint64_t>(dim) * 2;
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(dim), static_cast<cuuint64_t>(heads),
                              static_cast<cuuint64_t>(tokens)};
  const cuuint64_t strides[2] = {heads > 1 ? static_cast<cuuint64_t>(head_stride) * 2 : row,
                                 tokens > 1 ? static_cast<cuuint64_t>(token_stride) * 2 : row};
  const cuuint32_t box[3] = {64, static_cast<cuuint32_t>(box_heads), static_cast<cuuint32_t>(box_tokens)};
  const cuuint32_t estr[3] = {1, 1, 1};
  const CUresult r = fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box, estr,
                        CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                        CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) return fail(CSA2_ERR_CUDA, "cuTensorMapEncodeTiled failed (%d)", int(r));
  return CSA2_OK;
}

}  // namespace csa2

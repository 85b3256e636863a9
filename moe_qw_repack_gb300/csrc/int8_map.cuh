// int8_map.cuh - tensor maps of the INT8 products: two dimensions, 128-byte swizzle, zeros outside.
#pragma once
#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_runtime.h>

namespace qw {

inline PFN_cuTensorMapEncodeTiled_v12000 int8_encode_fn() {
  static const PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault,
                                         &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      f = nullptr;
    return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f);
  }();
  return fn;
}

inline bool encode_int8_2d(CUtensorMap* map, CUtensorMapDataType type, const void* base,
                           uint64_t inner, uint64_t rows, uint64_t pitch_bytes, uint32_t box_inner,
                           uint32_t box_rows) {
  auto enc = int8_encode_fn();
  if (!enc) return false;
  cuuint64_t dim[2] = {inner, rows};
  cuuint64_t str[1] = {pitch_bytes};
  cuuint32_t box[2] = {box_inner, box_rows};
  cuuint32_t es[2] = {1, 1};
  return enc(map, type, 2, const_cast<void*>(base), dim, str, box, es,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace qw

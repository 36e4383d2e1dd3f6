// Tensor maps of the gated delta rule's chunked kernels (internal to libmamba2).
#pragma once

#include <cuda.h>

#include <cstring>

#include "kernels.h"

namespace mamba2 {

// Maps of a chunk's keys and queries (64 rows of 64 columns, 128-byte swizzle) and of 16 columns of its values or their
// gradients (32-byte swizzle). A head's columns are a dimension of their own, so that what lies behind them reads as zeros.
struct DeltaMaps {
  CUtensorMap k, q, v;
};

inline bool delta_map(CUtensorMap* tm, const void* base, int64_t rows, int heads, int width, int64_t ld, int columns) {
  using Encode = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                              const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                              CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
  static const Encode encode = []() -> Encode {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      return nullptr;
    return reinterpret_cast<Encode>(p);
  }();
  std::memset(tm, 0, sizeof *tm);
  if (!encode) return false;
  const cuuint64_t dims[3] = {(cuuint64_t)width, (cuuint64_t)heads, (cuuint64_t)rows};
  const cuuint64_t strides[2] = {(cuuint64_t)width * 2, (cuuint64_t)ld * 2};
  const cuuint32_t box[3] = {(cuuint32_t)columns, 1, MAMBA2_DELTA_CHUNK}, one[3] = {1, 1, 1};
  return encode(tm, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box, one,
                CU_TENSOR_MAP_INTERLEAVE_NONE, columns == 64 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_32B,
                CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Of a call's keys, queries and (with their stride) values or gradients of y.
inline bool delta_maps(DeltaMaps* m, const DeltaArgs& a, const void* v, int64_t ld_v) {
  const int64_t rows = a.tab.cu[a.tab.n];
  return delta_map(&m->k, a.k, rows, a.groups, a.dk, a.ld_k, 64) && delta_map(&m->q, a.q, rows, a.groups, a.dk, a.ld_q, 64) &&
         delta_map(&m->v, v, rows, a.heads, a.dv, ld_v, 16);
}

}  // namespace mamba2

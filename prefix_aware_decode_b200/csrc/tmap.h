// Tensor maps of the session-cache operators, encoded per call (host).
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <cudaTypedefs.h>

#include <cstdint>

namespace pa {

inline PFN_cuTensorMapEncodeTiled_v12000 tmap_encoder() {
  // magic static: looked up once
  static const PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult q;
    const cudaError_t e = cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &f, cudaEnableDefault, &q);
    return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(e == cudaSuccess && q == cudaDriverEntryPointSuccess ? f
                                                                                                                   : nullptr);
  }();
  return fn;
}

// bf16 tensor, contiguous, dims innermost first; boxes with the 128-byte
// swizzle (box[0] = 64 elements); reads out of range give zeros.
inline bool tmap_bf16(CUtensorMap* out, const void* base, int rank, const uint64_t* dims, const uint32_t* box) {
  auto fn = tmap_encoder();
  if (!fn) return false;
  cuuint64_t d[3], st[2];
  cuuint32_t bx[3], es[3] = {1, 1, 1};
  uint64_t stride = 2;
  for (int i = 0; i < rank; ++i) {
    d[i] = dims[i];
    bx[i] = box[i];
    stride *= dims[i];
    if (i < rank - 1) st[i] = stride;
  }
  return fn(out, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, (cuuint32_t)rank, const_cast<void*>(base), d, st, bx, es,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// A pool [num_pages][Hkv][16][D] as rows x D, boxes of one page x 64 dims.
inline bool tmap_pool(CUtensorMap* out, const void* pool, int num_pages, int Hkv, int D) {
  const uint64_t dims[2] = {(uint64_t)D, (uint64_t)num_pages * Hkv * 16};
  const uint32_t box[2] = {64, 16};
  return tmap_bf16(out, pool, 2, dims, box);
}

// q [rows][Hq][D], boxes of (rows_per_box rows) x (G heads) x 64 dims.
inline bool tmap_q(CUtensorMap* out, const void* q, int rows, int Hq, int D, int G, int rows_per_box) {
  const uint64_t dims[3] = {(uint64_t)D, (uint64_t)Hq, (uint64_t)rows};
  const uint32_t box[3] = {64, (uint32_t)G, (uint32_t)rows_per_box};
  return tmap_bf16(out, q, 3, dims, box);
}

}  // namespace pa

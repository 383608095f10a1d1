// Tensor-core paged decode over whole contexts (decode_tc_kernel.cuh), and the
// tensor maps of the pools.
#include <cudaTypedefs.h>
#include <mutex>

#include "decode_tc_kernel.cuh"

namespace pkv {

PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault,
                                         &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f);
  });
  return fn;
}

// Tensor map of one pool: 2-D with one box per 128-byte chunk of a page, or
// 3-D with one box per whole page (declared in tc_common.cuh).
int encode_pool_map(CUtensorMap* out, const void* base, int64_t rows, int D, int BS, bool fp8,
                    bool whole_page) {
  auto enc = tensor_map_encoder();
  if (!enc) return PKV_ERR_CUDA;
  const int esz = fp8 ? 1 : 2;
  const cuuint32_t chunk = static_cast<cuuint32_t>(128 / esz);  // elements per 128 bytes
  CUtensorMap m;
  CUresult r;
  const auto dtype = fp8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  if (!whole_page) {
    cuuint64_t dims[2] = {static_cast<cuuint64_t>(D), static_cast<cuuint64_t>(rows)};
    cuuint64_t strides[1] = {static_cast<cuuint64_t>(D) * esz};
    cuuint32_t box[2] = {chunk, static_cast<cuuint32_t>(BS)};
    cuuint32_t estr[2] = {1u, 1u};
    r = enc(&m, dtype, 2, const_cast<void*>(base), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  } else {
    const cuuint64_t nchunks = static_cast<cuuint64_t>(D) * esz / 128;
    cuuint64_t dims[3] = {chunk, static_cast<cuuint64_t>(rows), nchunks};
    cuuint64_t strides[2] = {static_cast<cuuint64_t>(D) * esz, 128u};
    cuuint32_t box[3] = {chunk, static_cast<cuuint32_t>(BS), static_cast<cuuint32_t>(nchunks)};
    cuuint32_t estr[3] = {1u, 1u, 1u};
    r = enc(&m, dtype, 3, const_cast<void*>(base), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  }
  if (r != CUDA_SUCCESS) return PKV_ERR_CUDA;
  *out = m;
  return PKV_OK;
}

// The same, cached per (pointer, shape, kind).
int pool_tensor_map(CUtensorMap* out, const void* base, int64_t rows, int D, int BS,
                    bool fp8, bool whole_page) {
  struct Entry {
    const void* base;
    int64_t rows;
    int d, bs;
    bool fp8, whole_page;
    CUtensorMap map;
  };
  static std::mutex mu;
  static Entry cache[32];
  static int used = 0, next = 0;
  {
    std::lock_guard<std::mutex> lock(mu);
    for (int i = 0; i < used; ++i)
      if (cache[i].base == base && cache[i].rows == rows && cache[i].d == D &&
          cache[i].bs == BS && cache[i].fp8 == fp8 && cache[i].whole_page == whole_page) {
        *out = cache[i].map;
        return PKV_OK;
      }
  }
  CUtensorMap m;
  const int rc = encode_pool_map(&m, base, rows, D, BS, fp8, whole_page);
  if (rc != PKV_OK) return rc;
  std::lock_guard<std::mutex> lock(mu);
  Entry& e = cache[next];
  e = Entry{base, rows, D, BS, fp8, whole_page, m};
  next = (next + 1) % 32;
  if (used < 32) ++used;
  *out = m;
  return PKV_OK;
}

int launch_decode_tc(const DecodeParams& p, const void* k_cache, const void* v_cache,
                     int head_dim, int block_size, bool fp8, dim3 grid, cudaStream_t st) {
  return fp8 ? dispatch_tc<true, kWhole>(p, k_cache, v_cache, head_dim, block_size, grid, st)
             : dispatch_tc<false, kWhole>(p, k_cache, v_cache, head_dim, block_size, grid, st);
}

}  // namespace pkv

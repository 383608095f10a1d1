// kv_cache_read: the rows that given slots of a cache hold, as bf16.
//
// Thread (h, c8) of a token's threads reads channels [8*c8, 8*c8+8) of head h
// from both pools (16, 8 or 4 bytes) and writes 16 bytes each: the reads and
// writes of a warp are whole rows. Bound by HBM where there are many tokens, by
// latency at a step's few.
#include "common.cuh"
#include "fp4.cuh"
#include "host_util.h"

namespace pkv {

__device__ __forceinline__ uint32_t bf16x2_of(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}

// Channels [8*c8, 8*c8+8) of token `off` of a page.
template <int DTYPE, int D>
__device__ __forceinline__ uint4 read8(const uint8_t* page, int off, int c8, float scale) {
  if constexpr (DTYPE == PKV_DTYPE_BF16) {
    return *reinterpret_cast<const uint4*>(page + (off * D + 8 * c8) * 2);
  } else {
    float x[8];
    if constexpr (DTYPE == PKV_DTYPE_FP8_E4M3) {
      const uint2 w = *reinterpret_cast<const uint2*>(page + off * D + 8 * c8);
#pragma unroll
      for (int i = 0; i < 8; ++i)
        x[i] = e4m3_f32(static_cast<uint8_t>((i < 4 ? w.x : w.y) >> (8 * (i & 3)))) * scale;
    } else {
      const uint32_t w =
          *reinterpret_cast<const uint32_t*>(page + fp4_codes_at<D>(off) + 4 * c8);
      const float s = e4m3_f32(page[fp4_scales_at<D>(off) + c8 / 2]);
      uint32_t f[4];
      e2m1x8_f16x2(w, f);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 y = __half22float2(*reinterpret_cast<const __half2*>(&f[i]));
        x[2 * i] = y.x * s * scale;  // y * s is exact
        x[2 * i + 1] = y.y * s * scale;
      }
    }
    return make_uint4(bf16x2_of(x[0], x[1]), bf16x2_of(x[2], x[3]), bf16x2_of(x[4], x[5]),
                      bf16x2_of(x[6], x[7]));
  }
}

template <int DTYPE, int D>
__global__ void __launch_bounds__(1024) kv_cache_read_kernel(
    uint4* __restrict__ k, uint4* __restrict__ v, const int64_t* __restrict__ slot_mapping,
    const uint8_t* __restrict__ k_cache, const uint8_t* __restrict__ v_cache, int num_blocks,
    int block_size, int num_kv_heads, int64_t page_bytes, const float* __restrict__ k_scale,
    const float* __restrict__ v_scale, int* err) {
  wait_prerequisite();
  const int token = blockIdx.x;
  const int h = threadIdx.x / (D / 8);
  const int c8 = threadIdx.x % (D / 8);
  const int64_t slot = slot_mapping[token];
  const int64_t at = (static_cast<int64_t>(token) * num_kv_heads + h) * (D / 8) + c8;
  uint4 kr = make_uint4(0, 0, 0, 0), vr = kr;
  if (slot >= static_cast<int64_t>(num_blocks) * block_size) {
    if (threadIdx.x == 0) report_error(err, PKV_DEVERR_SLOT);
  } else if (slot >= 0) {
    const int64_t page = (slot / block_size * num_kv_heads + h) * page_bytes;
    const int off = static_cast<int>(slot % block_size);
    const bool coded = DTYPE != PKV_DTYPE_BF16;
    kr = read8<DTYPE, D>(k_cache + page, off, c8, coded ? k_scale[h] : 1.f);
    vr = read8<DTYPE, D>(v_cache + page, off, c8, coded ? v_scale[h] : 1.f);
  }
  k[at] = kr;
  v[at] = vr;
}

}  // namespace pkv

extern "C" int pkv_kv_cache_read(void* k, void* v, const int64_t* slot_mapping, int num_tokens,
                                 const void* k_cache, const void* v_cache, pkv_cache_desc cache,
                                 const float* k_scale, const float* v_scale, void* stream) {
  using namespace pkv;
  int rc = check_cache_desc(cache, true);
  if (rc != PKV_OK) return rc;
  if (num_tokens < 0) return PKV_ERR_INVALID_ARG;
  if (num_tokens == 0) return PKV_OK;
  if (!k || !v || !slot_mapping || !k_cache || !v_cache) return PKV_ERR_INVALID_ARG;
  if (!aligned16(k) || !aligned16(v) || !aligned16(k_cache) || !aligned16(v_cache))
    return PKV_ERR_INVALID_ARG;
  if (cache.dtype != PKV_DTYPE_BF16 && (!k_scale || !v_scale)) return PKV_ERR_INVALID_ARG;
  const int threads = cache.num_kv_heads * (cache.head_dim / 8);
  if (threads > 1024) return PKV_ERR_UNSUPPORTED;
  const size_t rows = static_cast<size_t>(num_tokens) * cache.num_kv_heads * cache.head_dim * 2;
  const size_t pool = static_cast<size_t>(cache.num_blocks) * cache.num_kv_heads *
                      page_bytes(cache);
  const size_t slots = static_cast<size_t>(num_tokens) * sizeof(int64_t);
  for (void* w : {k, v})
    if (overlap(w, rows, k_cache, pool) || overlap(w, rows, v_cache, pool) ||
        overlap(w, rows, slot_mapping, slots))
      return PKV_ERR_INVALID_ARG;
  if (overlap(k, rows, v, rows)) return PKV_ERR_INVALID_ARG;
  auto go = [&](auto kern) {
    return launch_dependent(kern, dim3(num_tokens), dim3(threads), 0,
                            static_cast<cudaStream_t>(stream), static_cast<uint4*>(k),
                            static_cast<uint4*>(v), slot_mapping,
                            static_cast<const uint8_t*>(k_cache),
                            static_cast<const uint8_t*>(v_cache), cache.num_blocks,
                            cache.block_size, cache.num_kv_heads, page_bytes(cache), k_scale,
                            v_scale, device_error_ptr());
  };
  const bool wide = cache.head_dim == 256;
  switch (cache.dtype) {
    case PKV_DTYPE_BF16:
      return wide ? go(kv_cache_read_kernel<PKV_DTYPE_BF16, 256>)
                  : go(kv_cache_read_kernel<PKV_DTYPE_BF16, 128>);
    case PKV_DTYPE_FP8_E4M3:
      return wide ? go(kv_cache_read_kernel<PKV_DTYPE_FP8_E4M3, 256>)
                  : go(kv_cache_read_kernel<PKV_DTYPE_FP8_E4M3, 128>);
    default:
      return wide ? go(kv_cache_read_kernel<PKV_DTYPE_FP4_E2M1, 256>)
                  : go(kv_cache_read_kernel<PKV_DTYPE_FP4_E2M1, 128>);
  }
}

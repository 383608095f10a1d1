// kv_cache_read: the rows that given slots of a cache hold, as bf16.
//
// A thread has channels [8 c8, 8 c8 + 8) of a head of U tokens, their loads in flight
// together: 16, 8 or 4 bytes of each pool, 16 bytes of each result; a warp's are whole
// rows. Many tokens are bound by HBM and, on 4-bit pools, as much by the conversions'
// instructions: 32768 tokens, 8 heads, d = 128, from HBM, bf16 42.4 us, 94 % of the copy
// rate, E4M3 32.6 (91 %), 4-bit 32.1 (80 %; 30.4 right after they were written). A step's
// few are bound by latency (64 tokens: 2.4 us, 1.5 right behind a write).
#include <type_traits>

#include "common.cuh"
#include "fp4.cuh"
#include "host_util.h"
#include "quotients.cuh"

namespace pkv {

__device__ __forceinline__ uint32_t bf16x2_of(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}

// Channels [8*c8, 8*c8+8) of token `off` of a page, as stored.
template <int DTYPE, int D>
struct Eight {
  uint4 w;
  uint8_t s;

  __device__ __forceinline__ void load(const uint8_t* page, int off, int c8) {
    if constexpr (DTYPE == PKV_DTYPE_BF16) {
      w = *reinterpret_cast<const uint4*>(page + (off * D + 8 * c8) * 2);
    } else if constexpr (DTYPE == PKV_DTYPE_FP8_E4M3) {
      const uint2 x = *reinterpret_cast<const uint2*>(page + off * D + 8 * c8);
      w = make_uint4(x.x, x.y, 0, 0);
    } else {
      w.x = *reinterpret_cast<const uint32_t*>(page + fp4_codes_at<D>(off) + 4 * c8);
      s = page[fp4_scales_at<D>(off) + c8 / 2];
    }
  }

  __device__ __forceinline__ uint4 values(float scale) const {
    if constexpr (DTYPE == PKV_DTYPE_BF16) {
      return w;
    } else {
      uint32_t f[4], out[4];
      if constexpr (DTYPE == PKV_DTYPE_FP8_E4M3) {
        f[0] = e4m3x2_f16x2_lo(w.x), f[1] = e4m3x2_f16x2_lo(w.x >> 16);
        f[2] = e4m3x2_f16x2_lo(w.y), f[3] = e4m3x2_f16x2_lo(w.y >> 16);
      } else {
        // code * s is an f16 number
        e2m1x8_f16x2(w.x, f);
        const uint32_t by = e4m3x2_f16x2_lo(s | (static_cast<uint32_t>(s) << 8));
#pragma unroll
        for (int i = 0; i < 4; ++i) asm("mul.rn.f16x2 %0, %0, %1;" : "+r"(f[i]) : "r"(by));
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 y = __half22float2(*reinterpret_cast<const __half2*>(&f[i]));
        const float2 z = of_pair(mul_pair(pair_of(y.x, y.y), pair_of(scale, scale)));
        out[i] = bf16x2_of(z.x, z.y);
      }
      return make_uint4(out[0], out[1], out[2], out[3]);
    }
  }
};

template <int DTYPE, int D, int U>
__global__ void __launch_bounds__(1024) kv_cache_read_kernel(
    uint4* __restrict__ k, uint4* __restrict__ v, const int64_t* __restrict__ slot_mapping,
    const uint8_t* __restrict__ k_cache, const uint8_t* __restrict__ v_cache, int64_t num_slots,
    int log_block, int num_kv_heads, uint32_t page_bytes, uint32_t num_tokens, RowsOfCta deal,
    const float* __restrict__ k_scale, const float* __restrict__ v_scale, int* err) {
  wait_prerequisite();
  const uint32_t row = deal.row_of(threadIdx.x);
  if (row >= deal.rows) return;
  const uint32_t rest = threadIdx.x - row * deal.per;
  const int h = rest / (D / 8), c8 = rest % (D / 8);
  const uint32_t first = blockIdx.x * (U * deal.rows) + row;
  constexpr bool kCoded = DTYPE != PKV_DTYPE_BF16;
  const float ks = kCoded ? k_scale[h] : 1.f, vs = kCoded ? v_scale[h] : 1.f;
  Eight<DTYPE, D> ke[U], ve[U];
  bool some[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const uint32_t token = first + u * deal.rows;
    const int64_t slot = token < num_tokens ? slot_mapping[token] : -1;
    if (slot >= num_slots && rest == 0) report_error(err, PKV_DEVERR_SLOT);
    some[u] = slot >= 0 && slot < num_slots;
    if (some[u]) {
      const uint32_t blk = static_cast<uint32_t>(slot >> log_block);
      const uint64_t page = static_cast<uint64_t>(blk * num_kv_heads + h) * page_bytes;
      const int off = static_cast<int>(slot) & ((1 << log_block) - 1);
      ke[u].load(k_cache + page, off, c8);
      ve[u].load(v_cache + page, off, c8);
    }
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const uint32_t token = first + u * deal.rows;
    if (token >= num_tokens) continue;
    const uint4 zero = make_uint4(0, 0, 0, 0);
    const uint32_t i = token * deal.per + rest;
    k[i] = some[u] ? ke[u].values(ks) : zero;
    v[i] = some[u] ? ve[u].values(vs) : zero;
  }
}

template <int DTYPE, int D, typename... Args>
static int launch_read(int num_tokens, const RowsOfCta& deal, cudaStream_t st, Args... args) {
  auto go = [&](auto kern, int u) {
    const int per = u * static_cast<int>(deal.rows);
    return launch_dependent(kern, dim3((num_tokens + int64_t{per} - 1) / per),
                            dim3(deal.threads()), 0, st, args...);
  };
  // two tokens to a thread once they fill the SMs (2048 threads each): 32768 tokens right
  // after they were written, 4-bit, 8 heads, d = 128 32 us; one 39, four 34
  return int64_t{num_tokens} * deal.per >= 2 * 2048 * 152
             ? go(kv_cache_read_kernel<DTYPE, D, 2>, 2)
             : go(kv_cache_read_kernel<DTYPE, D, 1>, 1);
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
  const RowsOfCta deal(threads);
  if (static_cast<int64_t>(num_tokens) * threads >= (int64_t{1} << 32) - 4096 ||
      static_cast<int64_t>(cache.num_blocks) * cache.num_kv_heads >= int64_t{1} << 32)
    return PKV_ERR_UNSUPPORTED;
  auto go = [&](auto launch) {
    return launch(num_tokens, deal, static_cast<cudaStream_t>(stream), static_cast<uint4*>(k),
                  static_cast<uint4*>(v), slot_mapping, static_cast<const uint8_t*>(k_cache),
                  static_cast<const uint8_t*>(v_cache),
                  static_cast<int64_t>(cache.num_blocks) * cache.block_size,
                  cache.block_size == 16 ? 4 : 5, cache.num_kv_heads,
                  static_cast<uint32_t>(page_bytes(cache)),
                  static_cast<uint32_t>(num_tokens), deal, k_scale, v_scale,
                  device_error_ptr());
  };
  const bool wide = cache.head_dim == 256;
  auto at = [&](auto dtype) {
    constexpr int kType = decltype(dtype)::value;
    return wide ? go([](auto... a) { return launch_read<kType, 256>(a...); })
                : go([](auto... a) { return launch_read<kType, 128>(a...); });
  };
  switch (cache.dtype) {
    case PKV_DTYPE_BF16: return at(std::integral_constant<int, PKV_DTYPE_BF16>{});
    case PKV_DTYPE_FP8_E4M3: return at(std::integral_constant<int, PKV_DTYPE_FP8_E4M3>{});
    default: return at(std::integral_constant<int, PKV_DTYPE_FP4_E2M1>{});
  }
}

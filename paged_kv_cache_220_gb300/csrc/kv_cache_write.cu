// kv_cache_write: scatter this step's K/V rows into their cache slots.
//
// Blocks are filled as tokens are produced ("How vLLM gets real throughput on
// H100s ...", section "PagedAttention borrows from operating systems";
// "vLLM architecture, memory and benchmarks deep dive", section
// "PagedAttention: a 1960s idea for modern GPUs"): token i goes to physical
// block slot_mapping[i] / B at offset slot_mapping[i] % B, all KV heads.
//
// One CTA per token; thread (h, c8) moves the 8 elements [8*c8, 8*c8+8) of
// head h for both K and V: one 16-byte load and one 16-byte (bf16) or 8-byte
// (fp8) store each, so a token's row of a head is a coalesced 256/512-byte
// access. The work is a few hundred kilobytes per step; it is latency-bound.
#include "common.cuh"
#include "fp4.cuh"
#include "host_util.h"

namespace pkv {

template <bool FP8>
__global__ void __launch_bounds__(1024) kv_cache_write_kernel(
    const uint4* __restrict__ k, const uint4* __restrict__ v,
    const int64_t* __restrict__ slot_mapping, uint8_t* __restrict__ k_cache,
    uint8_t* __restrict__ v_cache, int num_blocks, int block_size, int num_kv_heads,
    int head_dim, const float* __restrict__ k_scale, const float* __restrict__ v_scale,
    int* err) {
  // the decode launched next may start its set-up now; it waits for this
  // grid's completion before it reads the cache
  allow_dependents();
  const int token = blockIdx.x;
  const int64_t slot = slot_mapping[token];
  if (slot < 0) return;
  if (slot >= static_cast<int64_t>(num_blocks) * block_size) {
    if (threadIdx.x == 0) report_error(err, PKV_DEVERR_SLOT);
    return;
  }
  const int vec_per_head = head_dim / 8;
  const int h = threadIdx.x / vec_per_head;
  const int c8 = threadIdx.x % vec_per_head;
  if (h >= num_kv_heads) return;
  const int64_t blk = slot / block_size;
  const int off = static_cast<int>(slot % block_size);
  // element index of (blk, h, off, 8*c8) in [NB][Hk][B][D]
  const int64_t dst = ((blk * num_kv_heads + h) * block_size + off) * head_dim + 8 * c8;
  const int64_t src = (static_cast<int64_t>(token) * num_kv_heads + h) * vec_per_head + c8;
  const uint4 kv = k[src];
  const uint4 vv = v[src];
  if constexpr (!FP8) {
    *reinterpret_cast<uint4*>(k_cache + dst * 2) = kv;
    *reinterpret_cast<uint4*>(v_cache + dst * 2) = vv;
  } else {
    const float ks = k_scale[h];
    const float vs = v_scale[h];
    const uint32_t kw[4] = {kv.x, kv.y, kv.z, kv.w};
    const uint32_t vw[4] = {vv.x, vv.y, vv.z, vv.w};
    uint32_t ko[2] = {0, 0}, vo[2] = {0, 0};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint32_t kb = (i & 1) ? (kw[i / 2] & 0xFFFF0000u) : (kw[i / 2] << 16);
      const uint32_t vb = (i & 1) ? (vw[i / 2] & 0xFFFF0000u) : (vw[i / 2] << 16);
      // IEEE fp32 quotient, then round-to-nearest-even with saturation.
      const float kq = __fdiv_rn(__uint_as_float(kb), ks);
      const float vq = __fdiv_rn(__uint_as_float(vb), vs);
      const uint32_t kc = __nv_cvt_float_to_fp8(kq, __NV_SATFINITE, __NV_E4M3);
      const uint32_t vc = __nv_cvt_float_to_fp8(vq, __NV_SATFINITE, __NV_E4M3);
      ko[i / 4] |= (kc & 0xFFu) << (8 * (i % 4));
      vo[i / 4] |= (vc & 0xFFu) << (8 * (i % 4));
    }
    *reinterpret_cast<uint2*>(k_cache + dst) = make_uint2(ko[0], ko[1]);
    *reinterpret_cast<uint2*>(v_cache + dst) = make_uint2(vo[0], vo[1]);
  }
}

// The larger of two, NaN if one is.
__device__ __forceinline__ float max_nan(float a, float b) {
  float d;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}

// Eight channels of a row -> their codes (a word) and the scale of their 16; the
// lane next to this one has the group's other eight.
__device__ __forceinline__ uint32_t quantize_fp4(const uint4& x, float scale, uint8_t& s_code) {
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
  float y[8];
  float a = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    y[i] = __fdiv_rn((i & 1) ? bf16hi(w[i / 2]) : bf16lo(w[i / 2]), scale);
    a = max_nan(a, fabsf(y[i]));
  }
  a = max_nan(a, __shfl_xor_sync(0xffffffffu, a, 1));
  s_code = static_cast<uint8_t>(
      __nv_cvt_float_to_fp8(__fdiv_rn(a, 6.f), __NV_SATFINITE, __NV_E4M3));
  const float s = e4m3_f32(s_code);
  if (!(s > 0.f)) return 0;  // zero or NaN
  uint32_t codes = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    codes |= e2m1x2_of(__fdiv_rn(y[2 * i], s), __fdiv_rn(y[2 * i + 1], s)) << (8 * i);
  return codes;
}

// 4-bit pools: thread (h, c8) has channels [8*c8, 8*c8+8) of a row; two threads
// share a scale. Every warp has a whole row of a head (D = 256) or two (128).
template <int D>
__global__ void __launch_bounds__(1024) kv_cache_write_fp4_kernel(
    const uint4* __restrict__ k, const uint4* __restrict__ v,
    const int64_t* __restrict__ slot_mapping, uint8_t* __restrict__ k_cache,
    uint8_t* __restrict__ v_cache, int num_blocks, int block_size, int num_kv_heads,
    const float* __restrict__ k_scale, const float* __restrict__ v_scale, int* err) {
  allow_dependents();
  const int token = blockIdx.x;
  const int64_t slot = slot_mapping[token];
  if (slot < 0) return;
  if (slot >= static_cast<int64_t>(num_blocks) * block_size) {
    if (threadIdx.x == 0) report_error(err, PKV_DEVERR_SLOT);
    return;
  }
  // blockDim.x is a multiple of a row's threads; whole rows fall out, so the
  // two lanes of a group stay together (a warp's idle half at D = 128 takes
  // part in the shuffle with zeros)
  const int h = threadIdx.x / (D / 8);
  const int c8 = threadIdx.x % (D / 8);
  const bool live = h < num_kv_heads;
  const int64_t blk = slot / block_size;
  const int off = static_cast<int>(slot % block_size);
  const int64_t page = (blk * num_kv_heads + h) * (block_size * (D / 16 * 9));
  const int64_t src = (static_cast<int64_t>(token) * num_kv_heads + h) * (D / 8) + c8;
  const uint4 zero = make_uint4(0, 0, 0, 0);
  const uint4 kv = live ? k[src] : zero;
  const uint4 vv = live ? v[src] : zero;
  uint8_t ks, vs;
  const uint32_t kc = quantize_fp4(kv, live ? k_scale[h] : 1.f, ks);
  const uint32_t vc = quantize_fp4(vv, live ? v_scale[h] : 1.f, vs);
  if (!live) return;
  const int64_t codes = page + fp4_codes_at<D>(off) + 4 * c8;
  *reinterpret_cast<uint32_t*>(k_cache + codes) = kc;
  *reinterpret_cast<uint32_t*>(v_cache + codes) = vc;
  if ((c8 & 1) == 0) {
    const int64_t scales = page + fp4_scales_at<D>(off) + c8 / 2;
    k_cache[scales] = ks;
    v_cache[scales] = vs;
  }
}

}  // namespace pkv

extern "C" int pkv_kv_cache_write(const void* k, const void* v, const int64_t* slot_mapping,
                                  int num_tokens, void* k_cache, void* v_cache,
                                  pkv_cache_desc cache, const float* k_scale,
                                  const float* v_scale, void* stream) {
  using namespace pkv;
  int rc = check_cache_desc(cache, true);
  if (rc != PKV_OK) return rc;
  if (num_tokens < 0) return PKV_ERR_INVALID_ARG;
  if (num_tokens == 0) return PKV_OK;
  if (!k || !v || !slot_mapping || !k_cache || !v_cache) return PKV_ERR_INVALID_ARG;
  if (!aligned16(k) || !aligned16(v) || !aligned16(k_cache) || !aligned16(v_cache))
    return PKV_ERR_INVALID_ARG;
  const bool fp8 = cache.dtype == PKV_DTYPE_FP8_E4M3;
  const bool fp4 = cache.dtype == PKV_DTYPE_FP4_E2M1;
  if ((fp8 || fp4) && (!k_scale || !v_scale)) return PKV_ERR_INVALID_ARG;
  const int threads = cache.num_kv_heads * (cache.head_dim / 8);
  if (threads > 1024) return PKV_ERR_UNSUPPORTED;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const int bs = cache.block_size, nb = cache.num_blocks, hk = cache.num_kv_heads,
            hd = cache.head_dim;
  auto* kc = static_cast<uint8_t*>(k_cache);
  auto* vc = static_cast<uint8_t*>(v_cache);
  if (fp4) {
    auto kern = hd == 256 ? kv_cache_write_fp4_kernel<256> : kv_cache_write_fp4_kernel<128>;
    kern<<<num_tokens, (threads + 31) / 32 * 32, 0, st>>>(
        static_cast<const uint4*>(k), static_cast<const uint4*>(v), slot_mapping, kc, vc, nb, bs,
        hk, k_scale, v_scale, device_error_ptr());
  } else if (fp8)
    kv_cache_write_kernel<true><<<num_tokens, threads, 0, st>>>(
        static_cast<const uint4*>(k), static_cast<const uint4*>(v), slot_mapping, kc, vc, nb,
        bs, hk, hd, k_scale, v_scale, device_error_ptr());
  else
    kv_cache_write_kernel<false><<<num_tokens, threads, 0, st>>>(
        static_cast<const uint4*>(k), static_cast<const uint4*>(v), slot_mapping, kc, vc, nb,
        bs, hk, hd, nullptr, nullptr, device_error_ptr());
  return launch_status();
}

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

// a / b rounded to nearest from r = 1/b rounded to nearest, by two corrections with
// the exact remainder (Markstein, IBM J. Res. Dev. 34, 1990): the first leaves at most
// one unit in the last place, the second none. Holds while b, r, the quotient and
// the remainder's last bit are normal numbers.
__device__ __forceinline__ float quotient(float a, float b, float r) {
  float q = a * r;
  q = fmaf(fmaf(-b, q, a), r, q);
  return fmaf(fmaf(-b, q, a), r, q);
}

// Eight channels of a row -> their codes (a word) and the scale of their 16; the
// lane next to this one has the group's other eight. inv: 1 / scale; plain: scale is
// in 2^-40 .. 2^40.
//
// 17 divisions to 8 channels are what this costs, so they are made from the
// divisors' reciprocals where that is exact: with a scale as above and the group's
// largest |x| in 2^-40 .. 2^60 all that count are far inside the normal numbers.
// Channels that are smaller by 2^20 get the code 0 however y is rounded.
__device__ __forceinline__ uint32_t quantize_fp4(const uint4& x, float scale, float inv,
                                                 bool plain, uint8_t& s_code) {
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
  float top = 0.f;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    top = max_nan(top, max_nan(fabsf(bf16lo(w[i])), fabsf(bf16hi(w[i]))));
  top = max_nan(top, __shfl_xor_sync(0xffffffffu, top, 1));
  float y[8], z[8];
  if (plain && top >= 0x1p-40f && top <= 0x1p60f) {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      y[i] = quotient((i & 1) ? bf16hi(w[i / 2]) : bf16lo(w[i / 2]), scale, inv);
    // rounded quotients grow with their numerators: the largest is the largest's
    const float a = quotient(top, scale, inv);
    s_code = static_cast<uint8_t>(
        __nv_cvt_float_to_fp8(quotient(a, 6.f, 1.f / 6.f), __NV_SATFINITE, __NV_E4M3));
    const float s = e4m3_f32(s_code);
    if (!(s > 0.f)) return 0;
    const float inv_s = __frcp_rn(s);
#pragma unroll
    for (int i = 0; i < 8; ++i) z[i] = quotient(y[i], s, inv_s);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      y[i] = __fdiv_rn((i & 1) ? bf16hi(w[i / 2]) : bf16lo(w[i / 2]), scale);
    const float a = fabsf(__fdiv_rn(top, scale));
    s_code = static_cast<uint8_t>(
        __nv_cvt_float_to_fp8(__fdiv_rn(a, 6.f), __NV_SATFINITE, __NV_E4M3));
    const float s = e4m3_f32(s_code);
    if (!(s > 0.f)) return 0;  // zero or NaN
#pragma unroll
    for (int i = 0; i < 8; ++i) z[i] = __fdiv_rn(y[i], s);
  }
  uint32_t codes = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) codes |= e2m1x2_of(z[2 * i], z[2 * i + 1]) << (8 * i);
  return codes;
}

// 4-bit pools. Item i is channels [8 c8, 8 c8 + 8) of head h of a token, c8 fastest:
// rows of k and v are read straight through, a thread U items THREADS apart with
// their loads in flight together. Two lanes share a scale.
constexpr int kFp4WriteThreads = 256;

template <int D, int U>
__global__ void __launch_bounds__(kFp4WriteThreads) kv_cache_write_fp4_kernel(
    const uint4* __restrict__ k, const uint4* __restrict__ v,
    const int64_t* __restrict__ slot_mapping, uint8_t* __restrict__ k_cache,
    uint8_t* __restrict__ v_cache, int64_t num_slots, int log_block, int num_kv_heads,
    uint32_t items, const float* __restrict__ k_scale, const float* __restrict__ v_scale,
    int* err) {
  allow_dependents();
  wait_prerequisite();
  const uint32_t per_token = num_kv_heads * (D / 8);
  const uint32_t first = blockIdx.x * (U * kFp4WriteThreads) + threadIdx.x;
  int64_t slot[U];
  int rest[U];
  uint4 kv[U], vv[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const uint32_t i = first + u * kFp4WriteThreads;
    const bool live = i < items;
    const uint32_t token = live ? i / per_token : 0;
    rest[u] = live ? static_cast<int>(i - token * per_token) : 0;
    slot[u] = live ? slot_mapping[token] : -1;
    kv[u] = live ? k[i] : make_uint4(0, 0, 0, 0);
    vv[u] = live ? v[i] : make_uint4(0, 0, 0, 0);
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int h = rest[u] / (D / 8), c8 = rest[u] % (D / 8);
    const float ks = k_scale[h], vs = v_scale[h];
    uint8_t k8, v8;
    const uint32_t kc = quantize_fp4(kv[u], ks, __frcp_rn(ks), ks >= 0x1p-40f && ks <= 0x1p40f, k8);
    const uint32_t vc = quantize_fp4(vv[u], vs, __frcp_rn(vs), vs >= 0x1p-40f && vs <= 0x1p40f, v8);
    if (slot[u] < 0) continue;
    if (slot[u] >= num_slots) {
      if (rest[u] == 0) report_error(err, PKV_DEVERR_SLOT);
      continue;
    }
    const int64_t blk = slot[u] >> log_block;
    const int off = static_cast<int>(slot[u] - (blk << log_block));
    const int64_t page = ((blk * num_kv_heads + h) << log_block) * (D / 16 * 9);
    const int64_t codes = page + fp4_codes_at<D>(off) + 4 * c8;
    *reinterpret_cast<uint32_t*>(k_cache + codes) = kc;
    *reinterpret_cast<uint32_t*>(v_cache + codes) = vc;
    if ((c8 & 1) == 0) {
      const int64_t scales = page + fp4_scales_at<D>(off) + c8 / 2;
      k_cache[scales] = k8;
      v_cache[scales] = v8;
    }
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
    const int64_t items = static_cast<int64_t>(num_tokens) * threads;
    if (items >= (int64_t{1} << 32) - 4 * kFp4WriteThreads) return PKV_ERR_UNSUPPORTED;
    auto go = [&](auto kern, int u) {
      const int64_t per = static_cast<int64_t>(u) * kFp4WriteThreads;
      return launch_dependent(kern, dim3(static_cast<unsigned>((items + per - 1) / per)),
                              dim3(kFp4WriteThreads), 0, st, static_cast<const uint4*>(k),
                              static_cast<const uint4*>(v), slot_mapping, kc, vc,
                              static_cast<int64_t>(nb) * bs, bs == 16 ? 4 : 5, hk,
                              static_cast<uint32_t>(items), k_scale, v_scale,
                              device_error_ptr());
    };
    // two items to a thread once they fill the SMs (8 CTAs each)
    if (items >= 2 * 8 * 152 * kFp4WriteThreads)
      return hd == 256 ? go(kv_cache_write_fp4_kernel<256, 2>, 2)
                       : go(kv_cache_write_fp4_kernel<128, 2>, 2);
    return hd == 256 ? go(kv_cache_write_fp4_kernel<256, 1>, 1)
                     : go(kv_cache_write_fp4_kernel<128, 1>, 1);
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

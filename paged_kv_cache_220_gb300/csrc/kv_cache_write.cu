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
#include "quotients.cuh"

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

// The larger magnitude of each of two bf16 pairs, NaN if one is; some sign.
__device__ __forceinline__ uint32_t max2_abs(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("max.NaN.xorsign.abs.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}

// Eight channels of a row -> their codes (a word) and the scale of their 16; the
// lane next to this one has the group's other eight. inv: 1 / scale to nearest;
// plain: scale is in 2^-40 .. 2^40.
//
// 17 divisions to 8 channels are what this would cost. With a scale as above and the
// group's largest |x| in 2^-40 .. 2^60 all that count are far inside the normal
// numbers (channels smaller than that by 2^20 get the code 0 however they are
// rounded), and a product with reciprocals is off by less than 2^-21 of the rounded
// quotient of the rounded quotient: the same product 2^-20 lower and 2^-20 higher
// have it between them, and rounding to a code keeps the order. Where both get the
// same code, that is the one (8192 tokens, 8 heads, d = 128: 14.1 -> 12.1 us).
// Elsewhere, near a midpoint between two codes, the quotients are made exact, in
// pairs. Of y / s only the side of a midpoint counts. s has 4 significant bits and a
// midpoint m 3, so m s is an fp32 number: y / s rounds to m only if y = m s, the next y
// is off by at least 1.6 % of a unit in the last place more than half a unit, and one
// correction of an approximate reciprocal's quotient, off by 2^-20 of a unit before
// it is rounded, decides the same.
__device__ __forceinline__ uint32_t quantize_fp4(const uint4& x, float scale, float inv,
                                                 bool plain, uint8_t& s_code) {
  constexpr float kLess = 1.f - 0x1p-20f, kMore = 1.f + 0x1p-20f, kSixth = 1.f / 6.f;
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
  uint32_t t2 = max2_abs(max2_abs(w[0], w[1]), max2_abs(w[2], w[3]));
  t2 = max2_abs(t2, __shfl_xor_sync(0xffffffffu, t2, 1));
  const float top = fabsf(bf16lo(max2_abs(t2, t2 >> 16)));
  float z8[8];
  if (plain && top >= 0x1p-40f && top <= 0x1p60f) {
    const uint64_t r = pair_of(inv, inv), b = pair_of(-scale, -scale);
    const float t6 = top * inv * kSixth;
    const uint32_t both = __nv_cvt_float2_to_fp8x2(make_float2(t6 * kLess, t6 * kMore),
                                                   __NV_SATFINITE, __NV_E4M3);
    s_code = static_cast<uint8_t>(both);
    if (s_code != both >> 8) {
      // rounded quotients grow with their numerators: the largest is the largest's
      const float a = of_pair(quotients<2>(pair_of(top, top), b, r)).x;
      const float a6 = of_pair(quotients<2>(pair_of(a, a), pair_of(-6.f, -6.f),
                                            pair_of(kSixth, kSixth))).x;
      s_code = static_cast<uint8_t>(__nv_cvt_float_to_fp8(a6, __NV_SATFINITE, __NV_E4M3));
    }
    const float s = e4m3_f32(s_code);
    if (!(s > 0.f)) return 0;
    float inv_s;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(inv_s) : "f"(s));
    // (with a scale that is a power of two x meets midpoints exactly all the time)
    if ((__float_as_uint(scale) & 0x007FFFFFu) != 0) {
      const float f = inv * inv_s, less = f * kLess, more = f * kMore;
      const uint64_t f_less = pair_of(less, less), f_more = pair_of(more, more);
      float y8[8];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint64_t xs = pair_of(bf16lo(w[i]), bf16hi(w[i]));
        const float2 y = of_pair(mul_pair(xs, f_less)), z = of_pair(mul_pair(xs, f_more));
        y8[2 * i] = y.x, y8[2 * i + 1] = y.y;
        z8[2 * i] = z.x, z8[2 * i + 1] = z.y;
      }
      const uint32_t codes = e2m1x8_of(y8);
      if (codes == e2m1x8_of(z8)) return codes;
    }
    const uint64_t rs = pair_of(inv_s, inv_s), bs = pair_of(-s, -s);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint64_t y = quotients<2>(pair_of(bf16lo(w[i]), bf16hi(w[i])), b, r);
      const float2 z = of_pair(quotients<1>(y, bs, rs));
      // (a correction turns -0 into 0; the quotient has x's sign)
      z8[2 * i] = __uint_as_float(__float_as_uint(z.x) | ((w[i] << 16) & 0x80000000u));
      z8[2 * i + 1] = __uint_as_float(__float_as_uint(z.y) | (w[i] & 0x80000000u));
    }
    return e2m1x8_of(z8);
  }
  s_code = static_cast<uint8_t>(__nv_cvt_float_to_fp8(
      __fdiv_rn(fabsf(__fdiv_rn(top, scale)), 6.f), __NV_SATFINITE, __NV_E4M3));
  const float s = e4m3_f32(s_code);
  if (!(s > 0.f)) return 0;  // zero or NaN
#pragma unroll
  for (int i = 0; i < 8; ++i)
    z8[i] = __fdiv_rn(__fdiv_rn((i & 1) ? bf16hi(w[i / 2]) : bf16lo(w[i / 2]), scale), s);
  return e2m1x8_of(z8);
}

// 4-bit pools. A thread has channels [8 c8, 8 c8 + 8) of a head of U tokens, their loads
// in flight together; rows of k and v are read straight through. Two lanes share a
// scale. No pipe is full: loads and instructions (conversions, packing, addresses; the
// integer pipe is 66 % busy, the issue slots 64 %) wait for one another. 32768 tokens, 8
// heads, d = 128 38.0 us, 4.5 TB/s, 47.5 with scales that are powers of two; 64 tokens 1.5
// us. (One token to a thread: 8192 tokens 11.6 us, two 11.2, three 12.0, four 13.5.)
template <int D, int U>
__global__ void __launch_bounds__(1024) kv_cache_write_fp4_kernel(
    const uint4* __restrict__ k, const uint4* __restrict__ v,
    const int64_t* __restrict__ slot_mapping, uint8_t* __restrict__ k_cache,
    uint8_t* __restrict__ v_cache, int64_t num_slots, int log_block, int num_kv_heads,
    uint32_t num_tokens, RowsOfCta deal, const float* __restrict__ k_scale,
    const float* __restrict__ v_scale, int* err) {
  allow_dependents();
  wait_prerequisite();
  const uint32_t row = deal.row_of(threadIdx.x);
  const bool some = row < deal.rows;
  const uint32_t rest = some ? threadIdx.x - row * deal.per : 0;
  const int h = rest / (D / 8), c8 = rest % (D / 8);
  const uint32_t first = blockIdx.x * (U * deal.rows) + row;
  int64_t slot[U];
  uint4 kv[U], vv[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const uint32_t token = first + u * deal.rows;
    const bool live = some && token < num_tokens;
    const uint32_t i = token * deal.per + rest;
    slot[u] = live ? slot_mapping[token] : -1;
    kv[u] = live ? k[i] : make_uint4(0, 0, 0, 0);
    vv[u] = live ? v[i] : make_uint4(0, 0, 0, 0);
  }
  const float ks = k_scale[h], vs = v_scale[h];
  const float k_inv = __frcp_rn(ks), v_inv = __frcp_rn(vs);
  const bool k_plain = ks >= 0x1p-40f && ks <= 0x1p40f;
  const bool v_plain = vs >= 0x1p-40f && vs <= 0x1p40f;
#pragma unroll
  for (int u = 0; u < U; ++u) {
    uint8_t k8, v8;
    const uint32_t kc = quantize_fp4(kv[u], ks, k_inv, k_plain, k8);
    const uint32_t vc = quantize_fp4(vv[u], vs, v_inv, v_plain, v8);
    if (slot[u] < 0) continue;
    if (slot[u] >= num_slots) {
      if (rest == 0) report_error(err, PKV_DEVERR_SLOT);
      continue;
    }
    const uint32_t blk = static_cast<uint32_t>(slot[u] >> log_block);
    const int off = static_cast<int>(slot[u]) & ((1 << log_block) - 1);
    const int64_t page = static_cast<uint64_t>(blk * num_kv_heads + h) *
                         static_cast<uint32_t>((D / 16 * 9) << log_block);
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
    const int64_t pieces = static_cast<int64_t>(num_tokens) * threads;
    if (pieces >= (int64_t{1} << 32) - 4096 ||
        static_cast<int64_t>(nb) * hk >= int64_t{1} << 32)
      return PKV_ERR_UNSUPPORTED;
    const RowsOfCta deal(threads);
    auto go = [&](auto kern, int u) {
      const int per = u * static_cast<int>(deal.rows);
      return launch_dependent(kern, dim3((num_tokens + int64_t{per} - 1) / per),
                              dim3(deal.threads()), 0, st, static_cast<const uint4*>(k),
                              static_cast<const uint4*>(v), slot_mapping, kc, vc,
                              static_cast<int64_t>(nb) * bs, bs == 16 ? 4 : 5, hk,
                              static_cast<uint32_t>(num_tokens), deal, k_scale, v_scale,
                              device_error_ptr());
    };
    // two tokens to a thread once they fill the SMs (2048 threads each)
    if (pieces >= 2 * 2048 * 152)
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

// block_bounds: the lowest and highest K of every channel of a block, as whole
// multiples of a step per head.
//
// One warp per (block, head) page: lane l has D/32 consecutive channels and
// keeps their running minimum and maximum over the page's cached rows, the rows'
// loads (up to 64 words a lane) in flight together; a row of a page is one coalesced
// access. The extremes are taken two channels at a time of what is stored, bf16
// pairs, or f16 pairs that hold a code times its 16 channels' scale exactly: the
// head's scale, floor and ceil of a quotient by a positive step grow with the value
// (or all fall, for a negative scale), so only the extremes go through them. A
// third running value, a maximum that keeps NaN, says where a zero has to join.
// Bound by HBM over whole prompts, by latency at one block per sequence.
#include <algorithm>

#include "common.cuh"
#include "fp4.cuh"
#include "host_util.h"

namespace pkv {

constexpr int kBoundsWarps = 4;

struct BoundsParams {
  int8_t* bounds;
  const uint8_t* k_cache;
  const float* k_scale;
  const float* step;
  const int32_t* block_tables;
  const int32_t* context_lens;
  const int32_t* num_new;
  int* err;
  int num_blocks, num_kv_heads, max_blocks_per_seq, max_new;
  int per_seq;      // most blocks of a sequence that its newest tokens touch
  int64_t items;    // num_seqs * per_seq * num_kv_heads
};

// Row r's channels [C*lane, C*lane + C) of a page, as loaded, and as pairs.
template <int DTYPE, int D>
struct BoundsRow {
  static constexpr int C = D / 32;
  static constexpr int kWords = DTYPE == PKV_DTYPE_BF16 ? C / 2 : (C + 3) / 4;
  uint32_t w[kWords];
  uint8_t s;

  __device__ __forceinline__ void load(const uint8_t* page, int r, int lane) {
    if constexpr (DTYPE == PKV_DTYPE_BF16) {
      const uint8_t* p = page + (r * D + C * lane) * 2;
      if constexpr (C == 8) {
        const uint4 x = *reinterpret_cast<const uint4*>(p);
        w[0] = x.x, w[1] = x.y, w[2] = x.z, w[3] = x.w;
      } else {
        const uint2 x = *reinterpret_cast<const uint2*>(p);
        w[0] = x.x, w[1] = x.y;
      }
    } else if constexpr (DTYPE == PKV_DTYPE_FP8_E4M3) {
      const uint8_t* p = page + r * D + C * lane;
      if constexpr (C == 8) {
        const uint2 x = *reinterpret_cast<const uint2*>(p);
        w[0] = x.x, w[1] = x.y;
      } else {
        w[0] = *reinterpret_cast<const uint32_t*>(p);
      }
    } else {
      const uint8_t* p = page + fp4_codes_at<D>(r) + C / 2 * lane;
      if constexpr (C == 8)
        w[0] = *reinterpret_cast<const uint32_t*>(p);
      else
        w[0] = *reinterpret_cast<const uint16_t*>(p);
      s = page[fp4_scales_at<D>(r) + C * lane / kFp4Group];
    }
  }

  __device__ __forceinline__ void pairs(uint32_t (&x)[C / 2]) const {
    if constexpr (DTYPE == PKV_DTYPE_BF16) {
#pragma unroll
      for (int i = 0; i < C / 2; ++i) x[i] = w[i];
    } else if constexpr (DTYPE == PKV_DTYPE_FP8_E4M3) {
#pragma unroll
      for (int i = 0; i < C / 2; ++i) x[i] = e4m3x2_f16x2_lo(w[i / 2] >> (16 * (i & 1)));
    } else {
      uint32_t f[4];
      e2m1x8_f16x2(w[0], f);
      const uint32_t by = e4m3x2_f16x2_lo(s | (static_cast<uint32_t>(s) << 8));
#pragma unroll
      for (int i = 0; i < C / 2; ++i)
        asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(x[i]) : "r"(f[i]), "r"(by));
    }
  }
};

// Extremes of pairs: bf16 pairs if BF, else f16 ones.
template <bool BF>
__device__ __forceinline__ uint32_t min2(uint32_t a, uint32_t b) {
  uint32_t d;
  if constexpr (BF)
    asm("min.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  else
    asm("min.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
template <bool BF>
__device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b) {
  uint32_t d;
  if constexpr (BF)
    asm("max.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  else
    asm("max.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
template <bool BF>
__device__ __forceinline__ uint32_t max2_nan(uint32_t a, uint32_t b) {
  uint32_t d;
  if constexpr (BF)
    asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  else
    asm("max.NaN.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
template <bool BF>
__device__ __forceinline__ float2 to_f32(uint32_t a) {
  if constexpr (BF) return make_float2(bf16lo(a), bf16hi(a));
  return __half22float2(*reinterpret_cast<const __half2*>(&a));
}

template <int DTYPE, int D, int BS>
__global__ void __launch_bounds__(kBoundsWarps * 32) block_bounds_kernel(const BoundsParams p) {
  wait_prerequisite();
  const int lane = threadIdx.x & 31;
  const int64_t item = static_cast<int64_t>(blockIdx.x) * kBoundsWarps + (threadIdx.x >> 5);
  if (item >= p.items) return;
  const int h = static_cast<int>(item % p.num_kv_heads);
  const int64_t sj = item / p.num_kv_heads;
  const int j = static_cast<int>(sj % p.per_seq);
  const int s = static_cast<int>(sj / p.per_seq);
  const int ctx = p.context_lens[s];
  int n = p.num_new != nullptr ? p.num_new[s] : p.max_new;
  if (ctx < 0 || ctx > static_cast<int64_t>(p.max_blocks_per_seq) * BS || n < 0 ||
      n > p.max_new) {
    if (lane == 0 && h == 0 && j == 0) report_error(p.err, PKV_DEVERR_CONTEXT);
    return;
  }
  n = min(n, ctx);
  const int blk = (ctx - n) / BS + j;
  const int rows = min(BS, ctx - blk * BS);
  if (n == 0 || rows <= 0) return;
  const int32_t pb = p.block_tables[static_cast<int64_t>(s) * p.max_blocks_per_seq + blk];
  if (pb < 0 || pb >= p.num_blocks) {
    if (lane == 0 && h == 0) report_error(p.err, PKV_DEVERR_BLOCK_ID);
    return;
  }
  constexpr int kPage = DTYPE == PKV_DTYPE_BF16       ? BS * D * 2
                        : DTYPE == PKV_DTYPE_FP8_E4M3 ? BS * D
                                                      : BS * D / 16 * 9;
  constexpr bool BF = DTYPE == PKV_DTYPE_BF16;
  const uint8_t* page = p.k_cache + (static_cast<int64_t>(pb) * p.num_kv_heads + h) * kPage;
  using Row = BoundsRow<DTYPE, D>;
  constexpr int C = Row::C;
  constexpr int kTogether = Row::kWords * BS <= 64 ? BS : 64 / Row::kWords;  // rows
  constexpr uint32_t kPlus = BF ? 0x7F807F80u : 0x7C007C00u;                 // +inf twice
  uint32_t lo[C / 2], hi[C / 2], any[C / 2];
#pragma unroll
  for (int i = 0; i < C / 2; ++i) {
    lo[i] = kPlus;
    hi[i] = any[i] = kPlus | 0x80008000u;
  }
#pragma unroll 1
  for (int r0 = 0; r0 < rows; r0 += kTogether) {
    Row row[kTogether];
    // rows behind the last cached one are read as that one once more
#pragma unroll
    for (int r = 0; r < kTogether; ++r) row[r].load(page, min(r0 + r, rows - 1), lane);
#pragma unroll
    for (int r = 0; r < kTogether; ++r) {
      uint32_t x[C / 2];
      row[r].pairs(x);
#pragma unroll
      for (int i = 0; i < C / 2; ++i) {
        lo[i] = min2<BF>(lo[i], x[i]);
        hi[i] = max2<BF>(hi[i], x[i]);
        any[i] = max2_nan<BF>(any[i], x[i]);
      }
    }
  }
  const float scale = BF ? 1.f : p.k_scale[h];
  const float step = p.step[h];
  uint32_t wl[(C + 3) / 4] = {}, wh[(C + 3) / 4] = {};
#pragma unroll
  for (int i = 0; i < C; ++i) {
    const float2 l2 = to_f32<BF>(lo[i / 2]), h2 = to_f32<BF>(hi[i / 2]);
    const float2 a2 = to_f32<BF>(any[i / 2]);
    float l = (i & 1) ? l2.y : l2.x, u = (i & 1) ? h2.y : h2.x;
    const float a = (i & 1) ? a2.y : a2.x;
    if (a != a) {  // a NaN counts as 0
      l = fminf(l, 0.f);
      u = fmaxf(u, 0.f);
    }
    if (!BF) {
      // (infinities times a scale of 0 are NaN, which count as 0)
      l *= scale;
      u *= scale;
      l = l == l ? l : 0.f;
      u = u == u ? u : 0.f;
      if (scale < 0.f) {
        const float t = l;
        l = u;
        u = t;
      }
    }
    const float x = fminf(fmaxf(floorf(__fdiv_rn(l, step)), -127.f), 127.f);
    const float y = fminf(fmaxf(ceilf(__fdiv_rn(u, step)), -127.f), 127.f);
    wl[i / 4] |= (static_cast<uint32_t>(static_cast<int>(x)) & 0xFFu) << (8 * (i & 3));
    wh[i / 4] |= (static_cast<uint32_t>(static_cast<int>(y)) & 0xFFu) << (8 * (i & 3));
  }
  int8_t* out = p.bounds + (static_cast<int64_t>(pb) * p.num_kv_heads + h) * (2 * D) + C * lane;
  if constexpr (C == 8) {
    *reinterpret_cast<uint2*>(out) = make_uint2(wl[0], wl[1]);
    *reinterpret_cast<uint2*>(out + D) = make_uint2(wh[0], wh[1]);
  } else {
    *reinterpret_cast<uint32_t*>(out) = wl[0];
    *reinterpret_cast<uint32_t*>(out + D) = wh[0];
  }
}

template <int DTYPE>
static int launch_bounds(const BoundsParams& p, int head_dim, int block_size, cudaStream_t st) {
  const dim3 grid(static_cast<unsigned>((p.items + kBoundsWarps - 1) / kBoundsWarps));
  const dim3 block(kBoundsWarps * 32);
  if (head_dim == 256)
    return block_size == 16
               ? launch_dependent(block_bounds_kernel<DTYPE, 256, 16>, grid, block, 0, st, p)
               : launch_dependent(block_bounds_kernel<DTYPE, 256, 32>, grid, block, 0, st, p);
  return block_size == 16
             ? launch_dependent(block_bounds_kernel<DTYPE, 128, 16>, grid, block, 0, st, p)
             : launch_dependent(block_bounds_kernel<DTYPE, 128, 32>, grid, block, 0, st, p);
}

}  // namespace pkv

extern "C" int pkv_block_bounds(int8_t* bounds, const void* k_cache, pkv_cache_desc cache,
                                const float* k_scale, const float* step,
                                const int32_t* block_tables, int max_blocks_per_seq,
                                const int32_t* context_lens, const int32_t* num_new, int max_new,
                                int num_seqs, void* stream) {
  using namespace pkv;
  int rc = check_cache_desc(cache, true);
  if (rc != PKV_OK) return rc;
  if (num_seqs < 0 || max_new < 0 || max_blocks_per_seq <= 0) return PKV_ERR_INVALID_ARG;
  const int64_t cap = static_cast<int64_t>(max_blocks_per_seq) * cache.block_size;
  if (cap > (1 << 30)) return PKV_ERR_UNSUPPORTED;
  if (num_seqs == 0 || max_new == 0) return PKV_OK;
  if (!bounds || !k_cache || !step || !block_tables || !context_lens) return PKV_ERR_INVALID_ARG;
  if (!aligned16(bounds) || !aligned16(k_cache)) return PKV_ERR_INVALID_ARG;
  if (cache.dtype != PKV_DTYPE_BF16 && !k_scale) return PKV_ERR_INVALID_ARG;
  const size_t pages = static_cast<size_t>(cache.num_blocks) * cache.num_kv_heads;
  const size_t out = pages * 2 * cache.head_dim, heads = cache.num_kv_heads * sizeof(float);
  const size_t seqs = static_cast<size_t>(num_seqs) * sizeof(int32_t);
  if (overlap(bounds, out, k_cache, pages * page_bytes(cache)) ||
      overlap(bounds, out, step, heads) || (k_scale && overlap(bounds, out, k_scale, heads)) ||
      overlap(bounds, out, block_tables, seqs * max_blocks_per_seq) ||
      overlap(bounds, out, context_lens, seqs) ||
      (num_new && overlap(bounds, out, num_new, seqs)))
    return PKV_ERR_INVALID_ARG;
  BoundsParams p{};
  p.bounds = bounds;
  p.k_cache = static_cast<const uint8_t*>(k_cache);
  p.k_scale = k_scale;
  p.step = step;
  p.block_tables = block_tables;
  p.context_lens = context_lens;
  p.num_new = num_new;
  p.err = device_error_ptr();
  p.num_blocks = cache.num_blocks;
  p.num_kv_heads = cache.num_kv_heads;
  p.max_blocks_per_seq = max_blocks_per_seq;
  p.max_new = max_new;
  // n tokens that end anywhere in a block touch at most (n - 2) / B + 2 blocks
  p.per_seq = static_cast<int>(std::min<int64_t>(
      max_blocks_per_seq, (static_cast<int64_t>(max_new) + cache.block_size - 2) /
                              cache.block_size + 1));
  p.items = static_cast<int64_t>(num_seqs) * p.per_seq * cache.num_kv_heads;
  if ((p.items + kBoundsWarps - 1) / kBoundsWarps > INT32_MAX) return PKV_ERR_UNSUPPORTED;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  switch (cache.dtype) {
    case PKV_DTYPE_BF16:
      return launch_bounds<PKV_DTYPE_BF16>(p, cache.head_dim, cache.block_size, st);
    case PKV_DTYPE_FP8_E4M3:
      return launch_bounds<PKV_DTYPE_FP8_E4M3>(p, cache.head_dim, cache.block_size, st);
    default:
      return launch_bounds<PKV_DTYPE_FP4_E2M1>(p, cache.head_dim, cache.block_size, st);
  }
}

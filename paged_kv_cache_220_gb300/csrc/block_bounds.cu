// block_bounds: the lowest and highest K of every channel of a block, as whole
// multiples of a step per head.
//
// One warp per (block, head) page, in lines of 256 values (one token at d = 256, two
// at d = 128): a lane has 8 channels of one token of every line, a line is one
// coalesced access, and up to 32 words a lane are in flight together. The extremes
// are taken two channels at a time of what is stored, bf16 pairs, or f16 pairs that
// hold a code times its 16 channels' scale exactly: the head's scale, floor and ceil of a
// quotient by a positive step grow with the value (or all fall, for a negative
// scale), so only the extremes go through them. Extremes that keep a NaN say which
// lanes have to take theirs once more, value by value.
//
// Bound by HBM on bf16 pools (8 x 16384 tokens, 4 heads, d = 256, B = 16: 45 us, 93 % of
// the copy rate), by latency and the instructions of the extremes and conversions on
// coded ones (E4M3 26.3 us, 85 %; 4-bit 27.9 us, 49 %), and by latency alone at one block
// per sequence (2.5 us). Two to eight pages to a warp, with their blocks looked up
// together, took longer (E4M3, d = 128: 25 us with one, 34 to 63).
#include <algorithm>

#include "common.cuh"
#include "fp4.cuh"
#include "host_util.h"
#include "quotients.cuh"

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
};

// Eight channels of a token, as loaded from a line of a page, and as pairs.
template <int DTYPE, int D>
struct BoundsEight {
  static constexpr int kWords = DTYPE == PKV_DTYPE_BF16 ? 4 : DTYPE == PKV_DTYPE_FP8_E4M3 ? 2 : 1;
  static constexpr int kLine = DTYPE == PKV_DTYPE_FP4_E2M1 ? kFp4Line : 64 * 2 * kWords;
  uint32_t w[kWords];
  uint32_t s;

  // piece: which 8 of the line's 256 values. Loads stay in program order, so that a
  // batch of them is issued before the first is used (left to the compiler, few
  // registers: 8 x 8192 tokens, 8 heads, d = 128, bf16 27.5 us, 24.2 so)
  __device__ __forceinline__ void load(const uint8_t* line, int piece) {
    const uint8_t* p = line + 4 * kWords * piece;
    if constexpr (kWords == 4) {
      asm volatile("ld.global.v4.u32 {%0,%1,%2,%3}, [%4];"
                   : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
                   : "l"(p));
    } else if constexpr (kWords == 2) {
      asm volatile("ld.global.v2.u32 {%0,%1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "l"(p));
    } else {
      asm volatile("ld.global.u32 %0, [%1];" : "=r"(w[0]) : "l"(p));
      asm volatile("ld.global.u8 %0, [%1];" : "=r"(s) : "l"(line + 128 + piece / 2));
    }
  }

  __device__ __forceinline__ void pairs(uint32_t (&x)[4]) const {
    if constexpr (DTYPE == PKV_DTYPE_BF16) {
#pragma unroll
      for (int i = 0; i < 4; ++i) x[i] = w[i];
    } else if constexpr (DTYPE == PKV_DTYPE_FP8_E4M3) {
#pragma unroll
      for (int i = 0; i < 4; ++i) x[i] = e4m3x2_f16x2_lo(w[i / 2] >> (16 * (i & 1)));
    } else {
      uint32_t f[4];
      e2m1x8_f16x2(w[0], f);
      const uint32_t by = e4m3x2_f16x2_lo(s * 0x0101u);
#pragma unroll
      for (int i = 0; i < 4; ++i)
        asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(x[i]) : "r"(f[i]), "r"(by));
    }
  }
};

// Extremes of pairs, NaN where one is: bf16 pairs if BF, else f16 ones.
template <bool BF>
__device__ __forceinline__ uint32_t min2_nan(uint32_t a, uint32_t b) {
  uint32_t d;
  if constexpr (BF)
    asm("min.NaN.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  else
    asm("min.NaN.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
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

// The two numbers' whole steps below and above, clamped. plain: step in 2^-40 .. 2^16
// and l, u within a factor of 2^60 of it, whose quotients by it inv gives to nearest.
__device__ __forceinline__ void whole_steps(float l, float u, float step, float inv, bool plain,
                                            uint32_t& lo, uint32_t& hi) {
  float2 q;
  if (plain)
    q = of_pair(quotients<2>(pair_of(l, u), pair_of(-step, -step), pair_of(inv, inv)));
  else
    q = make_float2(__fdiv_rn(l, step), __fdiv_rn(u, step));
  // added to 1.5 * 2^23 a number below 2^22 leaves its whole part in the low bits
  constexpr float kWhole = 12582912.f;
  lo = __float_as_uint(__fadd_rd(fminf(fmaxf(q.x, -127.f), 127.f), kWhole)) & 0xFFu;
  hi = __float_as_uint(__fadd_ru(fminf(fmaxf(q.y, -127.f), 127.f), kWhole)) & 0xFFu;
}

template <int DTYPE, int D, int BS>
__global__ void __launch_bounds__(kBoundsWarps * 32, 8) block_bounds_kernel(const BoundsParams p) {
  wait_prerequisite();
  const int lane = threadIdx.x & 31;
  const uint32_t jh = blockIdx.x * kBoundsWarps + (threadIdx.x >> 5);
  const uint32_t heads = p.num_kv_heads;
  const int s = blockIdx.y;
  if (jh >= p.per_seq * heads) return;
  const int h = jh % heads, j = jh / heads;
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
  using Eight = BoundsEight<DTYPE, D>;
  constexpr int R = 256 / D;        // tokens of a line
  constexpr int NL = BS / R;        // lines of a page
  constexpr int P = 32 / R;         // lanes to a token
  constexpr int kTogether = Eight::kWords * NL <= 32 ? NL : 32 / Eight::kWords;
  constexpr bool BF = DTYPE == PKV_DTYPE_BF16;
  const int64_t at = static_cast<int64_t>(pb) * p.num_kv_heads + h;
  const uint8_t* page = p.k_cache + at * (NL * Eight::kLine);
  const float scale = BF ? 1.f : p.k_scale[h];
  const float step = p.step[h];
  const int off = lane / P;  // this lane's token of a line
  uint32_t lo[4], hi[4];
  auto take = [&](const Eight& e, bool first) {
    uint32_t x[4];
    e.pairs(x);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      lo[i] = first ? x[i] : min2_nan<BF>(lo[i], x[i]);
      hi[i] = first ? x[i] : max2_nan<BF>(hi[i], x[i]);
    }
  };
  if (rows == BS) {
#pragma unroll
    for (int l0 = 0; l0 < NL; l0 += kTogether) {
      Eight e[kTogether];
#pragma unroll
      for (int l = 0; l < kTogether; ++l) e[l].load(page + (l0 + l) * Eight::kLine, lane);
#pragma unroll
      for (int l = 0; l < kTogether; ++l) take(e[l], l0 + l == 0);
    }
  } else {
    // tokens behind the last cached one are read as that one once more
    constexpr int kSome = kTogether < 8 ? kTogether : 8;
#pragma unroll 1
    for (int t0 = 0; t0 < rows; t0 += kSome * R) {
      Eight e[kSome];
#pragma unroll
      for (int l = 0; l < kSome; ++l) {
        const int t = min(t0 + l * R + off, rows - 1);
        e[l].load(page + t / R * Eight::kLine, t % R * P + lane % P);
      }
#pragma unroll
      for (int l = 0; l < kSome; ++l) take(e[l], t0 == 0 && l == 0);
    }
  }
  // ---- the tokens of a line are joined; a lane goes on with 8 / R channels
  constexpr int NP = 4 / R;
  if constexpr (R == 2) {
#pragma unroll
    for (int i = 0; i < NP; ++i) {
      const uint32_t l = __shfl_xor_sync(0xffffffffu, off ? lo[i] : lo[NP + i], P);
      const uint32_t u = __shfl_xor_sync(0xffffffffu, off ? hi[i] : hi[NP + i], P);
      lo[i] = min2_nan<BF>(off ? lo[NP + i] : lo[i], l);
      hi[i] = max2_nan<BF>(off ? hi[NP + i] : hi[i], u);
    }
  }
  const int c0 = lane % P * 8 + off * (2 * NP);
  const float inv = __frcp_rn(step);
  // a code times its scale is 0 or in 2^-10 .. 2688
  const bool plain = step >= 0x1p-40f && step <= 0x1p16f &&
                     (BF || (scale >= 0x1p-20f && scale <= 0x1p20f));
  uint32_t wl[(NP + 1) / 2] = {}, wh[(NP + 1) / 2] = {};
#pragma unroll
  for (int i = 0; i < 2 * NP; ++i) {
    const float2 l2 = to_f32<BF>(lo[i / 2]), h2 = to_f32<BF>(hi[i / 2]);
    float l = (i & 1) ? l2.y : l2.x, u = (i & 1) ? h2.y : h2.x;
    if (l != l) {
      // a NaN counts as 0
      l = INFINITY;
      u = -INFINITY;
#pragma unroll 1
      for (int t = 0; t < rows; ++t) {
        Eight e;
        uint32_t x[4];
        e.load(page + t / R * Eight::kLine, t % R * P + lane % P);
        e.pairs(x);
        const float2 v2 = to_f32<BF>(R == 2 && off ? x[(NP + i / 2) & 3] : x[i / 2]);
        float v = (i & 1) ? v2.y : v2.x;
        v = v == v ? v : 0.f;
        l = fminf(l, v);
        u = fmaxf(u, v);
      }
    }
    if (BF) {
      if (plain) {
        // far outside the bounds' range before, far outside after
        l = fminf(fmaxf(l, -512.f * step), 512.f * step);
        u = fminf(fmaxf(u, -512.f * step), 512.f * step);
      }
    } else {
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
    uint32_t bl, bh;
    whole_steps(l, u, step, inv, plain, bl, bh);
    wl[i / 4] |= bl << (8 * (i & 3));
    wh[i / 4] |= bh << (8 * (i & 3));
  }
  int8_t* out = p.bounds + at * (2 * D) + c0;
  if constexpr (R == 1) {
    *reinterpret_cast<uint2*>(out) = make_uint2(wl[0], wl[1]);
    *reinterpret_cast<uint2*>(out + D) = make_uint2(wh[0], wh[1]);
  } else {
    *reinterpret_cast<uint32_t*>(out) = wl[0];
    *reinterpret_cast<uint32_t*>(out + D) = wh[0];
  }
}

template <int DTYPE>
static int launch_bounds(const BoundsParams& p, int num_seqs, int head_dim, int block_size, cudaStream_t st) {
  const int64_t pages = static_cast<int64_t>(p.per_seq) * p.num_kv_heads;  // up to 2^31
  const dim3 grid(static_cast<unsigned>((pages + kBoundsWarps - 1) / kBoundsWarps), num_seqs);
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
  if (cap > (1 << 30) || num_seqs > 65535) return PKV_ERR_UNSUPPORTED;
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
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  switch (cache.dtype) {
    case PKV_DTYPE_BF16:
      return launch_bounds<PKV_DTYPE_BF16>(p, num_seqs, cache.head_dim, cache.block_size, st);
    case PKV_DTYPE_FP8_E4M3:
      return launch_bounds<PKV_DTYPE_FP8_E4M3>(p, num_seqs, cache.head_dim, cache.block_size, st);
    default:
      return launch_bounds<PKV_DTYPE_FP4_E2M1>(p, num_seqs, cache.head_dim, cache.block_size, st);
  }
}

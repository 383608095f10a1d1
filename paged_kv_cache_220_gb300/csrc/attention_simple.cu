// Attention of one query token per sequence over a 4-bit cache, and over listed
// blocks of any cache: one warp per query head and partition, fp32 throughout.
#include "common.cuh"
#include "decode_params.h"
#include "fp4.cuh"
#include "host_util.h"

namespace pkv {

// Channels [C*lane, C*lane + C) of token t of a page, C = D/32.
template <int DTYPE, int D>
__device__ __forceinline__ void load_row(const uint8_t* page, int t, int lane,
                                         float (&x)[D / 32]) {
  constexpr int C = D / 32;
  if constexpr (DTYPE == PKV_DTYPE_BF16) {
    const uint16_t* p = reinterpret_cast<const uint16_t*>(page) + t * D + C * lane;
#pragma unroll
    for (int i = 0; i < C; ++i) x[i] = bf16lo(p[i]);
  } else if constexpr (DTYPE == PKV_DTYPE_FP8_E4M3) {
    const uint8_t* p = page + t * D + C * lane;
#pragma unroll
    for (int i = 0; i < C; ++i) x[i] = e4m3_f32(p[i]);
  } else {
    const uint8_t* p = page + fp4_codes_at<D>(t) + C / 2 * lane;
    uint32_t w = 0, f[4];
#pragma unroll
    for (int i = 0; i < C / 2; ++i) w |= static_cast<uint32_t>(p[i]) << (8 * i);
    e2m1x8_f16x2(w, f);
    const float s = e4m3_f32(page[fp4_scales_at<D>(t) + C * lane / kFp4Group]);
#pragma unroll
    for (int i = 0; i < C; ++i) {
      const float2 y = __half22float2(*reinterpret_cast<const __half2*>(&f[i / 2]));
      x[i] = ((i & 1) ? y.y : y.x) * s;
    }
  }
}

template <int DTYPE, int D>
__global__ void __launch_bounds__(32) attention_simple_kernel(const DecodeParams p, int block_size,
                                                              int64_t page_bytes) {
  constexpr int C = D / 32;
  wait_prerequisite();
  const int lane = threadIdx.x;
  const int part = blockIdx.x, j = blockIdx.y;
  int s = blockIdx.z;
  if (p.seq_order != nullptr) {
    s = p.seq_order[blockIdx.z];
    if (s < 0 || s >= static_cast<int>(gridDim.z)) {
      if (lane == 0) report_error(p.err, PKV_DEVERR_ORDER);
      return;
    }
  }
  const int h = j / p.group;
  int ctx = p.context_lens[s];
  const int cap = p.max_blocks_per_seq * block_size;
  if (ctx < 0 || ctx > cap) {
    if (lane == 0) report_error(p.err, PKV_DEVERR_CONTEXT);
    ctx = ctx < 0 ? 0 : cap;
  }
  const int32_t* list = nullptr;
  int b0 = 0, b1 = (ctx + block_size - 1) / block_size;
  const int all = b1;
  if (p.list != nullptr) {
    const int64_t row = static_cast<int64_t>(s) * p.num_kv_heads + h;
    list = p.list + row * p.max_selected;
    b1 = p.counts[row];
    if (b1 < 0 || b1 > p.max_selected) {
      if (lane == 0) report_error(p.err, PKV_DEVERR_SELECT);
      b1 = b1 < 0 ? 0 : p.max_selected;
    }
  } else if (p.partition_blocks > 0) {
    b0 = part * p.partition_blocks;
    if (b0 >= b1) return;
    b1 = min(b1, b0 + p.partition_blocks);
  }
  const int64_t qrow = static_cast<int64_t>(s) * p.num_heads + j;
  float q[C], o[C];
#pragma unroll
  for (int i = 0; i < C; ++i) {
    q[i] = bf16lo(p.q[qrow * D + C * lane + i]) * p.qscale *
           (DTYPE == PKV_DTYPE_BF16 ? 1.f : p.k_scale[h]);
    o[i] = 0.f;
  }
  float m = -INFINITY, l = 0.f;
  for (int v = b0; v < b1; ++v) {
    const int b = list ? list[v] : v;
    if (b < 0 || b >= all) {
      if (lane == 0) report_error(p.err, PKV_DEVERR_SELECT);
      continue;
    }
    const int32_t pb = p.block_tables[static_cast<int64_t>(s) * p.max_blocks_per_seq + b];
    if (pb < 0 || pb >= p.num_blocks) {
      if (lane == 0) report_error(p.err, PKV_DEVERR_BLOCK_ID);
      continue;
    }
    const int64_t page = (static_cast<int64_t>(pb) * p.num_kv_heads + h) * page_bytes;
    const int rows = min(block_size, ctx - b * block_size);
    for (int t = 0; t < rows; ++t) {
      float x[C];
      load_row<DTYPE, D>(p.k_cache + page, t, lane, x);
      float z = 0.f;
#pragma unroll
      for (int i = 0; i < C; ++i) z = fmaf(q[i], x[i], z);
#pragma unroll
      for (int off = 16; off > 0; off >>= 1) z += __shfl_xor_sync(0xffffffffu, z, off);
      load_row<DTYPE, D>(p.v_cache + page, t, lane, x);
      const float mn = fmaxf(m, z);
      const float c = fast_exp2(m - mn), w = fast_exp2(z - mn);
      l = l * c + w;
#pragma unroll
      for (int i = 0; i < C; ++i) o[i] = fmaf(w, x[i], o[i] * c);
      m = mn;
    }
  }
  const float f = (l > 0.f ? 1.f / l : 0.f) * (DTYPE == PKV_DTYPE_BF16 ? 1.f : p.v_scale[h]);
  if (p.list == nullptr && p.partition_blocks > 0) {
    const int64_t slot = qrow * p.np_max + part;
#pragma unroll
    for (int i = 0; i < C; ++i) p.tmp_out[slot * D + C * lane + i] = o[i] * f;
    if (lane == 0) {
      p.max_logits[slot] = m * 0.6931471805599453f;
      p.exp_sums[slot] = l;
    }
  } else {
#pragma unroll
    for (int i = 0; i < C; ++i)
      p.out[qrow * D + C * lane + i] = float_to_bf16_bits(l > 0.f ? o[i] * f : 0.f);
  }
}

int launch_attention_simple(const DecodeParams& p, const pkv_cache_desc& cache, dim3 grid,
                            cudaStream_t st) {
  grid.y = p.num_heads;
  auto go = [&](auto kern) {
    return launch_dependent(kern, grid, dim3(32), 0, st, p, cache.block_size, page_bytes(cache));
  };
  const bool wide = cache.head_dim == 256;
  if (cache.dtype == PKV_DTYPE_BF16)
    return wide ? go(attention_simple_kernel<PKV_DTYPE_BF16, 256>)
                : go(attention_simple_kernel<PKV_DTYPE_BF16, 128>);
  if (cache.dtype == PKV_DTYPE_FP8_E4M3)
    return wide ? go(attention_simple_kernel<PKV_DTYPE_FP8_E4M3, 256>)
                : go(attention_simple_kernel<PKV_DTYPE_FP8_E4M3, 128>);
  return wide ? go(attention_simple_kernel<PKV_DTYPE_FP4_E2M1, 256>)
              : go(attention_simple_kernel<PKV_DTYPE_FP4_E2M1, 128>);
}

}  // namespace pkv

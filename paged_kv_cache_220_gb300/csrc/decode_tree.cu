// Attention of several query tokens per sequence (drafted tokens, a chain or
// a tree) over the paged cache.
//
// One CTA per (query row, query head); its warps take the visible tokens in
// turn, each lane 1/32 of the head dimension, with an online softmax in fp32
// per warp, merged through shared memory.
#include <algorithm>
#include <climits>
#include <cmath>

#include "common.cuh"
#include "host_util.h"

namespace pkv {

struct RowsParams {
  const uint16_t* q;
  uint16_t* out;
  const uint8_t* k_cache;
  const uint8_t* v_cache;
  const float* k_scale;
  const float* v_scale;
  const int32_t* block_tables;
  const int32_t* context_lens;
  const int32_t* q_start;
  const uint64_t* tree_mask;
  int* err;
  int num_seqs, num_blocks, num_kv_heads, num_heads, group, block_size, max_blocks_per_seq;
  int max_draft;
  float qscale;
};

constexpr int kRowsWarps = 4;

template <int D, bool FP8>
__device__ __forceinline__ void load_row(const uint8_t* base, int64_t elem, int lane, float* x) {
  constexpr int E = D / 32;
  const int64_t at = elem + lane * E;
  if constexpr (FP8) {
    uint32_t w[E / 4];
#pragma unroll
    for (int i = 0; i < E / 4; ++i) w[i] = reinterpret_cast<const uint32_t*>(base + at)[i];
#pragma unroll
    for (int i = 0; i < E; ++i) {
      const __half_raw h = __nv_cvt_fp8_to_halfraw((w[i / 4] >> (8 * (i % 4))) & 0xFFu, __NV_E4M3);
      x[i] = __half2float(__half(h));
    }
  } else {
#pragma unroll
    for (int i = 0; i < E / 2; ++i) {
      const uint32_t w = reinterpret_cast<const uint32_t*>(base + 2 * at)[i];
      x[2 * i] = bf16lo(w);
      x[2 * i + 1] = bf16hi(w);
    }
  }
}

template <int D, bool FP8>
__global__ void __launch_bounds__(kRowsWarps * 32) rows_kernel(const RowsParams p) {
  constexpr int E = D / 32;
  __shared__ float sm_m[kRowsWarps], sm_l[kRowsWarps];
  __shared__ float sm_o[kRowsWarps][D];
  const int j = blockIdx.y, h = j / p.group;
  const int64_t row = blockIdx.x;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // the sequence of this row: the last one that starts at or before it
  if (row < p.q_start[0] || row >= p.q_start[p.num_seqs]) return;
  int s = 0, hi = p.num_seqs;
  while (hi - s > 1) {
    const int mid = (s + hi) / 2;
    if (p.q_start[mid] <= row) s = mid; else hi = mid;
  }
  const int i = static_cast<int>(row) - p.q_start[s];
  const int n = p.q_start[s + 1] - p.q_start[s];
  int ctx = p.context_lens[s];
  const int64_t cap = static_cast<int64_t>(p.max_blocks_per_seq) * p.block_size;
  if (ctx < 0 || ctx > cap) {
    if (threadIdx.x == 0) report_error(p.err, PKV_DEVERR_CONTEXT);
    ctx = ctx < 0 ? 0 : static_cast<int>(cap);
  }
  if (n > p.max_draft || n > ctx || i >= n) {
    if (threadIdx.x == 0) report_error(p.err, PKV_DEVERR_DRAFT);
    return;
  }
  const int base = ctx - n;
  const uint64_t mask = p.tree_mask != nullptr ? p.tree_mask[row] : (2ull << i) - 1;
  float q[E], o[E], m = -INFINITY, l = 0.f;
  load_row<D, false>(reinterpret_cast<const uint8_t*>(p.q), (row * p.num_heads + j) * D, lane, q);
#pragma unroll
  for (int e = 0; e < E; ++e) o[e] = 0.f;
  const float qs = FP8 ? p.qscale * p.k_scale[h] : p.qscale;
  for (int t = warp; t < ctx; t += kRowsWarps) {
    const bool see = t < base || ((mask >> (t - base)) & 1);
    if (!see) continue;
    const int32_t b = p.block_tables[static_cast<int64_t>(s) * p.max_blocks_per_seq +
                                     t / p.block_size];
    if (b < 0 || b >= p.num_blocks) {
      if (lane == 0) report_error(p.err, PKV_DEVERR_BLOCK_ID);
      continue;
    }
    const int64_t at = ((static_cast<int64_t>(b) * p.num_kv_heads + h) * p.block_size +
                        t % p.block_size) * D;
    float x[E], z = 0.f;
    load_row<D, FP8>(p.k_cache, at, lane, x);
#pragma unroll
    for (int e = 0; e < E; ++e) z = fmaf(q[e], x[e], z);
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) z += __shfl_xor_sync(0xffffffffu, z, off);
    z *= qs;
    load_row<D, FP8>(p.v_cache, at, lane, x);
    const float mn = fmaxf(m, z);
    const float c = fast_exp2(m - mn), w = fast_exp2(z - mn);
    m = mn;
    l = fmaf(l, c, w);
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] = fmaf(o[e], c, w * x[e]);
  }
  if (lane == 0) {
    sm_m[warp] = m;
    sm_l[warp] = l;
  }
#pragma unroll
  for (int e = 0; e < E; ++e) sm_o[warp][lane * E + e] = o[e];
  __syncthreads();
  float M = -INFINITY, L = 0.f;
  for (int w = 0; w < kRowsWarps; ++w) M = fmaxf(M, sm_m[w]);
  float a[kRowsWarps];
  for (int w = 0; w < kRowsWarps; ++w) {
    a[w] = sm_l[w] > 0.f ? fast_exp2(sm_m[w] - M) : 0.f;
    L += a[w] * sm_l[w];
  }
  const float vs = FP8 ? p.v_scale[h] : 1.f;
  for (int c = threadIdx.x; c < D; c += kRowsWarps * 32) {
    float r = 0.f;
    for (int w = 0; w < kRowsWarps; ++w)
      if (a[w] > 0.f) r += a[w] * sm_o[w][c];
    p.out[(row * p.num_heads + j) * D + c] = float_to_bf16_bits(L > 0.f ? r / L * vs : 0.f);
  }
}

static int launch_rows(const RowsParams& p, int head_dim, bool fp8, int rows, cudaStream_t st) {
  const dim3 grid(rows, p.num_heads), block(kRowsWarps * 32);
  if (head_dim == 128)
    fp8 ? rows_kernel<128, true><<<grid, block, 0, st>>>(p)
        : rows_kernel<128, false><<<grid, block, 0, st>>>(p);
  else
    fp8 ? rows_kernel<256, true><<<grid, block, 0, st>>>(p)
        : rows_kernel<256, false><<<grid, block, 0, st>>>(p);
  return launch_status();
}

}  // namespace pkv

extern "C" size_t pkv_tree_workspace_bytes(int num_seqs, int num_queries, int num_heads,
                                           int num_kv_heads, int head_dim, int max_context,
                                           int max_draft) {
  return 0;
}

extern "C" int pkv_paged_attention_tree(
    void* out, const void* q, const void* k_cache, const void* v_cache, pkv_cache_desc cache,
    const float* k_scale, const float* v_scale, const int32_t* block_tables,
    int max_blocks_per_seq, const int32_t* context_lens, const int32_t* q_start, int num_seqs,
    int num_queries, int max_draft, const uint64_t* tree_mask, int num_heads, int max_context,
    float scale, void* workspace, size_t workspace_bytes, void* stream) {
  using namespace pkv;
  int g = 0;
  int rc = check_attention(cache, out, q, k_cache, v_cache, k_scale, v_scale, block_tables,
                      max_blocks_per_seq, context_lens, num_queries > 0 ? num_seqs : 0, num_heads,
                      max_context, scale, &g);
  if (rc != PKV_OK) return rc;
  if (num_queries < 0 || max_draft < 1 || max_draft > PKV_MAX_DRAFT) return PKV_ERR_INVALID_ARG;
  if (num_seqs == 0 || num_queries == 0) return PKV_OK;
  if (!q_start) return PKV_ERR_INVALID_ARG;
  RowsParams p{};
  p.q = static_cast<const uint16_t*>(q);
  p.out = static_cast<uint16_t*>(out);
  p.k_cache = static_cast<const uint8_t*>(k_cache);
  p.v_cache = static_cast<const uint8_t*>(v_cache);
  p.k_scale = k_scale;
  p.v_scale = v_scale;
  p.block_tables = block_tables;
  p.context_lens = context_lens;
  p.q_start = q_start;
  p.tree_mask = tree_mask;
  p.err = device_error_ptr();
  p.num_seqs = num_seqs;
  p.num_blocks = cache.num_blocks;
  p.num_kv_heads = cache.num_kv_heads;
  p.num_heads = num_heads;
  p.group = g;
  p.block_size = cache.block_size;
  p.max_blocks_per_seq = max_blocks_per_seq;
  p.max_draft = max_draft;
  p.qscale = scale * 1.4426950408889634f;
  return launch_rows(p, cache.head_dim, cache.dtype == PKV_DTYPE_FP8_E4M3, num_queries,
                     static_cast<cudaStream_t>(stream));
}

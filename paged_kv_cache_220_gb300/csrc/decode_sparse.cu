// paged_attention_sparse: the C entry points of decode attention over listed
// blocks, each (sequence, KV head) pair its own list. The kernels are the decode's
// in their listed forms (decode_tc_kernel.cuh for bf16 and E4M3 pools, decode_fp4.cu
// for 4-bit ones) and the merge is its merge (reduce.cu): what a list changes is
// which blocks are walked, each with the two look-ups (entry, table) of a batch of
// entries made ahead of its copies.
//
// Measured: bf16, d = 256, 256 pairs of 128 blocks of 16 85.5 to 86.7 us (92 % of the copy
// rate); d = 128, 256 pairs of 256 blocks 89 us (89 %), 1024 of 64 blocks of 32 162 (98 %);
// E4M3 d = 128 49 us (81 %) and 85 (93 %); 4-bit, 32 pairs of 512 blocks of 32, d = 256,
// 36.8 us (61 %: one wave of short shares and the merge).
#include <algorithm>

#include "decode_tc_kernel.cuh"

namespace pkv {

static int launch_decode_listed(const DecodeParams& p, const void* k_cache, const void* v_cache,
                                int head_dim, int block_size, bool fp8, dim3 grid,
                                cudaStream_t st) {
  return fp8 ? dispatch_tc<true, kListed>(p, k_cache, v_cache, head_dim, block_size, grid, st)
             : dispatch_tc<false, kListed>(p, k_cache, v_cache, head_dim, block_size, grid, st);
}

// CTAs that run at once on 152 SMs: four to an SM at d = 256, eight at d = 128.
static int64_t listed_wave(int head_dim) { return head_dim == 256 ? 600 : 1200; }

// Entries to a partition of lists of up to max_selected, 0 = one pass.
static int64_t listed_split(const pkv_cache_desc& cache, int num_seqs, int max_selected,
                            int* cluster) {
  const int64_t pairs = static_cast<int64_t>(num_seqs) * cache.num_kv_heads;
  if (cache.dtype != PKV_DTYPE_FP4_E2M1)
    return parts_split(pairs, max_selected, listed_wave(cache.head_dim), cluster);
  const int unit = fp4_unit(cache.head_dim);
  const int64_t ub = unit / cache.block_size;
  const Fp4Split f = fp4_split(pairs, (max_selected + ub - 1) / ub, unit);
  *cluster = f.cluster;
  return f.per * ub;
}

}  // namespace pkv

extern "C" size_t pkv_sparse_workspace_bytes(pkv_cache_desc cache, int num_seqs, int num_heads,
                                             int max_selected) {
  using namespace pkv;
  if (check_cache_desc(cache, true) != PKV_OK || num_seqs <= 0 || num_heads <= 0 ||
      max_selected <= 0)
    return 0;
  int cluster = 1;
  const int64_t per = listed_split(cache, num_seqs, max_selected, &cluster);
  if (per == 0) return 0;
  return static_cast<size_t>(num_seqs) * num_heads * ((max_selected + per - 1) / per) *
         (cache.head_dim + 2) * sizeof(float);
}

extern "C" int pkv_paged_attention_sparse(
    void* out, const void* q, const void* k_cache, const void* v_cache, pkv_cache_desc cache,
    const float* k_scale, const float* v_scale, const int32_t* block_tables,
    int max_blocks_per_seq, const int32_t* context_lens, const int32_t* blocks,
    const int32_t* counts, int max_selected, int num_seqs, int num_heads, float scale,
    void* workspace, size_t workspace_bytes, void* stream) {
  using namespace pkv;
  int g = 0;
  int rc = check_attention(cache, out, q, k_cache, v_cache, k_scale, v_scale, block_tables,
                           max_blocks_per_seq, context_lens, num_seqs, num_heads, 0, scale, &g,
                           true);
  if (rc != PKV_OK) return rc;
  if (max_selected < 1) return PKV_ERR_INVALID_ARG;
  if (max_selected > 1 << 20) return PKV_ERR_UNSUPPORTED;
  if (num_seqs == 0) return PKV_OK;
  if (!blocks || !counts) return PKV_ERR_INVALID_ARG;
  const size_t q_bytes = static_cast<size_t>(num_seqs) * num_heads * cache.head_dim * 2;
  if (overlap(out, q_bytes, q, q_bytes)) return PKV_ERR_INVALID_ARG;
  const size_t need = pkv_sparse_workspace_bytes(cache, num_seqs, num_heads, max_selected);
  if (need > 0 && (!workspace || !aligned16(workspace) || workspace_bytes < need))
    return PKV_ERR_INVALID_ARG;
  DecodeParams p{};
  p.q = static_cast<const uint16_t*>(q);
  p.k_cache = static_cast<const uint8_t*>(k_cache);
  p.v_cache = static_cast<const uint8_t*>(v_cache);
  p.k_scale = k_scale;
  p.v_scale = v_scale;
  p.block_tables = block_tables;
  p.context_lens = context_lens;
  p.out = static_cast<uint16_t*>(out);
  p.err = device_error_ptr();
  p.num_blocks = cache.num_blocks;
  p.num_kv_heads = cache.num_kv_heads;
  p.num_heads = num_heads;
  p.group = g;
  p.max_blocks_per_seq = max_blocks_per_seq;
  p.qscale = scale * 1.4426950408889634f;
  p.list = blocks;
  p.counts = counts;
  p.max_selected = max_selected;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const int64_t per = listed_split(cache, num_seqs, max_selected, &p.cluster);
  dim3 grid(1, cache.num_kv_heads, num_seqs);
  int np = 0;
  if (per > 0) {
    np = static_cast<int>((max_selected + per - 1) / per);
    const int64_t rows = static_cast<int64_t>(num_seqs) * num_heads * np;
    p.partition_blocks = static_cast<int>(per);
    p.np_max = np;
    p.tmp_out = static_cast<float*>(workspace);
    p.max_logits = p.tmp_out + rows * cache.head_dim;
    p.exp_sums = p.max_logits + rows;
    grid.x = np;
  }
  rc = cache.dtype == PKV_DTYPE_FP4_E2M1
           ? launch_decode_fp4(p, cache.head_dim, cache.block_size, grid, st)
           : launch_decode_listed(p, k_cache, v_cache, cache.head_dim, cache.block_size,
                                  cache.dtype == PKV_DTYPE_FP8_E4M3, grid, st);
  if (rc != PKV_OK || per == 0) return rc;
  return launch_reduce_listed(out, p.tmp_out, p.max_logits, p.exp_sums, counts, num_seqs,
                              num_heads, cache.num_kv_heads, cache.head_dim, np,
                              static_cast<int>(per), st);
}

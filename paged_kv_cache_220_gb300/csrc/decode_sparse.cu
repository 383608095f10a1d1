// paged_attention_sparse: the C entry points of decode attention over listed
// blocks.
#include <algorithm>

#include "common.cuh"
#include "decode_params.h"
#include "host_util.h"

extern "C" size_t pkv_sparse_workspace_bytes(pkv_cache_desc cache, int num_seqs, int num_heads,
                                             int max_selected) {
  using namespace pkv;
  if (check_cache_desc(cache, true) != PKV_OK || num_seqs <= 0 || num_heads <= 0 ||
      max_selected <= 0)
    return 0;
  if (cache.dtype == PKV_DTYPE_FP4_E2M1)
    return fp4_workspace_bytes(cache, num_seqs, max_selected, true);
  return 0;
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
  if (cache.dtype == PKV_DTYPE_FP4_E2M1)
    return launch_decode_fp4(p, cache, num_seqs, max_blocks_per_seq * cache.block_size, workspace,
                             static_cast<cudaStream_t>(stream));
  return launch_attention_simple(p, cache, dim3(1, 1, num_seqs), static_cast<cudaStream_t>(stream));
}

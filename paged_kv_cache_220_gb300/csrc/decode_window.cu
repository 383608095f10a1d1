// paged_attention_window: the C entry points of decode attention through a
// sliding window with sink tokens. The kernel is the decode's (decode_tc.cu,
// its windowed form) and the merge is its merge (reduce.cu): what a window
// changes is which blocks are walked and which of their rows are masked.
#include <algorithm>

#include "common.cuh"
#include "decode_params.h"
#include "host_util.h"

namespace pkv {

// The most blocks that a context of at most max_context tokens has visible: a
// window of W tokens touches at most (W - 2) / B + 2 blocks.
static int64_t window_blocks_bound(int block_size, int max_context, int window, int sinks) {
  const int64_t b = block_size;
  const int64_t all = (max_context + b - 1) / b;
  const int64_t sink = (std::min(sinks, max_context) + b - 1) / b;
  return std::min(all, sink + (window + b - 2) / b + 1);
}

static int64_t window_partitions(int block_size, int max_context, int window, int sinks,
                                 int partition_size) {
  const int64_t per = partition_size / block_size;
  return (window_blocks_bound(block_size, max_context, window, sinks) + per - 1) / per;
}

// CTAs that run at once on GB300's 152 SMs: four to an SM at d = 256, three at
// d = 128, a few short of that.
static int64_t window_wave(int head_dim) { return head_dim == 256 ? 600 : 440; }

// CTAs of a pair's cluster in one pass: the smallest power of two, 8 at most,
// with two blocks or fewer for each, while one wave holds them. The shares are
// equal runs of pages rounded up, so some CTAs may get none; the longest share
// is what counts. Half as many CTAs where they would get less than two blocks
// each: 5 to 7 blocks 8.3 -> 10.7 .. 11.4 us (4 pairs, d = 256, B = 16), 11 to
// 15 blocks 7.8 -> 9.0 .. 9.6; 3 blocks 10.2 -> 7.7.
static int64_t window_cluster(int64_t pairs, int64_t blocks, int64_t wave) {
  int64_t c = 1;
  while (c < 8 && 2 * c < blocks && 2 * c * pairs <= wave) c <<= 1;
  return c;
}

}  // namespace pkv

extern "C" int pkv_window_partition_size(int num_seqs, int num_kv_heads, int head_dim,
                                         int block_size, int max_context, int window, int sinks) {
  using namespace pkv;
  if (head_dim != 128 && head_dim != 256) return PKV_ERR_UNSUPPORTED;
  if (num_seqs < 0 || num_kv_heads <= 0 || (block_size != 16 && block_size != 32) ||
      max_context < 0 || window <= 0 || sinks < 0)
    return PKV_ERR_INVALID_ARG;
  const int64_t blocks = window_blocks_bound(block_size, max_context, window, sinks);
  const int64_t pairs = static_cast<int64_t>(num_seqs) * num_kv_heads;
  if (pairs == 0) return 0;
  // One pass, a cluster of CTAs to a pair, saves the merge (64 pairs of 40
  // blocks, bf16, d = 256, B = 16: 12.3 us against 16.6 in 8 partitions), as
  // long as its CTAs have little to do each or fill most of a wave (64 pairs of
  // 520 blocks: 85 against 90). Few pairs of many blocks are cut into as many
  // partitions as a wave holds (4 pairs of 520 blocks: 17 us in 130, 46 in one
  // pass; 8: 20 us in 58, 29 in 87, which do not fit one wave). Where one CTA
  // to a pair leaves much of a wave empty or spills into the next one, about
  // three waves even it out (256 pairs of 160 blocks, d = 128: 85 us in 5
  // partitions, 101 in one pass; 512 pairs, 1.2 waves: 161 in 4, 225; but
  // 1024 pairs of up to 34 blocks, d = 256, 1.7 waves: 103 in 2, 99).
  const int64_t wave = window_wave(head_dim), c = window_cluster(pairs, blocks, wave);
  const int64_t waves = (pairs * c + wave - 1) / wave;
  if (blocks <= 12 * c || 10 * pairs * c >= (waves == 1 ? 6 : 7 * waves) * wave) return 0;
  const int64_t np = 2 * pairs <= wave
                         ? std::min(wave / pairs, blocks / 2)
                         : std::min((3 * wave + pairs / 2) / pairs, blocks / 4);
  if (np <= 1) return 0;
  const int64_t per = (blocks + np - 1) / np;
  return static_cast<int>(std::min<int64_t>(per, (INT32_MAX - 64) / block_size) * block_size);
}

extern "C" size_t pkv_window_workspace_bytes(int num_seqs, int num_heads, int head_dim,
                                             int block_size, int max_context, int window,
                                             int sinks, int partition_size) {
  using namespace pkv;
  if (num_seqs <= 0 || num_heads <= 0 || head_dim <= 0 || block_size <= 0 || max_context <= 0 ||
      window <= 0 || sinks < 0 || partition_size < block_size)
    return 0;
  const size_t np = window_partitions(block_size, max_context, window, sinks, partition_size);
  return static_cast<size_t>(num_seqs) * num_heads * np * (head_dim + 2) * sizeof(float);
}

extern "C" int pkv_paged_attention_window(
    void* out, const void* q, const void* k_cache, const void* v_cache, pkv_cache_desc cache,
    const float* k_scale, const float* v_scale, const int32_t* block_tables,
    int max_blocks_per_seq, const int32_t* context_lens, int num_seqs, int num_heads,
    int max_context, float scale, int window, int sinks, int partition_size, void* workspace,
    size_t workspace_bytes, const int32_t* seq_order, void* stream) {
  using namespace pkv;
  int g = 0;
  int rc = check_attention(cache, out, q, k_cache, v_cache, k_scale, v_scale, block_tables,
                           max_blocks_per_seq, context_lens, num_seqs, num_heads, max_context,
                           scale, &g);
  if (rc != PKV_OK) return rc;
  if (window <= 0 || sinks < 0 || partition_size < 0 || partition_size % cache.block_size != 0)
    return PKV_ERR_INVALID_ARG;
  if (num_seqs == 0) return PKV_OK;
  const size_t q_bytes = static_cast<size_t>(num_seqs) * num_heads * cache.head_dim * 2;
  if (overlap(out, q_bytes, q, q_bytes)) return PKV_ERR_INVALID_ARG;
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
  p.seq_order = seq_order;
  p.qscale = scale * 1.4426950408889634f;
  p.window = window;
  p.sinks = sinks;
  const bool fp8 = cache.dtype == PKV_DTYPE_FP8_E4M3;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  dim3 grid(1, cache.num_kv_heads, num_seqs);
  const int64_t blocks = window_blocks_bound(cache.block_size, max_context, window, sinks);
  if (partition_size == 0) {
    p.cluster = static_cast<int>(window_cluster(
        static_cast<int64_t>(num_seqs) * cache.num_kv_heads, blocks, window_wave(cache.head_dim)));
    return launch_decode_window(p, k_cache, v_cache, cache.head_dim, cache.block_size, fp8, grid,
                                st);
  }
  const int64_t np = window_partitions(cache.block_size, max_context, window, sinks,
                                       partition_size);
  if (np > 32767) return PKV_ERR_UNSUPPORTED;
  float* ws = static_cast<float*>(workspace);
  const int64_t rows = static_cast<int64_t>(num_seqs) * num_heads * np;
  if (np > 0) {
    const size_t need =
        pkv_window_workspace_bytes(num_seqs, num_heads, cache.head_dim, cache.block_size,
                                   max_context, window, sinks, partition_size);
    if (!workspace || !aligned16(workspace) || workspace_bytes < need) return PKV_ERR_INVALID_ARG;
    p.partition_blocks = partition_size / cache.block_size;
    p.np_max = static_cast<int>(np);
    p.tmp_out = ws;
    p.max_logits = ws + rows * cache.head_dim;
    p.exp_sums = p.max_logits + rows;
    grid.x = static_cast<unsigned>(np);
    rc = launch_decode_window(p, k_cache, v_cache, cache.head_dim, cache.block_size, fp8, grid,
                              st);
    if (rc != PKV_OK) return rc;
  }
  // with every context empty (np = 0) the merge writes zeros
  return launch_reduce_window(out, p.tmp_out, p.max_logits, p.exp_sums, context_lens, num_seqs,
                              num_heads, cache.head_dim, static_cast<int>(np), partition_size,
                              cache.block_size, window, sinks, st);
}

// kv_cache_accept: the rows of a sequence's accepted drafts move up behind its
// committed tokens, in every layer's pools.
//
// Sequence s has base committed tokens and n drafts behind them; the accepted
// drafts a_0 < a_1 < ... give row base + k <- row base + a_k. Every 16-byte
// column of a row moves on its own, and one thread owns a column for all the
// moves of its sequence, so no thread reads what another writes. Within a
// thread the moves go in order, several reads before their writes: a_k >= k
// (the list increases), so a row that move k overwrites, base + k, is read by
// no later move (base + a_m, m > k, lies behind it), and reading early is
// always safe.
#include <algorithm>
#include <functional>

#include "common.cuh"
#include "host_util.h"

namespace pkv {

constexpr int kAcceptThreads = 128;
constexpr int kAcceptList = 64;    // moves whose rows are looked up at once
constexpr int kAcceptUnroll = 8;   // rows in flight per thread
constexpr int kAcceptLayers = 64;  // layers of one launch (their pointers are kernel arguments)

struct AcceptParams {
  uint4* pool[2 * kAcceptLayers];  // K of each layer, then V of each layer
  const int32_t* block_tables;
  const int32_t* context_lens;
  const int32_t* q_start;
  const int32_t* accepted;
  const int32_t* num_accepted;
  int32_t* new_context_lens;
  int* err;
  int num_blocks, num_kv_heads, block_size;
  int row_vecs;  // 16-byte vectors of one head's row
  int max_blocks_per_seq;
  int max_accepted;
};

__global__ void __launch_bounds__(kAcceptThreads) kv_cache_accept_kernel(
    const __grid_constant__ AcceptParams p) {
  __shared__ int64_t src_row[kAcceptList], dst_row[kAcceptList];  // of head 0; -1 = no move
  const int s = blockIdx.x;
  const bool first = blockIdx.y == 0 && blockIdx.z == 0;  // this sequence's reporting CTA
  const int ctx = p.context_lens[s];
  const int n = p.q_start[s + 1] - p.q_start[s];
  const int m = p.num_accepted[s];
  const int base = ctx - n;
  const int32_t* list = p.accepted + static_cast<int64_t>(s) * p.max_accepted;
  const bool ctx_ok = ctx >= 0 && ctx <= static_cast<int64_t>(p.max_blocks_per_seq) * p.block_size;
  bool ok = ctx_ok && n >= 0 && base >= 0 && m >= 0 && m <= p.max_accepted && m <= n;
  if (ok) {
    // the whole list is checked before any row moves
    bool bad = false;
    for (int k = threadIdx.x; k < m; k += kAcceptThreads) {
      const int a = list[k];
      bad = bad || a < 0 || a >= n || (k > 0 && list[k - 1] >= a);
    }
    ok = __syncthreads_or(bad) == 0;
  }
  if (first && threadIdx.x == 0) {
    if (!ok) report_error(p.err, ctx_ok ? PKV_DEVERR_DRAFT : PKV_DEVERR_CONTEXT);
    if (p.new_context_lens != nullptr)
      p.new_context_lens[s] = ok ? base + m : (ctx_ok && n >= 0 && base >= 0 ? base : ctx);
  }
  if (!ok) return;

  uint4* pool = p.pool[blockIdx.y];
  const int col = blockIdx.z * kAcceptThreads + threadIdx.x;  // (head, vector) of a token
  const bool live = col < p.num_kv_heads * p.row_vecs;
  const int64_t off = static_cast<int64_t>(col / p.row_vecs) * p.block_size * p.row_vecs +
                      col % p.row_vecs;
  const int32_t* table = p.block_tables + static_cast<int64_t>(s) * p.max_blocks_per_seq;
  // row of head 0 of token t, in vectors; -1 for a bad block id
  auto row_of = [&](int t) -> int64_t {
    const int32_t b = table[t / p.block_size];
    if (b < 0 || b >= p.num_blocks) {
      if (first) report_error(p.err, PKV_DEVERR_BLOCK_ID);
      return -1;
    }
    return (static_cast<int64_t>(b) * p.num_kv_heads * p.block_size + t % p.block_size) *
           p.row_vecs;
  };
  for (int k0 = 0; k0 < m; k0 += kAcceptList) {
    const int cnt = min(kAcceptList, m - k0);
    __syncthreads();  // the rows of the chunk before are no longer needed
    for (int i = threadIdx.x; i < cnt; i += kAcceptThreads) {
      const int k = k0 + i, a = list[k];
      src_row[i] = a == k ? -1 : row_of(base + a);
      dst_row[i] = a == k ? -1 : row_of(base + k);
    }
    __syncthreads();
    if (!live) continue;
    for (int i0 = 0; i0 < cnt; i0 += kAcceptUnroll) {
      uint4 r[kAcceptUnroll];
#pragma unroll
      for (int u = 0; u < kAcceptUnroll; ++u) {
        const int i = i0 + u;
        if (i < cnt && src_row[i] >= 0 && dst_row[i] >= 0) r[u] = pool[src_row[i] + off];
      }
#pragma unroll
      for (int u = 0; u < kAcceptUnroll; ++u) {
        const int i = i0 + u;
        if (i < cnt && src_row[i] >= 0 && dst_row[i] >= 0) pool[dst_row[i] + off] = r[u];
      }
    }
  }
}

}  // namespace pkv

extern "C" int pkv_kv_cache_accept(void* const* k_caches, void* const* v_caches, int num_layers,
                                   pkv_cache_desc cache, const int32_t* block_tables,
                                   int max_blocks_per_seq, const int32_t* context_lens,
                                   const int32_t* q_start, int num_seqs,
                                   const int32_t* accepted, int max_accepted,
                                   const int32_t* num_accepted, int32_t* new_context_lens,
                                   void* stream) {
  using namespace pkv;
  int rc = check_cache_desc(cache);
  if (rc != PKV_OK) return rc;
  if (num_layers < 1 || num_seqs < 0 || max_blocks_per_seq <= 0 || max_accepted < 0)
    return PKV_ERR_INVALID_ARG;
  if (num_seqs == 0) return PKV_OK;
  if (!k_caches || !v_caches || !block_tables || !context_lens || !q_start || !num_accepted ||
      (max_accepted > 0 && !accepted))
    return PKV_ERR_INVALID_ARG;
  for (int l = 0; l < num_layers; ++l)
    if (!k_caches[l] || !v_caches[l] || !aligned16(k_caches[l]) || !aligned16(v_caches[l]))
      return PKV_ERR_INVALID_ARG;
  // the new lengths are written by one CTA of a sequence while others read
  if (new_context_lens) {
    const size_t n = static_cast<size_t>(num_seqs), w = sizeof(int32_t);
    if (overlap(new_context_lens, n * w, context_lens, n * w) ||
        overlap(new_context_lens, n * w, q_start, (n + 1) * w) ||
        overlap(new_context_lens, n * w, num_accepted, n * w) ||
        overlap(new_context_lens, n * w, accepted, n * max_accepted * w) ||
        overlap(new_context_lens, n * w, block_tables, n * max_blocks_per_seq * w))
      return PKV_ERR_INVALID_ARG;
  }
  // rows of pools that overlap, the same pool twice among them, would be moved
  // by CTAs that do not wait for each other
  const int pools = 2 * num_layers;
  const size_t pool_bytes = static_cast<size_t>(cache.num_blocks) * cache.num_kv_heads *
                            cache.block_size * cache.head_dim * elem_bytes(cache.dtype);
  auto pool_at = [&](int i) -> const void* {
    return i < num_layers ? k_caches[i] : v_caches[i - num_layers];
  };
  auto clash = [&](const void* a, const void* b) {
    return overlap(a, pool_bytes, b, pool_bytes);
  };
  const void* sorted[4 * kAcceptLayers];
  if (pools <= 4 * kAcceptLayers) {
    for (int i = 0; i < pools; ++i) sorted[i] = pool_at(i);
    std::sort(sorted, sorted + pools, std::less<const void*>());
    if (std::adjacent_find(sorted, sorted + pools, clash) != sorted + pools)
      return PKV_ERR_INVALID_ARG;
  } else {
    for (int i = 0; i < pools; ++i)
      for (int j = 0; j < i; ++j)
        if (clash(pool_at(i), pool_at(j))) return PKV_ERR_INVALID_ARG;
  }
  AcceptParams p{};
  p.block_tables = block_tables;
  p.context_lens = context_lens;
  p.q_start = q_start;
  p.accepted = accepted;
  p.num_accepted = num_accepted;
  p.err = device_error_ptr();
  p.num_blocks = cache.num_blocks;
  p.num_kv_heads = cache.num_kv_heads;
  p.block_size = cache.block_size;
  p.row_vecs = cache.head_dim * elem_bytes(cache.dtype) / 16;
  p.max_blocks_per_seq = max_blocks_per_seq;
  p.max_accepted = max_accepted;
  const int cols = cache.num_kv_heads * p.row_vecs;
  for (int l0 = 0; l0 < num_layers; l0 += kAcceptLayers) {
    const int nl = std::min(kAcceptLayers, num_layers - l0);
    for (int l = 0; l < nl; ++l) {
      p.pool[l] = static_cast<uint4*>(k_caches[l0 + l]);
      p.pool[nl + l] = static_cast<uint4*>(v_caches[l0 + l]);
    }
    p.new_context_lens = l0 == 0 ? new_context_lens : nullptr;
    const dim3 grid(num_seqs, 2 * nl, (cols + kAcceptThreads - 1) / kAcceptThreads);
    kv_cache_accept_kernel<<<grid, kAcceptThreads, 0, static_cast<cudaStream_t>(stream)>>>(p);
    rc = launch_status();
    if (rc != PKV_OK) return rc;
  }
  return PKV_OK;
}

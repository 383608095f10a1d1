// select_blocks: the blocks of each context whose logits may be the highest.
//
// The score of a block is sum_j sum_d max(c_j[d] lo[d], c_j[d] hi[d]) over the g
// query heads j of a KV head, c_j the query in whole steps of 1/127 of the
// group's largest element. With u = sum_j max(c_j, 0) and w = sum_j max(-c_j, 0)
// that is <u, hi> - <w, lo>: two products however many heads there are, and in
// whole numbers (u, w <= 127 g, |lo|, |hi| <= 127: below 2^26), so no order of
// summation shows in the choice.
//
// Two kernels. The first streams the bounds, 2 D bytes per (block, head) picked
// through the block table: eight lanes to a block with u and w in registers as
// 16-bit pairs, 16-bit x 8-bit dot products (two multiply-adds an instruction, 64
// a clock and SM; HBM leaves 24 bytes a clock and SM), three shuffles to join
// them. The second takes one CTA per (sequence, KV head): the scores go to shared
// memory, a histogram over the range that is left finds the lowest chosen score
// in two or three rounds, and ballots over runs of blocks write the list in order.
//
// Measured: 64 x 8192 tokens (B = 16, 4 heads, d = 256) 19.5 us, 8 x 131072 (B = 32)
// 21.2 us, of which HBM has 10 us and the second kernel 5 to 7; the rest is the chain
// of a CTA's loads (length, table, bounds) at the start of the first. Four heads to
// a CTA, whose bounds of a block are one run, took longer (25, 27 us): 128
// registers, and the queries' sums of four heads before the first product.
#include <algorithm>

#include "common.cuh"
#include "host_util.h"

namespace pkv {

struct SelectParams {
  const uint16_t* q;
  const int8_t* bounds;
  const int32_t* block_tables;
  const int32_t* context_lens;
  int32_t* scores;  // [S][Hk][blocks_max]
  int32_t* blocks;
  int32_t* counts;
  int* err;
  int num_blocks, num_kv_heads, group, max_blocks_per_seq, max_context;
  int blocks_max;  // ceil(max_context / B)
  int max_selected, first, last, block_size;
};

// Blocks of sequence s's context, at most blocks_max.
__device__ __forceinline__ int context_blocks(const SelectParams& p, int s, bool report) {
  int ctx = p.context_lens[s];
  if (ctx < 0 || ctx > p.max_context) {
    if (report) report_error(p.err, PKV_DEVERR_CONTEXT);
    ctx = ctx < 0 ? 0 : p.max_context;
  }
  return (ctx + p.block_size - 1) / p.block_size;
}

constexpr int kScoreThreads = 128;
constexpr int kScoreLanes = 8;                            // lanes to a block
constexpr int kScoreStep = kScoreThreads / kScoreLanes;   // blocks of a CTA at a time

// `rounds` rounds of STEPS * kScoreStep blocks of one pair to a CTA. The table's entries
// are asked for first, then the first bounds, and the query is made into whole
// numbers while those are on their way; later entries come a round ahead.
template <int D, int STEPS>
__global__ void __launch_bounds__(kScoreThreads)
    block_scores_kernel(const SelectParams p, int rounds) {
  constexpr int NV = D / (16 * kScoreLanes);  // 16-byte pieces of lo (and of hi) to a lane
  constexpr int CT = D / kScoreThreads;       // channels of a thread in the query's sums
  constexpr int U = STEPS < 2 ? STEPS : 2;    // blocks of a lane whose loads are in flight
  __shared__ float red[kScoreThreads / 32];
  __shared__ __align__(16) int16_t up[D], down[D];
  wait_prerequisite();
  const int h = blockIdx.x % p.num_kv_heads;
  const int s = blockIdx.y;
  const int tid = threadIdx.x;
  const int n = context_blocks(p, s, false);  // (the second kernel reports)
  const int b0 = blockIdx.x / p.num_kv_heads * (rounds * STEPS * kScoreStep);
  if (n <= p.max_selected || b0 >= n) return;  // all of them are chosen, or none is here
  const int g8 = tid % kScoreLanes;
  const int32_t* table = p.block_tables + static_cast<int64_t>(s) * p.max_blocks_per_seq;
  int mine = b0 + tid / kScoreLanes;  // this lane's first block of the round
  int id[STEPS], id_next[STEPS];
  auto ask = [&](int (&x)[STEPS], int from) {
#pragma unroll
    for (int k = 0; k < STEPS; ++k) {
      const int i = from + k * kScoreStep;
      x[k] = i < n ? table[i] : 0;
    }
  };
  ask(id, mine);
  // the queries' channels of this thread, a head after another
  const uint16_t* q =
      p.q + (static_cast<int64_t>(s) * p.num_kv_heads + h) * p.group * D + tid * CT;
  float x[8][CT];
  float top = 0.f;
#pragma unroll
  for (int j = 0; j < 8; ++j)
#pragma unroll
    for (int i = 0; i < CT; ++i) {
      x[j][i] = j < p.group ? bf16lo(q[j * D + i]) : 0.f;
      top = fmaxf(top, fabsf(x[j][i]));
    }
  uint4 lo[U][NV], hi[U][NV];
  auto load = [&](int k, int block) {
    const bool ok = block >= 0 && block < p.num_blocks;
    const uint4* src = reinterpret_cast<const uint4*>(
        p.bounds + (static_cast<int64_t>(ok ? block : 0) * p.num_kv_heads + h) * (2 * D));
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      lo[k % U][v] = __ldg(src + v * kScoreLanes + g8);
      hi[k % U][v] = __ldg(src + D / 16 + v * kScoreLanes + g8);
    }
  };
#pragma unroll
  for (int k = 0; k < U; ++k) load(k, id[k]);

  // ---- the group's queries as whole numbers, summed by sign
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
  if ((tid & 31) == 0) red[tid >> 5] = top;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kScoreThreads / 32; ++w) top = fmaxf(top, red[w]);
#pragma unroll
  for (int i = 0; i < CT; ++i) {
    int u = 0, w = 0;
    if (top > 0.f)
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        if (j >= p.group) break;
        // x * 127 is exact, the quotient rounded once: an exact tie stays one
        const float c = rintf(__fdiv_rn(x[j][i] * 127.f, top));
        const int k = c == c ? static_cast<int>(fminf(fmaxf(c, -127.f), 127.f)) : 0;
        u += max(k, 0);
        w += min(k, 0);
      }
    up[tid * CT + i] = static_cast<int16_t>(u);
    down[tid * CT + i] = static_cast<int16_t>(w);
  }
  __syncthreads();

  // ---- this lane's channels: pieces g8, g8 + 8, .. of 16 channels
  int cu[NV][8], cw[NV][8];
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    const int c = (v * kScoreLanes + g8) * 16;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      *reinterpret_cast<int4*>(&cu[v][4 * i]) = *reinterpret_cast<const int4*>(&up[c + 8 * i]);
      *reinterpret_cast<int4*>(&cw[v][4 * i]) = *reinterpret_cast<const int4*>(&down[c + 8 * i]);
    }
  }
  int32_t* scores = p.scores + (static_cast<int64_t>(s) * p.num_kv_heads + h) * p.blocks_max;
#pragma unroll 1
  for (int round = 0; round < rounds && b0 + round * STEPS * kScoreStep < n; ++round) {
    if (round + 1 < rounds) ask(id_next, mine + STEPS * kScoreStep);
#pragma unroll
    for (int k = 0; k < STEPS; ++k) {
      int sum = 0;
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        const uint4 l = lo[k % U][v], u = hi[k % U][v];
        const int wl[4] = {static_cast<int>(l.x), static_cast<int>(l.y), static_cast<int>(l.z),
                           static_cast<int>(l.w)};
        const int wh[4] = {static_cast<int>(u.x), static_cast<int>(u.y), static_cast<int>(u.z),
                           static_cast<int>(u.w)};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          sum = __dp2a_lo(cu[v][2 * i], wh[i], sum);
          sum = __dp2a_hi(cu[v][2 * i + 1], wh[i], sum);
          sum = __dp2a_lo(cw[v][2 * i], wl[i], sum);
          sum = __dp2a_hi(cw[v][2 * i + 1], wl[i], sum);
        }
      }
      if (k + U < STEPS)
        load(k + U, id[k + U]);
      else if (round + 1 < rounds)
        load(k + U, id_next[k + U - STEPS]);
#pragma unroll
      for (int off = 1; off < kScoreLanes; off <<= 1)
        sum += __shfl_xor_sync(0xffffffffu, sum, off);
      const int i = mine + k * kScoreStep;
      if (g8 == 0 && i < n) {
        const bool ok = id[k] >= 0 && id[k] < p.num_blocks;
        if (!ok) report_error(p.err, PKV_DEVERR_BLOCK_ID);
        scores[i] = ok ? sum : INT32_MIN;
      }
    }
    mine += STEPS * kScoreStep;
#pragma unroll
    for (int k = 0; k < STEPS; ++k) id[k] = id_next[k];
  }
  allow_dependents();
}

template <int D>
static int launch_scores(const SelectParams& p, int num_seqs, cudaStream_t st) {
  // 128 blocks to a CTA, or 32 where that gives fewer than three CTAs to an SM (1 x 32768
  // tokens, 2 heads: 7.8 us; 64 x 8192, 4 heads: 20.4 us with 128, 22.0 with 32); a
  // CTA's start is 2 us, so rounds of 128 where there are still about three CTAs to an
  // SM (six at d = 128: half the bytes in flight): 64 x 8192, d = 256 20.4 -> 19.5 us,
  // 16 x 65536, 8 heads, d = 128 34.0 -> 32.7 in 4 rounds, 42.6 in 9
  const int64_t pairs = static_cast<int64_t>(num_seqs) * p.num_kv_heads;
  const int64_t all = (p.blocks_max + 127) / 128 * pairs;
  const bool large = all >= 456;
  const int rounds = large ? static_cast<int>(std::max<int64_t>(
                                 1, std::min<int64_t>(all / (D == 256 ? 450 : 900),
                                                         (p.blocks_max + 127) / 128)))
                           : 1;
  const int64_t blocks = large ? 128 * rounds : 32;
  const int64_t gx = (p.blocks_max + blocks - 1) / blocks * p.num_kv_heads;
  const dim3 grid(static_cast<unsigned>(gx), num_seqs), block(kScoreThreads);
  return large ? launch_dependent(block_scores_kernel<D, 8>, grid, block, 0, st, p, rounds)
               : launch_dependent(block_scores_kernel<D, 2>, grid, block, 0, st, p, rounds);
}

// Bins of a round: two rounds for the 2^22 different scores that a context has at most
// in practice (their range is below 2^27, three rounds)
constexpr int kSelectBins = 2048;
constexpr int kSelectSmem = 192 * 1024;  // scores of up to 49152 blocks

template <int T>
__global__ void __launch_bounds__(T) select_kernel(const SelectParams p, bool staged) {
  constexpr int W = T / 32;
  constexpr int BT = kSelectBins / T;  // bins of a thread
  extern __shared__ uint32_t keys_sh[];
  __shared__ __align__(16) int hist[kSelectBins];
  __shared__ uint32_t red_lo[W], red_hi[W];
  __shared__ int seg_over[W], seg_equal[W];
  __shared__ int found_bin, found_need, found_in;
  wait_prerequisite();
  const int h = blockIdx.x, s = blockIdx.y;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int64_t row = static_cast<int64_t>(s) * p.num_kv_heads + h;
  const int n = context_blocks(p, s, tid == 0 && h == 0);
  const int K = p.max_selected;
  int32_t* out = p.blocks + row * K;
  if (tid == 0) p.counts[row] = min(n, K);
  if (n <= K) {
    for (int i = tid; i < K; i += T) out[i] = i < n ? i : -1;
    return;
  }
  const int32_t* scores = p.scores + row * p.blocks_max;
  // scores as unsigned numbers of the same order
  auto key = [&](int i) {
    return staged ? keys_sh[i] : static_cast<uint32_t>(scores[i]) ^ 0x80000000u;
  };
  const int c0 = p.first, c1 = n - p.last;  // [c0, c1): by their score
  uint32_t lo = 0xFFFFFFFFu, hi = 0;
#pragma unroll 4
  for (int i = tid; i < n; i += T) {
    const uint32_t k = static_cast<uint32_t>(scores[i]) ^ 0x80000000u;
    if (staged) keys_sh[i] = k;
    if (i >= c0 && i < c1) {
      lo = min(lo, k);
      hi = max(hi, k);
    }
  }
#pragma unroll
  for (int i = 0; i < BT; ++i) hist[tid * BT + i] = 0;
  lo = __reduce_min_sync(0xffffffffu, lo);
  hi = __reduce_max_sync(0xffffffffu, hi);
  if (lane == 0) {
    red_lo[warp] = lo;
    red_hi[warp] = hi;
  }
  __syncthreads();
#pragma unroll
  for (int w = 0; w < W; ++w) {
    lo = min(lo, red_lo[w]);
    hi = max(hi, red_hi[w]);
  }
  // ---- the lowest chosen key `cut`, and how many of those equal to it are taken
  int need = K - p.first - p.last;
  uint32_t cut = 0xFFFFFFFFu;
  int equal = 0;
  while (need > 0) {
    const int bits = 32 - __clz(hi - lo);
    const int shift = bits > 11 ? bits - 11 : 0;
    for (int i = c0 + tid; i < c1; i += T) {
      const uint32_t k = key(i);
      if (k >= lo && k <= hi) atomicAdd(&hist[(k - lo) >> shift], 1);
    }
    __syncthreads();
    // from the top: thread t has bins [BT t, BT t + BT); how many keys lie above them
    int mine[BT], sum = 0;
#pragma unroll
    for (int i = 0; i < BT; ++i) {
      mine[i] = hist[tid * BT + i];
      sum += mine[i];
    }
    int above = sum;  // of this thread's bins and those above, in the warp
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int x = __shfl_down_sync(0xffffffffu, above, off);
      if (lane + off < 32) above += x;
    }
    if (lane == 0) seg_over[warp] = above;
    __syncthreads();
    // the bins are read: ready for the next round
#pragma unroll
    for (int i = 0; i < BT; ++i) hist[tid * BT + i] = 0;
    for (int w = warp + 1; w < W; ++w) above += seg_over[w];
    above -= sum;
    if (above < need && above + sum >= need) {
      int left = need - above;
      int b = BT - 1;
#pragma unroll
      for (int i = BT - 1; i > 0; --i)
        if (b == i && mine[i] < left) {
          left -= mine[i];
          b = i - 1;
        }
      int in = mine[0];
#pragma unroll
      for (int i = 1; i < BT; ++i) in = b == i ? mine[i] : in;
      found_bin = tid * BT + b;
      found_need = left;
      found_in = in;
    }
    __syncthreads();
    lo += static_cast<uint32_t>(found_bin) << shift;
    need = found_need;
    cut = lo;
    equal = need;
    if (found_in == need) {
      // the whole bin: every key from its lowest on
      equal = INT32_MAX;
      break;
    }
    if (shift == 0) break;
    hi = lo + ((1u << shift) - 1);
  }
  // ---- the list: every warp has a run of blocks
  auto over = [&](int i, uint32_t k) { return i < c0 || i >= c1 || (k > cut); };
  auto even = [&](int i, uint32_t k) { return i >= c0 && i < c1 && k == cut && equal > 0; };
  const int run = ((n + W - 1) / W + 31) / 32 * 32;
  const int r0 = min(n, warp * run), r1 = min(n, r0 + run);
  int no = 0, ne = 0;
  for (int i0 = r0; i0 < r1; i0 += 32) {
    const int i = i0 + lane;
    const uint32_t k = i < r1 ? key(i) : 0;
    no += __popc(__ballot_sync(0xffffffffu, i < r1 && over(i, k)));
    ne += __popc(__ballot_sync(0xffffffffu, i < r1 && even(i, k)));
  }
  if (lane == 0) {
    seg_over[warp] = no;
    seg_equal[warp] = ne;
  }
  __syncthreads();
  int at = 0;        // where this warp's part of the list begins
  int left = equal;  // equal keys that this warp and those behind it may take
  for (int w = 0; w < warp; ++w) {
    const int t = min(left, seg_equal[w]);
    at += seg_over[w] + t;
    left -= t;
  }
  for (int i0 = r0; i0 < r1; i0 += 32) {
    const int i = i0 + lane;
    const uint32_t k = i < r1 ? key(i) : 0;
    const bool e = i < r1 && even(i, k);
    const unsigned me = __ballot_sync(0xffffffffu, e);
    const bool take = i < r1 && (over(i, k) || (e && __popc(me & ((1u << lane) - 1)) < left));
    const unsigned mt = __ballot_sync(0xffffffffu, take);
    if (take) out[at + __popc(mt & ((1u << lane) - 1))] = i;
    at += __popc(mt);
    left -= min(left, __popc(me));
  }
}

}  // namespace pkv

extern "C" size_t pkv_select_workspace_bytes(int num_seqs, int num_kv_heads, int block_size,
                                             int max_context) {
  if (num_seqs <= 0 || num_kv_heads <= 0 || block_size <= 0 || max_context <= 0) return 0;
  const size_t n = (static_cast<size_t>(max_context) + block_size - 1) / block_size;
  return static_cast<size_t>(num_seqs) * num_kv_heads * n * sizeof(int32_t);
}

extern "C" int pkv_select_blocks(int32_t* blocks, int32_t* counts, const void* q,
                                 const int8_t* bounds, pkv_cache_desc cache,
                                 const int32_t* block_tables, int max_blocks_per_seq,
                                 const int32_t* context_lens, int num_seqs, int num_heads,
                                 int max_context, int max_selected, int first, int last,
                                 void* workspace, size_t workspace_bytes, void* stream) {
  using namespace pkv;
  int rc = check_cache_desc(cache, true);
  if (rc != PKV_OK) return rc;
  if (num_seqs < 0 || num_heads <= 0 || max_context < 0 || max_blocks_per_seq <= 0 ||
      max_selected < 1 || first < 0 || last < 0 ||
      static_cast<int64_t>(first) + last > max_selected || num_heads % cache.num_kv_heads != 0)
    return PKV_ERR_INVALID_ARG;
  const int group = num_heads / cache.num_kv_heads;
  const int64_t cap = static_cast<int64_t>(max_blocks_per_seq) * cache.block_size;
  if (max_context > cap) return PKV_ERR_INVALID_ARG;
  // positions in a context and in a list, a CTA's stride behind the last, are 32-bit numbers
  if (group > 8 || num_seqs > 65535 || cap > (1 << 30) || max_selected > (1 << 30))
    return PKV_ERR_UNSUPPORTED;
  if (num_seqs == 0) return PKV_OK;
  if (!blocks || !counts || !q || !bounds || !block_tables || !context_lens)
    return PKV_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(bounds)) return PKV_ERR_INVALID_ARG;
  const size_t need =
      pkv_select_workspace_bytes(num_seqs, cache.num_kv_heads, cache.block_size, max_context);
  if (need > 0 && (!workspace || !aligned16(workspace) || workspace_bytes < need))
    return PKV_ERR_INVALID_ARG;
  // what is written against what is read, and against each other
  const size_t pairs = static_cast<size_t>(num_seqs) * cache.num_kv_heads;
  struct Span {
    const void* at;
    size_t bytes;
  };
  const Span wr[3] = {{blocks, pairs * max_selected * 4}, {counts, pairs * 4}, {workspace, need}};
  const Span rd[4] = {
      {q, static_cast<size_t>(num_seqs) * num_heads * cache.head_dim * 2},
      {bounds, static_cast<size_t>(cache.num_blocks) * cache.num_kv_heads * 2 * cache.head_dim},
      {block_tables, static_cast<size_t>(num_seqs) * max_blocks_per_seq * 4},
      {context_lens, static_cast<size_t>(num_seqs) * 4}};
  for (int i = 0; i < 3; ++i) {
    for (const Span& r : rd)
      if (overlap(wr[i].at, wr[i].bytes, r.at, r.bytes)) return PKV_ERR_INVALID_ARG;
    for (int j = 0; j < i; ++j)
      if (overlap(wr[i].at, wr[i].bytes, wr[j].at, wr[j].bytes)) return PKV_ERR_INVALID_ARG;
  }
  SelectParams p{};
  p.q = static_cast<const uint16_t*>(q);
  p.bounds = bounds;
  p.block_tables = block_tables;
  p.context_lens = context_lens;
  p.scores = static_cast<int32_t*>(workspace);
  p.blocks = blocks;
  p.counts = counts;
  p.err = device_error_ptr();
  p.num_blocks = cache.num_blocks;
  p.num_kv_heads = cache.num_kv_heads;
  p.group = group;
  p.max_blocks_per_seq = max_blocks_per_seq;
  p.max_context = max_context;
  p.blocks_max = (max_context + cache.block_size - 1) / cache.block_size;
  p.max_selected = max_selected;
  p.first = first;
  p.last = last;
  p.block_size = cache.block_size;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (p.blocks_max > max_selected) {
    rc = cache.head_dim == 256 ? launch_scores<256>(p, num_seqs, st)
                               : launch_scores<128>(p, num_seqs, st);
    if (rc != PKV_OK) return rc;
  }
  const size_t smem = static_cast<size_t>(p.blocks_max) * 4;
  const bool staged = smem <= kSelectSmem;
  const dim3 grid(cache.num_kv_heads, num_seqs);
  // few warps pass a barrier sooner, more have fewer blocks each (8 x 4096 blocks, 4
  // heads, with the scores: 24.5 us with 256 threads, 22.4 with 1024; 64 x 512: 20.4, 22)
  if (p.blocks_max <= 1024)
    return launch_dependent(select_kernel<256>, grid, dim3(256), smem, st, p, staged);
  static DeviceFlags done;
  rc = ensure_smem(select_kernel<1024>, kSelectSmem, done);
  if (rc != PKV_OK) return rc;
  return launch_dependent(select_kernel<1024>, grid, dim3(1024), staged ? smem : 0, st, p, staged);
}

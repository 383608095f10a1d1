// Attention of several drafted tokens per sequence (a chain or a tree) over
// the paged cache.
//
// The drafts of a sequence share its context, so the query rows of a KV head
// (drafts x query group, up to 512) are multiplied with every cached row: a
// contraction for the 5th-generation tensor cores. Rows are taken in tiles of
// 128 (M = 128, row i in lane i of tensor memory), tokens in steps of 128:
//     S = Q.K^T    16 (d = 256) products of 128 x 128 x 16, Q and K in shared memory
//     P = 2^(S scale log2e - m), masked; m the row's reference maximum
//     O = O + P.V  8 products of 128 x d x 16, P in tensor memory over S's
//                  columns, V in shared memory
// with fp32 accumulators in tensor memory: O [d], S of two steps [2][128].
//
// Work split. A unit is (sequence, KV head, row tile); its steps are the 128-
// token runs of its context. All steps of all units form one line that is cut
// into equal shares, one per CTA, one CTA per SM: no tail whatever the lengths
// are. A CTA's share is a row of segments (runs of steps of one unit). A unit
// inside one share is finished there; a unit that is cut leaves a partial
// (normalised fp32 output, maximum, sum) per segment, at most two per CTA, and
// tree_merge_kernel joins them by log-sum-exp. The pipeline below runs on
// across segments, so the loads never pause.
//
// Shared memory: the row tile's Q and a ring of 32 KB slots that TMA fills
// (cp.async.bulk.tensor, whole pages, 128-byte swizzle). A slot is [8-row
// group][64-column chunk][8 rows][128 B]: the box of a page is 4-D (64
// columns, 8 rows, chunks, row groups), so pages land one behind the other in
// what is both K's operand layout (N = tokens, row groups at one stride) and
// V's (N = columns, MN-major). K of a step takes d/128 slots (128 columns
// each), V d/128 slots (64 or 128 tokens each). Slots are filled and used in
// the order K(0), K(1), V(0), K(2), V(1), ...
//
// E4M3 pools: TMA stages the codes in a second ring; converter warps turn
// them into their exact f16 values in the slots. Q is converted to f16, P is
// f16; k_scale goes into the logits, v_scale into the output.
//
// P is one bf16 part (2^-9 relative rounding of each weight, as many bits as
// the output; a second part would double the P.V products).
//
// Warps: 0-3 softmax (thread t of warp w owns query row 32 w + t), 4 issues
// the products, 5-6 load pages, 7(-8) load Q, 8-15 convert (E4M3).
#include <algorithm>
#include <cmath>

#include "common.cuh"
#include "host_util.h"
#include "tc_common.cuh"
#include "tmem.cuh"

namespace pkv {

constexpr int kTreeMaxCtas = 160;  // one per SM; the workspace is sized for it
constexpr int kTreeRows = 128;     // query rows of a tile
constexpr int kTreeTok = 128;      // tokens of a step

struct TreeMeta {  // what the merge needs of a unit that starts in a CTA and is cut
  int row0;        // first query row (of q and out) of the sequence
  int first;       // first (draft, group) row of the tile
  int rows;        // live rows of the tile
  int head;        // KV head
  int slot;        // the CTA's partial that holds the unit's first segment
  int parts;       // segments; 0: nothing to merge
};

struct TreeParams {
  const uint16_t* q;
  uint16_t* out;
  const float* k_scale;
  const float* v_scale;
  const int32_t* block_tables;
  const int32_t* context_lens;
  const int32_t* q_start;
  const uint64_t* tree_mask;
  int* err;
  TreeMeta* meta;   // [ctas]
  float* part_o;    // [ctas][2][128][d]
  float* part_m;    // [ctas][2][128]
  float* part_l;
  int num_seqs, num_queries, max_draft;
  int num_blocks, num_kv_heads, num_heads, group, block_size, max_blocks_per_seq;
  int min_steps;    // steps a CTA takes at least (fewer CTAs work on less)
  float qscale;
};

template <int D, bool FP8>
struct TreeGeom {
  static constexpr int kSlot = 32768;
  static constexpr int kQ = kTreeRows * D * 2;
  static constexpr int kKS = D / 128;        // slots of a step's K
  static constexpr int kVS = D / 128;        // slots of a step's V
  static constexpr int kVTok = kTreeTok / kVS;
  static constexpr int kNSlot = FP8 ? 4 : (D == 256 ? 5 : 6);
  static constexpr int kStage = kSlot / 2;   // E4M3: codes of a slot
  static constexpr int kNStage = FP8 ? (D == 256 ? 2 : 4) : 0;
  static constexpr int kProducers = 2;
  static constexpr int kQWarps = FP8 ? 1 : 2;  // E4M3: 512 threads, 128 registers each
  static constexpr int kConvWarps = FP8 ? 8 : 0;
  static constexpr int kThreads = (4 + 1 + kProducers + kQWarps + kConvWarps) * 32;
  static constexpr int kSmem = 2048 + kQ + kNSlot * kSlot + kNStage * kStage;
  static constexpr uint32_t kColS = D;       // S of step t at kColS + 128 * (t & 1)
  static constexpr uint32_t kCols = 512;
  static_assert(kSmem <= 232448, "shared memory of a CTA");
};

// D[tmem] (+)= A[smem] . B[smem]
__device__ __forceinline__ void umma_ss(uint32_t d_tmem, uint64_t a, uint64_t b, uint32_t idesc,
                                        uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}

// One box of a 4-D pool map: chunk c, 8-row group y.
__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap* map, int c, int y,
                                            uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(0), "r"(0), "r"(c), "r"(y), "r"(smem_addr(bar))
      : "memory");
}

// A sequence's part of the line of steps; n = 0 if it has none (no drafts, or
// drafts or a context that cannot be).
struct TreeSeq {
  int ctx, n, q0, tiles, steps;
  __device__ __forceinline__ void load(const TreeParams& p, int s, bool report) {
    q0 = p.q_start[s];
    const int q1 = p.q_start[s + 1];
    ctx = p.context_lens[s];
    const bool ctx_ok =
        ctx >= 0 && ctx <= static_cast<int64_t>(p.max_blocks_per_seq) * p.block_size;
    const bool ok = ctx_ok && q0 >= 0 && q1 >= q0 && q1 <= p.num_queries &&
                    q1 - q0 <= p.max_draft && q1 - q0 <= ctx;
    if (!ok && report) report_error(p.err, ctx_ok ? PKV_DEVERR_DRAFT : PKV_DEVERR_CONTEXT);
    n = ok ? q1 - q0 : 0;
    tiles = (n * p.group + kTreeRows - 1) / kTreeRows;
    steps = ok ? (ctx + kTreeTok - 1) / kTreeTok : 0;
  }
  __device__ __forceinline__ int64_t weight(const TreeParams& p) const {
    return static_cast<int64_t>(p.num_kv_heads) * tiles * steps;
  }
};

// Walks a CTA's share step by step.
struct TreeWalk {
  TreeSeq q;
  int s, h, tile, st;   // the current step
  int64_t left;         // steps left, this one included
  bool begins;          // first step of a segment
  __device__ __forceinline__ void start(const TreeParams& p, int s0, int64_t off, int64_t count) {
    s = s0;
    left = count;
    begins = true;
    if (count <= 0) return;
    q.load(p, s, false);
    const int64_t unit = off / q.steps;
    st = static_cast<int>(off - unit * q.steps);
    h = static_cast<int>(unit / q.tiles);
    tile = static_cast<int>(unit % q.tiles);
  }
  __device__ __forceinline__ bool ends() const { return left == 1 || st + 1 == q.steps; }
  __device__ __forceinline__ void next(const TreeParams& p) {
    begins = false;
    if (--left <= 0) return;
    if (++st < q.steps) return;
    st = 0;
    begins = true;
    if (++tile < q.tiles) return;
    tile = 0;
    if (++h < p.num_kv_heads) return;
    h = 0;
    do q.load(p, ++s, false);
    while (q.tiles == 0 && s + 1 < p.num_seqs);
  }
};

// A place in a ring of N: the producer waits for `empty` with parity ph ^ 1
// (passes at once in the first round), the reader for `full` with parity ph.
template <int N>
struct RingPos {
  int i = 0;
  uint32_t ph = 0;
  __device__ __forceinline__ void next() {
    if (++i == N) {
      i = 0;
      ph ^= 1;
    }
  }
};

// r / g for a row of a unit (r < 64 g, g <= 8): exact, no division.
__device__ __forceinline__ int div_group(int r, int g) { return (r * (65536 / g + 1)) >> 16; }

// 16 bytes global -> shared in the background; zeros if not `live`.
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool live) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
               "r"(live ? 16 : 0)
               : "memory");
}

// One lane of the warp, the same one every time.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}"
               : "=r"(p));
  return p != 0;
}

// The number of V's first slot of step t in the ring's order (the slot is that
// modulo the slots), of a CTA with `total` steps.
template <int KS, int VS>
__device__ __forceinline__ int64_t v_seq(int64_t t, int64_t total) {
  return KS + t * (KS + VS) + (t + 1 < total ? KS : 0);
}

template <int D, bool FP8>
__global__ void __launch_bounds__(TreeGeom<D, FP8>::kThreads, 1)
    tree_kernel(const __grid_constant__ CUtensorMap tmk, const __grid_constant__ CUtensorMap tmv,
                const __grid_constant__ TreeParams p) {
  using G = TreeGeom<D, FP8>;
  constexpr int NCH = D / 64;
  constexpr int KS = G::kKS, VS = G::kVS, NS = G::kNSlot;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_addr(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* sbase = smem_raw + (base - raw);
  uint64_t* full = reinterpret_cast<uint64_t*>(sbase);  // [NS] slot filled
  uint64_t* empty = full + 8;                            // [NS] slot read
  uint64_t* full8 = empty + 8;                           // [NST] codes staged
  uint64_t* empty8 = full8 + 4;                          // [NST] codes converted
  uint64_t* s_full = empty8 + 4;                         // [2]
  uint64_t* p_full = s_full + 2;                         // [2]
  uint64_t* o_done = p_full + 2;                         // [2]
  uint64_t* q_full = o_done + 2;
  uint64_t* q_empty = q_full + 1;
  uint64_t* o_free = q_empty + 1;
  uint64_t* drained = o_free + 1;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(sbase + 512);
  int64_t* found = reinterpret_cast<int64_t*>(sbase + 520);    // sequence, offset in it
  int64_t* wsum = reinterpret_cast<int64_t*>(sbase + 544);     // [warps + 1]
  const uint32_t sq = base + 1024;
  const uint32_t ring = sq + G::kQ;
  const uint32_t stage = ring + NS * G::kSlot;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int cta = blockIdx.x;
  if (threadIdx.x == 0) {
    for (int i = 0; i < NS; ++i) {
      mbar_init(&full[i], FP8 ? G::kConvWarps : G::kProducers);
      mbar_init(&empty[i], 1);
    }
    for (int i = 0; i < G::kNStage; ++i) {
      mbar_init(&full8[i], G::kProducers);
      mbar_init(&empty8[i], G::kConvWarps);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&s_full[i], 1);
      mbar_init(&p_full[i], 128);
      mbar_init(&o_done[i], 1);
    }
    mbar_init(q_full, G::kQWarps * 32);
    mbar_init(q_empty, 1);
    mbar_init(o_free, 128);
    mbar_init(drained, 1);
    fence_mbar_init();
    found[0] = 0;
    found[1] = 0;
  }
  if (warp == 4) tmem_alloc(tmem_slot, G::kCols);
  wait_prerequisite();
  if (threadIdx.x == 0) p.meta[cta] = TreeMeta{0, 0, 0, 0, 0, 0};

  // ---- this CTA's share of the line: every thread sums a run of sequences,
  // the thread whose run holds the share's first step finds its sequence
  const int per = (p.num_seqs + G::kThreads - 1) / G::kThreads;
  const int s_lo = min(p.num_seqs, static_cast<int>(threadIdx.x) * per);
  const int s_hi = min(p.num_seqs, s_lo + per);
  int64_t mine = 0;
  for (int s = s_lo; s < s_hi; ++s) {
    TreeSeq q;
    q.load(p, s, cta == 0);
    mine += q.weight(p);
  }
  int64_t incl = mine;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int64_t x = __shfl_up_sync(0xffffffffu, incl, off);
    if (lane >= off) incl += x;
  }
  if (lane == 31) wsum[warp] = incl;
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  int64_t before = 0, total = 0;
  for (int w = 0; w < G::kThreads / 32; ++w) {
    if (w < warp) before += wsum[w];
    total += wsum[w];
  }
  const int64_t excl = before + incl - mine;
  const int64_t ctas = min(static_cast<int64_t>(gridDim.x),
                           (total + p.min_steps - 1) / p.min_steps);
  const int64_t begin = cta < ctas ? cta * total / ctas : 0;
  const int64_t end = cta < ctas ? (cta + 1) * total / ctas : 0;
  const int64_t count = end - begin;
  if (count > 0 && excl <= begin && begin < excl + mine) {
    int64_t at = excl;
    for (int s = s_lo; s < s_hi; ++s) {
      TreeSeq q;
      q.load(p, s, false);
      const int64_t w = q.weight(p);
      if (begin < at + w) {
        found[0] = s;
        found[1] = begin - at;
        break;
      }
      at += w;
    }
  }
  __syncthreads();
  const uint32_t tmem = *tmem_slot;
  const uint32_t t_o = tmem;
  const uint32_t t_s = tmem + G::kColS;
  TreeWalk walk;
  walk.start(p, static_cast<int>(found[0]), found[1], count);

  int64_t issued = 0;  // producers: slots (E4M3: stages) whose copies were started
  if (warp == 5 || warp == 6) {
    // ---------------- producers: the block table walk and the TMA copies
    if (lane == 0) {
      const int prod = warp - 5;  // takes the step's pages prod, prod + 2, ...
      const int B = p.block_size;
      const int per_v = G::kVTok / B;  // pages of a V slot
      RingPos<FP8 ? G::kNStage : NS> at;
      // this producer's block ids of one step, read well before they are used
      struct Step {
        int id[4];
        int head, pages;
      };
      auto read = [&](const TreeWalk& w) {
        Step x;
        x.head = w.h;
        x.pages = w.left > 0 ? (min(kTreeTok, w.q.ctx - w.st * kTreeTok) + B - 1) / B : 0;
        const int32_t* bt = p.block_tables + static_cast<int64_t>(w.s) * p.max_blocks_per_seq +
                            w.st * (kTreeTok / B);
#pragma unroll
        for (int j = 0; j < 4; ++j) x.id[j] = 2 * j + prod < x.pages ? bt[2 * j + prod] : 0;
        return x;
      };
      // the copies of one slot: K columns [128 part, 128 part + 128) of the
      // step's pages, or its pages of V slot `part`
      auto slot_copy = [&](const Step& x, bool is_v, int part) {
        const int i = at.i;
        uint64_t* f = FP8 ? &full8[i] : &full[i];
        uint64_t* e = FP8 ? &empty8[i] : &empty[i];
        if (!mbar_wait(e, at.ph ^ 1, p.err)) return false;
        const int first = is_v ? part * per_v : 0;
        const int last = min(x.pages, is_v ? first + per_v : x.pages);
        const int page_bytes = B * (is_v ? D : 128) * (FP8 ? 1 : 2);
        int good = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int pg = 2 * j + prod;
          if (pg < first || pg >= last) continue;
          if (x.id[j] >= 0 && x.id[j] < p.num_blocks) ++good;
          else report_error(p.err, PKV_DEVERR_BLOCK_ID);
        }
        mbar_arrive_expect_tx(f, good * page_bytes);
        const uint32_t dst = FP8 ? stage + i * G::kStage : ring + i * G::kSlot;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int pg = 2 * j + prod;
          if (pg < first || pg >= last || x.id[j] < 0 || x.id[j] >= p.num_blocks) continue;
          const int y = (x.id[j] * p.num_kv_heads + x.head) * B;
          const uint32_t to = dst + (pg - first) * page_bytes;
          if constexpr (!FP8) {
            tma_load_4d(to, is_v ? &tmv : &tmk, is_v ? 0 : 2 * part, y / 8, f);
          } else if (is_v) {
#pragma unroll
            for (int c = 0; c < D / 128; ++c)
              tma_load_2d(to + c * B * 128, &tmv, c * 128, y, f);
          } else {
            tma_load_2d(to, &tmk, part * 128, y, f);
          }
        }
        at.next();
        ++issued;
        return true;
      };
      if (walk.left > 0) {
        // V of step t, K of step t + 1, ids of step t + 2
        Step now = read(walk), ahead;
        bool ok = true;
        for (int ks = 0; ks < KS && ok; ++ks) ok = slot_copy(now, false, ks);
        walk.next(p);
        ahead = read(walk);
        for (int64_t t = 0; t < count && ok; ++t) {
          if (t + 1 < count)
            for (int ks = 0; ks < KS && ok; ++ks) ok = slot_copy(ahead, false, ks);
          walk.next(p);
          const Step far = read(walk);
          for (int vs = 0; vs < VS && ok; ++vs) ok = slot_copy(now, true, vs);
          now = ahead;
          ahead = far;
        }
      }
    }
  } else if (warp == 4) {
    // ---------------- the products: the whole warp walks, one lane issues.
    // Operand descriptors are a constant plus the address: one addition each
    // (built one by one they cost the issuing lane about as much as the
    // tensor core takes for a product).
    constexpr uint32_t idesc_qk = FP8 ? umma_idesc_f16(128, kTreeTok, false)
                                      : umma_idesc_bf16(128, kTreeTok, false);
    constexpr uint32_t idesc_pv = FP8 ? umma_idesc_f16(128, D, true)
                                      : umma_idesc_bf16(128, D, true);
    const bool lead = elect_one();
    const uint64_t qd = umma_sdesc(sq, 16, NCH * 1024, 2);
    const uint64_t kd0 = umma_sdesc(ring, 16, 2048, 2);
    const uint64_t vd0 = umma_sdesc(ring, 1024, NCH * 1024, 2);
    RingPos<NS> at;
    uint32_t segs = 0;     // segments whose S has begun
    uint32_t pv_segs = 0;  // segments whose P.V has begun
    bool prev_begins = false;
    int prev_tok = 0;      // valid tokens of the step before
    auto wait = [&](uint64_t* bar, uint32_t parity) {
      return __all_sync(0xffffffffu, mbar_wait(bar, parity, p.err)) != 0;
    };
    for (uint32_t t = 0;; ++t) {
      const bool have = walk.left > 0;
      if (have) {
        const int b = t & 1;
        // S of step t overwrites P of step t - 2
        if (t >= 2 && !wait(&o_done[b], ((t - 2) >> 1) & 1)) break;
        if (walk.begins && !wait(q_full, segs++ & 1)) break;
        bool ok = true;
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) {
          if (!(ok = wait(&full[at.i], at.ph))) break;
          tc_fence_after();
          if (lead) {
            const uint64_t kd = kd0 + ((at.i * G::kSlot) >> 4);
#pragma unroll
            for (int k = 0; k < 8; ++k)
              umma_ss(t_s + b * kTreeTok, qd + (((ks * 2 + (k >> 2)) * 1024 + (k & 3) * 32) >> 4),
                      kd + (((k >> 2) * 1024 + (k & 3) * 32) >> 4), idesc_qk,
                      (ks > 0 || k > 0) ? 1u : 0u);
            umma_commit(&empty[at.i]);
          }
          at.next();
        }
        if (!ok) break;
        if (lead) {
          umma_commit(&s_full[b]);
          if (walk.ends()) umma_commit(q_empty);
        }
      }
      if (t >= 1) {
        const uint32_t j = t - 1;
        const int b = j & 1;
        if (!wait(&p_full[b], (j >> 1) & 1)) break;
        // the segment before has left O
        if (prev_begins && pv_segs++ > 0 && !wait(o_free, (pv_segs - 2) & 1)) break;
        bool ok = true;
#pragma unroll
        for (int vs = 0; vs < VS; ++vs) {
          if (!(ok = wait(&full[at.i], at.ph))) break;
          tc_fence_after();
          if (lead) {
            constexpr int kPer = G::kVTok / 16;  // k-steps of a slot
            const uint64_t vd = vd0 + ((at.i * G::kSlot) >> 4);
            const uint32_t pa = t_s + b * kTreeTok + 8 * vs * kPer;
            const int k1 = (prev_tok + 15) / 16 - vs * kPer;
            const uint32_t keep = !prev_begins || vs > 0 ? 1u : 0u;
            if (k1 >= kPer) {
#pragma unroll
              for (int kk = 0; kk < kPer; ++kk)
                umma_bf16_ta(t_o, pa + 8 * kk, vd + ((kk * 2 * NCH * 1024) >> 4), idesc_pv,
                             kk > 0 ? 1u : keep);
            } else {
              for (int kk = 0; kk < k1; ++kk)
                umma_bf16_ta(t_o, pa + 8 * kk, vd + ((kk * 2 * NCH * 1024) >> 4), idesc_pv,
                             kk > 0 ? 1u : keep);
            }
            umma_commit(&empty[at.i]);
          }
          at.next();
        }
        if (!ok) break;
        if (lead) umma_commit(&o_done[b]);
      }
      if (!have) break;
      prev_begins = walk.begins;
      prev_tok = min(kTreeTok, walk.q.ctx - walk.st * kTreeTok);
      walk.next(p);
    }
    // every product issued here has finished before tensor memory is released
    if (lead) umma_commit(drained);
    (void)wait(drained, 0);
  } else if (warp < 4) {
    // ---------------- softmax: one query row per thread
    const int row = 32 * warp + lane;
    const uint32_t lane_off = static_cast<uint32_t>(32 * warp) << 16;
    const int g = p.group;
    float m = -INFINITY, l = 0.f, qs = p.qscale;
    uint64_t mask = 0;
    bool live = false;
    int draft = 0, head = 0;
    int seg_st = 0;         // the segment's first step in its unit
    bool first_seg = true;  // of this share
    for (int64_t t = 0; walk.left > 0; ++t) {
      const int b = static_cast<int>(t & 1);
      const int base_tok = walk.q.ctx - walk.q.n;
      const bool begins = walk.begins;
      if (begins) {
        const int r = walk.tile * kTreeRows + row;
        live = r < walk.q.n * g;
        draft = live ? div_group(r, g) : 0;
        head = walk.h * g + (live ? r - draft * g : 0);
        mask = p.tree_mask != nullptr ? p.tree_mask[walk.q.q0 + draft] : (2ull << draft) - 1;
        if (walk.q.n < 64) mask &= (1ull << walk.q.n) - 1;
        if constexpr (FP8) qs = p.qscale * p.k_scale[walk.h];
        m = -INFINITY;
        l = 0.f;
        seg_st = walk.st;
      }
      if (!__all_sync(0xffffffffu, mbar_wait(&s_full[b], (t >> 1) & 1, p.err))) break;
      tc_fence_after();
      const uint32_t ts = t_s + lane_off + b * kTreeTok;
      const int tok0 = walk.st * kTreeTok;
      const bool clean = tok0 + kTreeTok <= base_tok;  // committed tokens only
      // visible columns of this row, 32 to a word
      uint32_t see[4] = {~0u, ~0u, ~0u, ~0u};
      if (!clean) {
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          const int sh = tok0 + 32 * w - base_tok;  // draft of the word's first column
          if (sh >= 64) see[w] = 0;
          else if (sh >= 0) see[w] = static_cast<uint32_t>(mask >> sh);
          else if (sh > -32) see[w] = static_cast<uint32_t>(mask << -sh) | ((1u << -sh) - 1);
        }
      }
      float sv[64];
      float mx = -INFINITY;
      {
        float m4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int hf = 1; hf >= 0; --hf) {
          tmem_ld64(ts + 64 * hf, sv);
          if (clean) {
#pragma unroll
            for (int i = 0; i < 64; ++i) m4[i & 3] = fmaxf(m4[i & 3], sv[i] * qs);
          } else {
#pragma unroll
            for (int i = 0; i < 64; ++i) {
              sv[i] = (see[2 * hf + i / 32] >> (i % 32)) & 1 ? sv[i] * qs : -INFINITY;
              m4[i & 3] = fmaxf(m4[i & 3], sv[i]);
            }
          }
        }
        mx = fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3]));
      }
      // O is rescaled when the maximum grows by more than 2^8 (loads and
      // stores of tensor memory are warp-collective: all lanes or none)
      const bool want = mx > m + 8.f;
      if (__any_sync(0xffffffffu, want) && !begins) {
        if (!__all_sync(0xffffffffu,
                        mbar_wait(&o_done[(t - 1) & 1], ((t - 1) >> 1) & 1, p.err)))
          break;
        tc_fence_after();
        const float alpha = want ? fast_exp2(m - mx) : 1.f;  // 0 while m is -inf
#pragma unroll 1
        for (int c = 0; c < D; c += 16) {
          float ov[16];
          tmem_ld16(t_o + lane_off + c, ov);
#pragma unroll
          for (int i = 0; i < 16; ++i) ov[i] *= alpha;
          tmem_st16(t_o + lane_off + c, ov);
        }
        if (want) l *= alpha;
      }
      if (want) m = mx;
      const float ref = m == -INFINITY ? 0.f : m;
      // P over S's columns: the first half (still in registers) goes to columns
      // 0..31, then the second, read again, to columns 32..63
      float l4[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int hf = 0; hf < 2; ++hf) {
        if (hf == 1) tmem_ld64(ts + 64, sv);
        uint32_t pw[32];
        if (clean) {
#pragma unroll
          for (int i = 0; i < 32; ++i) {
            const float a = fast_exp2(fmaf(sv[2 * i], qs, -ref));
            const float c = fast_exp2(fmaf(sv[2 * i + 1], qs, -ref));
            l4[(2 * i) & 3] += a;
            l4[(2 * i + 1) & 3] += c;
            pw[i] = FP8 ? pack_f16(a, c) : pack_bf16(a, c);
          }
        } else {
#pragma unroll
          for (int i = 0; i < 32; ++i) {
            const uint32_t word = see[2 * hf + i / 16] >> ((2 * i) % 32);
            // the first half was scaled and masked in place above
            const float x = hf == 0 ? sv[2 * i] : word & 1 ? sv[2 * i] * qs : -INFINITY;
            const float y = hf == 0 ? sv[2 * i + 1] : word & 2 ? sv[2 * i + 1] * qs : -INFINITY;
            const float a = fast_exp2(x - ref), c = fast_exp2(y - ref);
            l4[(2 * i) & 3] += a;
            l4[(2 * i + 1) & 3] += c;
            pw[i] = FP8 ? pack_f16(a, c) : pack_bf16(a, c);
          }
        }
        tmem_st16_nowait(ts + 32 * hf, pw);
        tmem_st16_nowait(ts + 32 * hf + 16, pw + 16);
      }
      l += (l4[0] + l4[1]) + (l4[2] + l4[3]);
      const int valid = walk.q.ctx - tok0;
      if (valid < kTreeTok && (valid & 15) != 0) {
        // the rows behind the context that the last product of P.V covers
        // hold whatever was there: zero them, P is zero there
        const int64_t seq = v_seq<KS, VS>(t, count) + valid / G::kVTok;
        const int i = static_cast<int>(seq % NS);
        if (!__all_sync(0xffffffffu, mbar_wait(&full[i], (seq / NS) & 1, p.err))) break;
        const uint32_t vp = ring + i * G::kSlot;
        const int r0 = valid % G::kVTok, r1 = (r0 + 15) & ~15;
        constexpr int U = NCH * 8;  // 16-byte units of a row
        for (int x = threadIdx.x; x < (r1 - r0) * U; x += 128) {
          const int r = r0 + x / U, u = x % U;
          const uint32_t at =
              vp + ((r / 8) * NCH + u / 8) * 1024 + (r % 8) * 128 + (u % 8) * 16;
          asm volatile("st.shared.v4.u32 [%0], {%1,%1,%1,%1};" ::"r"(at ^ (((at >> 7) & 7u) << 4)),
                       "r"(0u)
                       : "memory");
        }
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      }
      tmem_wait_st();
      tc_fence_before();
      mbar_arrive(&p_full[b]);
      if (walk.ends()) {
        // ---- the segment's result
        if (!__all_sync(0xffffffffu, mbar_wait(&o_done[b], (t >> 1) & 1, p.err))) break;
        tc_fence_after();
        const float inv = l > 0.f ? (FP8 ? p.v_scale[walk.h] : 1.f) / l : 0.f;
        const bool whole = seg_st == 0 && walk.st + 1 == walk.q.steps;
        if (whole) {
          uint16_t* dst = p.out + (static_cast<int64_t>(walk.q.q0 + draft) * p.num_heads + head) * D;
#pragma unroll 1
          for (int c = 0; c < D; c += 16) {
            float ov[16];
            tmem_ld16(t_o + lane_off + c, ov);
            if (live) {
              uint32_t w[8];
#pragma unroll
              for (int i = 0; i < 8; ++i) w[i] = pack_bf16(ov[2 * i] * inv, ov[2 * i + 1] * inv);
              reinterpret_cast<uint4*>(dst + c)[0] = make_uint4(w[0], w[1], w[2], w[3]);
              reinterpret_cast<uint4*>(dst + c)[1] = make_uint4(w[4], w[5], w[6], w[7]);
            }
          }
        } else {
          const int slot = first_seg ? 0 : 1;
          const int64_t at = (static_cast<int64_t>(cta) * 2 + slot) * kTreeRows + row;
          float* dst = p.part_o + at * D;
#pragma unroll 1
          for (int c = 0; c < D; c += 16) {
            float ov[16];
            tmem_ld16(t_o + lane_off + c, ov);
            if (live) {
#pragma unroll
              for (int i = 0; i < 16; i += 4)
                *reinterpret_cast<float4*>(dst + c + i) =
                    make_float4(ov[i] * inv, ov[i + 1] * inv, ov[i + 2] * inv, ov[i + 3] * inv);
            }
          }
          if (live) {
            p.part_m[at] = m;
            p.part_l[at] = l;
          }
        }
        tc_fence_before();
        mbar_arrive(o_free);
        if (threadIdx.x == 0 && !whole && seg_st == 0) {
          // the unit starts here and goes on, up to the share that holds its end
          const int64_t u_end = end + (walk.q.steps - 1 - walk.st);
          int64_t last = cta + 1;
          while ((last + 1) * total / ctas < u_end) ++last;
          TreeMeta md;
          md.row0 = walk.q.q0;
          md.first = walk.tile * kTreeRows;
          md.rows = min(kTreeRows, walk.q.n * g - md.first);
          md.head = walk.h;
          md.slot = first_seg ? 0 : 1;
          md.parts = static_cast<int>(last - cta + 1);
          p.meta[cta] = md;
        }
        first_seg = false;
      }
      walk.next(p);
    }
  } else if (warp < 7 + G::kQWarps) {
    // ---------------- Q of each segment into shared memory (K-major, 128-byte
    // swizzle); rows past the tile's query rows are zero
    const int i0 = threadIdx.x - 7 * 32;
    const int g = p.group;
    constexpr int U = D / 8;  // 16-byte units of a row
    constexpr int kStep = G::kQWarps * 32;
    const int inv = 65536 / g + 1;
    uint32_t seg = 0;
    while (walk.left > 0) {
      const int r0 = walk.tile * kTreeRows;
      const int rows = min(kTreeRows, walk.q.n * g - r0);
      const uint16_t* q0 = p.q + (static_cast<int64_t>(walk.q.q0) * p.num_heads + walk.h * g) * D;
      // row r of the tile: draft (r0 + r) / g, group row (r0 + r) % g
      auto row_of = [&](int r) {
        const int dr = ((r0 + r) * inv) >> 16;
        return q0 + (static_cast<int64_t>(dr) * p.num_heads + (r0 + r - dr * g)) * D;
      };
      // into L2 while the segment before is still being multiplied
      for (int x = i0; x < rows * (D / 64); x += kStep)
        asm volatile("prefetch.global.L2 [%0];" ::"l"(row_of(x / (D / 64)) + x % (D / 64) * 64));
      if (!__all_sync(0xffffffffu, mbar_wait(q_empty, (seg & 1) ^ 1, p.err))) break;
      auto place = [&](int r, int u) {
        const uint32_t at = sq + ((r / 8) * NCH + u / 8) * 1024 + (r % 8) * 128 + (u % 8) * 16;
        return at ^ (((at >> 7) & 7u) << 4);
      };
#pragma unroll 4
      for (int x = i0; x < kTreeRows * U; x += kStep) {
        const int r = x / U, u = x % U;
        cp_async16(place(r, u), row_of(r < rows ? r : 0) + u * 8, r < rows);
      }
      asm volatile("cp.async.wait_all;" ::: "memory");
      if constexpr (FP8) {
        // f16 operands: each thread converts the units it brought
#pragma unroll 4
        for (int x = i0; x < kTreeRows * U; x += kStep) {
          const uint32_t at = place(x / U, x % U);
          uint4 v;
          asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
                       : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                       : "r"(at));
          asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(at),
                       "r"(pack_f16(bf16lo(v.x), bf16hi(v.x))),
                       "r"(pack_f16(bf16lo(v.y), bf16hi(v.y))),
                       "r"(pack_f16(bf16lo(v.z), bf16hi(v.z))),
                       "r"(pack_f16(bf16lo(v.w), bf16hi(v.w)))
                       : "memory");
        }
      }
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      mbar_arrive(q_full);
      ++seg;
      while (!walk.ends()) walk.next(p);
      walk.next(p);
    }
  } else if constexpr (FP8) {
    // ---------------- converters: codes of a stage -> the f16 values of a slot
    const int ct = threadIdx.x - (7 + G::kQWarps) * 32;
    const int B = p.block_size;
    RingPos<FP8 ? G::kNStage : 1> from;
    RingPos<NS> to;
    // order of the slots: K(0), then K(t + 1) and V(t) for each step t
    int64_t k_left = count * KS, v_left = count * VS;
    int run = KS;  // slots of the kind at hand before the other kind's turn
    bool is_v = false;
    while (k_left + v_left > 0) {
      const int i8 = from.i, i = to.i;
      if (!__all_sync(0xffffffffu, mbar_wait(&full8[i8], from.ph, p.err))) break;
      if (!__all_sync(0xffffffffu, mbar_wait(&empty[i], to.ph ^ 1, p.err))) break;
      const uint32_t src0 = stage + i8 * G::kStage, dst0 = ring + i * G::kSlot;
      // codes per row: 128 (K; V at d = 128) or 256 (V at d = 256)
      const int nch = is_v ? NCH : 2;
      const int upr = is_v ? D / 16 : 8;  // 16-code units of a row
      for (int x = ct; x < G::kStage / 16; x += G::kConvWarps * 32) {
        const int u = x % upr, r = x / upr;
        // staged page: [128-code chunk][B rows][128 B]
        const int pg = r / B, rr = r % B;
        uint32_t src = src0 + pg * B * upr * 16 + (u >> 3) * B * 128 + rr * 128 + (u & 7) * 16;
        src ^= ((src >> 7) & 7u) << 4;
        uint32_t dst = dst0 + ((r / 8) * nch + u / 4) * 1024 + (r % 8) * 128 + (u % 4) * 32;
        const uint32_t sw = ((dst >> 7) & 7u) << 4;
        uint32_t c0, c1, c2, c3;
        asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
                     : "=r"(c0), "=r"(c1), "=r"(c2), "=r"(c3)
                     : "r"(src));
        asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(dst ^ sw),
                     "r"(e4m3x2_f16x2(c0, 0)), "r"(e4m3x2_f16x2(c0, 1)), "r"(e4m3x2_f16x2(c1, 0)),
                     "r"(e4m3x2_f16x2(c1, 1))
                     : "memory");
        asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"((dst + 16) ^ sw),
                     "r"(e4m3x2_f16x2(c2, 0)), "r"(e4m3x2_f16x2(c2, 1)), "r"(e4m3x2_f16x2(c3, 0)),
                     "r"(e4m3x2_f16x2(c3, 1))
                     : "memory");
      }
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(&full[i]);
        mbar_arrive(&empty8[i8]);
      }
      from.next();
      to.next();
      (is_v ? v_left : k_left) -= 1;
      if (--run == 0) {
        // after K(0) comes K(1); V(t) follows K(t + 1), or stands alone at the end
        is_v = k_left == 0 || (!is_v && k_left != (count - 1) * KS);
        run = is_v ? VS : KS;
      }
    }
  }

  allow_dependents();  // the merge may be scheduled; it waits for this grid
  tc_fence_before();
  __syncthreads();
  if ((warp == 5 || warp == 6) && lane == 0) {
    // no copy may still be writing this CTA's shared memory when it exits
    const int n = FP8 ? G::kNStage : NS;
    for (int64_t seq = issued > n ? issued - n : 0; seq < issued; ++seq)
      if (!mbar_wait(FP8 ? &full8[seq % n] : &full[seq % n], (seq / n) & 1, p.err)) break;
  }
  if (warp == 4) {
    tc_fence_after();
    tmem_dealloc(tmem, G::kCols);
  }
}

// Joins the partials of the units that were cut: CTA (c, y) takes rows
// 8 y .. 8 y + 7 of the unit that starts in share c, one warp per row. With
// m_i, l_i, o_i of the unit's segments in order, M = max m_i (base 2) and
// w_i = l_i 2^(m_i - M): out = sum (w_i / sum w) o_i.
template <int D>
__global__ void __launch_bounds__(256) tree_merge_kernel(const __grid_constant__ TreeParams p) {
  wait_prerequisite();
  const int c = blockIdx.x;
  const TreeMeta md = p.meta[c];
  const int row = blockIdx.y * 8 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  if (md.parts == 0 || row >= md.rows) return;
  // partial i: the first is share c's, the others are slot 0 of the next shares
  auto at = [&](int i) {
    return (static_cast<int64_t>(c + i) * 2 + (i == 0 ? md.slot : 0)) * kTreeRows + row;
  };
  float M = -INFINITY;
  for (int i = lane; i < md.parts; i += 32) M = fmaxf(M, p.part_m[at(i)]);
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, off));
  const float ref = M == -INFINITY ? 0.f : M;
  float W = 0.f;
  for (int i = lane; i < md.parts; i += 32) W += p.part_l[at(i)] * fast_exp2(p.part_m[at(i)] - ref);
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) W += __shfl_xor_sync(0xffffffffu, W, off);
  const float inv = W > 0.f ? 1.f / W : 0.f;
  constexpr int V4 = D / 128;
  float4 acc[V4];
#pragma unroll
  for (int v = 0; v < V4; ++v) acc[v] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
  for (int i = 0; i < md.parts; ++i) {
    const float w = p.part_l[at(i)] * fast_exp2(p.part_m[at(i)] - ref) * inv;
    const float4* src = reinterpret_cast<const float4*>(p.part_o + at(i) * D);
#pragma unroll
    for (int v = 0; v < V4; ++v) {
      const float4 x = src[lane + 32 * v];
      acc[v].x = fmaf(w, x.x, acc[v].x);
      acc[v].y = fmaf(w, x.y, acc[v].y);
      acc[v].z = fmaf(w, x.z, acc[v].z);
      acc[v].w = fmaf(w, x.w, acc[v].w);
    }
  }
  const int r = md.first + row;
  const int64_t hq = static_cast<int64_t>(md.row0 + r / p.group) * p.num_heads +
                     md.head * p.group + r % p.group;
  uint2* dst = reinterpret_cast<uint2*>(p.out + hq * D);
#pragma unroll
  for (int v = 0; v < V4; ++v)
    dst[lane + 32 * v] = make_uint2(pack_bf16(acc[v].x, acc[v].y), pack_bf16(acc[v].z, acc[v].w));
}

// ---------------------------------------------------------------- host side

// 4-D map of a bf16 pool, [8-row group][64-column chunk][8 rows][64 columns],
// boxes of `chunks` chunks of one page.
static int tree_pool_map(CUtensorMap* out, const void* base, int64_t rows, int D, int B,
                         int chunks) {
  auto enc = tensor_map_encoder();
  if (!enc) return PKV_ERR_CUDA;
  const cuuint64_t row = static_cast<cuuint64_t>(D) * 2;
  cuuint64_t dims[4] = {64, 8, static_cast<cuuint64_t>(D / 64), static_cast<cuuint64_t>(rows / 8)};
  cuuint64_t strides[3] = {row, 128, 8 * row};
  cuuint32_t box[4] = {64, 8, static_cast<cuuint32_t>(chunks), static_cast<cuuint32_t>(B / 8)};
  cuuint32_t estr[4] = {1, 1, 1, 1};
  const CUresult r =
      enc(out, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(base), dims, strides, box,
          estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
          CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? PKV_OK : PKV_ERR_CUDA;
}

template <int D, bool FP8>
static int launch_tree(const TreeParams& p, const void* k_cache, const void* v_cache, int ctas,
                       cudaStream_t st) {
  using G = TreeGeom<D, FP8>;
  const int64_t rows = static_cast<int64_t>(p.num_blocks) * p.num_kv_heads * p.block_size;
  CUtensorMap tk, tv;
  int rc = FP8 ? encode_pool_map(&tk, k_cache, rows, D, p.block_size, true, false)
               : tree_pool_map(&tk, k_cache, rows, D, p.block_size, 2);
  if (rc != PKV_OK) return rc;
  rc = FP8 ? encode_pool_map(&tv, v_cache, rows, D, p.block_size, true, false)
           : tree_pool_map(&tv, v_cache, rows, D, p.block_size, D / 64);
  if (rc != PKV_OK) return rc;
  static DeviceFlags done;
  auto kern = tree_kernel<D, FP8>;
  rc = ensure_smem(kern, G::kSmem, done);
  if (rc != PKV_OK) return rc;
  rc = launch_dependent(kern, dim3(ctas), dim3(G::kThreads), G::kSmem, st, tk, tv, p);
  if (rc != PKV_OK) return rc;
  return launch_dependent(tree_merge_kernel<D>, dim3(ctas, kTreeRows / 8), dim3(256), 0, st, p);
}

}  // namespace pkv

extern "C" size_t pkv_tree_workspace_bytes(int num_seqs, int num_queries, int num_heads,
                                           int num_kv_heads, int head_dim, int max_context,
                                           int max_draft) {
  using namespace pkv;
  if (num_seqs <= 0 || num_queries <= 0 || num_heads <= 0 || num_kv_heads <= 0 || head_dim <= 0 ||
      max_context <= 0 || max_draft <= 0)
    return 0;
  // per CTA: what the merge needs, two partial tiles
  return static_cast<size_t>(kTreeMaxCtas) *
         (sizeof(TreeMeta) + 2u * kTreeRows * (static_cast<size_t>(head_dim) + 2) * sizeof(float));
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
                           max_blocks_per_seq, context_lens, num_queries > 0 ? num_seqs : 0,
                           num_heads, max_context, scale, &g);
  if (rc != PKV_OK) return rc;
  if (num_queries < 0 || num_seqs < 0 || max_draft < 1 || max_draft > PKV_MAX_DRAFT)
    return PKV_ERR_INVALID_ARG;
  if (num_seqs == 0 || num_queries == 0) return PKV_OK;
  const size_t need = pkv_tree_workspace_bytes(num_seqs, num_queries, num_heads,
                                               cache.num_kv_heads, cache.head_dim,
                                               std::max(1, max_context), max_draft);
  if (!q_start || !workspace || !aligned16(workspace) || workspace_bytes < need)
    return PKV_ERR_INVALID_ARG;
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return PKV_ERR_CUDA;
  TreeParams p{};
  p.q = static_cast<const uint16_t*>(q);
  p.out = static_cast<uint16_t*>(out);
  p.k_scale = k_scale;
  p.v_scale = v_scale;
  p.block_tables = block_tables;
  p.context_lens = context_lens;
  p.q_start = q_start;
  p.tree_mask = tree_mask;
  p.err = device_error_ptr();
  const size_t tiles = static_cast<size_t>(kTreeMaxCtas) * 2 * kTreeRows;
  p.part_o = static_cast<float*>(workspace);
  p.part_m = p.part_o + tiles * cache.head_dim;
  p.part_l = p.part_m + tiles;
  p.meta = reinterpret_cast<TreeMeta*>(p.part_l + tiles);
  p.num_seqs = num_seqs;
  p.num_queries = num_queries;
  p.max_draft = max_draft;
  p.num_blocks = cache.num_blocks;
  p.num_kv_heads = cache.num_kv_heads;
  p.num_heads = num_heads;
  p.group = g;
  p.block_size = cache.block_size;
  p.max_blocks_per_seq = max_blocks_per_seq;
  p.min_steps = 2;
  p.qscale = scale * 1.4426950408889634f;
  // no more CTAs than the call's bounds can give work
  const int64_t tiles_most =
      num_seqs + static_cast<int64_t>(num_queries) * g / kTreeRows;
  const int64_t steps_most = tiles_most * cache.num_kv_heads *
                             ((static_cast<int64_t>(max_context) + kTreeTok - 1) / kTreeTok);
  const int ctas = static_cast<int>(std::max<int64_t>(
      1, std::min<int64_t>(std::min(sms, kTreeMaxCtas),
                           (steps_most + p.min_steps - 1) / p.min_steps)));
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const bool fp8 = cache.dtype == PKV_DTYPE_FP8_E4M3;
  if (cache.head_dim == 128)
    return fp8 ? launch_tree<128, true>(p, k_cache, v_cache, ctas, st)
               : launch_tree<128, false>(p, k_cache, v_cache, ctas, st);
  return fp8 ? launch_tree<256, true>(p, k_cache, v_cache, ctas, st)
             : launch_tree<256, false>(p, k_cache, v_cache, ctas, st);
}

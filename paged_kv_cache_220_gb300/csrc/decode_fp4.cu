// Attention of one query token per sequence over a 4-bit cache: over the whole
// context (paged_attention_fp4) or over listed blocks (paged_attention_sparse).
//
// The batch's work is one line of units of tokens (TU = 64, 32 at D = 256), pair
// (sequence, KV head) after pair, cut into equal shares, one per resident warp.
// Every warp works alone: lane 0 keeps a ring of K and V of its next units in
// flight with bulk copies, one per block and pool (a page's codes and scales are
// one contiguous run), through the ends of pairs too. A pair inside a share is
// written to the result; of a pair that is cut each warp leaves (maxima, sums,
// output) in its slots, at most two, and a second kernel joins them.
//
// Arithmetic, with mma.m16n8k16 (f16 in, fp32 out): tokens are the M side of
// S^T = K Q^T and the head's channels that of O^T = V^T P^T; the padded query
// group is the N side.
// - An operand value is E2M1 code * E4M3 scale, which f16 holds exactly (6
//   significant bits, 2^-10 to 2688): cvt.f16x2.e2m1x2 (a byte of codes, 64 lanes a
//   clock and SM, the pipe of the integer instructions) and one f16x2 product.
// - S sums over channels, in any order: lane (r, c) of a fragment (row r = lane /
//   4, column pair c = lane % 4) takes a quarter of the row's channels, D/4 c on, 16
//   bytes at a time, and Q's fragments have the same order. Nothing is moved
//   between lanes.
// - O's rows are channels: lane (r, c) takes channels D/8 r on of four tokens; the
//   codes of two tokens are put into one byte (even channels, then odd ones) with
//   a shift and a three-input logic instruction, so that a conversion gives the
//   pair the fragment wants. The scale is that of the two tokens.
// - Which token is which row of S is free as long as P has the same: at D = 128,
//   where two tokens share a line, tokens 4c .. 4c + 3 are rows 2c, 2c + 1, 2c + 8,
//   2c + 9, so that 16 lanes of the V loads meet 16 different 8-byte banks.
// - Rows of q are scaled by a power of two to below 2 before they become f16; the
//   weights are 2^15 times as large, so that f16 loses what is below 2^-40 of the
//   largest and not 2^-25. Both factors leave exactly.
// - A hidden token (behind the context, of a skipped block) gets the logit -inf and
//   V's scale 0: codes are always finite, only a scale can be NaN.
#include <algorithm>

#include "common.cuh"
#include "decode_params.h"
#include "fp4.cuh"
#include "host_util.h"
#include "tc_common.cuh"

namespace pkv {

constexpr float kUpFp4 = 15.f;    // log2 of the factor on the weights
constexpr int kFp4Warps = 4;      // warps of a CTA
constexpr int kFp4Ctas = 3;       // CTAs to an SM
constexpr int kFp4Stages = 2;     // units in a warp's ring
constexpr int kFp4MaxCtas = 456;  // of a launch: the residents of 152 SMs

template <int D>
struct Fp4Geom {
  static constexpr int TU = D == 256 ? 32 : 64;       // tokens of a unit
  static constexpr int kBytes = TU * D / 16 * 9;      // K (or V) of a unit
  static constexpr int kStage = 2 * kBytes;
  static constexpr int kThreads = kFp4Warps * 32;
  // barriers, the rows' first units by thread, the look-up cursors, the ends' states
  static constexpr int kHead = kFp4Warps * kFp4Stages * 16 + (kThreads + 4) * 4 +
                               kFp4Warps * (16 + 64 + 4);
  static constexpr int kRingAt = (kHead + 127) / 128 * 128;
  static constexpr int kSmem = kRingAt + kFp4Warps * kFp4Stages * kStage;
  // a slot: O as the lanes hold it, [D/16][32] float4, then 8 maxima (base 2) and 8 sums
  static constexpr int kSlot = 8 * D + 16;            // floats
};

struct Fp4Params {
  const uint16_t* q;
  const uint8_t* k_cache;
  const uint8_t* v_cache;
  const float* k_scale;
  const float* v_scale;
  const int32_t* block_tables;
  const int32_t* context_lens;
  const int32_t* list;     // the listed form: [S][Hk][max_selected], [S][Hk]
  const int32_t* counts;
  uint16_t* out;
  int32_t* first;          // first unit of every row (sequence, or pair if listed), and the end
  float* slots;            // [workers][2][kSlot]
  int* err;
  int num_seqs, num_blocks, num_kv_heads, group, max_blocks_per_seq;
  int max_context, max_selected;
  int workers;             // warps of the launch
  float qscale;            // scale * log2(e)
};

// First unit of worker w of n, T units in all.
__device__ __forceinline__ int share_begin(int w, int n, int T) {
  return static_cast<int>(static_cast<int64_t>(w) * T / n);
}

// One contiguous run of global memory into shared memory; evict-first in L2, a
// page is read once.
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes,
                                          uint64_t* bar, uint64_t policy) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint"
      " [%0], [%1], %2, [%3], %4;" ::"r"(dst),
      "l"(src), "r"(bytes), "r"(smem_addr(bar)), "l"(policy)
      : "memory");
}

__device__ __forceinline__ uint4 lds128(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(a));
  return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t a) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a));
  return v;
}
__device__ __forceinline__ uint32_t lds32(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(a));
  return v;
}
__device__ __forceinline__ uint32_t lds16(uint32_t a) {
  uint16_t v;
  asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(a));
  return v;
}
__device__ __forceinline__ uint32_t lds8(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared.u8 %0, [%1];" : "=r"(v) : "r"(a));
  return v;
}

__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, __half2 b) {
  const __half2 d = __hmul2(*reinterpret_cast<const __half2*>(&a), b);
  return *reinterpret_cast<const uint32_t*>(&d);
}
// Two E4M3 codes (the low or the high 16 bits of w) as f16x2
__device__ __forceinline__ __half2 scales_of(uint32_t w, int hi) {
  const uint32_t d = e4m3x2_f16x2(w, hi);
  return *reinterpret_cast<const __half2*>(&d);
}

template <int D, int BS, bool LIST>
__global__ void __launch_bounds__(Fp4Geom<D>::kThreads, kFp4Ctas)
    decode_fp4_kernel(const Fp4Params p) {
  using G = Fp4Geom<D>;
  constexpr int TU = G::TU, W = kFp4Warps, NST = kFp4Stages, THREADS = G::kThreads;
  constexpr int UB = TU / BS;             // blocks of a unit
  constexpr int NT = TU / 16;             // 16-token tiles of a unit
  constexpr int PAGE = BS * D / 16 * 9;   // bytes of a block's page
  constexpr int KW = D / 16;              // k-steps of S, row tiles of O
  extern __shared__ __align__(128) uint8_t smem_raw[];
  uint64_t* my_k = reinterpret_cast<uint64_t*>(smem_raw) + (threadIdx.x >> 5) * NST;
  uint64_t* my_v = my_k + W * NST;
  int* pre = reinterpret_cast<int*>(smem_raw + W * NST * 16);  // [THREADS + 4]
  int4* my_cursor = reinterpret_cast<int4*>(pre + THREADS + 4) + (threadIdx.x >> 5);
  float* ends_m = reinterpret_cast<float*>(pre + THREADS + 4) + W * 4;  // [W][8]
  float* ends_l = ends_m + W * 8;                                       // [W][8]
  int* ends_pair = reinterpret_cast<int*>(ends_l + W * 8);              // [W]
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int r = lane >> 2, c = lane & 3;
  if (lane == 0) {
    for (int i = 0; i < NST; ++i) {
      mbar_init(&my_k[i], 1);
      mbar_init(&my_v[i], 1);
    }
    fence_mbar_init();
  }
  wait_prerequisite();
  const int Hk = p.num_kv_heads, g = p.group;

  // ---- the line of units: rows are sequences (all heads alike) or, listed, pairs
  auto context = [&](int s) {
    const int ctx = p.context_lens[s];
    if (ctx >= 0 && ctx <= p.max_context) return ctx;
    report_error(p.err, PKV_DEVERR_CONTEXT);
    return ctx < 0 ? 0 : p.max_context;
  };
  // blocks of a pair of the row: the context's or the list's
  auto blocks_of = [&](int row) {
    if (!LIST) return (context(row) + BS - 1) / BS;
    const int n = p.counts[row];
    if (n >= 0 && n <= p.max_selected) return n;
    report_error(p.err, PKV_DEVERR_SELECT);
    return n < 0 ? 0 : p.max_selected;
  };
  const int rows = LIST ? p.num_seqs * Hk : p.num_seqs;
  const int per_row = LIST ? 1 : Hk;                       // pairs of a row
  const int chunk = (rows + THREADS - 1) / THREADS;        // rows of a thread
  int T = 0;
  {
    const int row0 = min(rows, static_cast<int>(threadIdx.x) * chunk);
    const int row1 = min(rows, row0 + chunk);
    int sum = 0;
    for (int row = row0; row < row1; ++row) sum += per_row * ((blocks_of(row) + UB - 1) / UB);
    int incl = sum;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int x = __shfl_up_sync(0xffffffffu, incl, off);
      if (lane >= off) incl += x;
    }
    if (lane == 31) pre[THREADS + warp] = incl;
    __syncthreads();
    int before = 0;
#pragma unroll
    for (int w = 0; w < W; ++w) {
      if (w < warp) before += pre[THREADS + w];
      T += pre[THREADS + w];
    }
    int at = before + incl - sum;
    pre[threadIdx.x] = at;
    if (blockIdx.x == 0) {
      for (int row = row0; row < row1; ++row) {
        p.first[row] = at;
        at += per_row * ((blocks_of(row) + UB - 1) / UB);
      }
      if (threadIdx.x == 0) p.first[rows] = T;
    }
    __syncthreads();
  }
  // the merge launched next may be scheduled; it waits for this grid's end
  allow_dependents();
  const int n_workers = min(p.workers, T);
  const int me = blockIdx.x * W + warp;
  if (blockIdx.x * W >= n_workers) return;
  const int u0 = me < n_workers ? share_begin(me, n_workers, T) : T;
  // units of this warp, one at least if it is one of the workers
  const int mine = me < n_workers ? share_begin(me + 1, n_workers, T) - u0 : 0;
  // the pair and unit that u0 is
  int pair = -1, unit = 0, units = 0;
  if (mine > 0) {
    int t = 0;
#pragma unroll
    for (int k = 0; k < W; ++k)
      t += __popc(__ballot_sync(0xffffffffu, pre[k * 32 + lane] <= u0));
    int row = (t - 1) * chunk;
    int left = u0 - pre[t - 1];
    for (;; ++row) {
      units = (blocks_of(row) + UB - 1) / UB;
      if (left < per_row * units) break;
      left -= per_row * units;
    }
    pair = row * per_row + left / units;
    unit = left % units;
  }

  // ---- look-ups: lanes look up the blocks of the next units of one pair, 32 / UB at
  // most, together: lane l block l % UB of unit l / UB. pb: the block, -1 if there
  // is none; vis: how many tokens of each of the unit's blocks are visible, a byte
  // each. The cursor: pair, its next unit, its units, units left for this warp
  constexpr int kBatch = 32 / UB;
  constexpr uint32_t kWhole = BS * (UB == 1 ? 1u : UB == 2 ? 0x0101u : 0x01010101u);
  if (lane == 0) *my_cursor = make_int4(pair, unit, units, mine);
  __syncwarp();
  auto look_up = [&](int& pb, uint32_t& vis) {  // -> units looked up
    int4 u = *my_cursor;
    pb = -1;
    vis = 0;
    if (u.w == 0) return 0;
    while (u.y == u.z) {  // the next pair that has a unit
      ++u.x;
      u.y = 0;
      u.z = (blocks_of(LIST ? u.x : u.x / Hk) + UB - 1) / UB;
    }
    const int n = min(min(kBatch, u.z - u.y), u.w);
    const int s = u.x / Hk;
    const int ctx = context(s);
    const int v = UB * (u.y + lane / UB) + lane % UB;
    if (lane / UB < n && v < (LIST ? blocks_of(u.x) : (ctx + BS - 1) / BS)) {
      const int b = LIST ? p.list[static_cast<int64_t>(u.x) * p.max_selected + v] : v;
      if (LIST && (b < 0 || b >= (ctx + BS - 1) / BS)) {
        report_error(p.err, PKV_DEVERR_SELECT);
      } else {
        const int32_t x = p.block_tables[static_cast<int64_t>(s) * p.max_blocks_per_seq + b];
        if (x < 0 || x >= p.num_blocks) {
          report_error(p.err, PKV_DEVERR_BLOCK_ID);
        } else {
          pb = x * Hk + u.x % Hk;  // the page
          vis = static_cast<uint32_t>(min(BS, ctx - b * BS)) << (8 * (lane % UB));
        }
      }
    }
    __syncwarp();
    if (lane == 0) *my_cursor = make_int4(u.x, u.y + n, u.z, u.w - n);
    __syncwarp();
#pragma unroll
    for (int off = 1; off < UB; off <<= 1) vis |= __shfl_xor_sync(0xffffffffu, vis, off);
    return n;
  };
  int pb_now, pb_next;
  uint32_t vis_now, vis_next;
  int n_now = look_up(pb_now, vis_now), n_next = 0;
  int at = 0;  // units of the current batch that are loaded
  const uint32_t my_ring = smem_addr(smem_raw) + G::kRingAt + warp * NST * G::kStage;
  uint64_t policy;
  asm volatile("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(policy));
  // the unit whose K was loaded last (its V comes next)
  int ids[UB];
  uint32_t vis[NST] = {};  // of the units in the ring, the oldest first
  auto load = [&](uint32_t dst, const uint8_t* pool, uint64_t* bar) {
    if (lane != 0) return;
    uint32_t bytes = 0;
#pragma unroll
    for (int b = 0; b < UB; ++b) bytes += ids[b] >= 0 ? PAGE : 0;
    mbar_arrive_expect_tx(bar, bytes);
#pragma unroll
    for (int b = 0; b < UB; ++b)
      if (ids[b] >= 0)
        bulk_load(dst + b * PAGE, pool + static_cast<uint64_t>(ids[b]) * PAGE, PAGE, bar, policy);
  };
  // K of the next unit into slot st
  auto load_k = [&](int st) {
    if (at == n_now) {
      pb_now = pb_next;
      vis_now = vis_next;
      n_now = n_next;
      n_next = look_up(pb_next, vis_next);
      at = 0;
    }
#pragma unroll
    for (int b = 0; b < UB; ++b) ids[b] = __shfl_sync(0xffffffffu, pb_now, at * UB + b);
    vis[NST - 1] = __shfl_sync(0xffffffffu, vis_now, at * UB);
    ++at;
    load(my_ring + st * G::kStage, p.k_cache, &my_k[st]);
  };
  auto load_v = [&](int st) { load(my_ring + st * G::kStage + G::kBytes, p.v_cache, &my_v[st]); };
#pragma unroll
  for (int i = 0; i < NST; ++i) {
#pragma unroll
    for (int k = 0; k + 1 < NST; ++k) vis[k] = vis[k + 1];
    if (i < mine) load_k(i);
    if (i < mine && i + 1 < NST) load_v(i);
    // the second batch's look-up behind the first unit's loads
    if (i == 0) n_next = look_up(pb_next, vis_next);
  }

  // ---- the pair at hand: units of it that are left, whether it is this warp's alone
  int seg = min(units - unit, mine);
  bool alone = unit == 0 && seg == units;
  bool fresh = true;
  uint32_t bq[KW][2];
  float f0 = 0.f, f1 = 0.f;  // logit factors of queries 2c, 2c + 1 (base 2), not negative
  // running maxima of the products before their factor, sums, outputs
  float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.f, l1 = 0.f;
  float o[KW][4];
  // the sums over the eight lanes that share a query pair
  auto sum_rows = [&] {
#pragma unroll
    for (int off = 4; off < 32; off <<= 1) {
      l0 += __shfl_xor_sync(0xffffffffu, l0, off);
      l1 += __shfl_xor_sync(0xffffffffu, l1, off);
    }
  };
  // a maximum as a base-2 logit
  auto log2_max = [](float m, float f) { return m == -INFINITY ? m : m * f; };
  // token of the unit that row x of tile t stands for
  auto token = [](int t, int x) {
    return 16 * t + (D == 256 ? x : ((x & 7) >> 1) * 4 + (x & 1) + (x >= 8 ? 2 : 0));
  };
  int done = 0;          // units done
  bool v_late = false;  // the wait that ran out, if one did, was V's
  int st = 0;
  uint32_t parity = 0;
  for (; done < mine; ++done) {
    if (fresh) {
      fresh = false;
      m0 = m1 = -INFINITY;
      l0 = l1 = 0.f;
#pragma unroll
      for (int k = 0; k < KW; ++k) o[k][0] = o[k][1] = o[k][2] = o[k][3] = 0.f;
      // Q^T fragments: lane (n = r, c) has channels D/4 c + 4 j + {0, 1} and {2, 3} of
      // query n for k-step j, as f16, in units of a power of two of its row, with
      // the logit factor's sign
      const uint2* qrow = reinterpret_cast<const uint2*>(
          p.q + (static_cast<int64_t>(pair) * g + r) * D + D / 4 * c);
      float top = 0.f;
#pragma unroll
      for (int j = 0; j < KW; ++j) {
        const uint2 w = r < g ? __ldg(qrow + j) : make_uint2(0, 0);
        bq[j][0] = w.x;
        bq[j][1] = w.y;
        top = fmaxf(top, fmaxf(fmaxf(fabsf(bf16lo(w.x)), fabsf(bf16hi(w.x))),
                               fmaxf(fabsf(bf16lo(w.y)), fabsf(bf16hi(w.y)))));
      }
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
      const float qs = p.qscale * p.k_scale[pair % Hk];
      const int e = min(max(static_cast<int>(__float_as_uint(top) >> 23), 1), 253);
      const float down = copysignf(__uint_as_float(static_cast<uint32_t>(254 - e) << 23), qs);
      const float up = __uint_as_float(static_cast<uint32_t>(e) << 23);
#pragma unroll
      for (int j = 0; j < KW; ++j)
#pragma unroll
        for (int i = 0; i < 2; ++i)
          bq[j][i] = pack_f16(bf16lo(bq[j][i]) * down, bf16hi(bq[j][i]) * down);
      f0 = fabsf(qs) * __shfl_sync(0xffffffffu, up, 8 * c);
      f1 = fabsf(qs) * __shfl_sync(0xffffffffu, up, 8 * c + 4);
    }
    if (!__all_sync(0xffffffffu, mbar_wait(&my_k[st], parity, p.err))) break;
    const uint32_t kp = my_ring + st * G::kStage, vp = kp + G::kBytes;
    const uint32_t seen = vis[0];
    const bool whole = seen == kWhole;
    auto sees = [&](int t) { return t % BS < static_cast<int>(seen >> (8 * (t / BS)) & 0xFFu); };

    // ---- S^T = K Q^T
    float sc[NT][4];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      constexpr int NW = D / 32;  // words of codes of a lane and row
      uint32_t wa[NW], wb[NW], sa, sb;
      const int ta = token(t, r), tb = token(t, r + 8);
      if constexpr (D == 256) {
        const uint32_t ra = kp + ta * kFp4Line, rb = kp + tb * kFp4Line;
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const uint4 a = lds128(ra + 32 * c + 16 * x), b = lds128(rb + 32 * c + 16 * x);
          wa[4 * x] = a.x, wa[4 * x + 1] = a.y, wa[4 * x + 2] = a.z, wa[4 * x + 3] = a.w;
          wb[4 * x] = b.x, wb[4 * x + 1] = b.y, wb[4 * x + 2] = b.z, wb[4 * x + 3] = b.w;
        }
        sa = lds32(ra + 128 + 4 * c);
        sb = lds32(rb + 128 + 4 * c);
      } else {
        const uint4 a = lds128(kp + fp4_codes_at<D>(ta) + 16 * c);
        const uint4 b = lds128(kp + fp4_codes_at<D>(tb) + 16 * c);
        wa[0] = a.x, wa[1] = a.y, wa[2] = a.z, wa[3] = a.w;
        wb[0] = b.x, wb[1] = b.y, wb[2] = b.z, wb[3] = b.w;
        sa = lds16(kp + fp4_scales_at<D>(ta) + 2 * c);
        sb = lds16(kp + fp4_scales_at<D>(tb) + 2 * c);
      }
      sc[t][0] = sc[t][1] = sc[t][2] = sc[t][3] = 0.f;
#pragma unroll
      for (int x = 0; x < NW; ++x) {
        // two words (16 channels) to a scale
        const int gr = x / 2;
        const __half2 pa = scales_of(sa, gr / 2), pb = scales_of(sb, gr / 2);
        const __half2 fa = gr & 1 ? __high2half2(pa) : __low2half2(pa);
        const __half2 fb = gr & 1 ? __high2half2(pb) : __low2half2(pb);
        uint32_t a[4], b[4];
        e2m1x8_f16x2(wa[x], a);
        e2m1x8_f16x2(wb[x], b);
#pragma unroll
        for (int y = 0; y < 2; ++y)
          mma_f16(sc[t], mul_f16x2(a[2 * y], fa), mul_f16x2(b[2 * y], fb),
                  mul_f16x2(a[2 * y + 1], fa), mul_f16x2(b[2 * y + 1], fb), bq[2 * x + y][0],
                  bq[2 * x + y][1]);
      }
    }
    if (!whole) {
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        if (!sees(token(t, r))) sc[t][0] = sc[t][1] = -INFINITY;
        if (!sees(token(t, r + 8))) sc[t][2] = sc[t][3] = -INFINITY;
      }
    }
    // ---- online softmax: rows are tokens, columns queries
    float x0 = m0, x1 = m1;
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      x0 = fmaxf(x0, fmaxf(sc[t][0], sc[t][2]));
      x1 = fmaxf(x1, fmaxf(sc[t][1], sc[t][3]));
    }
#pragma unroll
    for (int off = 4; off < 32; off <<= 1) {
      x0 = fmaxf(x0, __shfl_xor_sync(0xffffffffu, x0, off));
      x1 = fmaxf(x1, __shfl_xor_sync(0xffffffffu, x1, off));
    }
    // Every lane's products have met in the shuffles, so every lane has read this
    // unit's K, and (loads of a warp return in order) the unit before's V: both
    // slots can take their next unit's
    __syncwarp();
    if (done + NST - 1 < mine) load_v(st == 0 ? NST - 1 : st - 1);
#pragma unroll
    for (int k = 0; k + 1 < NST; ++k) vis[k] = vis[k + 1];
    if (done + NST < mine) load_k(st);
    if (__any_sync(0xffffffffu, x0 > m0 || x1 > m1)) {
      // nothing has been summed where the maximum was -inf
      const float c0 = m0 == -INFINITY ? 0.f : fast_exp2((m0 - x0) * f0);
      const float c1 = m1 == -INFINITY ? 0.f : fast_exp2((m1 - x1) * f1);
      l0 *= c0;
      l1 *= c1;
#pragma unroll
      for (int k = 0; k < KW; ++k) {
        o[k][0] *= c0;
        o[k][1] *= c1;
        o[k][2] *= c0;
        o[k][3] *= c1;
      }
      m0 = x0;
      m1 = x1;
    }
    const float ref0 = kUpFp4 - (m0 == -INFINITY ? 0.f : m0 * f0);
    const float ref1 = kUpFp4 - (m1 == -INFINITY ? 0.f : m1 * f1);
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      sc[t][0] = fast_exp2(fmaf(sc[t][0], f0, ref0));
      sc[t][1] = fast_exp2(fmaf(sc[t][1], f1, ref1));
      sc[t][2] = fast_exp2(fmaf(sc[t][2], f0, ref0));
      sc[t][3] = fast_exp2(fmaf(sc[t][3], f1, ref1));
    }
    if (!whole) {
      // (a factor of 0 makes the -inf a NaN)
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        if (!sees(token(t, r))) sc[t][0] = sc[t][1] = 0.f;
        if (!sees(token(t, r + 8))) sc[t][2] = sc[t][3] = 0.f;
      }
    }
    if (!__all_sync(0xffffffffu, mbar_wait(&my_v[st], parity, p.err))) {
      v_late = true;
      break;
    }
    // ---- O^T += V^T P^T
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      l0 += sc[t][0] + sc[t][2];
      l1 += sc[t][1] + sc[t][3];
      const uint32_t q0 = movm_t(pack_f16(sc[t][0], sc[t][1]));
      const uint32_t q1 = movm_t(pack_f16(sc[t][2], sc[t][3]));
      constexpr int NW = D / 64;  // words of codes of a lane and token
      uint32_t w[4][NW], e8[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int tk = token(t, 2 * c + (k & 1) + (k >= 2 ? 8 : 0));
        if constexpr (D == 256) {
          const uint4 a = lds128(vp + tk * kFp4Line + 16 * r);
          w[k][0] = a.x, w[k][1] = a.y, w[k][2] = a.z, w[k][3] = a.w;
          e8[k] = lds16(vp + tk * kFp4Line + 128 + 2 * r);
        } else {
          const uint2 a = lds64(vp + fp4_codes_at<D>(tk) + 8 * r);
          w[k][0] = a.x, w[k][1] = a.y;
          e8[k] = lds8(vp + fp4_scales_at<D>(tk) + r);
        }
      }
      if (!whole) {
#pragma unroll
        for (int k = 0; k < 4; ++k)
          if (!sees(token(t, 2 * c + (k & 1) + (k >= 2 ? 8 : 0)))) e8[k] = 0;
      }
#pragma unroll
      for (int x = 0; x < NW; ++x) {
        // the word's scale: byte x / 2 of each token's
        const uint32_t sel = x / 2 ? 0x51 : 0x40;
        const __half2 s01 = scales_of(__byte_perm(e8[0], e8[1], sel), 0);
        const __half2 s23 = scales_of(__byte_perm(e8[2], e8[3], sel), 0);
        constexpr uint32_t kLow = 0x0F0F0F0Fu;
        uint32_t ev01[4], od01[4], ev23[4], od23[4];
        e2m1x8_f16x2((w[0][x] & kLow) | ((w[1][x] << 4) & ~kLow), ev01);
        e2m1x8_f16x2(((w[0][x] >> 4) & kLow) | (w[1][x] & ~kLow), od01);
        e2m1x8_f16x2((w[2][x] & kLow) | ((w[3][x] << 4) & ~kLow), ev23);
        e2m1x8_f16x2(((w[2][x] >> 4) & kLow) | (w[3][x] & ~kLow), od23);
#pragma unroll
        for (int y = 0; y < 4; ++y)
          mma_f16(o[4 * x + y], mul_f16x2(ev01[y], s01), mul_f16x2(od01[y], s01),
                  mul_f16x2(ev23[y], s23), mul_f16x2(od23[y], s23), q0, q1);
      }
    }
    if (++st == NST) {
      st = 0;
      parity ^= 1;
    }
    --seg;
    if (seg > 0 || (done + 1 == mine && !alone)) continue;
    // ---- the pair's end before the share's, or a pair of this warp alone
    sum_rows();
    if (alone) {
      const float vsc = p.v_scale[pair % Hk];
      const float i0 = l0 != 0.f ? vsc / l0 : 0.f, i1 = l1 != 0.f ? vsc / l1 : 0.f;
      uint16_t* dst = p.out + (static_cast<int64_t>(pair) * g + 2 * c) * D + D / 8 * r;
#pragma unroll
      for (int k = 0; k < KW; ++k) {
        if (2 * c < g)
          *reinterpret_cast<uint32_t*>(dst + 2 * k) = pack_bf16(o[k][0] * i0, o[k][2] * i0);
        if (2 * c + 1 < g)
          *reinterpret_cast<uint32_t*>(dst + D + 2 * k) = pack_bf16(o[k][1] * i1, o[k][3] * i1);
      }
    } else {
      float* dst = p.slots + static_cast<int64_t>(me) * 2 * G::kSlot;
      if (2 * c < g) {
#pragma unroll
        for (int k = 0; k < KW; ++k)
          reinterpret_cast<float4*>(dst)[k * 32 + lane] =
              make_float4(o[k][0], o[k][1], o[k][2], o[k][3]);
      }
      if (lane < 4) {
        *reinterpret_cast<float2*>(dst + 8 * D + 2 * c) = make_float2(log2_max(m0, f0), log2_max(m1, f1));
        *reinterpret_cast<float2*>(dst + 8 * D + 8 + 2 * c) = make_float2(l0, l1);
      }
    }
    fresh = true;
    if (done + 1 < mine) {
      do {
        ++pair;
        units = (blocks_of(LIST ? pair : pair / Hk) + UB - 1) / UB;
      } while (units == 0);
      seg = min(units, mine - done - 1);
      alone = seg == units;
    }
  }
  if (done < mine && lane == 0) {
    // a wait ran out: what is in flight has to land before the CTA's memory goes
    const int nk = min(mine, done + NST + (v_late ? 1 : 0));
    const int nv = min(mine, done + NST - (v_late ? 0 : 1));
    for (int i = max(done, nk - NST); i < nk; ++i)
      (void)mbar_wait(&my_k[i % NST], (i / NST) & 1, p.err);
    for (int i = max(done, nv - NST); i < nv; ++i)
      (void)mbar_wait(&my_v[i % NST], (i / NST) & 1, p.err);
  }
  // ---- what the warps' shares end with, unless a warp has written it: warps of
  // one pair are neighbours; their states are summed in their order
  const bool open = mine > 0 && !fresh;
  if (open) sum_rows();
  if (lane < 4) {
    ends_m[warp * 8 + 2 * c] = log2_max(m0, f0);
    ends_m[warp * 8 + 2 * c + 1] = log2_max(m1, f1);
    ends_l[warp * 8 + 2 * c] = l0;
    ends_l[warp * 8 + 2 * c + 1] = l1;
  }
  if (lane == 0) ends_pair[warp] = open ? pair : -1 - warp;
  __syncthreads();  // every warp's copies have landed and are read: the rings are free
  float4* ends_o = reinterpret_cast<float4*>(smem_raw + G::kRingAt);  // [W][KW][32]
  if (open) {
    float t0 = -INFINITY, t1 = -INFINITY;
#pragma unroll
    for (int w = 0; w < W; ++w) {
      if (ends_pair[w] != pair) continue;
      t0 = fmaxf(t0, ends_m[w * 8 + 2 * c]);
      t1 = fmaxf(t1, ends_m[w * 8 + 2 * c + 1]);
    }
    const float a0 = m0 == -INFINITY ? 0.f : fast_exp2(m0 * f0 - t0);
    const float a1 = m1 == -INFINITY ? 0.f : fast_exp2(m1 * f1 - t1);
#pragma unroll
    for (int k = 0; k < KW; ++k)
      ends_o[(warp * KW + k) * 32 + lane] =
          make_float4(o[k][0] * a0, o[k][1] * a1, o[k][2] * a0, o[k][3] * a1);
  }
  __syncthreads();
#pragma unroll 1
  for (int w = 0; w < W; ++w) {
    const int of = ends_pair[w];
    if (of < 0 || (w > 0 && ends_pair[w - 1] == of)) continue;  // not the first that has it
    int last = w;
    while (last + 1 < W && ends_pair[last + 1] == of) ++last;
    float* dst = p.slots + (static_cast<int64_t>(blockIdx.x * W + w) * 2 + 1) * G::kSlot;
    if (2 * c < g) {
      for (int k = warp; k < KW; k += W) {
        float4 sum = ends_o[(w * KW + k) * 32 + lane];
        for (int x = w + 1; x <= last; ++x) {
          const float4 y = ends_o[(x * KW + k) * 32 + lane];
          sum.x += y.x;
          sum.y += y.y;
          sum.z += y.z;
          sum.w += y.w;
        }
        reinterpret_cast<float4*>(dst)[k * 32 + lane] = sum;
      }
    }
    if (threadIdx.x < 8) {
      const int j = threadIdx.x;
      float M = -INFINITY, L = 0.f;
      for (int x = w; x <= last; ++x) M = fmaxf(M, ends_m[x * 8 + j]);
      for (int x = w; x <= last; ++x) {
        const float m = ends_m[x * 8 + j];
        L = fmaf(ends_l[x * 8 + j], m == -INFINITY ? 0.f : fast_exp2(m - M), L);
      }
      dst[8 * D + j] = M;
      dst[8 * D + 8 + j] = L;
    }
  }
}

// The pairs that several warps had parts of: out = sum_i e_i O_i / sum_i e_i l_i with e_i
// = 2^(m_i - max m). A CTA of 16 warps has 16 / SPLIT of the slots' D/16 pieces of a
// pair, SPLIT warps to a piece: all pieces in one CTA where there are many pairs,
// one piece (SPLIT = 16) where few pairs have many parts.
constexpr int kMergeWarps = 16;

template <int D, int SPLIT, bool LIST>
__global__ void __launch_bounds__(kMergeWarps * 32)
    merge_fp4_kernel(uint16_t* __restrict__ out, const int32_t* __restrict__ first,
                     const float* __restrict__ slots, const float* __restrict__ v_scale,
                     int num_rows, int Hk, int g, int workers) {
  using G = Fp4Geom<D>;
  constexpr int U = 8;  // parts of a warp whose loads are in flight together
  extern __shared__ float weights[];  // [n][8], and the parts' sums [n][8]
  __shared__ float4 acc_sh[kMergeWarps][32];
  __shared__ float inv_sum[8];
  wait_prerequisite();
  const int pair = blockIdx.x;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int r = lane >> 2, c = lane & 3;
  const int piece = (blockIdx.y * kMergeWarps + warp) / SPLIT, split = warp % SPLIT;
  const int T = first[num_rows];
  int u, units;
  if (LIST) {
    u = first[pair];
    units = first[pair + 1] - u;
  } else {
    const int s = pair / Hk;
    u = first[s];
    units = (first[s + 1] - u) / Hk;
    u += pair % Hk * units;
  }
  uint16_t* dst = out + (static_cast<int64_t>(pair) * g + 2 * c) * D + D / 8 * r + 2 * piece;
  if (units == 0) {
    if (split == 0) {
      if (2 * c < g) *reinterpret_cast<uint32_t*>(dst) = 0u;
      if (2 * c + 1 < g) *reinterpret_cast<uint32_t*>(dst + D) = 0u;
    }
    return;
  }
  const int nw = min(workers, T);
  // the worker that has unit x: the last whose first one is not behind it
  auto worker_of = [&](int x) {
    return static_cast<int>((static_cast<int64_t>(x + 1) * nw - 1) / T);
  };
  const int w0 = worker_of(u), w1 = worker_of(u + units - 1);
  if (w0 == w1) return;  // written already
  // slot 1 of w0 and of the first warps of the CTAs behind it, as long as shares
  // end with this pair; then slot 0 of w1 if its share ends with another one
  const bool more = share_begin(w1 + 1, nw, T) > u + units;
  const int c0 = w0 / kFp4Warps, ends = (more ? w1 - 1 : w1) / kFp4Warps - c0 + 1;
  const int n = ends + (more ? 1 : 0);
  auto part = [&](int i) {
    const int64_t at = i == ends ? 2 * static_cast<int64_t>(w1)
                       : 2 * static_cast<int64_t>(i == 0 ? w0 : (c0 + i) * kFp4Warps) + 1;
    return slots + at * G::kSlot;
  };
  const bool live = 2 * c < g;
  auto piece_of = [&](int i) {
    return live && i < n ? reinterpret_cast<const float4*>(part(i))[piece * 32 + lane]
                         : make_float4(0.f, 0.f, 0.f, 0.f);
  };
  // the first parts are on their way while the weights are made
  float4 x[U];
#pragma unroll
  for (int k = 0; k < U; ++k) x[k] = piece_of(split + k * SPLIT);
  // weights[i][0..8): the maxima, then the weights; sums[i][8]
  float* sums = weights + 8 * n;
#pragma unroll 4
  for (int i = threadIdx.x; i < 16 * n; i += kMergeWarps * 32) {
    const float y = part(i / 16)[8 * D + i % 16];
    (i % 16 < 8 ? weights : sums)[i / 16 * 8 + i % 8] = y;
  }
  __syncthreads();
  if (warp < 8) {
    // query `warp`, lane i the parts i, i + 32, ..
    float M = -INFINITY;
    for (int i = lane; i < n; i += 32) M = fmaxf(M, weights[i * 8 + warp]);
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, off));
    float L = 0.f;
    for (int i = lane; i < n; i += 32) {
      const float m = weights[i * 8 + warp];
      const float e = m == -INFINITY ? 0.f : fast_exp2(m - M);
      weights[i * 8 + warp] = e;
      L = fmaf(e, sums[i * 8 + warp], L);
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) L += __shfl_xor_sync(0xffffffffu, L, off);
    if (lane == 0) inv_sum[warp] = L != 0.f ? v_scale[pair % Hk] / L : 0.f;
  }
  __syncthreads();
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int i0 = split; i0 < n; i0 += U * SPLIT) {
    if (i0 != split) {
#pragma unroll
      for (int k = 0; k < U; ++k) x[k] = piece_of(i0 + k * SPLIT);
    }
#pragma unroll
    for (int k = 0; k < U; ++k) {
      if (i0 + k * SPLIT >= n) continue;
      const float2 e = *reinterpret_cast<const float2*>(&weights[(i0 + k * SPLIT) * 8 + 2 * c]);
      acc.x = fmaf(e.x, x[k].x, acc.x);
      acc.y = fmaf(e.y, x[k].y, acc.y);
      acc.z = fmaf(e.x, x[k].z, acc.z);
      acc.w = fmaf(e.y, x[k].w, acc.w);
    }
  }
  if constexpr (SPLIT > 1) {
    acc_sh[warp][lane] = acc;
    __syncthreads();
    if (split != 0) return;
#pragma unroll
    for (int k = 1; k < SPLIT; ++k) {
      const float4 x = acc_sh[warp + k][lane];
      acc.x += x.x;
      acc.y += x.y;
      acc.z += x.z;
      acc.w += x.w;
    }
  }
  const float i0 = inv_sum[2 * c], i1 = inv_sum[2 * c + 1];
  if (2 * c < g) *reinterpret_cast<uint32_t*>(dst) = pack_bf16(acc.x * i0, acc.z * i0);
  if (2 * c + 1 < g) *reinterpret_cast<uint32_t*>(dst + D) = pack_bf16(acc.y * i1, acc.w * i1);
}

// CTAs of a launch over at most `bound` units: residents of 152 SMs, no more
// than one to a unit.
static int fp4_ctas(int64_t bound) {
  return static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(bound, kFp4MaxCtas)));
}

// Units of all pairs at most.
static int64_t fp4_units(const pkv_cache_desc& cache, int64_t pairs, int64_t blocks) {
  const int64_t ub = (cache.head_dim == 256 ? 32 : 64) / cache.block_size;
  return pairs * ((blocks + ub - 1) / ub);
}

size_t fp4_workspace_bytes(const pkv_cache_desc& cache, int num_seqs, int64_t blocks,
                           bool listed) {
  const int64_t pairs = static_cast<int64_t>(num_seqs) * cache.num_kv_heads;
  const int64_t rows = listed ? pairs : num_seqs;
  const int64_t workers =
      static_cast<int64_t>(fp4_ctas(fp4_units(cache, pairs, blocks))) * kFp4Warps;
  // first units (padded to 16 bytes), then the slots
  return static_cast<size_t>((rows + 1 + 3) / 4 * 16 +
                             workers * 2 * (8 * cache.head_dim + 16) * 4);
}

template <int D, int BS, bool LIST>
static int launch_fp4(Fp4Params p, int64_t bound, void* workspace, cudaStream_t st) {
  using G = Fp4Geom<D>;
  const int ctas = fp4_ctas(bound);
  const int rows = LIST ? p.num_seqs * p.num_kv_heads : p.num_seqs;
  const int pairs = p.num_seqs * p.num_kv_heads;
  p.workers = ctas * kFp4Warps;
  p.first = static_cast<int32_t*>(workspace);
  p.slots = reinterpret_cast<float*>(p.first + (rows + 1 + 3) / 4 * 4);
  static DeviceFlags done, done_merge;
  auto kern = decode_fp4_kernel<D, BS, LIST>;
  int rc = ensure_smem(kern, G::kSmem, done);
  if (rc != PKV_OK) return rc;
  rc = launch_dependent(kern, dim3(ctas), dim3(G::kThreads), G::kSmem, st, p);
  if (rc != PKV_OK) return rc;
  // a pair has at most a part of every CTA and one more
  const size_t smem = static_cast<size_t>(ctas + 1) * 16 * sizeof(float);
  constexpr size_t kMaxSmem = static_cast<size_t>(kFp4MaxCtas + 1) * 16 * sizeof(float);
  if (pairs < 152) {
    auto wide = merge_fp4_kernel<D, kMergeWarps, LIST>;
    static DeviceFlags done_wide;
    rc = ensure_smem(wide, kMaxSmem, done_wide);
    if (rc != PKV_OK) return rc;
    return launch_dependent(wide, dim3(pairs, D / 16), dim3(kMergeWarps * 32), smem, st, p.out,
                            static_cast<const int32_t*>(p.first),
                            static_cast<const float*>(p.slots), p.v_scale, rows, p.num_kv_heads,
                            p.group, p.workers);
  }
  auto merge = merge_fp4_kernel<D, kMergeWarps * 16 / D, LIST>;
  rc = ensure_smem(merge, kMaxSmem, done_merge);
  if (rc != PKV_OK) return rc;
  return launch_dependent(merge, dim3(pairs), dim3(kMergeWarps * 32), smem, st, p.out,
                          static_cast<const int32_t*>(p.first),
                          static_cast<const float*>(p.slots), p.v_scale, rows, p.num_kv_heads,
                          p.group, p.workers);
}

int launch_decode_fp4(const DecodeParams& d, const pkv_cache_desc& cache, int num_seqs,
                      int max_context, void* workspace, cudaStream_t st) {
  Fp4Params p{};
  p.q = d.q;
  p.k_cache = d.k_cache;
  p.v_cache = d.v_cache;
  p.k_scale = d.k_scale;
  p.v_scale = d.v_scale;
  p.block_tables = d.block_tables;
  p.context_lens = d.context_lens;
  p.list = d.list;
  p.counts = d.counts;
  p.out = d.out;
  p.err = d.err;
  p.num_seqs = num_seqs;
  p.num_blocks = d.num_blocks;
  p.num_kv_heads = d.num_kv_heads;
  p.group = d.group;
  p.max_blocks_per_seq = d.max_blocks_per_seq;
  p.max_context = max_context;
  p.max_selected = d.max_selected;
  p.qscale = d.qscale;
  const bool listed = d.list != nullptr;
  const int64_t blocks = listed ? d.max_selected
                                : (static_cast<int64_t>(max_context) + cache.block_size - 1) /
                                      cache.block_size;
  const int64_t pairs = static_cast<int64_t>(num_seqs) * cache.num_kv_heads;
  const int64_t bound = fp4_units(cache, pairs, blocks);
  if (bound > INT32_MAX ||
      static_cast<int64_t>(cache.num_blocks) * cache.num_kv_heads > INT32_MAX)
    return PKV_ERR_UNSUPPORTED;
  auto go = [&](auto one, auto two) { return cache.block_size == 16 ? one() : two(); };
  if (listed) {
    if (cache.head_dim == 256)
      return go([&] { return launch_fp4<256, 16, true>(p, bound, workspace, st); },
                [&] { return launch_fp4<256, 32, true>(p, bound, workspace, st); });
    return go([&] { return launch_fp4<128, 16, true>(p, bound, workspace, st); },
              [&] { return launch_fp4<128, 32, true>(p, bound, workspace, st); });
  }
  if (cache.head_dim == 256)
    return go([&] { return launch_fp4<256, 16, false>(p, bound, workspace, st); },
              [&] { return launch_fp4<256, 32, false>(p, bound, workspace, st); });
  return go([&] { return launch_fp4<128, 16, false>(p, bound, workspace, st); },
            [&] { return launch_fp4<128, 32, false>(p, bound, workspace, st); });
}

}  // namespace pkv

extern "C" size_t pkv_fp4_workspace_bytes(pkv_cache_desc cache, int num_seqs, int max_context) {
  using namespace pkv;
  if (check_cache_desc(cache, true) != PKV_OK || cache.dtype != PKV_DTYPE_FP4_E2M1 ||
      num_seqs <= 0 || max_context < 0)
    return 0;
  return fp4_workspace_bytes(
      cache, num_seqs, (static_cast<int64_t>(max_context) + cache.block_size - 1) / cache.block_size,
      false);
}

extern "C" int pkv_paged_attention_fp4(void* out, const void* q, const void* k_cache,
                                       const void* v_cache, pkv_cache_desc cache,
                                       const float* k_scale, const float* v_scale,
                                       const int32_t* block_tables, int max_blocks_per_seq,
                                       const int32_t* context_lens, int num_seqs, int num_heads,
                                       int max_context, float scale, void* workspace,
                                       size_t workspace_bytes, void* stream) {
  using namespace pkv;
  if (cache.dtype != PKV_DTYPE_FP4_E2M1) return PKV_ERR_INVALID_ARG;
  int g = 0;
  const int rc = check_attention(cache, out, q, k_cache, v_cache, k_scale, v_scale, block_tables,
                                 max_blocks_per_seq, context_lens, num_seqs, num_heads,
                                 max_context, scale, &g, true);
  if (rc != PKV_OK) return rc;
  if (num_seqs == 0) return PKV_OK;
  const size_t q_bytes = static_cast<size_t>(num_seqs) * num_heads * cache.head_dim * 2;
  if (overlap(out, q_bytes, q, q_bytes)) return PKV_ERR_INVALID_ARG;
  if (!workspace || !aligned16(workspace) ||
      workspace_bytes < pkv_fp4_workspace_bytes(cache, num_seqs, max_context))
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
  return launch_decode_fp4(p, cache, num_seqs, max_context, workspace,
                           static_cast<cudaStream_t>(stream));
}

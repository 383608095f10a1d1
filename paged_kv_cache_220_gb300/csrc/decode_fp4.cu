// Attention of one query token per sequence over a 4-bit cache: over the whole
// context (paged_attention_decode) or over listed blocks (paged_attention_sparse).
//
// Every warp works alone on units of 64 tokens (32 at D = 256), the CTA's in turn:
// one lane keeps a ring of their K and V in flight with bulk copies, one per block
// and pool, a page's codes and scales being one contiguous run; the warps of a
// CTA, and the CTAs of a cluster, are merged once at the end. Nothing is
// exchanged per unit.
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
// - A logit that is NaN passes the maxima by and reaches the sums: a query whose logits
//   are all NaN has the maximum -inf of one without a token, a sum of NaN in the place
//   of 0, and every merge multiplies and adds them as any other state's.
//
// Bound by HBM in whole waves (8 x 131072 tokens, 4 heads, d = 256 186 us with the merge,
// 6.5 TB/s of codes and scales, 96 % of the copy rate); 64 x 8192 112 us (5.4 TB/s):
// 2.25 waves, whose starts, ends and uneven last part three warps to a scheduler
// (168 registers, 55 % of the issue slots) do not hide. About 1040 instructions to a
// warp's unit, 750 of them conversions, products by scales and the mma.
#include <algorithm>

#include "common.cuh"
#include "decode_params.h"
#include "fp4.cuh"
#include "host_util.h"
#include "tc_common.cuh"

namespace pkv {

constexpr float kUpFp4 = 15.f;  // log2 of the factor on the weights

template <int D, int TU, int W, int NST>
struct Fp4Geom {
  static constexpr int kBytes = TU * D / 16 * 9;  // K (or V) of a unit of TU tokens
  static constexpr int kStage = 2 * kBytes;
  static constexpr int kRing = W * NST * kStage;
  // merge: the warps' O, padded against bank conflicts, then the CTA's
  static constexpr int kRow8 = D / 8 + 4;        // channels of one fragment row
  static constexpr int kRowQ = 8 * kRow8 + 8;    // of one query
  static constexpr int kMerge = (W * 8 * kRowQ + 8 * D) * 4;
  static constexpr int kHead = (W * NST * 16 + W * 64 + 96 + 127) / 128 * 128;  // barriers, maxima and sums
  static constexpr int kSmem = kHead + (kRing > kMerge ? kRing : kMerge);
  static constexpr int kThreads = W * 32;
};

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

// True in one lane of a converged warp. (The compiler knows that it is one, and takes a
// copy's addresses from it without a loop over lanes: 64 x 8192, d = 256 115.1 -> 112.3 us
// with it in the place of lane == 0, 8 x 131072, d = 128 207.9 -> 198.8)
__device__ __forceinline__ bool elected() {
  uint32_t e;
  asm volatile(
      "{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(e));
  return e != 0;
}

// 16 bytes of the cluster's CTA `rank`, at this CTA's address a
__device__ __forceinline__ float4 ld_dsmem4(uint32_t a, int rank) {
  uint32_t at;
  float4 v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(a), "r"(rank));
  asm volatile("ld.shared::cluster.v4.f32 {%0,%1,%2,%3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(at));
  return v;
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
// D += A B as mma_f16, free to move between the others' instructions.
__device__ __forceinline__ void mma_f16_free(float* d, uint32_t a0, uint32_t a1, uint32_t a2,
                                             uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// Two E4M3 codes (the low or the high 16 bits of w) as f16x2
__device__ __forceinline__ __half2 scales_of(uint32_t w, int hi) {
  const uint32_t d = e4m3x2_f16x2(w, hi);
  return *reinterpret_cast<const __half2*>(&d);
}

// The bits of a where mask has ones, those of b elsewhere (written as an expression it
// became two instructions)
__device__ __forceinline__ uint32_t bits_of(uint32_t mask, uint32_t a, uint32_t b) {
  uint32_t d;
  asm("lop3.b32 %0, %1, %2, %3, 0xCA;" : "=r"(d) : "r"(mask), "r"(a), "r"(b));
  return d;
}

template <int D, int BS, bool LIST, int TU, int W, int NST, int CTAS>
__global__ void __launch_bounds__(W * 32, CTAS) decode_fp4_kernel(const DecodeParams p) {
  using G = Fp4Geom<D, TU, W, NST>;
  constexpr int UB = TU / BS;             // blocks of a unit
  constexpr int NT = TU / 16;             // 16-token tiles of a unit
  constexpr int PAGE = BS * D / 16 * 9;   // bytes of a block's page
  constexpr int KW = D / 16;              // k-steps of S, row tiles of O
  extern __shared__ __align__(128) uint8_t smem_raw[];
  uint64_t* kfull = reinterpret_cast<uint64_t*>(smem_raw);       // [W][NST]
  uint64_t* vfull = kfull + W * NST;                             // [W][NST]
  float* sm_m = reinterpret_cast<float*>(vfull + W * NST);       // [W][8]
  float* sm_l = sm_m + W * 8;                                    // [W][8]
  uint8_t* ring_p = smem_raw + G::kHead;

  const int part = blockIdx.x;
  const int h = blockIdx.y;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int r = lane >> 2, c = lane & 3;
  uint64_t* my_k = kfull + warp * NST;
  uint64_t* my_v = vfull + warp * NST;
  if (lane == 0) {
    for (int i = 0; i < NST; ++i) {
      mbar_init(&my_k[i], 1);
      mbar_init(&my_v[i], 1);
    }
    fence_mbar_init();
  }
  __syncwarp();
  wait_prerequisite();
  int s = static_cast<int>(blockIdx.z);
  if (p.seq_order != nullptr) {
    s = p.seq_order[blockIdx.z];
    if (s < 0 || s >= static_cast<int>(gridDim.z)) {
      if (threadIdx.x == 0 && part == 0 && h == 0) report_error(p.err, PKV_DEVERR_ORDER);
      return;
    }
  }
  const int g = p.group;
  int ctx = p.context_lens[s];
  const int cap = p.max_blocks_per_seq * BS;
  if (ctx < 0 || ctx > cap) {
    if (threadIdx.x == 0 && part == 0 && h == 0) report_error(p.err, PKV_DEVERR_CONTEXT);
    ctx = ctx < 0 ? 0 : cap;
  }
  // the run [b0, b1) of the context's blocks, or of the list's entries
  const int nctx = (ctx + BS - 1) / BS;
  int b0 = 0, b1 = nctx;
  const int32_t* list = nullptr;
  if constexpr (LIST) {
    const int64_t row = static_cast<int64_t>(s) * p.num_kv_heads + h;
    list = p.list + row * p.max_selected;
    b1 = p.counts[row];
    if (b1 < 0 || b1 > p.max_selected) {
      if (threadIdx.x == 0 && part == 0) report_error(p.err, PKV_DEVERR_SELECT);
      b1 = b1 < 0 ? 0 : p.max_selected;
    }
  }
  if (p.partition_blocks > 0) {
    b0 = part * p.partition_blocks;
    if (b0 >= b1) return;  // a partition past the end: nothing to store
    b1 = min(b1, b0 + p.partition_blocks);
  } else if (p.cluster > 1) {
    const int share = (b1 + p.cluster - 1) / p.cluster;
    b0 = min(b1, part * share);
    b1 = min(b1, b0 + share);
  }
  const int units = (b1 - b0 + UB - 1) / UB;
  const int mine = units > warp ? (units - warp + W - 1) / W : 0;  // units of this warp
  const int32_t* table = p.block_tables + static_cast<int64_t>(s) * p.max_blocks_per_seq;

  // ---- lanes look up the blocks of the warp's next 32 / UB units together: lane l
  // block l % UB of unit l / UB. pb: the block, -1 if there is none; vis: how
  // many tokens of each of the unit's blocks are visible, a byte each
  constexpr int kBatch = 32 / UB;
  constexpr uint32_t kWhole = BS * (UB == 1 ? 1u : UB == 2 ? 0x0101u : 0x01010101u);
  int id_next = -1;
  uint32_t vis_next = 0;
  auto ask = [&](int batch) {
    const int i = batch * kBatch + lane / UB;
    const int v = b0 + UB * (warp + W * i) + lane % UB;
    id_next = -1;
    vis_next = 0;
    if (i >= mine || v >= b1) return;
    const int b = LIST ? list[v] : v;
    if (LIST && (b < 0 || b >= nctx)) {
      report_error(p.err, PKV_DEVERR_SELECT);
      return;
    }
    id_next = table[b];
    vis_next = static_cast<uint32_t>(min(BS, ctx - b * BS)) << (8 * (lane % UB));
  };
  int pb_now = -1;
  uint32_t vis_now = 0;
  auto take = [&] {
    pb_now = -1;
    vis_now = 0;
    if (vis_next != 0) {  // there is a block
      if (id_next < 0 || id_next >= p.num_blocks) {
        report_error(p.err, PKV_DEVERR_BLOCK_ID);
      } else {
        pb_now = id_next;
        vis_now = vis_next;
      }
    }
    __syncwarp();
#pragma unroll
    for (int off = 1; off < UB; off <<= 1)
      vis_now |= __shfl_xor_sync(0xffffffffu, vis_now, off);
  };
  ask(0);
  take();
  const uint32_t my_ring = smem_addr(ring_p) + warp * NST * G::kStage;
  uint64_t policy;
  asm volatile("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(policy));
  const uint32_t block_bytes = p.num_kv_heads * PAGE;
  const uint8_t* k_head = p.k_cache + h * PAGE;
  const uint8_t* v_head = p.v_cache + h * PAGE;
  // the unit whose K was loaded last (its V comes behind it)
  int ids[UB];
  uint32_t vis[NST] = {};  // of the units in the ring, the oldest first
  auto load = [&](uint32_t dst, const uint8_t* head, uint64_t* bar) {
    if (!elected()) return;
    uint32_t bytes = 0;
#pragma unroll
    for (int b = 0; b < UB; ++b) bytes += ids[b] >= 0 ? PAGE : 0;
    mbar_arrive_expect_tx(bar, bytes);
#pragma unroll
    for (int b = 0; b < UB; ++b)
      if (ids[b] >= 0)
        bulk_load(dst + b * PAGE, head + static_cast<uint64_t>(ids[b]) * block_bytes, PAGE, bar,
                  policy);
  };
  // K of unit i into slot st
  auto load_k = [&](int i, int st) {
    const int at = i % kBatch;
    if (at == 0 && i > 0) {
      take();
      ask(i / kBatch + 1);
    }
#pragma unroll
    for (int b = 0; b < UB; ++b) ids[b] = __shfl_sync(0xffffffffu, pb_now, at * UB + b);
    vis[NST - 1] = __shfl_sync(0xffffffffu, vis_now, at * UB);
    load(my_ring + st * G::kStage, k_head, &my_k[st]);
  };
  auto load_v = [&](int st) { load(my_ring + st * G::kStage + G::kBytes, v_head, &my_v[st]); };
#pragma unroll
  for (int i = 0; i < NST; ++i) {
#pragma unroll
    for (int k = 0; k + 1 < NST; ++k) vis[k] = vis[k + 1];
    if (i < mine) load_k(i, i);
    if (i < mine) load_v(i);
    // the second batch's ids behind the first unit's loads
    if (i == 0) ask(1);
  }

  // ---- Q^T fragments: lane (n = r, c) has channels D/4 c + 4 j + {0, 1} and {2, 3}
  // of query n for k-step j, as f16, in units of a power of two of its row, with
  // the logit factor's sign
  uint32_t bq[KW][2];
  float f0, f1;  // logit factors of queries 2c, 2c + 1 (base 2), not negative
  {
    const uint2* qrow = reinterpret_cast<const uint2*>(
        p.q + (static_cast<int64_t>(s) * p.num_heads + h * g + r) * D + D / 4 * c);
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
    const float qs = p.qscale * p.k_scale[h];
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
  // running maxima of the products before their factor, sums, outputs
  float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.f, l1 = 0.f;
  float o[KW][4];
#pragma unroll
  for (int k = 0; k < KW; ++k) o[k][0] = o[k][1] = o[k][2] = o[k][3] = 0.f;
  // token of the unit that row x of tile t stands for
  auto token = [](int t, int x) {
    return 16 * t + (D == 256 ? x : ((x & 7) >> 1) * 4 + (x & 1) + (x >= 8 ? 2 : 0));
  };

  int done = 0;          // units done
  bool v_late = false;  // the wait that ran out, if one did, was V's
  int st = 0;
  uint32_t parity = 0;
  for (; done < mine; ++done) {
    if (!__all_sync(0xffffffffu, mbar_wait(&my_k[st], parity, p.err))) break;
    const uint32_t kp = my_ring + st * G::kStage, vp = kp + G::kBytes;
    const uint32_t seen = vis[0];
    const bool whole = seen == kWhole;
    auto sees = [&](int t) { return t % BS < static_cast<int>(seen >> (8 * (t / BS)) & 0xFFu); };

    // ---- S^T = K Q^T: two tiles at a time, word by word, two sums each, so that four
    // chains of products are under way
    float sc[NT][4];
#pragma unroll
    for (int t0 = 0; t0 < NT; t0 += 2) {
      float u[2][4], v[2][4];
      uint32_t sa[2], sb[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int ta = token(t0 + i, r), tb = token(t0 + i, r + 8);
        u[i][0] = u[i][1] = u[i][2] = u[i][3] = 0.f;
        v[i][0] = v[i][1] = v[i][2] = v[i][3] = 0.f;
        if constexpr (D == 256) {
          sa[i] = lds32(kp + ta * kFp4Line + 128 + 4 * c);
          sb[i] = lds32(kp + tb * kFp4Line + 128 + 4 * c);
        } else {
          sa[i] = lds16(kp + fp4_scales_at<D>(ta) + 2 * c);
          sb[i] = lds16(kp + fp4_scales_at<D>(tb) + 2 * c);
        }
      }
#pragma unroll
      for (int y = 0; y < D / 128; ++y) {  // 16 bytes of codes of a lane and row
        uint32_t wa[2][4], wb[2][4];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int ta = token(t0 + i, r), tb = token(t0 + i, r + 8);
          const uint4 a = lds128(kp + fp4_codes_at<D>(ta) + D / 8 * c + 16 * y);
          const uint4 b = lds128(kp + fp4_codes_at<D>(tb) + D / 8 * c + 16 * y);
          wa[i][0] = a.x, wa[i][1] = a.y, wa[i][2] = a.z, wa[i][3] = a.w;
          wb[i][0] = b.x, wb[i][1] = b.y, wb[i][2] = b.z, wb[i][3] = b.w;
        }
#pragma unroll
        for (int x = 0; x < 4; ++x) {
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            // two words (16 channels) to a scale
            const __half2 pa = scales_of(sa[i], y), pb = scales_of(sb[i], y);
            const __half2 fa = x / 2 ? __high2half2(pa) : __low2half2(pa);
            const __half2 fb = x / 2 ? __high2half2(pb) : __low2half2(pb);
            uint32_t a[4], b[4];
            e2m1x8_f16x2(wa[i][x], a);
            e2m1x8_f16x2(wb[i][x], b);
            const int k = 8 * y + 2 * x;
            mma_f16_free(u[i], mul_f16x2(a[0], fa), mul_f16x2(b[0], fb), mul_f16x2(a[1], fa),
                         mul_f16x2(b[1], fb), bq[k][0], bq[k][1]);
            mma_f16_free(v[i], mul_f16x2(a[2], fa), mul_f16x2(b[2], fb), mul_f16x2(a[3], fa),
                         mul_f16x2(b[3], fb), bq[k + 1][0], bq[k + 1][1]);
          }
        }
      }
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int k = 0; k < 4; ++k) sc[t0 + i][k] = u[i][k] + v[i][k];
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
    // every lane's products have met in the shuffles, so every lane has read this
    // unit's K: its slot can take the next one
    __syncwarp();
#pragma unroll
    for (int k = 0; k + 1 < NST; ++k) vis[k] = vis[k + 1];
    if (done + NST < mine) load_k(done + NST, st);
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
        e2m1x8_f16x2(bits_of(kLow, w[0][x], w[1][x] << 4), ev01);
        e2m1x8_f16x2(bits_of(kLow, w[0][x] >> 4, w[1][x]), od01);
        e2m1x8_f16x2(bits_of(kLow, w[2][x], w[3][x] << 4), ev23);
        e2m1x8_f16x2(bits_of(kLow, w[2][x] >> 4, w[3][x]), od23);
#pragma unroll
        for (int y = 0; y < 4; ++y)
          mma_f16(o[4 * x + y], mul_f16x2(ev01[y], s01), mul_f16x2(od01[y], s01),
                  mul_f16x2(ev23[y], s23), mul_f16x2(od23[y], s23), q0, q1);
      }
    }
    // every lane has issued its products, whose operands its V had to be: the slot
    // can take the next one
    __syncwarp();
    if (done + NST < mine) load_v(st);
    if (++st == NST) {
      st = 0;
      parity ^= 1;
    }
  }
  if (done < mine && lane == 0) {
    // a wait ran out: what is in flight has to land before the ring is used again
    const int nk = min(mine, done + NST + (v_late ? 1 : 0));
    const int nv = min(mine, done + NST);
    for (int i = max(done, nk - NST); i < nk; ++i)
      (void)mbar_wait(&my_k[i % NST], (i / NST) & 1, p.err);
    for (int i = max(done, nv - NST); i < nv; ++i)
      (void)mbar_wait(&my_v[i % NST], (i / NST) & 1, p.err);
  }
  // the maxima as base-2 logits
  m0 = m0 == -INFINITY ? m0 : m0 * f0;
  m1 = m1 == -INFINITY ? m1 : m1 * f1;
#pragma unroll
  for (int off = 4; off < 32; off <<= 1) {
    l0 += __shfl_xor_sync(0xffffffffu, l0, off);
    l1 += __shfl_xor_sync(0xffffffffu, l1, off);
  }
  if (lane < 4) {
    sm_m[warp * 8 + 2 * c] = m0;
    sm_m[warp * 8 + 2 * c + 1] = m1;
    sm_l[warp * 8 + 2 * c] = l0;
    sm_l[warp * 8 + 2 * c + 1] = l1;
  }
  __syncthreads();
  // the merge launched next may be scheduled; it waits for this grid's end
  allow_dependents();

  // ---- the warps' states become the CTA's: sums over the warps in their order
  float* os = reinterpret_cast<float*>(ring_p);       // [W][8][kRowQ]
  float* cs_o = os + W * 8 * G::kRowQ;                // [8][D]
  float* cs_m = sm_m + 2 * W * 8;                     // [8]
  float* cs_l = cs_m + 8;                             // [8]
  float* cs_f = cs_l + 8;                             // [8] v's scale over the sum
  const float vsc = p.v_scale[h];
  if (threadIdx.x < 8) {
    const int j = threadIdx.x;
    float M = sm_m[j], L = 0.f;
#pragma unroll
    for (int w = 1; w < W; ++w) M = fmaxf(M, sm_m[w * 8 + j]);
    const float ref = M == -INFINITY ? 0.f : M;
#pragma unroll
    for (int w = 0; w < W; ++w) L = fmaf(sm_l[w * 8 + j], fast_exp2(sm_m[w * 8 + j] - ref), L);
    cs_m[j] = M;
    cs_l[j] = L;
    cs_f[j] = L != 0.f ? vsc / L : 0.f;
  }
  {
    float t0 = sm_m[2 * c], t1 = sm_m[2 * c + 1];
#pragma unroll
    for (int w = 1; w < W; ++w) {
      t0 = fmaxf(t0, sm_m[w * 8 + 2 * c]);
      t1 = fmaxf(t1, sm_m[w * 8 + 2 * c + 1]);
    }
    const float a0 = m0 == -INFINITY ? 0.f : fast_exp2(m0 - t0);
    const float a1 = m1 == -INFINITY ? 0.f : fast_exp2(m1 - t1);
    float* d0 = os + (warp * 8 + 2 * c) * G::kRowQ + r * G::kRow8;
    float* d1 = d0 + G::kRowQ;
#pragma unroll
    for (int k = 0; k < KW; ++k) {
      *reinterpret_cast<float2*>(d0 + 2 * k) = make_float2(o[k][0] * a0, o[k][2] * a0);
      *reinterpret_cast<float2*>(d1 + 2 * k) = make_float2(o[k][1] * a1, o[k][3] * a1);
    }
  }
  __syncthreads();
  const int64_t hq0 = static_cast<int64_t>(s) * p.num_heads + h * g;
#pragma unroll 2
  for (int idx = threadIdx.x; idx < g * (D / 4); idx += G::kThreads) {
    const int j = idx / (D / 4), col = idx % (D / 4) * 4;
    const int at = j * G::kRowQ + col / (D / 8) * G::kRow8 + col % (D / 8);
    float4 sum = *reinterpret_cast<const float4*>(os + at);
#pragma unroll
    for (int w = 1; w < W; ++w) {
      const float4 x = *reinterpret_cast<const float4*>(os + w * 8 * G::kRowQ + at);
      sum.x += x.x;
      sum.y += x.y;
      sum.z += x.z;
      sum.w += x.w;
    }
    if (p.cluster > 1) {
      *reinterpret_cast<float4*>(cs_o + j * D + col) = sum;
      continue;
    }
    const float f = cs_f[j];
    sum.x *= f;
    sum.y *= f;
    sum.z *= f;
    sum.w *= f;
    if (p.partition_blocks == 0) {
      *reinterpret_cast<uint2*>(p.out + (hq0 + j) * D + col) =
          make_uint2(pack_bf16(sum.x, sum.y), pack_bf16(sum.z, sum.w));
    } else {
      const int64_t slot = (hq0 + j) * p.np_max + part;
      *reinterpret_cast<float4*>(p.tmp_out + slot * D + col) = sum;
      if (col == 0) {
        // the sums have the weights' factor; the merge only compares them
        p.max_logits[slot] = cs_m[j] * kLn2Tc;
        p.exp_sums[slot] = cs_l[j];
      }
    }
  }
  if (p.cluster <= 1) return;
  // ---- the CTAs of the cluster: rank k has channels [k D/C, (k + 1) D/C) of the
  // result, from every rank's state in rank order
  cluster_sync_all();
  const int C = p.cluster, SL = D / C;  // up to 8 ranks
  const uint32_t o_addr = smem_addr(cs_o), m_addr = smem_addr(cs_m), l_addr = smem_addr(cs_l);
  for (int idx = threadIdx.x; idx < g * SL / 4; idx += G::kThreads) {
    const int j = idx / (SL / 4), col = part * SL + idx % (SL / 4) * 4;
    // all ranks' loads in flight together; -inf and zeros for ranks that there are not
    float m[8], l[8];
    float4 x[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      m[k] = k < C ? ld_dsmem(m_addr + 4 * j, k) : -INFINITY;
      l[k] = k < C ? ld_dsmem(l_addr + 4 * j, k) : 0.f;
      x[k] = k < C ? ld_dsmem4(o_addr + 4 * (j * D + col), k) : make_float4(0.f, 0.f, 0.f, 0.f);
    }
    float M = m[0], L = 0.f;
#pragma unroll
    for (int k = 1; k < 8; ++k) M = fmaxf(M, m[k]);
    const float ref = M == -INFINITY ? 0.f : M;
    float4 O = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const float a = fast_exp2(m[k] - ref);
      L = fmaf(l[k], a, L);
      O.x = fmaf(x[k].x, a, O.x);
      O.y = fmaf(x[k].y, a, O.y);
      O.z = fmaf(x[k].z, a, O.z);
      O.w = fmaf(x[k].w, a, O.w);
    }
    const bool any = L != 0.f;
    *reinterpret_cast<uint2*>(p.out + (hq0 + j) * D + col) = make_uint2(
        pack_bf16(any ? O.x / L * vsc : 0.f, any ? O.y / L * vsc : 0.f),
        pack_bf16(any ? O.z / L * vsc : 0.f, any ? O.w / L * vsc : 0.f));
  }
  cluster_sync_all();  // this CTA's state lives until every rank has read it
}

// 456 CTAs run at once on 152 SMs, and a CTA costs 5 to 6 us besides its units
// (start, first loads, merge), which the SM's other two hide in part. Figures are d =
// 256, "u units" are those of a pair, of 32 tokens.
// - One pass where a warp has four units or fewer, with a cluster of CTAs to a pair as long
//   as there is one CTA to an SM or less (32 pairs of 64 units: 11.8 us with 4 CTAs, 13.5
//   with 8, 12.3 in 8 partitions; 120 of 16: 11.4 with 1, 13.2 with 2), none up to 8 units
//   (100 pairs: 7.7, with two CTAs 9.3); and where the pairs fill half a wave by
//   themselves and have 64 units or fewer (256 pairs of 64: 36.6 us, 42.6 in 2 partitions).
//   Pairs that leave no room for two CTAs each get four if a warp then has two units or
//   fewer (96 of 17 units of 64 tokens, d = 128: 9.3 us, 11.6 in 2 partitions).
// - Else partitions: of 8 units up to two CTAs to an SM, of 16 up to a wave (64 pairs of 64:
//   16.9 us in 4, 18.7 in 7, 22 in 8; 160 of 32: 20.6 in 2, 29.4 in 7; 32 pairs of 131072
//   tokens: 186 us in 14, 207 in 56); 16 or fewer are made a multiple of the four warps.
// - Where whole partitions leave more than a quarter of a wave empty and the pairs are long,
//   somewhat over two waves, whose end is short (256 pairs of 256: 112 us in 4, 118 in 3,
//   117 in 8, 123 in one pass; 160 of 256: 82 in 7, 88 in 2, but 160 of 128: 52.6, 49.7),
//   in partitions of at most 2048 tokens, as contexts may differ (768 pairs of 16 to
//   16384 tokens, d = 128: 65 us, 70 in partitions of 4096; with the sequences longest
//   first 60 and 56. Ranking them in every CTA cost more than it gave from about 100
//   sequences on).
// A pass that the caller asks for has a cluster as long as that fits a wave (100 pairs of
// 256: 51 us with 4 CTAs, 93 with 1).
Fp4Split fp4_split(int64_t pairs, int64_t units, int unit) {
  constexpr int64_t kWave = 456, kSms = 152;
  if (pairs <= 0 || units <= 0) return {1, 0};
  auto cluster = [&](int64_t ctas) {
    int c = 1;
    while (c < 8 && kFp4Warps * c < units && 2 * c * pairs <= ctas) c <<= 1;
    return c;
  };
  const int c = units <= 2 * kFp4Warps ? 1 : cluster(kSms);
  if (units <= std::min(4 * kFp4Warps * c, 64) || (2 * pairs >= kWave && units <= 64))
    return {c, 0};
  const int wide = cluster(kWave);
  if (c == 1 && wide >= 4 && units <= 2 * kFp4Warps * wide) return {wide, 0};
  const int64_t one = kWave / pairs;
  int64_t np = std::max(std::min(units / 8, 2 * kSms / pairs), std::min(units / 16, one));
  if (one * pairs < kWave * 3 / 4 && one <= units / 16 && (units > 128 || one == 0))
    np = std::max((11 * kWave / 5 + pairs - 1) / pairs, (units * unit + 2047) / 2048);
  np = std::min<int64_t>(np, 8192);  // the merge takes 32767
  if (np <= 1) return {c, 0};
  int64_t per = (units + np - 1) / np;
  if (per <= 16) per = (per + kFp4Warps - 1) / kFp4Warps * kFp4Warps;
  return {wide, per};
}

template <int D, int BS, bool LIST>
static int launch_fp4(const DecodeParams& p_in, dim3 grid, cudaStream_t st) {
  constexpr int TU = fp4_unit(D), W = kFp4Warps, NST = 2, CTAS = 3;
  using G = Fp4Geom<D, TU, W, NST>;
  auto kern = decode_fp4_kernel<D, BS, LIST, TU, W, NST, CTAS>;
  static DeviceFlags done;
  int rc = ensure_smem(kern, G::kSmem, done);
  if (rc != PKV_OK) return rc;
  DecodeParams p = p_in;
  if (p.partition_blocks > 0 || p.cluster <= 1) {
    p.cluster = 1;
    return launch_dependent(kern, grid, dim3(G::kThreads), G::kSmem, st, p);
  }
  grid.x = p.cluster;
  // clusters of up to 8 CTAs are portable
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  cfg.gridDim = grid;
  cfg.blockDim = dim3(G::kThreads);
  cfg.dynamicSmemBytes = G::kSmem;
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = p.cluster;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  if (cudaLaunchKernelEx(&cfg, kern, p) != cudaSuccess) return PKV_ERR_CUDA;
  return launch_status();
}

int launch_decode_fp4(const DecodeParams& p, int head_dim, int block_size, dim3 grid,
                      cudaStream_t st) {
  if (p.list != nullptr) {
    if (head_dim == 256)
      return block_size == 16 ? launch_fp4<256, 16, true>(p, grid, st)
                              : launch_fp4<256, 32, true>(p, grid, st);
    return block_size == 16 ? launch_fp4<128, 16, true>(p, grid, st)
                            : launch_fp4<128, 32, true>(p, grid, st);
  }
  if (head_dim == 256)
    return block_size == 16 ? launch_fp4<256, 16, false>(p, grid, st)
                            : launch_fp4<256, 32, false>(p, grid, st);
  return block_size == 16 ? launch_fp4<128, 16, false>(p, grid, st)
                          : launch_fp4<128, 32, false>(p, grid, st);
}

}  // namespace pkv

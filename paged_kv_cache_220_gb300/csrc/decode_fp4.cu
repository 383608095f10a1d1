// Attention of one query token per sequence over a 4-bit cache: over the whole
// context (paged_attention_decode) or over listed blocks (paged_attention_sparse).
//
// Every warp works alone on units of 32 tokens (one block, or two of 16 tokens):
// lane 0 keeps a ring of their K and V in flight with bulk copies, one per block
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
#include <algorithm>

#include "common.cuh"
#include "decode_params.h"
#include "fp4.cuh"
#include "host_util.h"
#include "tc_common.cuh"

namespace pkv {

constexpr int kUnit = 32;               // tokens of a unit
constexpr int kNoToken = 0x7F000000;    // first "token" of a block that is not there
constexpr float kUpFp4 = 15.f;          // log2 of the factor on the weights

template <int D, int W, int NST>
struct Fp4Geom {
  static constexpr int kBytes = kUnit * D / 16 * 9;  // K (or V) of a unit
  static constexpr int kStage = 2 * kBytes;
  static constexpr int kRing = W * NST * kStage;
  // merge: the warps' O, padded against bank conflicts, then the CTA's
  static constexpr int kRow8 = D / 8 + 4;        // channels of one fragment row
  static constexpr int kRowQ = 8 * kRow8 + 8;    // of one query
  static constexpr int kMerge = (W * 8 * kRowQ + 8 * D) * 4;
  static constexpr int kHead = 1024;  // barriers, units' blocks, maxima and sums
  static constexpr int kSmem = kHead + (kRing > kMerge ? kRing : kMerge);
  static constexpr int kThreads = W * 32;
  static_assert(W * NST * (16 + 16) + W * 64 + 64 <= kHead, "head of the shared memory");
};

// One contiguous run of global memory into shared memory; evict-first in L2, a
// page is read once.
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes,
                                          uint64_t* bar) {
  uint64_t policy;
  asm volatile("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(policy));
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

__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
// (x.lo, x.lo) and (x.hi, x.hi)
__device__ __forceinline__ uint32_t dup_lo(uint32_t x) { return __byte_perm(x, 0, 0x1010); }
__device__ __forceinline__ uint32_t dup_hi(uint32_t x) { return __byte_perm(x, 0, 0x3232); }

template <int D, int BS, bool LIST, int W, int NST>
__global__ void __launch_bounds__(W * 32, (D == 256 ? 12 : 16) / W)
    decode_fp4_kernel(const DecodeParams p) {
  using G = Fp4Geom<D, W, NST>;
  constexpr int UB = kUnit / BS;          // blocks of a unit
  constexpr int PAGE = BS * D / 16 * 9;   // bytes of a block's page
  constexpr int KW = D / 16;              // k-steps of S, row tiles of O
  extern __shared__ __align__(128) uint8_t smem_raw[];
  uint64_t* kfull = reinterpret_cast<uint64_t*>(smem_raw);       // [W][NST]
  uint64_t* vfull = kfull + W * NST;                             // [W][NST]
  int4* meta = reinterpret_cast<int4*>(vfull + W * NST);         // [W][NST] block, first token; twice
  float* sm_m = reinterpret_cast<float*>(meta + W * NST);        // [W][8]
  float* sm_l = sm_m + W * 8;                                    // [W][8]
  uint8_t* ring_p = smem_raw + G::kHead;
  const uint32_t ring = smem_addr(ring_p);

  const int part = blockIdx.x;
  const int h = blockIdx.y;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int r = lane >> 2, c = lane & 3;
  if (lane == 0) {
    for (int i = 0; i < NST; ++i) {
      mbar_init(&kfull[warp * NST + i], 1);
      mbar_init(&vfull[warp * NST + i], 1);
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

  // ---- lanes look up the blocks of the warp's next 32 / UB units together
  constexpr int kBatch = 32 / UB;
  auto look_up = [&](int batch, int& pb, int& tok) {
    const int i = batch * kBatch + lane / UB;
    const int v = b0 + UB * (warp + W * i) + lane % UB;
    pb = -1;
    tok = kNoToken;
    if (i >= mine || v >= b1) return;
    const int b = LIST ? list[v] : v;
    if (LIST && (b < 0 || b >= nctx)) {
      report_error(p.err, PKV_DEVERR_SELECT);
      return;
    }
    const int32_t x = table[b];
    if (x < 0 || x >= p.num_blocks) {
      report_error(p.err, PKV_DEVERR_BLOCK_ID);
      return;
    }
    pb = x;
    tok = b * BS;
  };
  int pb_now, tok_now, pb_next = -1, tok_next = kNoToken;
  look_up(0, pb_now, tok_now);
  if (mine > kBatch) look_up(1, pb_next, tok_next);
  uint64_t* my_k = kfull + warp * NST;
  uint64_t* my_v = vfull + warp * NST;
  int4* my_meta = meta + warp * NST;
  const uint32_t my_ring = ring + warp * NST * G::kStage;
  auto load = [&](uint32_t dst, const uint8_t* pool, const int4& m, uint64_t* bar) {
    const int n = (m.x >= 0 ? 1 : 0) + (UB == 2 && m.z >= 0 ? 1 : 0);
    if (n == 0) {
      mbar_arrive(bar);
      return;
    }
    mbar_arrive_expect_tx(bar, n * PAGE);
    if (m.x >= 0)
      bulk_load(dst, pool + (static_cast<int64_t>(m.x) * p.num_kv_heads + h) * PAGE, PAGE, bar);
    if (UB == 2 && m.z >= 0)
      bulk_load(dst + PAGE, pool + (static_cast<int64_t>(m.z) * p.num_kv_heads + h) * PAGE, PAGE,
                bar);
  };
  // K of unit i into its slot, and what the unit is; all lanes
  auto load_k = [&](int i) {
    if (i >= mine) return;
    const int at = i % kBatch * UB;
    if (at == 0 && i > 0) {
      pb_now = pb_next;
      tok_now = tok_next;
      if (i + kBatch < mine) look_up(i / kBatch + 1, pb_next, tok_next);
    }
    int4 m;
    m.x = __shfl_sync(0xffffffffu, pb_now, at);
    m.y = __shfl_sync(0xffffffffu, tok_now, at);
    m.z = UB == 2 ? __shfl_sync(0xffffffffu, pb_now, at + UB - 1) : -1;
    m.w = UB == 2 ? __shfl_sync(0xffffffffu, tok_now, at + UB - 1) : kNoToken;
    if (lane == 0) {
      my_meta[i % NST] = m;
      load(my_ring + i % NST * G::kStage, p.k_cache, m, &my_k[i % NST]);
    }
  };
  // its V; after load_k of the same unit
  auto load_v = [&](int i) {
    if (i < mine && lane == 0)
      load(my_ring + i % NST * G::kStage + G::kBytes, p.v_cache, my_meta[i % NST], &my_v[i % NST]);
  };
  for (int i = 0; i < NST; ++i) {
    load_k(i);
    load_v(i);
  }

  // ---- Q^T fragments: lane (n = r, c) has channels D/4 c + 4 j + {0, 1} and {2, 3}
  // of query n for k-step j, as f16, in units of a power of two of its row
  uint32_t bq[KW][2];
  float f0, f1;  // logit factors of queries 2c, 2c + 1 (base 2)
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
    const int e = min(max(static_cast<int>(__float_as_uint(top) >> 23), 1), 253);
    const float down = __uint_as_float(static_cast<uint32_t>(254 - e) << 23);
    const float up = __uint_as_float(static_cast<uint32_t>(e) << 23);
#pragma unroll
    for (int j = 0; j < KW; ++j)
#pragma unroll
      for (int i = 0; i < 2; ++i)
        bq[j][i] = pack_f16(bf16lo(bq[j][i]) * down, bf16hi(bq[j][i]) * down);
    const float qs = p.qscale * p.k_scale[h];
    f0 = qs * __shfl_sync(0xffffffffu, up, 8 * c);
    f1 = qs * __shfl_sync(0xffffffffu, up, 8 * c + 4);
  }
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
  for (; done < mine; ++done) {
    const int i = done, st = i % NST;
    const uint32_t parity = (i / NST) & 1;
    if (!__all_sync(0xffffffffu, mbar_wait(&my_k[st], parity, p.err))) break;
    const int4 m = my_meta[st];
    const uint32_t kp = my_ring + st * G::kStage, vp = kp + G::kBytes;
    // visible tokens of the unit's blocks
    const int n0 = ctx - m.y, n1 = UB == 2 ? ctx - m.w : 0;
    const bool whole = n0 >= BS && (UB == 1 || n1 >= BS);
    auto sees = [&](int t) { return UB == 1 || t < BS ? t < n0 : t - BS < n1; };

    // ---- S^T = K Q^T
    float sc[2][4];
#pragma unroll
    for (int t = 0; t < 2; ++t) {
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
      float u[4] = {0.f, 0.f, 0.f, 0.f}, v[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int x = 0; x < NW; ++x) {
        // two words (16 channels) to a scale
        const int gr = x / 2;
        const uint32_t pa = e4m3x2_f16x2(sa, gr / 2), pb = e4m3x2_f16x2(sb, gr / 2);
        const uint32_t fa = gr & 1 ? dup_hi(pa) : dup_lo(pa);
        const uint32_t fb = gr & 1 ? dup_hi(pb) : dup_lo(pb);
        uint32_t a[4], b[4];
        e2m1x8_f16x2(wa[x], a);
        e2m1x8_f16x2(wb[x], b);
#pragma unroll
        for (int y = 0; y < 4; ++y) {
          a[y] = mul_f16x2(a[y], fa);
          b[y] = mul_f16x2(b[y], fb);
        }
        mma_f16(u, a[0], b[0], a[1], b[1], bq[2 * x][0], bq[2 * x][1]);
        mma_f16(v, a[2], b[2], a[3], b[3], bq[2 * x + 1][0], bq[2 * x + 1][1]);
      }
      const bool see_a = whole || sees(ta), see_b = whole || sees(tb);
      sc[t][0] = see_a ? (u[0] + v[0]) * f0 : -INFINITY;
      sc[t][1] = see_a ? (u[1] + v[1]) * f1 : -INFINITY;
      sc[t][2] = see_b ? (u[2] + v[2]) * f0 : -INFINITY;
      sc[t][3] = see_b ? (u[3] + v[3]) * f1 : -INFINITY;
    }
    // ---- online softmax: rows are tokens, columns queries
    float x0 = fmaxf(fmaxf(sc[0][0], sc[0][2]), fmaxf(sc[1][0], sc[1][2]));
    float x1 = fmaxf(fmaxf(sc[0][1], sc[0][3]), fmaxf(sc[1][1], sc[1][3]));
#pragma unroll
    for (int off = 4; off < 32; off <<= 1) {
      x0 = fmaxf(x0, __shfl_xor_sync(0xffffffffu, x0, off));
      x1 = fmaxf(x1, __shfl_xor_sync(0xffffffffu, x1, off));
    }
    // Every lane's logits have met in the shuffles, so every lane has read this
    // unit's K, and (loads of a warp return in order) the unit before's V: both
    // slots take the next unit's
    __syncwarp();
    load_k(i + NST);
    if (i > 0) load_v(i - 1 + NST);
    const float y0 = fmaxf(m0, x0), y1 = fmaxf(m1, x1);
    if (__any_sync(0xffffffffu, y0 > m0 || y1 > m1)) {
      // 0 where the maximum was -inf, 1 where it stays that
      const float c0 = y0 > m0 ? fast_exp2(m0 - y0) : 1.f;
      const float c1 = y1 > m1 ? fast_exp2(m1 - y1) : 1.f;
      l0 *= c0;
      l1 *= c1;
#pragma unroll
      for (int k = 0; k < KW; ++k) {
        o[k][0] *= c0;
        o[k][1] *= c1;
        o[k][2] *= c0;
        o[k][3] *= c1;
      }
      m0 = y0;
      m1 = y1;
    }
    const float ref0 = (m0 == -INFINITY ? 0.f : m0) - kUpFp4;
    const float ref1 = (m1 == -INFINITY ? 0.f : m1) - kUpFp4;
    if (!__all_sync(0xffffffffu, mbar_wait(&my_v[st], parity, p.err))) {
      v_late = true;
      break;
    }
    // ---- O^T += V^T P^T
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      const float p00 = fast_exp2(sc[t][0] - ref0), p01 = fast_exp2(sc[t][1] - ref1);
      const float p10 = fast_exp2(sc[t][2] - ref0), p11 = fast_exp2(sc[t][3] - ref1);
      l0 += p00 + p10;
      l1 += p01 + p11;
      const uint32_t q0 = movm_t(pack_f16(p00, p01)), q1 = movm_t(pack_f16(p10, p11));
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
        if (!whole && !sees(tk)) e8[k] = 0;
      }
#pragma unroll
      for (int x = 0; x < NW; ++x) {
        // the word's scale: byte x / 2 of each token's
        const uint32_t sel = x / 2 ? 0x51 : 0x40;
        const uint32_t s01 = e4m3x2_f16x2(__byte_perm(e8[0], e8[1], sel), 0);
        const uint32_t s23 = e4m3x2_f16x2(__byte_perm(e8[2], e8[3], sel), 0);
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
  }
  if (done < mine && lane == 0) {
    // a wait ran out: what is in flight has to land before the ring is used again
    const int nk = min(mine, done + NST + (v_late ? 1 : 0));
    const int nv = min(mine, done + NST - (v_late || done == 0 ? 0 : 1));
    for (int i = max(done, nk - NST); i < nk; ++i)
      (void)mbar_wait(&my_k[i % NST], (i / NST) & 1, p.err);
    for (int i = max(done, nv - NST); i < nv; ++i)
      (void)mbar_wait(&my_v[i % NST], (i / NST) & 1, p.err);
  }
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
  const float vsc = p.v_scale[h];
  const int64_t hq0 = static_cast<int64_t>(s) * p.num_heads + h * g;
  // query j's maximum and sum over the warps
  auto state = [&](int j, float& M, float& L) {
    M = sm_m[j];
#pragma unroll
    for (int w = 1; w < W; ++w) M = fmaxf(M, sm_m[w * 8 + j]);
    L = 0.f;
    if (M != -INFINITY)
#pragma unroll
      for (int w = 0; w < W; ++w) L = fmaf(sm_l[w * 8 + j], fast_exp2(sm_m[w * 8 + j] - M), L);
  };
  for (int idx = threadIdx.x; idx < g * (D / 2); idx += G::kThreads) {
    const int j = idx / (D / 2), col = idx % (D / 2) * 2;
    const int at = j * G::kRowQ + col / (D / 8) * G::kRow8 + col % (D / 8);
    float2 sum = *reinterpret_cast<const float2*>(os + at);
#pragma unroll
    for (int w = 1; w < W; ++w) {
      const float2 x = *reinterpret_cast<const float2*>(os + w * 8 * G::kRowQ + at);
      sum.x += x.x;
      sum.y += x.y;
    }
    if (p.cluster > 1) {
      *reinterpret_cast<float2*>(cs_o + j * D + col) = sum;
      continue;
    }
    float M, L;
    state(j, M, L);
    const float ox = L > 0.f ? sum.x / L * vsc : 0.f, oy = L > 0.f ? sum.y / L * vsc : 0.f;
    if (p.partition_blocks == 0) {
      *reinterpret_cast<uint32_t*>(p.out + (hq0 + j) * D + col) = pack_bf16(ox, oy);
    } else {
      const int64_t slot = (hq0 + j) * p.np_max + part;
      *reinterpret_cast<float2*>(p.tmp_out + slot * D + col) = make_float2(ox, oy);
      if (col == 0) {
        // the sums have the weights' factor; the merge only compares them
        p.max_logits[slot] = M * kLn2Tc;
        p.exp_sums[slot] = L;
      }
    }
  }
  if (p.cluster <= 1) return;
  // ---- the CTAs of the cluster: rank k has channels [k D/C, (k + 1) D/C) of the
  // result, from every rank's state in rank order
  float* cs_m = sm_m + 2 * W * 8;  // [8]
  float* cs_l = cs_m + 8;          // [8]
  if (threadIdx.x < 8) state(threadIdx.x, cs_m[threadIdx.x], cs_l[threadIdx.x]);
  cluster_sync_all();
  const int C = p.cluster, SL = D / C;
  const uint32_t o_addr = smem_addr(cs_o), m_addr = smem_addr(cs_m), l_addr = smem_addr(cs_l);
  for (int idx = threadIdx.x; idx < g * SL; idx += G::kThreads) {
    const int j = idx / SL, col = part * SL + idx % SL;
    float M = -INFINITY;
    for (int k = 0; k < C; ++k) M = fmaxf(M, ld_dsmem(m_addr + 4 * j, k));
    float L = 0.f, O = 0.f;
    if (M != -INFINITY) {
      for (int k = 0; k < C; ++k) {
        const float a = fast_exp2(ld_dsmem(m_addr + 4 * j, k) - M);
        L = fmaf(ld_dsmem(l_addr + 4 * j, k), a, L);
        O = fmaf(ld_dsmem(o_addr + 4 * (j * D + col), k), a, O);
      }
    }
    p.out[(hq0 + j) * D + col] = float_to_bf16_bits(L > 0.f ? O / L * vsc : 0.f);
  }
  cluster_sync_all();  // this CTA's state lives until every rank has read it
}

template <int D, int BS, bool LIST>
static int launch_fp4(const DecodeParams& p_in, dim3 grid, cudaStream_t st) {
  constexpr int W = 4, NST = D == 256 ? 2 : 3;
  using G = Fp4Geom<D, W, NST>;
  auto kern = decode_fp4_kernel<D, BS, LIST, W, NST>;
  static DeviceFlags done;
  int rc = ensure_smem(kern, G::kSmem, done);
  if (rc != PKV_OK) return rc;
  DecodeParams p = p_in;
  if (p.partition_blocks > 0 || p.cluster <= 1) {
    p.cluster = 1;
    return launch_dependent(kern, grid, dim3(G::kThreads), G::kSmem, st, p);
  }
  grid.x = p.cluster;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  cfg.gridDim = grid;
  cfg.blockDim = dim3(G::kThreads);
  cfg.dynamicSmemBytes = G::kSmem;
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  // clusters of up to 8 CTAs are portable
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

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
// with fp32 accumulators in tensor memory: O [d], S of two or three steps [128].
//
// Work split. A unit is (sequence, KV head, row tile); its steps are the 128-
// token runs of its context. All steps of all units form one line that is cut
// into equal shares, one per CTA, one CTA per SM: no tail whatever the lengths
// are. A unit's start counts as three steps more (its Q has to come, its result
// to go: without that, 96 sequences of 16 .. 16384 tokens take 227 us instead
// of 150, because a few CTAs get all the short ones). A CTA's share is a row of
// segments (runs of steps of one unit). A unit inside one share is finished
// there; a unit that is cut leaves a partial (normalised fp32 output, maximum,
// sum) per segment, at most two per CTA, and tree_merge_kernel joins them by
// log-sum-exp. The pipeline below runs on across segments, so the loads never
// pause. Where every sequence has the same number T > 1 of row tiles, the CTAs
// work in teams of T: a team takes a share of the line of (sequence, KV head)
// steps, each member one row tile of it, so that the tiles' reads of a page
// fall together and all but the first find it in L2 (16 sequences x 4096
// tokens x 64 drafts, d = 256: 161 -> 133 us when it was introduced).
//
// Shared memory: the row tile's Q and a ring of 32 KB slots that TMA fills
// (cp.async.bulk.tensor, whole pages, 128-byte swizzle). A slot is [8-row
// group][64-column chunk][8 rows][128 B]: the box of a page is 4-D (64
// columns, 8 rows, chunks, row groups), so pages land one behind the other in
// what is both K's operand layout (N = tokens, row groups at one stride) and
// V's (N = columns, MN-major). K of a step takes d/128 slots (128 columns
// each), V d/128 slots (64 or 128 tokens each). Slots are filled in the order
// K(0) .. K(lead), V(0), K(lead + 1), V(1), ...; lead is 1 (d = 256) or 2.
//
// E4M3 pools: K's codes are the operand as they are (kind::f8f6f4). Q is split
// into two E4M3 parts, q 2^e = hi + lo with a power of two per row that puts
// the row's largest element in [128, 256): bf16 has 8 significant bits and
// each part 4, so elements down to 2^-9 of the largest are exact and the rest
// are off by at most 2^-17 of it. V's codes are staged by TMA and turned into
// their exact f16 values by converter warps; P is f16. k_scale and the row's
// 2^-e go into the logits, v_scale into the output. K and V have rings of their
// own.
//
// What V holds behind the context and in drafts that no row sees never counts:
// its weight is 0, and the row is zeroed in shared memory before P.V reads it,
// since 0 x NaN is NaN (16-bit pools: by the softmax warps, in place; E4M3: by
// the converters).
//
// P is one bf16 part, a rounding of each weight to as many bits as the output
// has. The one-token decode holds P in two parts. Here a second part (the
// remainders over the other half of S's columns, one more product each) takes
// the error against 64 bits from 0.0023 to 0.0017 of the output (the output's
// own rounding is 0.0017) and costs 1 % where HBM bounds the call (32 x 8192
// tokens x 16 drafts, d = 256: 171 -> 173 us), 7 % at d = 128 (96 ragged
// sequences 153 -> 164), 4 to 8 % of small calls and 17 to 26 % of calls with
// several row tiles (16 x 4096 x 64, d = 256: 94 -> 118): the softmax's
// instructions more than the products.
//
// Warps: 0-7 softmax (threads t and t + 128 own query row t, 64 of a step's
// columns each; they exchange maxima through shared memory), 8 issues Q.K^T, 9
// P.V; bf16: 10-13 load Q, 14-15 load pages; E4M3: 10 loads K, 11 V, 12-15
// convert V and load Q. 512 threads of up to 128 registers, all the SM has.
//
// What bounds it on GB300 (of 6788 GB/s copy, 1943 TFLOP/s bf16; calls in a
// graph; clocks of a step from calls of two lengths, at 2070 MHz):
//   few rows, bf16: HBM. 32 x 8192 tokens x 16 drafts, d = 256: 173 us, 92 %;
//     64 x 8192 x 1: 317 us, 100 %; 96 sequences of 16 .. 16384: 153 us, 91 %
//   many rows: at d = 128 a step takes 2000 clocks, the softmax's chain of one
//     row tile (load S, maximum, exchange with the row's other thread,
//     exponentials, P) on two warps a scheduler; 1040 of them are the tensor
//     core's and 512 the 128 x 128 exponentials at 32 a clock. 32 x 4096 x 64:
//     248 us, 57 % of the products' floor; 42 us are the starts and ends of
//     seven units per CTA and the merge. At d = 256 a step takes 3300 clocks,
//     2100 of them the tensor core's: P, S's two buffers and the reads of K and
//     V by all tiles of a team out of L2. 16 x 4096 x 64: 93 us, 57 %, 27 of
//     them starts, ends and the merge
//   E4M3: HBM leaves a step 3040 clocks at d = 256 and 1520 at d = 128; the
//     kernel takes 3400 and 2000. 8 x 65536 x 8, d = 256: 197 us, 80 % of HBM;
//     32 x 8192 x 4, d = 128: 127 us, 63 %; 64 x 4096 x 21, d = 256: 154 us, 55 %
//     (half the exponentials and loads of S would take 6 to 20 % off; every
//     instruction that the softmax's or the converters' loop gains or loses
//     shows)
//   one short sequence: latency. 1033 tokens x 5 drafts 11.2 us, 4 of them the
//     merge
#include <algorithm>
#include <climits>
#include <cmath>

#include "common.cuh"
#include "host_util.h"
#include "tc_common.cuh"
#include "tmem.cuh"

namespace pkv {

constexpr int kTreeMaxCtas = 160;  // one per SM; the workspace is sized for it
constexpr int kTreeRows = 128;     // query rows of a tile
constexpr int kTreeTok = 128;      // tokens of a step
constexpr int kTreeEven = 4;       // shares of at most so many steps are cut evenly
constexpr int kTreeStart = 3;      // steps that a unit's start counts for in longer ones
// E4M3 pools: P is 2^(z - m + kTreeUp) in f16, which holds 2^-24 to 2^16. The
// reference m may lie 8 below the maximum, so 2^15 is P's largest value, and
// what rounds to zero is below 2^-32 of 2^m: without the shift it was 2^-25,
// and of 65536 such weights 0.2 % of the row's sum were lost. All partials of
// a row have the shift in their sums, so it cancels.
constexpr float kTreeUp = 7.f;

struct TreeMeta {  // what the merge needs of a unit that starts in a CTA and is cut
  int row0;        // first query row (of q and out) of the sequence
  int first;       // first (draft, group) row of the tile
  int rows;        // live rows of the tile
  int head;        // KV head
  int slot;        // the CTA's partial that holds the unit's first segment
  int parts;       // segments; 0: nothing to merge
  int stride;      // CTAs from one of the unit's segments to the next
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
  float* part_o;    // [ctas][2][d][128]: a column's rows side by side
  float* part_m;    // [ctas][2][128]
  float* part_l;
  int num_seqs, num_queries, max_draft, max_context;
  int num_blocks, num_kv_heads, num_heads, group, block_size, max_blocks_per_seq;
  int ctas;         // of the grid
  float qscale;
};

template <int D, bool FP8>
struct TreeGeom {
  static constexpr int kQ = kTreeRows * D * 2;  // E4M3: two parts of one byte
  static constexpr int kKS = FP8 ? 1 : D / 128;  // slots of a step's K
  static constexpr int kVS = D / 128;           // slots of a step's V
  static constexpr int kVTok = kTreeTok / kVS;
  // the ring that TMA fills: K's and V's 16-bit values; E4M3: V's codes
  static constexpr int kSlot = FP8 ? 16384 : 32768;
  static constexpr int kNSlot = FP8 ? (D == 256 ? 2 : 4) : (D == 256 ? 5 : 6);
  // E4M3: K's codes, a step to a slot
  static constexpr int kK8 = kTreeTok * D;
  static constexpr int kNK8 = FP8 ? (D == 256 ? 2 : 4) : 0;
  // E4M3: V's f16 values, two slots
  static constexpr int kV16 = 32768;
  static constexpr int kNV16 = FP8 ? 2 : 0;
  static constexpr int kSoftWarps = 8;
  static constexpr int kSWarp = 8, kPvWarp = 9;
  static constexpr int kProdWarp = FP8 ? 10 : 14, kProducers = 2;
  static constexpr int kConvWarp = 12, kConvWarps = FP8 ? 4 : 0;
  // bf16: warps of their own load Q; E4M3: the converters do
  static constexpr int kQWarp = FP8 ? kConvWarp : 10, kQWarps = 4;
  static constexpr int kThreads = 16 * 32;
  static constexpr int kHead = 3072;  // barriers, exchange buffers
  static constexpr int kSmem = kHead + kQ + kNSlot * kSlot + kNK8 * kK8 + kNV16 * kV16;
  // S of step t at kColS + 128 * (t % kNB); three buffers where they fit (d =
  // 128: 32 x 4096 tokens x 64 drafts 294 -> 272 us when it was introduced)
  static constexpr int kNB = D == 128 ? 3 : 2;
  static constexpr int kLead = kNB - 1;  // steps that S runs ahead of P.V
  static constexpr uint32_t kColS = D;
  static constexpr uint32_t kCols = 512;
  static_assert(kColS + kNB * kTreeTok <= kCols, "tensor memory");
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

// The same on E4M3 operands (32 bytes of a row each).
__device__ __forceinline__ void umma_ss_e4m3(uint32_t d_tmem, uint64_t a, uint64_t b,
                                             uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}

// Instruction descriptor, kind::f8f6f4 with E4M3 A and B (both K-major), fp32
// accumulator.
__host__ __device__ constexpr uint32_t umma_idesc_e4m3(int M, int N) {
  return (1u << 4) | (static_cast<uint32_t>(N >> 3) << 17) | (static_cast<uint32_t>(M >> 4) << 24);
}

// One box of a 4-D pool map: chunk c, 8-row group y.
__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap* map, int c, int y,
                                            uint64_t* bar, uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      ".L2::cache_hint [%0], [%1, {%2, %3, %4, %5}], [%6], %7;" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(0), "r"(0), "r"(c), "r"(y), "r"(smem_addr(bar)),
      "l"(policy)
      : "memory");
}

// A sequence's part of the line of steps; n = 0 if it has none (no drafts, or
// drafts or a context that cannot be).
struct TreeSeq {
  int ctx, n, q0, tiles, steps;
  __device__ __forceinline__ void set(const TreeParams& p, int first, int next, int context,
                                      bool report) {
    q0 = first;
    ctx = context;
    const bool ctx_ok =
        ctx >= 0 && ctx <= p.max_context &&
        ctx <= static_cast<int64_t>(p.max_blocks_per_seq) * p.block_size;
    const bool ok = ctx_ok && q0 >= 0 && next >= q0 && next <= p.num_queries &&
                    next - q0 <= p.max_draft && next - q0 <= ctx;
    if (!ok && report) report_error(p.err, ctx_ok ? PKV_DEVERR_DRAFT : PKV_DEVERR_CONTEXT);
    n = ok ? next - q0 : 0;
    tiles = (n * p.group + kTreeRows - 1) / kTreeRows;
    steps = ok ? (ctx + kTreeTok - 1) / kTreeTok : 0;
  }
  __device__ __forceinline__ void load(const TreeParams& p, int s, bool report) {
    set(p, p.q_start[s], p.q_start[s + 1], p.context_lens[s], report);
  }
  __device__ __forceinline__ int units(const TreeParams& p) const {
    return p.num_kv_heads * tiles;
  }
};

// a / b for a >= 0, b > 0; the long division only where it is needed.
__device__ __forceinline__ int64_t quotient(int64_t a, int64_t b) {
  if (((a | b) >> 32) == 0) return static_cast<uint32_t>(a) / static_cast<uint32_t>(b);
  return a / b;
}

// Walks a CTA's share step by step.
struct TreeWalk {
  TreeSeq q;
  int s, h, tile, st;   // the current step
  int left;             // steps left, this one included
  bool begins;          // first step of a segment
  int next_q0, next_q1, next_ctx;  // of sequence s + 1, read when s is entered
  bool team;            // the tile is the CTA's for good (see tree_kernel)
  __device__ __forceinline__ void peek(const TreeParams& p) {
    const int x = min(s + 1, p.num_seqs - 1);
    next_q0 = p.q_start[x];
    next_q1 = p.q_start[x + 1];
    next_ctx = p.context_lens[x];
  }
  // at: the share's first step in unit `unit` of sequence s0; member: the
  // CTA's tile if it belongs to a team, else -1
  __device__ __forceinline__ void start(const TreeParams& p, const TreeSeq& q0, int s0, int unit,
                                        int at, int count, int member) {
    q = q0;
    s = s0;
    left = count;
    begins = true;
    team = member >= 0;
    h = tile = st = 0;
    if (count <= 0) return;
    peek(p);
    st = at;
    h = team ? unit : unit / q.tiles;
    tile = team ? member : unit - h * q.tiles;
  }
  __device__ __forceinline__ bool ends() const { return left == 1 || st + 1 == q.steps; }
  // steps of the segment from this one on, and over them
  __device__ __forceinline__ int run() const { return min(left, q.steps - st); }
  __device__ __forceinline__ void skip(const TreeParams& p, int n) {
    left -= n - 1;
    st += n - 1;
    next(p);
  }
  __device__ __forceinline__ void next(const TreeParams& p) {
    begins = false;
    if (--left <= 0) return;
    if (++st < q.steps) return;
    st = 0;
    begins = true;
    if (!team) {
      if (++tile < q.tiles) return;
      tile = 0;
    }
    if (++h < p.num_kv_heads) return;
    h = 0;
    q.set(p, next_q0, next_q1, next_ctx, false);
    ++s;
    while (q.tiles == 0 && s + 1 < p.num_seqs) q.load(p, ++s, false);
    peek(p);
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

// The drafts that some row of the sequence sees, by all lanes of a warp (given
// masks).
__device__ __forceinline__ uint64_t drafts_seen(const TreeParams& p, const TreeSeq& q, int lane) {
  uint64_t any = lane < q.n ? p.tree_mask[q.q0 + lane] : 0ull;
  any |= lane + 32 < q.n ? p.tree_mask[q.q0 + lane + 32] : 0ull;
  const uint32_t lo = __reduce_or_sync(0xffffffffu, static_cast<uint32_t>(any));
  const uint32_t hi = __reduce_or_sync(0xffffffffu, static_cast<uint32_t>(any >> 32));
  __syncwarp();
  return static_cast<uint64_t>(hi) << 32 | lo;
}

// r / g for a row of a unit (r < 64 g, g <= 8): exact, no division.
__device__ __forceinline__ int div_group(int r, int g) { return (r * (65536 / g + 1)) >> 16; }

// One lane of the warp, the same one every time.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}"
               : "=r"(p));
  return p != 0;
}

// Loads a segment's Q into shared memory (K-major, 128-byte swizzle) with NW
// warps; rows past the tile's query rows are zero.
template <int D, bool FP8, int NW>
struct TreeQ {
  static constexpr int U = D / 8;     // 16-byte units of a row of q
  static constexpr int RPW = 32 / U;  // rows a warp takes at a time
  static constexpr int kRowStep = NW * RPW;
  const uint16_t* q0;
  int64_t draft_stride;  // elements from a draft's rows to the next one's
  int r0, rows, inv, g, rl, rs, u;

  __device__ __forceinline__ TreeQ(const TreeParams& p, const TreeWalk& w, int wi, int lane) {
    g = p.group;
    inv = 65536 / g + 1;
    r0 = w.tile * kTreeRows;
    rows = min(kTreeRows, w.q.n * g - r0);
    rs = lane / U;
    rl = wi * RPW + rs;  // first row of this lane
    u = lane % U;
    draft_stride = static_cast<int64_t>(p.num_heads) * D;
    q0 = p.q + w.q.q0 * draft_stride + w.h * g * D + u * 8;
  }
  // this lane's unit of row r of the tile: draft (r0 + r) / g, group row (r0 + r) % g
  __device__ __forceinline__ const uint16_t* unit_of(int r) const {
    const int rr = r0 + (r < rows ? r : 0);
    const int dr = (rr * inv) >> 16;
    return q0 + dr * draft_stride + (rr - dr * g) * D;
  }
  // where it goes: a 16-byte unit; E4M3: 8 codes of the first part, half a unit
  __device__ __forceinline__ uint32_t place(uint32_t sq, int r) const {
    if constexpr (FP8)
      return sq + ((r / 8) * (D / 128) + u / 16) * 1024 + (r % 8) * 128 +
             ((((u % 16) / 2) ^ (r % 8)) * 16) + (u & 1) * 8;
    else
      return sq + ((r / 8) * (D / 64) + u / 8) * 1024 + (r % 8) * 128 + ((u % 8) ^ (r % 8)) * 16;
  }
  // exps (E4M3): [128] exponents of the rows' scales
  __device__ __forceinline__ void run(uint32_t sq, int8_t* exps) const {
    if constexpr (!FP8) {
      constexpr int kRows = (kTreeRows + kRowStep - 1) / kRowStep;  // of this lane
      constexpr int kBatch = kRows < 16 ? kRows : 11;
      for (int rb = rl; rb < kTreeRows; rb += kBatch * kRowStep) {
        const uint16_t* src[kBatch];
#pragma unroll
        for (int e = 0; e < kBatch; ++e) src[e] = unit_of(rb + e * kRowStep);
#pragma unroll
        for (int e = 0; e < kBatch; ++e) {
          const int r = rb + e * kRowStep;
          if (r < rows)
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(place(sq, r)),
                         "l"(src[e])
                         : "memory");
          else if (r < kTreeRows)
            asm volatile("st.shared.v4.u32 [%0], {%1,%1,%1,%1};" ::"r"(place(sq, r)), "r"(0u)
                         : "memory");
        }
      }
      asm volatile("cp.async.wait_all;" ::: "memory");
    } else {
      constexpr int kBatch = 8;
      // rows past the tile's: zero codes (their exponents are never used)
      for (int r = rl; r < kTreeRows; r += kRowStep)
        if (r >= rows) {
          const uint32_t at = place(sq, r);
          asm volatile("st.shared.v2.u32 [%0], {%1,%1};" ::"r"(at), "r"(0u) : "memory");
          asm volatile("st.shared.v2.u32 [%0], {%1,%1};" ::"r"(at + kTreeRows * D), "r"(0u)
                       : "memory");
          if (u == 0) exps[r] = 0;
        }
      for (int rb = rl; rb - rs < rows; rb += kBatch * kRowStep) {
        uint4 v[kBatch];
#pragma unroll
        for (int e = 0; e < kBatch; ++e) {
          const int r = rb + e * kRowStep;
          v[e] = make_uint4(0u, 0u, 0u, 0u);
          if (r < rows) v[e] = *reinterpret_cast<const uint4*>(unit_of(r));
        }
#pragma unroll
        for (int e = 0; e < kBatch; ++e) {
          const int r = rb + e * kRowStep;
          float x[8] = {bf16lo(v[e].x), bf16hi(v[e].x), bf16lo(v[e].y), bf16hi(v[e].y),
                        bf16lo(v[e].z), bf16hi(v[e].z), bf16lo(v[e].w), bf16hi(v[e].w)};
          // the row's largest magnitude; as bit patterns, so NaN counts as largest
          uint32_t top = 0;
#pragma unroll
          for (int i = 0; i < 8; ++i) top = max(top, __float_as_uint(x[i]) & 0x7FFFFFFFu);
#pragma unroll
          for (int off = U / 2; off > 0; off >>= 1)
            top = max(top, __shfl_xor_sync(0xffffffffu, top, off));
          // 2^ex puts it in [128, 256); zero and tiny rows are scaled by 2^100
          const int ex = max(-120, min(100, 134 - static_cast<int>(top >> 23)));
          const float up = __uint_as_float(static_cast<uint32_t>(ex + 127) << 23);
          uint32_t hi[2] = {0, 0}, lo[2] = {0, 0};
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float a = x[2 * i] * up, c = x[2 * i + 1] * up;
            const uint32_t h = __nv_cvt_float2_to_fp8x2(make_float2(a, c), __NV_SATFINITE,
                                                        __NV_E4M3);
            const uint32_t back = e4m3x2_f16x2(h, 0);
            const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&back));
            const uint32_t r2 = __nv_cvt_float2_to_fp8x2(make_float2(a - f.x, c - f.y),
                                                         __NV_SATFINITE, __NV_E4M3);
            hi[i / 2] |= (h & 0xFFFFu) << (16 * (i & 1));
            lo[i / 2] |= (r2 & 0xFFFFu) << (16 * (i & 1));
          }
          if (r < rows) {
            const uint32_t at = place(sq, r);
            asm volatile("st.shared.v2.u32 [%0], {%1,%2};" ::"r"(at), "r"(hi[0]), "r"(hi[1])
                         : "memory");
            asm volatile("st.shared.v2.u32 [%0], {%1,%2};" ::"r"(at + kTreeRows * D),
                         "r"(lo[0]), "r"(lo[1])
                         : "memory");
            if (u == 0)
              exps[r] = static_cast<int8_t>(top >= 0x7F800000u ? -128 : ex);
          }
        }
      }
    }
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  }
};

// The number of V's first slot of step t in the ring's order (the slot is that
// modulo the slots), of a CTA with `total` steps; `lead`: K of step t + lead
// comes before V of step t.
template <int KS, int VS>
__device__ __forceinline__ int v_seq(int t, int total, int lead) {
  return KS * min(total, t + lead + 1) + t * VS;
}

template <int D, bool FP8>
__global__ void __launch_bounds__(TreeGeom<D, FP8>::kThreads, 1)
    tree_kernel(const __grid_constant__ CUtensorMap tmk, const __grid_constant__ CUtensorMap tmv,
                const __grid_constant__ TreeParams p) {
  using G = TreeGeom<D, FP8>;
  constexpr int NCH = D / 64;    // 128-byte chunks of a 16-bit row
  constexpr int NC8 = D / 128;   // of a row of codes
  constexpr int KS = G::kKS, VS = G::kVS, NS = G::kNSlot;
  constexpr int NK8 = FP8 ? G::kNK8 : 1;
  constexpr int NB = G::kNB;
  extern __shared__ __align__(1024) uint8_t sbase[];  // no room to align it by hand
  const uint32_t base = smem_addr(sbase);
  uint64_t* full = reinterpret_cast<uint64_t*>(sbase);  // [NS] slot filled
  uint64_t* empty = full + 8;                            // [NS] slot read
  uint64_t* vfull = empty + 8;                           // [2] E4M3: V converted
  uint64_t* vempty = vfull + 2;                          // [2]
  uint64_t* kfull = vempty + 2;                          // [4] E4M3: K's codes in
  uint64_t* kempty = kfull + 4;                          // [4]
  uint64_t* s_full = kempty + 4;                         // [NB] S of a step is done
  uint64_t* p_full = s_full + 3;                         // [NB] its P is written
  uint64_t* o_done = p_full + 3;                         // [NB] its P.V is done
  uint64_t* pair = o_done + 3;                           // [4] the two threads of a row
  uint64_t* q_full = pair + 4;
  uint64_t* q_empty = q_full + 1;
  uint64_t* o_free = q_empty + 1;
  uint64_t* drained = o_free + 1;
  uint64_t* q_first = drained + 1;                       // Q of the share's first segment
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(sbase + 376);
  int* found = reinterpret_cast<int*>(sbase + 380);  // sequence, its TreeSeq, unit, step
  int* cut = reinterpret_cast<int*>(sbase + 368);              // steps before the share, its end
  int4* wsum = reinterpret_cast<int4*>(sbase + 416);           // [warps], until the share is known
  int8_t* q_exp = reinterpret_cast<int8_t*>(sbase + 416);      // [3][128] E4M3: e of Q's rows
  int32_t* ids = reinterpret_cast<int32_t*>(sbase + 800);      // [2][3][8] block ids of three steps
  uint64_t* seen = reinterpret_cast<uint64_t*>(sbase + 992);   // [4] bf16: drafts_seen
  float* xch = reinterpret_cast<float*>(sbase + 1024);         // [2][2][128]
  const uint32_t sq = base + G::kHead;
  const uint32_t ring = sq + G::kQ;
  const uint32_t k8 = ring + NS * G::kSlot;                   // E4M3: K's codes
  const uint32_t v16 = FP8 ? k8 + G::kNK8 * G::kK8 : ring;     // V's 16-bit values

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int cta = blockIdx.x;
  if (threadIdx.x == 0) {
    for (int i = 0; i < NS; ++i) {
      mbar_init(&full[i], FP8 ? 1 : G::kProducers);
      mbar_init(&empty[i], FP8 ? G::kConvWarps : 1);
    }
    for (int i = 0; i < G::kNK8; ++i) {
      mbar_init(&kfull[i], 1);
      mbar_init(&kempty[i], 1);
    }
    for (int i = 0; i < G::kNV16; ++i) {
      mbar_init(&vfull[i], G::kConvWarps);
      mbar_init(&vempty[i], 1);
    }
    for (int i = 0; i < G::kNB; ++i) {
      mbar_init(&s_full[i], 1);
      mbar_init(&p_full[i], G::kSoftWarps * 32);
      mbar_init(&o_done[i], 1);
    }
    for (int i = 0; i < 4; ++i) mbar_init(&pair[i], 64);
    mbar_init(q_full, G::kQWarps * 32);
    mbar_init(q_empty, 1);
    mbar_init(o_free, G::kSoftWarps * 32);
    mbar_init(drained, 2);
    mbar_init(q_first, G::kSoftWarps * 32);
    fence_mbar_init();
  }
  if (warp == G::kSWarp) tmem_alloc(tmem_slot, G::kCols);
  if (threadIdx.x == G::kProdWarp * 32) {
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&tmk)) : "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&tmv)) : "memory");
  }
  wait_prerequisite();
  if ((base & 1023u) != 0 && threadIdx.x == 0) report_error(p.err, PKV_DEVERR_WAIT_TIMEOUT);
  if (threadIdx.x == G::kProdWarp * 32) p.meta[cta] = TreeMeta{0, 0, 0, 0, 0, 0, 0};

  // ---- this CTA's share of the line: every thread sums a run of sequences,
  // the thread whose run holds the share's first step finds its sequence
  const int per = (p.num_seqs + G::kThreads - 1) / G::kThreads;
  const int s_lo = min(p.num_seqs, static_cast<int>(threadIdx.x) * per);
  const int s_hi = min(p.num_seqs, s_lo + per);
  int mine = 0, units = 0;  // steps, units
  int tiles_lo = INT_MAX, tiles_hi = 0;  // of sequences that have drafts
  TreeSeq seq;  // the run's last sequence (its only one, for small batches)
  for (int s = s_lo; s < s_hi; ++s) {
    seq.load(p, s, cta == 0);
    units += seq.units(p);
    mine += seq.units(p) * seq.steps;
    if (seq.tiles > 0) {
      tiles_lo = min(tiles_lo, seq.tiles);
      tiles_hi = max(tiles_hi, seq.tiles);
    }
  }
  tiles_lo = __reduce_min_sync(0xffffffffu, tiles_lo);
  tiles_hi = __reduce_max_sync(0xffffffffu, tiles_hi);
  int before = mine, before_u = units;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int x = __shfl_up_sync(0xffffffffu, before, off);
    const int y = __shfl_up_sync(0xffffffffu, before_u, off);
    if (lane >= off) {
      before += x;
      before_u += y;
    }
  }
  if (lane == 31) wsum[warp] = make_int4(before, before_u, tiles_lo, tiles_hi);
  before -= mine;
  before_u -= units;
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  int total = 0, total_u = 0;
#pragma unroll
  for (int w = 0; w < G::kThreads / 32; ++w) {
    const int4 x = wsum[w];
    if (w < warp) {
      before += x.x;
      before_u += x.y;
    }
    total += x.x;
    total_u += x.y;
    tiles_lo = min(tiles_lo, x.z);
    tiles_hi = max(tiles_hi, x.w);
  }
  // teams: shares in steps of (sequence, KV head), T CTAs to a share
  const int T = tiles_lo == tiles_hi && tiles_hi > 1 &&
                        tiles_hi <= static_cast<int>(gridDim.x) ? tiles_hi : 1;
  if (T > 1) {
    total /= T;
    before /= T;
    mine /= T;
    total_u /= T;
    before_u /= T;
    units /= T;
  }
  const int share = T > 1 ? cta / T : cta;
  // few steps to a CTA: as many CTAs as the longest share asks for, so that
  // fewer shares begin or end inside a unit
  const int most = static_cast<int>(T > 1 ? gridDim.x / T : gridDim.x);
  const int longest = (total + most - 1) / most;
  const int shares = longest > kTreeEven ? most
                     : longest > 0       ? (total + longest - 1) / longest
                                         : 0;
  // many: a unit's start counts as W steps (its Q, its result)
  const int W = longest > kTreeEven ? kTreeStart : 0;
  total += W * total_u;
  auto bound = [&](int x) {  // where share x of the line begins
    return static_cast<int>(quotient(static_cast<int64_t>(x) * total, shares));
  };
  int begin = 0, end = 0;
  if (share < shares) {
    begin = bound(share);
    end = bound(share + 1);
    // where it begins and ends: found in the runs that hold these places
    const int lo = before + W * before_u, hi = lo + mine + W * units;
    if (threadIdx.x == 0 && end == total) cut[1] = total - W * total_u;
#pragma unroll 1
    for (int e = 0; e < 2; ++e) {
      const int x = e == 0 ? begin : end;
      if (x < lo || x >= hi) continue;
      int at = lo, steps = before, s = s_lo;
      for (;; ++s) {
        if (per > 1) seq.load(p, s, false);
        const int n = seq.units(p) / T;
        if (per == 1 || x < at + n * (seq.steps + W)) break;
        at += n * (seq.steps + W);
        steps += n * seq.steps;
      }
      const int unit = (x - at) / (seq.steps + W);
      const int st = max(0, x - at - unit * (seq.steps + W) - W);
      cut[e] = steps + unit * seq.steps + st;
      if (e == 0) {
        found[0] = s;
        found[1] = seq.ctx;
        found[2] = seq.n;
        found[3] = seq.q0;
        found[4] = seq.tiles;
        found[5] = seq.steps;
        found[6] = unit;
        found[7] = st;
      }
    }
  }
  __syncthreads();
  const int count = begin < end ? cut[1] - cut[0] : 0;
  const uint32_t tmem = *tmem_slot;
  const uint32_t t_o = tmem;
  const uint32_t t_s = tmem + G::kColS;
  TreeWalk walk;
  walk.start(p, TreeSeq{found[1], found[2], found[3], found[4], found[5]}, found[0], found[6],
             found[7], count, T > 1 ? cta % T : -1);

  uint32_t issued = 0, issued_k = 0;  // producers: slots whose copies were started
  if (warp >= G::kProdWarp && warp < G::kProdWarp + G::kProducers) {
    // ---------------- producers: the block table walk and the TMA copies, a
    // page to a lane (one lane for all pages took about 3000 clocks a step: 8 x
    // 65536 tokens E4M3 267 us instead of 212). E4M3: the first warp loads
    // K, the second V; 16-bit pools: each warp its pages of both, in the order
    // of the one ring
    if (walk.left > 0) {
      constexpr int NP = FP8 ? 1 : G::kProducers;  // warps that share a slot
      const int prod = FP8 ? 0 : warp - G::kProdWarp;
      const bool loads_v = FP8 && warp != G::kProdWarp;  // else K (16-bit pools: both)
      const int page = NP * lane + prod;     // of a step
      const int B = p.block_size, lgB = B == 32 ? 5 : 4;
      const int per_v = G::kVTok >> lgB;     // pages of a V slot
      int32_t* my_ids = ids + (loads_v ? 24 : 0) + (page & 7);
      RingPos<NS> at;
      RingPos<NK8> at_k;  // E4M3: K has a ring of its own
      // pages of a single row tile are read once: they need not stay in L2
      uint64_t once, stay;
      asm volatile("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(once));
      asm volatile("createpolicy.fractional.L2::evict_normal.b64 %0, 1.0;" : "=l"(stay));
      int seg_st = walk.st;    // the segment's first step in its unit
      bool first_seg = true;   // of this share
      // on to the walk's next step; at the share's end, what the merge needs
      // if the unit starts here and goes on, up to the share that holds its end
      auto advance = [&] {
        if (walk.left == 1 && warp == G::kProdWarp && lane == 0 && seg_st == 0 &&
            walk.st + 1 < walk.q.steps) {
          const int u_end = end + (walk.q.steps - 1 - walk.st);
          int last = share + 1;
          while (bound(last + 1) < u_end) ++last;
          TreeMeta md;
          md.row0 = walk.q.q0;
          md.first = walk.tile * kTreeRows;
          md.rows = min(kTreeRows, walk.q.n * p.group - md.first);
          md.head = walk.h;
          md.slot = first_seg ? 0 : 1;
          md.parts = last - share + 1;
          md.stride = T;
          p.meta[cta] = md;
        }
        if (walk.left <= 0) return;
        walk.next(p);
        if (walk.begins) {
          seg_st = walk.st;
          first_seg = false;
        }
      };
      // What the copies of a step need. The block ids come through shared
      // memory in the background, two steps ahead: a load into registers would
      // be waited for as soon as the steps' registers change places.
      struct Step {
        int head, pages;
        bool once;
        int y;  // first 8-row group of this lane's page; -1 = no copy
      };
      int put = 0;  // ids: place of the step to be fetched
      auto fetch = [&] {
        Step x;
        x.y = -1;
        x.head = walk.h;
        x.once = walk.q.tiles == 1;
        x.pages = walk.left > 0
                      ? (min(kTreeTok, walk.q.ctx - walk.st * kTreeTok) + B - 1) >> lgB : 0;
        if (page < x.pages)
          asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(
                           smem_addr(my_ids + put * 8)),
                       "l"(p.block_tables +
                           static_cast<int64_t>(walk.s) * p.max_blocks_per_seq +
                           walk.st * (kTreeTok >> lgB) + page)
                       : "memory");
        asm volatile("cp.async.commit_group;" ::: "memory");
        put = put == 2 ? 0 : put + 1;
        return x;
      };
      int get = 0;  // ids: place of the next step to be loaded
      auto resolve = [&](Step& x) {
        if (page < x.pages) {
          const int id = my_ids[get * 8];
          if (id < 0 || id >= p.num_blocks)
            report_error(p.err, PKV_DEVERR_BLOCK_ID);
          else
            x.y = (id * p.num_kv_heads + x.head) << (lgB - 3);
        }
        get = get == 2 ? 0 : get + 1;
      };
      auto wait = [&](uint64_t* bar, uint32_t parity) {
        return __all_sync(0xffffffffu, mbar_wait(bar, parity, p.err)) != 0;
      };
      // a page into its place in the slot at dst, which `bar` announces
      auto copy = [&](const Step& x, const CUtensorMap* map, int chunk, bool mine, uint32_t dst,
                      int bytes, uint64_t* bar) {
        const uint32_t good = __ballot_sync(0xffffffffu, mine && x.y >= 0);
        if (lane == 0) mbar_arrive_expect_tx(bar, __popc(good) * bytes);
        if (mine && x.y >= 0) tma_load_4d(dst, map, chunk, x.y, bar, x.once ? once : stay);
      };
      // K of a step: columns [128 ks, 128 ks + 128) to a slot (E4M3: all)
      auto copy_k = [&](const Step& x) {
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) {
          const int bytes = (FP8 ? D : 256) << lgB;  // of one page
          if constexpr (FP8) {
            if (!wait(&kempty[at_k.i], at_k.ph ^ 1)) return false;
            copy(x, &tmk, 0, true, k8 + at_k.i * G::kK8 + page * bytes, bytes, &kfull[at_k.i]);
            at_k.next();
            ++issued_k;
          } else {
            if (!wait(&empty[at.i], at.ph ^ 1)) return false;
            copy(x, &tmk, 2 * ks, true, ring + at.i * G::kSlot + page * bytes, bytes,
                 &full[at.i]);
            at.next();
            ++issued;
          }
        }
        return true;
      };
      // V of a step, kVTok tokens to a slot
      auto copy_v = [&](const Step& x) {
#pragma unroll
        for (int vs = 0; vs < VS; ++vs) {
          if (!wait(&empty[at.i], at.ph ^ 1)) return false;
          const int bytes = D * (FP8 ? 1 : 2) << lgB;
          const int in = page - vs * per_v;  // its place in the slot
          copy(x, &tmv, 0, in >= 0 && in < per_v, ring + at.i * G::kSlot + in * bytes, bytes,
               &full[at.i]);
          at.next();
          ++issued;
        }
        return true;
      };
      // ids of step t + 2; E4M3: K or V of step t, else K of step t and V of
      // step t - kLead
      Step now = fetch();
      advance();
      Step ahead = fetch();
      Step before[G::kLead];
      bool ok = true;
      for (int t = 0; t < count && ok; ++t) {
        advance();
        const Step far = fetch();
        asm volatile("cp.async.wait_group 2;" ::: "memory");
        resolve(now);
        if constexpr (FP8) {
          ok = loads_v ? copy_v(now) : copy_k(now);
        } else {
          ok = copy_k(now);
          if (ok && t >= G::kLead) ok = copy_v(before[0]);
#pragma unroll
          for (int i = 0; i + 1 < G::kLead; ++i) before[i] = before[i + 1];
          before[G::kLead - 1] = now;
        }
        now = ahead;
        ahead = far;
      }
      if constexpr (!FP8) {
#pragma unroll
        for (int i = 0; i < G::kLead; ++i)
          if (ok && count - G::kLead + i >= 0) ok = copy_v(before[i]);
      }
      asm volatile("cp.async.wait_all;" ::: "memory");
    }
  } else if (warp == G::kSWarp) {
    // ---------------- the products S = Q.K^T, issued by one lane. P.V comes
    // from a lane of another warp: waits, commits and loops of both in one
    // lane took longer than the products (64 x 4096 x 21 drafts E4M3 180 us
    // instead of 164). Operand descriptors are a constant plus the address:
    // one addition each.
    if (elect_one()) {
      constexpr uint32_t idesc =
          FP8 ? umma_idesc_e4m3(128, kTreeTok) : umma_idesc_bf16(128, kTreeTok, false);
      const uint64_t qd = umma_sdesc(sq, 16, (FP8 ? NC8 : NCH) * 1024, 2);
      const uint64_t kd0 =
          FP8 ? umma_sdesc(k8, 16, NC8 * 1024, 2) : umma_sdesc(ring, 16, 2048, 2);
      RingPos<FP8 ? NK8 : NS> at;  // the next K's slot
      RingPos<NB> sb;
      int t = 0;
      bool ok = true;
      for (uint32_t seg = 0; walk.left > 0; ++seg) {
        ok = seg == 0 ? mbar_wait(q_first, 0, p.err) : mbar_wait(q_full, (seg - 1) & 1, p.err);
        const int n = walk.run();
        for (int i = 0; i < n && ok; ++i, ++t) {
          // over P of the step NB before. Its V is in then, so no wait for a
          // slot of the ring is two phases ahead of its barrier
          ok = mbar_wait(&o_done[sb.i], sb.ph ^ 1, p.err);
          const uint32_t ts = t_s + sb.i * kTreeTok;
          if constexpr (FP8) {
            ok = ok && mbar_wait(&kfull[at.i], at.ph, p.err);
            if (!ok) break;
            tc_fence_after();
            const uint64_t kd = kd0 + ((at.i * G::kK8) >> 4);
#pragma unroll
            for (int part = 0; part < 2; ++part)
#pragma unroll
              for (int k = 0; k < D / 32; ++k)
                umma_ss_e4m3(ts,
                             qd + ((part * kTreeRows * D + (k >> 2) * 1024 + (k & 3) * 32) >> 4),
                             kd + (((k >> 2) * 1024 + (k & 3) * 32) >> 4), idesc,
                             (part > 0 || k > 0) ? 1u : 0u);
            umma_commit(&s_full[sb.i]);
            umma_commit(&kempty[at.i]);
            at.next();
          } else {
#pragma unroll
            for (int ks = 0; ks < KS; ++ks) {
              ok = ok && mbar_wait(&full[at.i], at.ph, p.err);
              if (!ok) break;
              tc_fence_after();
              const uint64_t kd = kd0 + ((at.i * G::kSlot) >> 4);
#pragma unroll
              for (int k = 0; k < 8; ++k)
                umma_ss(ts, qd + (((ks * 2 + (k >> 2)) * 1024 + (k & 3) * 32) >> 4),
                        kd + (((k >> 2) * 1024 + (k & 3) * 32) >> 4), idesc,
                        (ks > 0 || k > 0) ? 1u : 0u);
              if (ks == KS - 1) umma_commit(&s_full[sb.i]);
              umma_commit(&empty[at.i]);
              at.next();
            }
            if (t >= G::kLead) {  // over V of step t - kLead
#pragma unroll
              for (int vs = 0; vs < VS; ++vs) at.next();
            }
          }
          sb.next();
        }
        if (!ok) break;
        umma_commit(q_empty);
        walk.skip(p, n);
      }
      // every product issued here has finished before tensor memory is released
      umma_commit(drained);
      (void)mbar_wait(drained, 0, p.err);
    }
  } else if (warp == G::kPvWarp) {
    // ---------------- the products O += P.V, issued by one lane
    if (elect_one()) {
      constexpr uint32_t idesc = FP8 ? umma_idesc_f16(128, D, true)
                                     : umma_idesc_bf16(128, D, true);
      const uint64_t vd0 = umma_sdesc(v16, 1024, NCH * 1024, 2);
      RingPos<FP8 ? 2 : NS> at;  // the next V's slot
      RingPos<NB> pb;
      if constexpr (!FP8)
        for (int i = v_seq<KS, VS>(0, count, G::kLead); i > 0; --i) at.next();
      int t = 0;
      bool ok = true;
      for (uint32_t seg = 0; walk.left > 0; ++seg) {
        // the segment before has left O
        if (seg > 0) ok = mbar_wait(o_free, (seg - 1) & 1, p.err);
        const int n = walk.run();
        const int tail = walk.q.ctx - (walk.st + n - 1) * kTreeTok;  // tokens of the last step
        for (int i = 0; i < n && ok; ++i, ++t) {
          // P first: S of the step is done then, so no wait for a slot of the
          // ring is two phases ahead of its barrier
          ok = mbar_wait(&p_full[pb.i], pb.ph, p.err);
          const uint32_t ps = t_s + pb.i * kTreeTok;
          // P of tokens 16 kk of the step: 8 columns, 32 to each half of S's columns
          auto pa = [&](int kk) { return ps + 64 * (kk / 4) + 8 * (kk % 4); };
          const int tok = i + 1 < n ? kTreeTok : tail;
#pragma unroll
          for (int vs = 0; vs < VS; ++vs) {
            uint64_t* f = FP8 ? &vfull[at.i] : &full[at.i];
            uint64_t* e = FP8 ? &vempty[at.i] : &empty[at.i];
            ok = ok && mbar_wait(f, at.ph, p.err);
            if (!ok) break;
            tc_fence_after();
            constexpr int kPer = G::kVTok / 16;  // k-steps of a slot
            const uint64_t vd = vd0 + ((at.i * (FP8 ? G::kV16 : G::kSlot)) >> 4);
            const uint32_t keep = i > 0 || vs > 0 ? 1u : 0u;
            if (tok >= kTreeTok) {
#pragma unroll
              for (int kk = 0; kk < kPer; ++kk)
                umma_bf16_ta(t_o, pa(vs * kPer + kk), vd + ((kk * 2 * NCH * 1024) >> 4), idesc,
                             kk > 0 ? 1u : keep);
            } else {
              const int k1 = min(kPer, (tok + 15) / 16 - vs * kPer);
              for (int kk = 0; kk < k1; ++kk)
                umma_bf16_ta(t_o, pa(vs * kPer + kk), vd + ((kk * 2 * NCH * 1024) >> 4), idesc,
                             kk > 0 ? 1u : keep);
            }
            if (vs == VS - 1) umma_commit(&o_done[pb.i]);
            umma_commit(e);
            at.next();
          }
          if (!FP8 && t + 1 + G::kLead < count) {  // over K of step t + 1 + kLead
#pragma unroll
            for (int ks = 0; ks < KS; ++ks) at.next();
          }
          pb.next();
        }
        if (!ok) break;
        walk.skip(p, n);
      }
      umma_commit(drained);
      (void)mbar_wait(drained, 0, p.err);
    }
  } else if (warp < G::kSoftWarps) {
    // ---------------- softmax: two threads per query row, 64 columns each, in
    // chunks of NC. d = 256: two, read twice, in loops that are not unrolled:
    // half the code and no spilled registers (64 x 4096 tokens x 21 drafts E4M3
    // 164 -> 148 us, 16 x 4096 x 64 94 -> 92 when it was introduced); d = 128:
    // one (in two 32 x 4096 x 64 drafts take 264 us instead of 249), at the
    // price of 12 bytes of spills (E4M3: 4)
    constexpr int NC = D == 256 ? 32 : 64;
    const int quad = warp & 3, half = warp >> 2;
    const int row = 32 * quad + lane;
    const uint32_t lane_off = static_cast<uint32_t>(32 * quad) << 16;
    const int g = p.group;
    bool first_seg = true;  // of this share
    uint32_t seg = 0;
    uint32_t swaps = 0;     // exchanges with the row's other thread so far
    if (walk.left > 0) {
      // Q of the share's first segment: these warps have nothing else to do yet
      const TreeQ<D, FP8, G::kSoftWarps> load(p, walk, warp, lane);
      load.run(sq, q_exp);
      mbar_arrive(q_first);
    }
    // v of the row's other thread; false if it does not come
    auto exchange = [&](float& v) {
      float* x = xch + (swaps & 1) * 256;
      x[half * 128 + row] = v;
      mbar_arrive(&pair[quad]);
      if (!__all_sync(0xffffffffu, mbar_wait(&pair[quad], swaps & 1, p.err))) return false;
      ++swaps;
      v = x[(half ^ 1) * 128 + row];
      return true;
    };
    RingPos<NB> sb, before_sb;  // S buffer of the step, of the step before
    bool ok = true;
    for (int t = 0; walk.left > 0 && ok;) {
      const int steps = walk.run();
      const int base_tok = walk.q.ctx - walk.q.n;
      const int r = walk.tile * kTreeRows + row;
      const bool live = r < walk.q.n * g;
      const int draft = live ? div_group(r, g) : 0;
      const int head = walk.h * g + (live ? r - draft * g : 0);
      uint64_t mask = p.tree_mask != nullptr ? p.tree_mask[walk.q.q0 + draft] : (2ull << draft) - 1;
      if (walk.q.n < 64) mask &= (1ull << walk.q.n) - 1;
      float m = -INFINITY, l = 0.f, qs = p.qscale;
      if constexpr (FP8) qs *= p.k_scale[walk.h];
      const int seg_st = walk.st;  // the segment's first step in its unit
      if (!FP8 && half == 0 && p.tree_mask != nullptr &&
          (seg_st + steps) * kTreeTok > base_tok) {
        // a segment with drafts. The exchange of its first step hands this to
        // the row's other thread, that of its sums keeps it until both have
        // read it
        const uint64_t any = drafts_seen(p, walk.q, lane);
        if (lane == 0) seen[quad] = any;
      }
      ok = false;  // until the segment is through
      int tok0 = seg_st * kTreeTok;
      for (int i = 0;; ++i, ++t, tok0 += kTreeTok) {
        const int b = sb.i;
        const bool begins = i == 0;
        if (!__all_sync(0xffffffffu, mbar_wait(&s_full[b], sb.ph, p.err))) break;
        tc_fence_after();
        if constexpr (FP8)
          if (begins) {
            // infinite or NaN queries give NaN
            const int ex = q_exp[seg % 3 * 128 + row];
            qs *= ex == -128 ? __uint_as_float(0x7FC00000u)
                             : __uint_as_float(static_cast<uint32_t>(127 - ex) << 23);
          }
        const uint32_t ts = t_s + lane_off + b * kTreeTok;
        const bool clean = tok0 + kTreeTok <= base_tok;  // committed tokens only
        // this thread's columns, 64 half .. 64 half + 63
        const uint32_t mine = ts + 64 * half;
        float sv[NC];
        // the logits of chunk c: raw, or (not clean) scaled and -inf where the
        // row does not see; it sees the committed tokens and those its mask names
        auto chunk = [&](int c) {
          if constexpr (NC == 64)
            tmem_ld64(mine, sv);
          else
            tmem_ld32(mine + NC * c, sv);
          if (clean) return;
#pragma unroll
          for (int w = 0; w < NC / 32; ++w) {
            const int sh = tok0 + 64 * half + NC * c + 32 * w - base_tok;  // first column's draft
            uint32_t see = ~0u;
            if (sh >= 64) see = 0;
            else if (sh >= 0) see = static_cast<uint32_t>(mask >> sh);
            else if (sh > -32) see = static_cast<uint32_t>(mask << -sh) | ((1u << -sh) - 1);
#pragma unroll
            for (int i = 0; i < 32; ++i)
              sv[32 * w + i] = (see >> i) & 1 ? sv[32 * w + i] * qs : -INFINITY;
          }
        };
        float m4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll 1
        for (int c = 0; c < 64 / NC; ++c) {
          chunk(c);
          if (!clean || qs >= 0.f) {
#pragma unroll
            for (int i = 0; i < NC; ++i) m4[i & 3] = fmaxf(m4[i & 3], sv[i]);
          } else {
#pragma unroll
            for (int i = 0; i < NC; ++i) m4[i & 3] = fmaxf(m4[i & 3], -sv[i]);
          }
        }
        float mx = fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3]));
        if (clean) mx *= fabsf(qs);
        float other = mx;
        if (!exchange(other)) break;
        mx = fmaxf(mx, other);
        // O is rescaled when the maximum grows by more than 2^8 (loads and
        // stores of tensor memory are warp-collective: all lanes or none)
        const bool want = mx > m + 8.f;
        if (__any_sync(0xffffffffu, want) && !begins) {
          if (!__all_sync(0xffffffffu,
                          mbar_wait(&o_done[before_sb.i], before_sb.ph, p.err)))
            break;
          tc_fence_after();
          const float alpha = want ? fast_exp2(m - mx) : 1.f;  // 0 while m is -inf
#pragma unroll 1
          for (int c = half * (D / 2); c < (half + 1) * (D / 2); c += 16) {
            float ov[16];
            tmem_ld16(t_o + lane_off + c, ov);
#pragma unroll
            for (int i = 0; i < 16; ++i) ov[i] *= alpha;
            tmem_st16(t_o + lane_off + c, ov);
          }
          if (want) l *= alpha;
        }
        if (want) m = mx;
        const float shift = (FP8 ? kTreeUp : 0.f) - (m == -INFINITY ? 0.f : m);
        // P over this thread's own columns of S, two tokens to a column (over
        // chunks that have been read)
        float l4[4] = {0.f, 0.f, 0.f, 0.f};
        const float by = clean ? qs : 1.f;
#pragma unroll 1
        for (int c = 0; c < 64 / NC; ++c) {
          if (NC < 64) chunk(c);
          uint32_t pw[NC / 2];
#pragma unroll
          for (int i = 0; i < NC / 2; ++i) {
            const float a = fast_exp2(fmaf(sv[2 * i], by, shift));
            const float e = fast_exp2(fmaf(sv[2 * i + 1], by, shift));
            l4[(2 * i) & 3] += a;
            l4[(2 * i + 1) & 3] += e;
            pw[i] = FP8 ? pack_f16(a, e) : pack_bf16(a, e);
          }
#pragma unroll
          for (int w = 0; w < NC / 32; ++w)
            tmem_st16_nowait(mine + NC / 2 * c + 16 * w, pw + 16 * w);
        }
        l += (l4[0] + l4[1]) + (l4[2] + l4[3]);
        if constexpr (!FP8) {
          // P is zero for the rows behind the context that the last product of
          // P.V covers and for the drafts that no row sees, but these rows
          // hold whatever was there, NaN included: zero them (E4M3: the
          // converters write zeros)
          const int valid = walk.q.ctx - tok0;
          const bool tail = valid < kTreeTok && (valid & 15) != 0;
          uint64_t hidden = 0;  // drafts of this step that no row sees
          if (!clean && p.tree_mask != nullptr) {
            const int b0 = max(0, tok0 - base_tok), b1 = min(walk.q.n, tok0 + kTreeTok - base_tok);
            hidden = ~seen[quad] & (~0ull << b0) & (~0ull >> (64 - b1));
          }
          if (tail || hidden != 0) {
            // the step before is waited for first: its V may have been the
            // slot's last use, and a wait must not be two phases ahead of its
            // barrier
            if (t >= 1 && !__all_sync(0xffffffffu, mbar_wait(&o_done[before_sb.i], before_sb.ph,
                                                             p.err)))
              break;
            const int v0 = v_seq<KS, VS>(t, count, G::kLead);
            // row r of the step, one warp to a row in turn
            int turn = 0;
            bool came = true;
            auto zero = [&](int r) {
              if (turn++ % G::kSoftWarps != warp || !came) return;
              const int at_v = v0 + r / G::kVTok, i = at_v % NS;
              came = __all_sync(0xffffffffu, mbar_wait(&full[i], (at_v / NS) & 1, p.err));
              if (!came || lane >= NCH * 8) return;  // 16-byte units of a row
              r %= G::kVTok;
              const uint32_t at = ring + i * G::kSlot + ((r / 8) * NCH + lane / 8) * 1024 +
                                  (r % 8) * 128 + ((lane % 8) ^ (r % 8)) * 16;
              asm volatile("st.shared.v4.u32 [%0], {%1,%1,%1,%1};" ::"r"(at), "r"(0u)
                           : "memory");
            };
            if (tail)
#pragma unroll 1
              for (int r = valid; r & 15; ++r) zero(r);
#pragma unroll 1
            for (uint64_t u = hidden; u != 0; u &= u - 1) zero(base_tok - tok0 + __ffsll(u) - 1);
            if (!came) break;
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
          }
        }
        tmem_wait_st();
        tc_fence_before();
        mbar_arrive(&p_full[b]);
        if (i + 1 == steps) {
          // ---- the segment's result, each thread d / 2 columns of its row
          other = l;
          if (!exchange(other)) break;
          const float sum = half == 0 ? l + other : other + l;
          if (!__all_sync(0xffffffffu, mbar_wait(&o_done[b], sb.ph, p.err))) break;
          tc_fence_after();
          const float inv = sum > 0.f ? (FP8 ? p.v_scale[walk.h] : 1.f) / sum : 0.f;
          const bool whole = seg_st == 0 && steps == walk.q.steps;
          const int c0 = half * (D / 2);
          const int64_t part = static_cast<int64_t>(cta) * 2 + (first_seg ? 0 : 1);
          if (whole) {
            uint16_t* dst = p.out +
                            (static_cast<int64_t>(walk.q.q0 + draft) * p.num_heads + head) * D + c0;
#pragma unroll 1
            for (int c = 0; c < D / 2; c += 16) {
              float ov[16];
              tmem_ld16(t_o + lane_off + c0 + c, ov);
              if (c + 16 == D / 2) {  // O is free; what is left are stores
                tc_fence_before();
                mbar_arrive(o_free);
              }
              if (live) {
                uint32_t w[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) w[i] = pack_bf16(ov[2 * i] * inv, ov[2 * i + 1] * inv);
                reinterpret_cast<uint4*>(dst + c)[0] = make_uint4(w[0], w[1], w[2], w[3]);
                reinterpret_cast<uint4*>(dst + c)[1] = make_uint4(w[4], w[5], w[6], w[7]);
              }
            }
          } else {
            // a partial, a column's rows side by side: full lines per store
            float* dst = p.part_o + (part * D + c0) * kTreeRows + row;
#pragma unroll 1
            for (int c = 0; c < D / 2; c += 16) {
              float ov[16];
              tmem_ld16(t_o + lane_off + c0 + c, ov);
              if (c + 16 == D / 2) {
                tc_fence_before();
                mbar_arrive(o_free);
              }
              if (live) {
#pragma unroll
                for (int i = 0; i < 16; ++i) dst[(c + i) * kTreeRows] = ov[i] * inv;
              }
            }
          }
          if (!whole && live && half == 0) {
            p.part_m[part * kTreeRows + row] = m;
            p.part_l[part * kTreeRows + row] = sum;
          }
          first_seg = false;
          ++seg;
          ok = true;
        }
        before_sb = sb;
        sb.next();
        if (ok) {
          ++t;
          break;
        }
      }
      walk.skip(p, steps);
    }
  } else if (!FP8 && warp >= G::kQWarp && warp < G::kQWarp + G::kQWarps) {
    // ---------------- Q of each segment but the first
    for (uint32_t seg = 1;; ++seg) {
      while (walk.left > 0 && !walk.ends()) walk.next(p);
      if (walk.left <= 1) break;
      walk.next(p);
      const TreeQ<D, FP8, G::kQWarps> load(p, walk, warp - G::kQWarp, lane);
      if (!__all_sync(0xffffffffu, mbar_wait(q_empty, (seg - 1) & 1, p.err))) break;
      load.run(sq, nullptr);
      mbar_arrive(q_full);
    }
  } else if constexpr (FP8) {
    // ---------------- converters: a staged V slot's codes -> their f16 values
    const int ct = threadIdx.x - G::kConvWarp * 32;
    constexpr int UPR = D / 16;  // 16-code units of a row
    constexpr int kCT = G::kConvWarps * 32;
    constexpr int kUnits = G::kSlot / 16 / kCT;
    // a thread's units lie kCT / UPR rows apart, a multiple of 8, at one place
    // of their rows: one swizzled address each and constant steps
    static_assert(kCT / UPR % 8 == 0, "row groups");
    constexpr uint32_t kSrcStep = kCT / UPR / 8 * NC8 * 1024, kDstStep = kCT / UPR / 8 * NCH * 1024;
    const int cu = ct % UPR, cr = ct / UPR;
    uint32_t src_at = ((cr / 8) * NC8 + cu / 8) * 1024 + (cr % 8) * 128 +
                      ((cu % 8) ^ (cr % 8)) * 16;
    uint32_t dst_at = ((cr / 8) * NCH + cu / 4) * 1024 + (cr % 8) * 128 +
                      ((2 * (cu % 4)) ^ (cr % 8)) * 16;
    // odd chunks store their second half first: the two chunks of a
    // quarter-warp then use different banks
    const uint32_t second = (cu >> 2) & 1;
    dst_at ^= second * 16;
    RingPos<NS> from;
    RingPos<2> to;
    // Q of a segment is loaded as soon as V of the segment before is converted
    // and its last S is done
    auto load_q = [&](uint32_t seg) {
      const TreeQ<D, FP8, G::kQWarps> load(p, walk, warp - G::kConvWarp, lane);
      if (!__all_sync(0xffffffffu, mbar_wait(q_empty, (seg - 1) & 1, p.err))) return false;
      load.run(sq, q_exp + seg % 3 * 128);
      mbar_arrive(q_full);
      return true;
    };
    uint32_t seg = 1;  // the first segment's Q is not theirs
    bool ok = true;
    for (int vs = 0; walk.left > 0 && ok;) {
      if (!(ok = __all_sync(0xffffffffu, mbar_wait(&full[from.i], from.ph, p.err)))) break;
      const uint32_t src0 = ring + from.i * G::kSlot, dst0 = v16 + to.i * G::kV16;
      uint32_t c[kUnits][4];
#pragma unroll
      for (int e = 0; e < kUnits; ++e) {
        asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
                     : "=r"(c[e][0]), "=r"(c[e][1]), "=r"(c[e][2]), "=r"(c[e][3])
                     : "r"(src0 + src_at + e * kSrcStep)
                     : "memory");
      }
      if (!(ok = __all_sync(0xffffffffu, mbar_wait(&vempty[to.i], to.ph ^ 1, p.err)))) break;
#pragma unroll
      for (int e = 0; e < kUnits; ++e) {
        if (second) {
          const uint32_t c0 = c[e][0], c1 = c[e][1];
          c[e][0] = c[e][2];
          c[e][1] = c[e][3];
          c[e][2] = c0;
          c[e][3] = c1;
        }
        uint32_t w[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) w[i] = e4m3x2_f16x2(c[e][i / 2], i & 1);
        const uint32_t dst = dst0 + dst_at + e * kDstStep;
        asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(dst), "r"(w[0]), "r"(w[1]),
                     "r"(w[2]), "r"(w[3])
                     : "memory");
        asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(dst ^ 16), "r"(w[4]),
                     "r"(w[5]), "r"(w[6]), "r"(w[7])
                     : "memory");
      }
      // the rows of drafts that no row sees and those behind the context that
      // the last product of P.V covers may hold anything, NaN included, and P =
      // 0 does not hide it: zeros. A rolled loop, each thread over its own
      // units: in registers before the conversion 64 x 4096 tokens x 21 drafts
      // take 157 us instead of 151
      const int draft0 = walk.q.ctx - walk.q.n - walk.st * kTreeTok;  // the first draft's row
      if (draft0 < kTreeTok) {
        const int valid = draft0 + walk.q.n;
        const uint64_t seen = p.tree_mask ? drafts_seen(p, walk.q, lane) : ~0ull;
#pragma unroll 1
        for (int e = 0; e < kUnits; ++e) {
          const int r = vs * G::kVTok + cr + e * (kCT / UPR);
          if (r >= valid ? r < ((valid + 15) & ~15) : r >= draft0 && !(seen >> (r - draft0) & 1)) {
            const uint32_t dst = dst0 + dst_at + e * kDstStep;
            asm volatile("st.shared.v4.u32 [%0], {%1,%1,%1,%1};" ::"r"(dst), "r"(0u) : "memory");
            asm volatile("st.shared.v4.u32 [%0], {%1,%1,%1,%1};" ::"r"(dst ^ 16), "r"(0u)
                         : "memory");
          }
        }
        __syncwarp();
      }
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      __syncwarp();
      // the codes' slot is given back only now that they have been used: an
      // arrival does not wait for loads that are merely issued, and the next
      // codes would overwrite what they are still to read
      if (lane == 0) {
        mbar_arrive(&vfull[to.i]);
        mbar_arrive(&empty[from.i]);
      }
      from.next();
      to.next();
      if (++vs == VS) {
        vs = 0;
        const bool last = walk.ends();
        walk.next(p);
        if (last && walk.left > 0) ok = load_q(seg++);
      }
    }
  }

  allow_dependents();  // the merge may be scheduled; it waits for this grid
  tc_fence_before();
  __syncthreads();
  if (warp >= G::kProdWarp && warp < G::kProdWarp + G::kProducers && lane == 0) {
    // no copy may still be writing this CTA's shared memory when it exits
    for (uint32_t i = issued > NS ? issued - NS : 0; i < issued; ++i)
      if (!mbar_wait(&full[i % NS], (i / NS) & 1, p.err)) break;
    for (uint32_t i = issued_k > NK8 ? issued_k - NK8 : 0; i < issued_k; ++i)
      if (!mbar_wait(&kfull[i % NK8], (i / NK8) & 1, p.err)) break;
  }
  if (warp == G::kSWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, G::kCols);
  }
}

// Joins the partials of the units that were cut: CTA (x, y) takes columns
// 8 y .. of a unit, thread (i, r) of it the parts i, i + GROUPS, ... of row r.
// With m_i, l_i, o_i of the unit's segments, M = max m_i (base 2) and w_i =
// l_i 2^(m_i - M): out = sum (w_i / sum w) o_i. GROUPS = 1 where units have few
// parts: x is the share that a unit starts in, as most have one. GROUPS = 4
// where few units are cut into many: x counts the units that were cut. Whole
// call, GROUPS 1 / 4: 1 x 8192 tokens, 32 parts a unit 23.1 / 18.2 us, 16 parts
// 18.1 / 16.3.
constexpr int kMergeCols = 8;

// A load that stays where it is: a plain one is moved next to its use to save
// registers, one latency after the other (the merge of 5 parts: 9.6 us, so 4.1).
__device__ __forceinline__ float load_now(const float* x) {
  float v;
  asm volatile("ld.relaxed.gpu.global.f32 %0, [%1];" : "=f"(v) : "l"(x) : "memory");
  return v;
}

template <int D, int GROUPS>
__global__ void __launch_bounds__(GROUPS * kTreeRows)
    tree_merge_kernel(const __grid_constant__ TreeParams p) {
  wait_prerequisite();
  int c = blockIdx.x;
  if constexpr (GROUPS > 1) {
    // the x-th share that has a unit to merge
    __shared__ int below[kTreeMaxCtas / 32], mine;
    static_assert(GROUPS * kTreeRows >= kTreeMaxCtas && kTreeMaxCtas % 32 == 0, "a thread each");
    const int t = threadIdx.x;
    const bool has = t < p.ctas && p.meta[t].parts > 0;
    const uint32_t with = __ballot_sync(0xffffffffu, has);
    if (t < kTreeMaxCtas && t % 32 == 0) below[t / 32] = __popc(with);
    if (t == 0) mine = -1;
    __syncthreads();
    if (has) {
      int rank = __popc(with & ((1u << (t % 32)) - 1));
      for (int w = 0; w < t / 32; ++w) rank += below[w];
      if (rank == c) mine = t;
    }
    __syncthreads();
    c = mine;
    if (c < 0) return;
  }
  const TreeMeta md = p.meta[c];
  if (md.parts == 0) return;
  const int row = threadIdx.x % kTreeRows, grp = threadIdx.x / kTreeRows;
  const int c0 = blockIdx.y * kMergeCols;
  const bool live = row < md.rows;
  constexpr int kMergeParts = GROUPS == 1 ? 4 : 5;  // parts whose loads are in flight at once
  // partial i: the first is share c's, the others are slot 0 of the next shares
  auto at = [&](int i) { return (c + i * md.stride) * 2 + (i == 0 ? md.slot : 0); };
  float M = -INFINITY, W = 0.f, acc[kMergeCols];
#pragma unroll
  for (int i = 0; i < kMergeCols; ++i) acc[i] = 0.f;
  if (live) {
    // several parts at a time, with a running maximum
    for (int i = grp; i < md.parts; i += kMergeParts * GROUPS) {
      float x[kMergeParts][kMergeCols], m[kMergeParts], l[kMergeParts];
#pragma unroll
      for (int k = 0; k < kMergeParts; ++k) {
        m[k] = -INFINITY;
        l[k] = 0.f;
#pragma unroll
        for (int e = 0; e < kMergeCols; ++e) x[k][e] = 0.f;
        if (i + k * GROUPS < md.parts) {
          const int64_t a = at(i + k * GROUPS);
          m[k] = load_now(p.part_m + a * kTreeRows + row);
          l[k] = load_now(p.part_l + a * kTreeRows + row);
#pragma unroll
          for (int e = 0; e < kMergeCols; ++e)
            x[k][e] = load_now(p.part_o + (a * D + c0 + e) * kTreeRows + row);
        }
      }
      float top = M;
#pragma unroll
      for (int k = 0; k < kMergeParts; ++k) top = fmaxf(top, m[k]);
      const float ref = top == -INFINITY ? 0.f : top;
      const float f = fast_exp2(M - ref);
      M = top;
      W *= f;
#pragma unroll
      for (int e = 0; e < kMergeCols; ++e) acc[e] *= f;
#pragma unroll
      for (int k = 0; k < kMergeParts; ++k) {
        const float w = l[k] * fast_exp2(m[k] - ref);
        W += w;
#pragma unroll
        for (int e = 0; e < kMergeCols; ++e) acc[e] = fmaf(w, x[k][e], acc[e]);
      }
    }
  }
  constexpr int E = kMergeCols / GROUPS;  // columns a thread writes
  float o[E], sum;
  if constexpr (GROUPS == 1) {
    if (!live) return;
    sum = W;
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] = acc[e];
  } else {
    __shared__ float sm_m[GROUPS][kTreeRows], sm_w[GROUPS][kTreeRows];
    __shared__ float sm_o[GROUPS][kMergeCols][kTreeRows];
    sm_m[grp][row] = M;
    sm_w[grp][row] = W;
#pragma unroll
    for (int e = 0; e < kMergeCols; ++e) sm_o[grp][e][row] = acc[e];
    __syncthreads();
    if (!live) return;
    float top = sm_m[0][row];
#pragma unroll
    for (int i = 1; i < GROUPS; ++i) top = fmaxf(top, sm_m[i][row]);
    float f[GROUPS];
    sum = 0.f;
#pragma unroll
    for (int i = 0; i < GROUPS; ++i) {
      f[i] = sm_m[i][row] == -INFINITY ? 0.f : fast_exp2(sm_m[i][row] - top);
      sum = fmaf(f[i], sm_w[i][row], sum);
    }
#pragma unroll
    for (int e = 0; e < E; ++e) {
      o[e] = 0.f;
#pragma unroll
      for (int i = 0; i < GROUPS; ++i) o[e] = fmaf(f[i], sm_o[i][grp * E + e][row], o[e]);
    }
  }
  const float inv = sum > 0.f ? 1.f / sum : 0.f;
  const int r = md.first + row, draft = div_group(r, p.group);
  const int64_t hq = static_cast<int64_t>(md.row0 + draft) * p.num_heads + md.head * p.group +
                     (r - draft * p.group);
  uint32_t* dst = reinterpret_cast<uint32_t*>(p.out + hq * D + c0 + (E > 1 ? grp * E : 0));
  if constexpr (E == 8) {
    *reinterpret_cast<uint4*>(dst) =
        make_uint4(pack_bf16(o[0] * inv, o[1] * inv), pack_bf16(o[2] * inv, o[3] * inv),
                   pack_bf16(o[4] * inv, o[5] * inv), pack_bf16(o[6] * inv, o[7] * inv));
  } else if constexpr (E == 2) {
    *dst = pack_bf16(o[0] * inv, o[1] * inv);
  } else {
    p.out[hq * D + c0 + grp] = float_to_bf16_bits(o[0] * inv);
  }
}

// ---------------------------------------------------------------- host side

// 4-D map of a pool, [8-row group][128-byte chunk][8 rows][128 bytes], boxes of
// `chunks` chunks of one page.
static int tree_pool_map(CUtensorMap* out, const void* base, int64_t rows, int D, int B, bool fp8,
                         int chunks) {
  auto enc = tensor_map_encoder();
  if (!enc) return PKV_ERR_CUDA;
  const cuuint64_t row = static_cast<cuuint64_t>(D) * (fp8 ? 1 : 2);
  const cuuint32_t elems = fp8 ? 128 : 64;
  cuuint64_t dims[4] = {elems, 8, row / 128, static_cast<cuuint64_t>(rows / 8)};
  cuuint64_t strides[3] = {row, 128, 8 * row};
  cuuint32_t box[4] = {elems, 8, static_cast<cuuint32_t>(chunks), static_cast<cuuint32_t>(B / 8)};
  cuuint32_t estr[4] = {1, 1, 1, 1};
  const CUresult r =
      enc(out, fp8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4,
          const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
          CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
          CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? PKV_OK : PKV_ERR_CUDA;
}

template <int D, bool FP8>
static int launch_tree(const TreeParams& p, const void* k_cache, const void* v_cache, int ctas,
                       int64_t units, cudaStream_t st) {
  using G = TreeGeom<D, FP8>;
  const int64_t rows = static_cast<int64_t>(p.num_blocks) * p.num_kv_heads * p.block_size;
  CUtensorMap tk, tv;
  int rc = tree_pool_map(&tk, k_cache, rows, D, p.block_size, FP8, FP8 ? D / 128 : 2);
  if (rc != PKV_OK) return rc;
  rc = tree_pool_map(&tv, v_cache, rows, D, p.block_size, FP8, FP8 ? D / 128 : D / 64);
  if (rc != PKV_OK) return rc;
  static DeviceFlags done;
  auto kern = tree_kernel<D, FP8>;
  rc = ensure_smem(kern, G::kSmem, done);
  if (rc != PKV_OK) return rc;
  rc = launch_dependent(kern, dim3(ctas), dim3(G::kThreads), G::kSmem, st, tk, tv, p);
  if (rc != PKV_OK) return rc;
  // parts of a unit, if all are equally long: at most ctas over the units
  const int64_t pairs = static_cast<int64_t>(p.num_seqs) * p.num_kv_heads;
  const bool many = ctas > 12 * pairs;
  const int few = static_cast<int>(std::min<int64_t>(ctas, units));
  constexpr int GR = 4, Y = D / kMergeCols;
  return many ? launch_dependent(tree_merge_kernel<D, GR>, dim3(few, Y), dim3(GR * kTreeRows), 0,
                                 st, p)
              : launch_dependent(tree_merge_kernel<D, 1>, dim3(ctas, Y), dim3(kTreeRows), 0, st,
                                 p);
}

}  // namespace pkv

extern "C" size_t pkv_tree_workspace_bytes(int num_seqs, int num_queries, int num_heads,
                                           int num_kv_heads, int head_dim, int max_context,
                                           int max_draft) {
  using namespace pkv;
  if (num_seqs <= 0 || num_queries <= 0 || num_heads <= 0 || num_kv_heads <= 0 || head_dim <= 0 ||
      max_context < 0 || max_draft <= 0)
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
                                               max_context, max_draft);
  if (!q_start || !workspace || !aligned16(workspace) || workspace_bytes < need)
    return PKV_ERR_INVALID_ARG;
  // the most that the call's bounds allow
  const int64_t tiles_most =
      num_seqs + static_cast<int64_t>(num_queries) * g / kTreeRows;
  const int64_t units = tiles_most * cache.num_kv_heads;
  const int64_t longest = (static_cast<int64_t>(max_context) + kTreeTok - 1) / kTreeTok;
  // places of the line are 32-bit numbers (a q_start that is not ascending may
  // ask for up to four times the work: a sequence has at most four row tiles)
  if (units * (longest + kTreeStart) >= (1 << 29)) return PKV_ERR_UNSUPPORTED;
  const size_t q_bytes = static_cast<size_t>(num_queries) * num_heads * cache.head_dim * 2;
  if (overlap(out, q_bytes, q, q_bytes)) return PKV_ERR_INVALID_ARG;
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
  p.max_context = max_context;
  p.num_blocks = cache.num_blocks;
  p.num_kv_heads = cache.num_kv_heads;
  p.num_heads = num_heads;
  p.group = g;
  p.block_size = cache.block_size;
  p.max_blocks_per_seq = max_blocks_per_seq;
  p.qscale = scale * 1.4426950408889634f;
  // no more CTAs than the call's bounds can give work
  const int ctas = static_cast<int>(std::max<int64_t>(
      1, std::min<int64_t>(std::min(sms, kTreeMaxCtas), units * longest)));
  p.ctas = ctas;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const bool fp8 = cache.dtype == PKV_DTYPE_FP8_E4M3;
  if (cache.head_dim == 128)
    return fp8 ? launch_tree<128, true>(p, k_cache, v_cache, ctas, units, st)
               : launch_tree<128, false>(p, k_cache, v_cache, ctas, units, st);
  return fp8 ? launch_tree<256, true>(p, k_cache, v_cache, ctas, units, st)
             : launch_tree<256, false>(p, k_cache, v_cache, ctas, units, st);
}

// attn_kernel.cuh -- attention of new tokens over a paged key-value cache.
//
// For a kv head and the rows r = (new token i, head g of the group) that read it,
//
//     out_r = sum_j p_rj v_j / sum_j p_rj,   p_rj = 2^(z_rj - m_r),   z = scale log2(e) q.k
//
// in one pass over the keys with a running maximum m and sum l. The keys and values are
// read once from HBM and carry 2 G multiply-adds a byte (G rows), so the copy rate bounds
// it; the work is cut so that every SM streams the same number of tokens:
//
//   - An item is one (sequence, kv head, tile of M = 8 NR WR rows). Its keys are cut into
//     stages of 64 tokens (128 with 8-bit elements). All stages of all items, in order, with
//     a fixed charge for every item's start and end, are divided evenly among the CTAs; a CTA
//     works through its range segment by segment (a segment is its part of one item).
//   - Two warps fill a ring of stages, looking up the pages; they run ahead across segments,
//     so the next item's keys stream while the last one is joined and written. Where pages
//     are made of whole blocks of 8 or more tokens, a lane issues one TMA box per block and
//     128 bytes of the head; otherwise 16-byte asynchronous copies, each row looked up by
//     itself, write the same layout.
//   - Four warps multiply. WR of them share the rows, 4 / WR the tokens of a stage: with few
//     rows each warp takes a quarter of the tokens with its own m, l and output accumulators
//     (no exchange until the segment ends), with 64 rows each takes 16 of them and all
//     tokens. Both products run on mma.sync m16n8k16 with the tokens (for the weights times
//     values: the head's elements) as M and the rows as N, eight at a time: a decode step
//     has 4 to 8 rows a kv head, and with the rows as M half of the products or more would
//     be padding. Scores and weights stay in registers.
//   - At the end of a segment the warps' (m, l, out) are joined in the memory of the
//     segment's last stage. An item that lies in one CTA is finished there; otherwise each
//     CTA stores its fp32 partial in the workspace, and the last to arrive at the item's
//     counter adds them in CTA order: the result depends on the lengths only.
//
// e4m3 caches are widened to f16 in registers (every e4m3 value is an f16 value); q is
// scaled by a power of two per row so that its largest element is in [2^14, 2^15) and converted
// to f16: exact but for elements 2^-31 below the row's largest. The key scale joins the
// score's factor, the value scale the last division.
//
// Measured with 8 rows a kv head (64 sequences of 0 to 8192 tokens, 8 kv heads of 128, 1045 MB):
// 161 to 163 us, 6.4 TB/s, where a plain copy moves 6.76; an e4m3 cache over 1024 to 16384
// tokens (951 MB) 150 to 152 us; one sequence of 131072 tokens (537 MB) 90 us. Short calls are
// chains of latencies: one sequence of 777 tokens takes 9.8 us where its bytes take 0.1 (start
// and lengths, the first stage from HBM, a stage or two of products, and the join's way
// through global memory: partial results, the counter, the parts read back).
//
// Every wait on an mbarrier is bounded; after a time-out the waits return at once, nothing
// more is copied, and the control flow, which depends on the lengths alone, runs to its end
// over stale data. Copies still on their way are waited for after the last wait of any warp.
#pragma once

#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "attn.h"
#include "common.cuh"

namespace ssd {
namespace {

constexpr int AT_CWARPS = 4;  // warps that multiply
constexpr int AT_PWARPS = 2;  // warps that copy
constexpr int AT_CTHREADS = 32 * AT_CWARPS;
constexpr int AT_THREADS = 32 * (AT_CWARPS + AT_PWARPS);
constexpr int AT_GROUP = 16;     // workers whose parts of a much split item are joined first
// An item costs what four stages do (its q, partial results, the join): with a charge of one,
// 28 sequences of 150 to 320 tokens with heads of 256 take 17.2 us instead of 16.1, 3 long ones under a
// window 24.8 instead of 23.0. Shares of two stages and more: with four, a single
// sequence of 1024 tokens takes 11.0 us instead of 9.8.
constexpr int AT_ITEM_COST = 4, AT_LEAST = 2;
// Weights are powers of two of a score less the running maximum, and as many times larger as
// these powers say: those that round to f16 (8-bit caches) then keep 11 bits down to 2^-21 of the
// largest, and are off by at most 2^-32 of it below (unscaled, 2^-25, and a long flat tail of
// weights under that was lost to the outputs, not to the sum they are divided by). Seven: the
// largest f16 is just below 2^16, weights under the maximum that lags by 8 (attn_tc.cuh) reach
// 2^15, and no rounding of a huge maximum less seven can be off by as much again.
constexpr float F16_POWERS = 7.0f;
constexpr float LOG2E = 1.4426950408889634f, LN2 = 0.6931471805599453f;

template <bool E4M3, int DP, int NR, int WR>
struct AttnCfg {
  static constexpr int ES = E4M3 ? 1 : 2;        // bytes of a cache element
  static constexpr int MW = 8 * NR;              // rows of a warp
  static constexpr int M = MW * WR;              // rows of an item
  static constexpr int SPAN = E4M3 ? 32 : 16;    // tokens of a stage for each warp
  static constexpr int TOK = AT_CWARPS * SPAN;   // tokens of a stage
  // Tokens of an inner step (e4m3, 16 rows a warp, 64 or, heads of 256, 24 ragged sequences; in
  // brackets bytes of spill stores a thread): heads of 128 140 us with 16 (56 to 76), 199 with
  // 32 (336 to 524); heads of 256 127 (432) and 200 (396 to 840). Heads up to 64 spill in
  // neither, and there 32 is the faster one, 73 us where 16 takes 92: not yet told apart.
  static constexpr int STEP = NR == 1 ? SPAN : 16;
  static constexpr int RB = DP * ES;             // bytes of a token's row in a stage
  static constexpr int CPR = RB / 16;            // 16-byte chunks of a row
  static constexpr int STAGE = 2 * TOK * RB;     // K then V
  static constexpr int ST = DP == 64 ? 4 : (DP == 128 && WR == 4 ? 2 : 3);
  static constexpr int QB = WR == 1 || (DP == 128 && WR == 4) ? 2 : 1;  // buffers of q
  static constexpr int QBYTES = M * DP * 2;
  static constexpr size_t SMEM = ST * STAGE + QB * QBYTES;
  static constexpr int CTAS = DP <= 128 ? 2 : 1;  // per SM
  // one partial result: M rows of DP outputs, then m and l of the rows
  static constexpr int SLOT = M * DP + 2 * M;
  // the join buffer, a row of DP floats for each row of each warp, fits a stage
  static_assert(STAGE >= AT_CWARPS * MW * DP * 4, "join buffer");
};

// True in one thread of the (converged) warp. Under this predicate the compiler knows that a
// single thread issues the copies and products, whose operands are uniform registers; under
// `lane == 0` it serialised them over the warp (125 clocks a product).
__device__ __forceinline__ bool elect_one() {
  uint32_t yes;
  asm volatile(
      "{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(yes));
  return yes != 0;
}
__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm4_t(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
template <bool F16>
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1) {
  if (F16)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// 16 bytes global -> shared; zeros where !valid (nothing is read).
__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src, bool valid) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
               "r"(valid ? 16 : 0)
               : "memory");
}
// Arrive on `bar` once this thread's copies so far have landed.
__device__ __forceinline__ void cp_async_arrive(uint64_t *bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar))
               : "memory");
}
__device__ __forceinline__ void cp_async_wait_all() {
  asm volatile("cp.async.wait_all;" ::: "memory");
}
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// two e4m3 (low 16 bits) -> two f16
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t x) {
  uint32_t y;
  asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, lo;\n\t}"
      : "=r"(y)
      : "r"(x));
  return y;
}
template <bool F16>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  uint32_t y;
  if (F16) asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(y) : "f"(hi), "f"(lo));
  else asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(y) : "f"(hi), "f"(lo));
  return y;
}
__device__ __forceinline__ float power_of_two(int e) {  // e in [-126, 127]
  return __uint_as_float(static_cast<uint32_t>(e + 127) << 23);
}
// The power of two that a row of q whose largest element is mx is divided by on its way to f16:
// the largest is then in [2^14, 2^15) (smaller where mx is below 2^-112; infinities leave
// finite elements finite), and elements down to 2^-31 of it are exact, as bf16's eight bits
// end above f16's last, 2^-24. At most 114.
__device__ __forceinline__ int q_exponent(float mx) {
  return max(static_cast<int>(__float_as_uint(mx) >> 23) - 127 - 14, -126);
}
// Transposes an 8 x 8 matrix of 16-bit elements held as one register a lane.
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
// One box (64 or 128 bytes of the head x tokens of one page and kv head) into shared memory.
__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap *map, uint64_t *bar,
                                            int c0, int c1, int c2, int c3) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(c0), "r"(c1), "r"(c2),
      "r"(c3)
      : "memory");
}
// Byte offset of 16-byte chunk `ch` of row `row` in a tile of ROWS rows of RB bytes: slabs of
// 128 bytes a row, the chunk's place in its 128 bytes exchanged by the row (TMA's 128-byte
// swizzle; the 64-byte one for rows of 64 bytes), so that eight rows' equal chunks lie in
// different banks.
template <int RB, int ROWS>
__device__ __forceinline__ uint32_t swz(int row, int ch) {
  if (RB == 64) return row * 64 + ((ch ^ ((row >> 1) & 3)) << 4);
  return (ch >> 3) * (ROWS * 128) + row * 128 + (((ch & 7) ^ (row & 7)) << 4);
}

// One sequence's rows and keys.
struct SeqInfo {
  int q0, n;       // first row, rows
  int len, begin;  // keys [begin, len) that some row can see
  int kt;          // stages of keys (at least 1: an empty row still has to be written)
  int rt;          // row tiles
  __device__ __forceinline__ long long units(int Hkv, int cost) const {
    return static_cast<long long>(Hkv) * rt * (kt + cost);
  }
};

template <int TOK, int M>
__device__ __forceinline__ SeqInfo seq_info(const AttnParams &p, int G, int s) {
  SeqInfo x;
  x.q0 = s;
  x.n = 1;
  if (p.q_start) {
    x.q0 = min(max(p.q_start[s], 0), p.T);
    x.n = max(0, min(max(p.q_start[s + 1], 0), p.T) - x.q0);
  }
  // what the table holds, and no token number of a stage's end passes 2^31
  const long long cap =
      min(static_cast<long long>(p.max_pages) * p.c.page_size, 0x7fffff00ll);
  x.len = static_cast<int>(min(static_cast<long long>(max(p.seq_len[s], 0)), cap));
  const int pos = x.len - x.n;  // the first row's
  x.begin = p.window > 0 && pos >= p.window ? pos - p.window + 1 : 0;
  if (p.box > 0) x.begin &= -p.box;  // whole boxes
  x.kt = x.len > x.begin ? (x.len - x.begin - 1) / TOK + 1 : 1;
  x.rt = (x.n * G + M - 1) / M;
  return x;
}

struct AttnPlan {
  float *partials;
  int *counters, *group_counters;
  unsigned *status;
  uint64_t wait_limit_ns;
  int hold;  // self-test: waits that run out (dec_debug_attn_timeout)
};

// All items' units in order (an item: its COST, then one per stage), and worker c's
// share of them: share_n, one more for the first share_r workers.
struct Shares {
  long long share_n, share_r;
  __device__ __forceinline__ int worker_of(long long unit) const {
    const long long longer = share_r * (share_n + 1);
    return static_cast<int>(unit < longer ? unit / (share_n + 1)
                                          : share_r + (unit - longer) / share_n);
  }
};

// Walks the segments of one CTA's range. TOK: tokens of a stage; M: rows of an item; COST:
// stages that an item's start and end are charged as; LEAST: units of the smallest share.
template <int TOK, int M, int COST, int LEAST>
struct Cursor {
  long long cur, end, item;  // next unit, end of the range, first unit of the item
  int s, hk, rt, t0, t1;     // segment: stages [t0, t1) of item (s, hk, rt)
  SeqInfo x;
  // The next segment that has a stage; false at the end of the range.
  __device__ __forceinline__ bool next(const AttnParams &p, int G) {
    while (cur < end) {
      const long long stop = item + COST + x.kt;
      if (cur == stop) {  // the next item
        item = cur;
        if (++rt == x.rt) {
          rt = 0;
          if (++hk == p.Hkv) {
            hk = 0;
            do x = seq_info<TOK, M>(p, G, ++s);
            while (x.rt == 0);
          }
        }
        continue;
      }
      const long long from = cur, to = stop < end ? stop : end;
      cur = to;
      t0 = static_cast<int>(max(from - item - COST, 0ll));
      t1 = static_cast<int>(to - item - COST);
      if (t1 > t0) return true;
    }
    return false;
  }
};

// This CTA's share of all units, found in one pass over the sequences by the whole CTA;
// false: the work does not reach this CTA. Holds a barrier before any shared memory written
// by one thread before the call is read by others after it.
template <int THREADS>
struct RangeStart {
  long long warp_sum[THREADS / 32];
  long long off;
  int seq;
};
template <int THREADS, int TOK, int M, int COST, int LEAST>
__device__ __forceinline__ bool begin_range(const AttnParams &p, int G,
                                            RangeStart<THREADS> &start, Shares &sh,
                                            Cursor<TOK, M, COST, LEAST> &c) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, me = blockIdx.x;
  const int per = (p.S + THREADS - 1) / THREADS;
  const int s_lo = min(tid * per, p.S), s_hi = min(s_lo + per, p.S);
  long long mine = 0;
  for (int s = s_lo; s < s_hi; ++s) mine += seq_info<TOK, M>(p, G, s).units(p.Hkv, COST);
  long long incl = mine;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, incl, d);
    if (lane >= d) incl += y;
  }
  if (lane == 31) start.warp_sum[warp] = incl;
  __syncthreads();
  long long total = 0, before = 0;
#pragma unroll
  for (int w = 0; w < THREADS / 32; ++w) {
    if (w < warp) before += start.warp_sum[w];
    total += start.warp_sum[w];
  }
  const long long most = (total + LEAST - 1) / LEAST;
  const int workers = static_cast<int>(most < gridDim.x ? most : gridDim.x);
  if (me >= workers) return false;
  sh.share_n = total / workers;
  sh.share_r = total % workers;
  c.cur = me * sh.share_n + min(static_cast<long long>(me), sh.share_r);
  c.end = c.cur + sh.share_n + (me < sh.share_r ? 1 : 0);
  long long at = before + incl - mine;  // units before this thread's sequences
  if (at <= c.cur && c.cur < at + mine) {
    for (int s = s_lo; s < s_hi; ++s) {
      const long long n = seq_info<TOK, M>(p, G, s).units(p.Hkv, COST);
      if (c.cur < at + n) {
        start.seq = s;
        start.off = c.cur - at;
        break;
      }
      at += n;
    }
  }
  __syncthreads();
  c.s = start.seq;
  c.x = seq_info<TOK, M>(p, G, c.s);
  const long long per_item = c.x.kt + COST, i = start.off / per_item;
  c.hk = static_cast<int>(i / c.x.rt);
  c.rt = static_cast<int>(i - static_cast<long long>(c.hk) * c.x.rt);
  c.item = c.cur - (start.off - i * per_item);
  return true;
}

// What a copying warp brings of a stage by TMA: HALF tokens of K and V in blocks of `box` tokens
// of one page. The pages of 32 blocks are looked up in one step, a step ahead, and the boxes
// leave from one thread with uniform operands. (With a look-up each stage and a box a lane, a
// warp took 0.6 us a stage, however few bytes it had: 64 ragged sequences with heads of 64
// and pages of 16 tokens took 100 us instead of 88.) Its loops stay loops: unrolled, their
// instructions crowd out the multiplying warps' (e4m3 heads of 256: 113 us instead of 107).
template <int RB, int TOK, int HALF, int ES>
struct Boxes {
  static constexpr int SLABS = RB == 64 ? 1 : RB / 128, ROW = RB == 64 ? 64 : 128;
  int lg, nb, per;  // log2 of the box, blocks of a stage, stages of a step
  int page, off, next_page, next_off;  // lane: block lane % nb of the step's stage lane / nb
  uint32_t exist;                      // blocks whose page exists
  __device__ __forceinline__ explicit Boxes(int box) {
    lg = 31 - __clz(box);
    nb = HALF >> lg;
    per = 32 / nb;
  }
  template <typename Cur>
  __device__ __forceinline__ void look_up(const AttnParams &p, const Cur &c, int from, int pw,
                                          int lane, int &pg, int &of) const {
    const int t = from + lane / nb;
    pg = -1;
    of = 0;
    if (t < c.t1) {
      const int j = c.x.begin + t * TOK + pw * HALF + ((lane & (nb - 1)) << lg);
      if (j < c.x.len) {
        const int i = j / p.c.page_size;
        of = j - i * p.c.page_size;
        pg = p.block_table[static_cast<long long>(c.s) * p.max_pages + i];
        if (pg >= p.c.num_pages) pg = -1;
      }
    }
  }
  // At each stage of a segment in turn, before issue().
  template <typename Cur>
  __device__ __forceinline__ void step(const AttnParams &p, const Cur &c, int t, int pw,
                                       int lane) {
    const int i = (t - c.t0) & (per - 1);
    if (i == 0) {
      if (t == c.t0) {
        look_up(p, c, t, pw, lane, page, off);
      } else {
        page = next_page;
        off = next_off;
      }
      exist = __ballot_sync(0xffffffffu, page >= 0);
    }
  }
  // After issue(): the next step's pages.
  template <typename Cur>
  __device__ __forceinline__ void ahead(const AttnParams &p, const Cur &c, int t, int pw,
                                        int lane) {
    if (((t - c.t0) & (per - 1)) == 0) look_up(p, c, t + per, pw, lane, next_page, next_off);
  }
  // The boxes of stage t into stage memory `dst` (K, then V TOK * RB bytes on). Writes the
  // bits of the tokens that exist and arrives on `full` with the bytes to come.
  template <typename Cur>
  __device__ __forceinline__ void issue(const CUtensorMap *kmap, const CUtensorMap *vmap,
                                        const Cur &c, int t, int pw, uint32_t dst,
                                        uint64_t *full, uint32_t *valid) const {
    const int i = (t - c.t0) & (per - 1);
    const uint32_t all = (1u << nb) - 1, blocks = exist >> (i * nb) & all;
    const int left = c.x.len - c.x.begin - t * TOK - pw * HALF;
    uint64_t bits = ~0ull;
    if (blocks != all || left < HALF) {
      bits = 0;
#pragma unroll 1
      for (int b = 0; b < nb; ++b)
        if (blocks >> b & 1) bits |= (~0ull >> (64 - (1 << lg))) << (b << lg);
      if (left < HALF) bits &= (1ull << max(left, 0)) - 1;
    }
    if (elect_one()) {
#pragma unroll
      for (int w = 0; w < HALF / 32; ++w)
        valid[pw * (HALF / 32) + w] = static_cast<uint32_t>(bits >> (32 * w));
      mbar_arrive_expect_tx(full, __popc(blocks) * (2 * SLABS * ROW << lg));
    }
#pragma unroll 1
    for (int b = 0; b < nb; ++b) {
      const int pg = __shfl_sync(0xffffffffu, page, i * nb + b);
      const int of = __shfl_sync(0xffffffffu, off, i * nb + b);
      if ((blocks >> b & 1) && elect_one()) {
#pragma unroll
        for (int slab = 0; slab < SLABS; ++slab) {
          const uint32_t to = dst + slab * (TOK * 128) + (pw * HALF + (b << lg)) * ROW;
          tma_load_4d(to, kmap, full, slab * (128 / ES), of, c.hk, pg);
          tma_load_4d(to + TOK * RB, vmap, full, slab * (128 / ES), of, c.hk, pg);
        }
      }
      __syncwarp();
    }
  }
};

// Four outputs of one row, divided, rounded and stored; the row's lse with its first four.
struct ItemOut {
  int q0, row0, head0, G;  // first row of the sequence; of the item; its first head
  float v_scale;
  // Four finished outputs.
  __device__ __forceinline__ void put_out(const AttnParams &p, int r, int d, float4 v) const {
    const int rr = row0 + r, i = rr / G, g = rr - i * G;
    uint2 u;
    u.x = pack2<false>(v.x, v.y);
    u.y = pack2<false>(v.z, v.w);
    const long long row = q0 + i, head = head0 + g;
    *reinterpret_cast<uint2 *>(p.out + row * p.out_stride + head * p.D + d) = u;
  }
  __device__ __forceinline__ void put_lse(const AttnParams &p, int r, float m, float l) const {
    const int rr = row0 + r, i = rr / G, g = rr - i * G;
    if (p.lse)
      p.lse[static_cast<long long>(q0 + i) * p.Hq + head0 + g] =
          l == 0.0f ? -INFINITY : (m + log2f(l)) * LN2;
  }
  // Four outputs to be divided by the row's sum (zero: nothing seen), with the first the lse.
  __device__ __forceinline__ void put(const AttnParams &p, int r, int d, float4 v, float m,
                                      float l) const {
    const float inv = v_scale / l;
    if (l == 0.0f) v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    else v = make_float4(v.x * inv, v.y * inv, v.z * inv, v.w * inv);
    put_out(p, r, d, v);
    if (d == 0) put_lse(p, r, m, l);
  }
};

struct PendingJoin {
  int c0, parts, group, n_rows;  // first worker, workers, group (-1: the whole item), rows
  ItemOut dst;
};

// Where workers leave their parts of an item: worker c has slot 2c for the item that began
// before its range and 2c + 1 for one that begins in it, and so do the counters of the groups.
__device__ __forceinline__ int part_slot(int c0, int q) { return 2 * (c0 + q) + (q == 0 ? 1 : 0); }

// Parts first, first + every, ... of an item (n of them), added in their order, into dst or
// (to != nullptr) as one part, by the first THREADS threads. Every (m, l) comes into shared memory `ml` in
// one round trip, then the outputs with 16 loads of a thread on their way (a round trip to
// the other die's L2 is 0.7 us; one load at a time took 0.25 us a part): NB blocks of four
// outputs x AHEAD parts. The threads meet at named barrier 2.
template <int M, int DP, int THREADS>
__device__ __forceinline__ void join_parts(const AttnParams &p, float *partials, float2 *ml,
                                           int c0, int first, int every, int n, int n_rows,
                                           float *to, const ItemOut &dst) {
  constexpr int SLOT = M * DP + 2 * M, NB = M <= 16 ? 2 : 4, AHEAD = 16 / NB;
  const int tid = threadIdx.x, cols = p.D / 4;
  auto part = [&](int i) {
    return partials + static_cast<size_t>(part_slot(c0, first + i * every)) * SLOT;
  };
#pragma unroll 4
  for (int i = tid; i < n * n_rows; i += THREADS)
    ml[i] = __ldcg(
        reinterpret_cast<const float2 *>(part(i / n_rows) + M * DP + 2 * (i % n_rows)));
  named_bar_sync(2, THREADS);
  const int all = n_rows * cols;
  for (int i = tid; i < all; i += NB * THREADS) {
    const int blocks = min(NB, (all - i - 1) / THREADS + 1);
    int r[NB], d[NB];
    float m[NB], l[NB], base[NB];
    float4 v[NB];
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      const int at = i + (b < blocks ? b : 0) * THREADS;
      r[b] = at / cols;
      d[b] = 4 * (at - r[b] * cols);
      v[b] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      m[b] = -INFINITY;
      l[b] = 0.0f;
    }
    for (int q0 = 0; q0 < n; q0 += AHEAD) {
      float4 u[NB][AHEAD];
#pragma unroll
      for (int e = 0; e < AHEAD; ++e)
#pragma unroll
        for (int b = 0; b < NB; ++b)
          if (q0 + e < n)
            u[b][e] = __ldcg(reinterpret_cast<const float4 *>(part(q0 + e) + r[b] * DP + d[b]));
      if (q0 == 0) {
#pragma unroll
        for (int b = 0; b < NB; ++b) {
#pragma unroll 4
          for (int q = 0; q < n; ++q) m[b] = fmaxf(m[b], ml[q * n_rows + r[b]].x);
          base[b] = m[b] == -INFINITY ? 0.0f : m[b];
        }
      }
#pragma unroll
      for (int e = 0; e < AHEAD; ++e)
#pragma unroll
        for (int b = 0; b < NB; ++b)
          if (q0 + e < n) {
            const float2 y = ml[(q0 + e) * n_rows + r[b]];
            const float f = ex2(y.x - base[b]);
            l[b] += f * y.y;
            v[b].x += f * u[b][e].x;
            v[b].y += f * u[b][e].y;
            v[b].z += f * u[b][e].z;
            v[b].w += f * u[b][e].w;
          }
    }
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      if (b >= blocks) continue;
      if (to == nullptr) {
        dst.put(p, r[b], d[b], v[b], m[b], l[b]);
      } else {  // `to` may be the first part: only this thread reads or writes these four
        *reinterpret_cast<float4 *>(to + r[b] * DP + d[b]) = v[b];
        if (d[b] == 0)
          *reinterpret_cast<float2 *>(to + M * DP + 2 * r[b]) = make_float2(m[b], l[b]);
      }
    }
  }
}

// Counts a worker's part of a split item, which threads in order before this one have stored.
// The last to arrive joins the item, once its own range is done. With many parts the last
// of each 16 neighbours joins those (in parallel on as many SMs: a single one would read
// them for longer than the products took), and the last group the groups.
__device__ __forceinline__ void count_part(const AttnPlan &pl, int me, int c0, int c1, int n_rows,
                                           const ItemOut &dst, PendingJoin *pending,
                                           int *n_pending) {
  const int parts = c1 - c0 + 1, q = me - c0;
  const bool grouped = parts > 2 * AT_GROUP;
  const int lead = q / AT_GROUP * AT_GROUP;
  int *counter = grouped ? pl.group_counters + part_slot(c0, lead) : pl.counters + c0;
  const int expected = grouped ? min(AT_GROUP, parts - lead) : parts;
  if (atom_add_acq_rel_gpu(counter, 1) == expected - 1) {
    *counter = 0;
    pending[(*n_pending)++] = {c0, parts, grouped ? lead : -1, n_rows, dst};
  }
}

// The joins that fell to this worker, by its first THREADS threads after the last segment, when
// neither registers nor stages hold anything else. `ml`: 2 AT_GROUP M pairs of shared memory.
template <int M, int DP, int THREADS>
__device__ __forceinline__ void run_joins(const AttnParams &p, const AttnPlan &pl, float2 *ml,
                                          const PendingJoin *pending, const int *n_pending,
                                          int *is_last) {
  constexpr int SLOT = M * DP + 2 * M;
  named_bar_sync(2, THREADS);
  for (int i = 0; i < *n_pending; ++i) {
    const PendingJoin j = pending[i];
    const int groups = (j.parts - 1) / AT_GROUP + 1;
    float *to = nullptr;
    int first = 0, every = 1, n = j.parts;
    if (j.group >= 0) {
      to = pl.partials + static_cast<size_t>(part_slot(j.c0, j.group)) * SLOT;
      first = j.group;
      n = min(AT_GROUP, j.parts - j.group);
    }
    for (;;) {  // one place of the join in the code: its first use is paid in fetches
      join_parts<M, DP, THREADS>(p, pl.partials, ml, j.c0, first, every, n, j.n_rows, to, j.dst);
      named_bar_sync(2, THREADS);
      if (to == nullptr) break;
      if (threadIdx.x == 0) {
        *is_last = atom_add_acq_rel_gpu(pl.counters + j.c0, 1) == groups - 1;
        if (*is_last) pl.counters[j.c0] = 0;
      }
      named_bar_sync(2, THREADS);
      if (!*is_last) break;
      to = nullptr;
      first = 0;
      every = AT_GROUP;
      n = groups;
    }
  }
}

// Whether a CTA's static shared memory (FIXED bytes of variables, 64 for gaps between them), which is
// filled up to the 1024 bytes that the dynamic one is aligned to, and the dynamic one fit
// the 227 KB that a CTA may have. Several shapes are full to the last KB, and a launch that
// asks for more fails.
template <size_t FIXED, size_t DYNAMIC>
constexpr bool fits_shared = (FIXED + 64 + 1023) / 1024 * 1024 + DYNAMIC <= 227 * 1024;

template <bool E4M3, int DP, int NR, int WR>
__global__ void __launch_bounds__(AT_THREADS, (AttnCfg<E4M3, DP, NR, WR>::CTAS))
    attn_decode_kernel(const __grid_constant__ CUtensorMap kmap,
                       const __grid_constant__ CUtensorMap vmap,
                       const __grid_constant__ AttnParams p, const AttnPlan pl) {
  using C = AttnCfg<E4M3, DP, NR, WR>;
  constexpr int TOK = C::TOK, STEP = C::STEP, RB = C::RB, M = C::M, MW = C::MW, ST = C::ST;
  constexpr int MT = STEP / 16;  // 16-token tiles of a step
  extern __shared__ __align__(1024) uint8_t at_smem[];
  __shared__ RangeStart<AT_THREADS> start;
  __shared__ __align__(8) uint64_t full[ST], empty[ST], qempty[C::QB];
  __shared__ float join_ml[AT_CWARPS * MW][2];         // m, l of each warp's rows
  __shared__ uint32_t stage_valid[ST][TOK / 32];       // tokens of the stage that exist
  __shared__ int abort_flag, n_pending, is_last;
  __shared__ PendingJoin pending[2];  // a range splits at most its first and last item
  static_assert(fits_shared<sizeof(start) + sizeof(full) + sizeof(empty) + sizeof(qempty) +
                                sizeof(join_ml) + sizeof(stage_valid) + 3 * sizeof(int) +
                                sizeof(pending),
                            C::SMEM>,
                "all of the above and the dynamic shared memory");
  uint8_t *q_smem = at_smem + ST * C::STAGE;

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (tid == 0) {
    abort_flag = 0;
    n_pending = 0;
    for (int i = 0; i < ST; ++i) {
      mbar_init(&full[i], AT_PWARPS * 33);  // every copying thread's copies, and each warp
      mbar_init(&empty[i], AT_CWARPS);
    }
    for (int i = 0; i < C::QB; ++i) mbar_init(&qempty[i], AT_CWARPS);
    fence_mbar_init();
    if (p.box > 0) {
      prefetch_tensormap(&kmap);
      prefetch_tensormap(&vmap);
    }
  }
  griddep_wait();
  griddep_launch_dependents();
  const int G = p.Hq / p.Hkv;

  Shares sh;
  Cursor<TOK, M, AT_ITEM_COST, AT_LEAST> c;
  if (!begin_range<AT_THREADS>(p, G, start, sh, c)) return;

  if (warp >= AT_CWARPS) {
    // ================================================================ copying warps
    constexpr int HALF = TOK / AT_PWARPS;  // tokens of this warp
    constexpr int WORDS = HALF / 32;
    const int pw = warp - AT_CWARPS;
    const char *kbase = static_cast<const char *>(p.c.k);
    const char *vbase = static_cast<const char *>(p.c.v);
    Boxes<RB, TOK, HALF, C::ES> boxes(p.box > 0 ? p.box : HALF);
    int k = 0, seg = 0;  // stages and segments so far
    bool go = true;      // until a time-out: no copy into a stage that may be in use
    while (go && c.next(p, G)) {
      const int32_t *table = p.block_table + static_cast<long long>(c.s) * p.max_pages;
      // 16-byte copies: first token of this warp in stage t, and the page of a lane's token
      auto token0 = [&](int t) { return c.x.begin + t * TOK + pw * HALF; };
      int page[WORDS], ahead[WORDS];  // of this stage and the next
      auto look_up = [&](int t, int (&to)[WORDS]) {
#pragma unroll
        for (int q = 0; q < WORDS; ++q) {
          const int j = token0(t) + q * 32 + lane;
          to[q] = p.box == 0 && t < c.t1 && j < c.x.len ? table[j / p.c.page_size] : -1;
        }
      };
      look_up(c.t0, page);
      look_up(c.t0 + 1, ahead);
      for (int t = c.t0; t < c.t1; ++t, ++k) {
        const int st = k % ST, j0 = token0(t);
        if (p.box > 0) boxes.step(p, c, t, pw, lane);
        if (k >= ST) {
          go = __all_sync(0xffffffffu, mbar_wait_bounded(&empty[st], ((k / ST) - 1) & 1, pl.status,
                                                         &abort_flag, pl.wait_limit_ns));
          if (!go) break;
        }
        const uint32_t dst = smem_u32(at_smem + st * C::STAGE);
        if (p.box > 0) {
          boxes.issue(&kmap, &vmap, c, t, pw, dst, &full[st], stage_valid[st]);
          boxes.ahead(p, c, t, pw, lane);
        } else {
#pragma unroll
          for (int q = 0; q < WORDS; ++q) {
            const bool ok = page[q] >= 0 && page[q] < p.c.num_pages;
            long long off = -1;
            if (ok)
              off = (page[q] * p.c.page_stride + c.hk * p.c.head_stride +
                     (j0 + q * 32 + lane) % p.c.page_size * p.c.token_stride) * C::ES;
            const uint32_t valid = __ballot_sync(0xffffffffu, ok);
            if (lane == 0) stage_valid[st][pw * WORDS + q] = valid;
#pragma unroll
            for (int i = 0; i < C::CPR; ++i) {
              const int row = (i * 32 + lane) / C::CPR, ch = (i * 32 + lane) % C::CPR;
              const long long o = __shfl_sync(0xffffffffu, off, row);
              const bool in = o >= 0 && ch * 16 < p.D * C::ES;
              const long long at = in ? o + ch * 16 : 0;
              const uint32_t d = dst + swz<RB, TOK>(pw * HALF + q * 32 + row, ch);
              cp_async16(d, kbase + at, in);
              cp_async16(d + TOK * RB, vbase + at, in);
            }
          }
        }
#pragma unroll
        for (int q = 0; q < WORDS; ++q) page[q] = ahead[q];
        look_up(t + 2, ahead);
        if (t == c.t0) {
          // the item's rows of q, zeros past them and past D
          const int qb = seg % C::QB;
          if (seg >= C::QB)
            mbar_wait_bounded(&qempty[qb], ((seg / C::QB) - 1) & 1, pl.status, &abort_flag,
                              pl.wait_limit_ns);
          const int n_rows = min(M, c.x.n * G - c.rt * M);
          const uint32_t qd = smem_u32(q_smem + qb * C::QBYTES);
#pragma unroll 4
          for (int i = pw * 32 + lane; i < M * DP / 8; i += 32 * AT_PWARPS) {
            const int r = i / (DP / 8), ch = i % (DP / 8);
            const bool in = r < n_rows && ch * 8 < p.D;
            const int rr = c.rt * M + (in ? r : 0), tok = rr / G, g = rr - tok * G;
            cp_async16(qd + swz<DP * 2, M>(r, ch),
                       p.q + (c.x.q0 + tok) * p.q_stride +
                           static_cast<long long>(c.hk * G + g) * p.D + (in ? ch * 8 : 0),
                       in);
          }
          ++seg;
        }
        cp_async_arrive(&full[st]);
        __syncwarp();
        if (lane == 0 && p.box == 0) mbar_arrive(&full[st]);
      }
    }
    cp_async_wait_all();
    // The multiplying warps' waits are over as well: a time-out of theirs after this warp's last
    // stage is known here, and boxes still on their way land before the CTA ends.
    named_bar_sync(3, AT_THREADS);
    if (*static_cast<volatile int *>(&abort_flag) && lane == 0) {
      for (int i = max(k - ST, 0); i < k; ++i)
        mbar_wait_drain(&full[i % ST], (i / ST) & 1, 10000000ull);
    }
    return;
  }

  // ================================================================ multiplying warps
  const int wr = warp % WR, wt = warp / WR;  // which rows, which tokens of a stage
  const int g8 = lane >> 2, c4 = lane & 3;   // a lane's place in the fragments
  int k = 0, seg = 0;
  // self-test: nobody but these warps, later, arrives here
  if (pl.hold)
    mbar_wait_bounded(&qempty[0], 0, pl.status, &abort_flag, pl.wait_limit_ns);
  while (c.next(p, G)) {
    const SeqInfo &x = c.x;
    const int n_rows = min(M, x.n * G - c.rt * M);   // of the item
    const int my_rows = min(MW, n_rows - wr * MW);   // of this warp, may be <= 0
    const int row0 = c.rt * M + wr * MW;             // this warp's first
    // what every row of this warp sees: [lo_all, hi_all]
    const int pos0 = x.len - x.n;
    const int hi_all = pos0 + row0 / G;
    const int hi_top = pos0 + (row0 + max(my_rows, 1) - 1) / G;
    const int lo_all = p.window > 0 && hi_top >= p.window ? hi_top - p.window + 1 : 0;

    // this thread's rows are nr * 8 + 2 c4 + e: score factor, what weights refer to (the
    // maximum, less F16_POWERS on an e4m3 cache), sum, outputs
    float zf[NR][2], m[NR][2], l[NR][2];
    float o[NR][DP / 16][4];
    const float z_all = p.scale * LOG2E * (p.c.k_scale ? p.c.k_scale[c.hk] : 1.0f);
#pragma unroll
    for (int r = 0; r < NR; ++r) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        zf[r][e] = z_all;
        m[r][e] = -INFINITY;
        l[r][e] = 0.0f;
      }
#pragma unroll
      for (int i = 0; i < DP / 16; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[r][i][e] = 0.0f;
    }
    uint32_t qf[NR][DP / 16][2];

    for (int t = c.t0; t < c.t1; ++t, ++k) {
      const int st = k % ST;
      mbar_wait_bounded(&full[st], (k / ST) & 1, pl.status, &abort_flag, pl.wait_limit_ns);
      uint8_t *stage = at_smem + st * C::STAGE;
      if (t == c.t0) {
        const uint8_t *qs = q_smem + (seg % C::QB) * C::QBYTES;
        if (!E4M3) {
#pragma unroll
          for (int r = 0; r < NR; ++r)
#pragma unroll
            for (int kk = 0; kk < DP / 16; kk += 2) {
              uint32_t v[4];
              ldsm4(v, smem_u32(qs) + swz<DP * 2, M>(wr * MW + r * 8 + (lane & 7),
                                                     2 * kk + (lane >> 3)));
              qf[r][kk][0] = v[0], qf[r][kk][1] = v[1];
              qf[r][kk + 1][0] = v[2], qf[r][kk + 1][1] = v[3];
            }
        } else {
          // f16 operands in the order in which the widened keys come out of their
          // registers: of each 16 elements of row g8 this lane holds 4 c4 .. 4 c4 + 3
#pragma unroll
          for (int r = 0; r < NR; ++r) {
            float mx = 0.0f;
            uint2 raw[DP / 16];
#pragma unroll
            for (int kk = 0; kk < DP / 16; ++kk) {
              raw[kk] = *reinterpret_cast<const uint2 *>(
                  qs + swz<DP * 2, M>(wr * MW + r * 8 + g8, 2 * kk + (c4 >> 1)) + (c4 & 1) * 8);
              mx = fmaxf(mx, fmaxf(fmaxf(fabsf(bf16lo(raw[kk].x)), fabsf(bf16hi(raw[kk].x))),
                                   fmaxf(fabsf(bf16lo(raw[kk].y)), fabsf(bf16hi(raw[kk].y)))));
            }
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
            const int e = q_exponent(mx);
            const float f = power_of_two(-e), back = power_of_two(e);
            zf[r][0] *= __shfl_sync(0xffffffffu, back, 8 * c4);
            zf[r][1] *= __shfl_sync(0xffffffffu, back, 8 * c4 + 4);
#pragma unroll
            for (int kk = 0; kk < DP / 16; ++kk) {
              qf[r][kk][0] = pack2<true>(bf16lo(raw[kk].x) * f, bf16hi(raw[kk].x) * f);
              qf[r][kk][1] = pack2<true>(bf16lo(raw[kk].y) * f, bf16hi(raw[kk].y) * f);
            }
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&qempty[seg % C::QB]);
      }
      if (my_rows > 0) {
#pragma unroll 1
        for (int sub = 0; sub < WR * (C::SPAN / STEP); ++sub) {
          const int tok0 = wt * WR * C::SPAN + sub * STEP;  // of the stage
          const uint32_t ks = smem_u32(stage), vs = ks + TOK * RB;
          const uint32_t valid = STEP == 32 ? stage_valid[st][tok0 >> 5]
                                            : stage_valid[st][tok0 >> 5] >> (tok0 & 31);
          const int j0 = x.begin + t * TOK + tok0;

          // ---- scores [STEP tokens, rows]
          float z[NR][MT][4];
#pragma unroll
          for (int r = 0; r < NR; ++r)
#pragma unroll
            for (int i = 0; i < MT; ++i)
#pragma unroll
              for (int e = 0; e < 4; ++e) z[r][i][e] = 0.0f;
          // a lone chain of products is as long as the head: two, added at the end
          float z2[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
          for (int kk = 0; kk < DP / 16; kk += E4M3 ? 2 : 1) {
#pragma unroll
            for (int i = 0; i < MT; ++i) {
              uint32_t v[4];
              ldsm4(v, ks + swz<RB, TOK>(tok0 + i * 16 + (lane & 15),
                                         (E4M3 ? kk : 2 * kk) + (lane >> 4)));
              if (E4M3) {
#pragma unroll
                for (int q = 0; q < 2; ++q) {  // k step
                  const uint32_t a[4] = {e4m3x2_to_f16x2(v[2 * q]), e4m3x2_to_f16x2(v[2 * q + 1]),
                                         e4m3x2_to_f16x2(v[2 * q] >> 16),
                                         e4m3x2_to_f16x2(v[2 * q + 1] >> 16)};
#pragma unroll
                  for (int r = 0; r < NR; ++r)
                    mma16816<true>(z[r][i], a, qf[r][E4M3 ? kk + q : 0][0],
                                   qf[r][E4M3 ? kk + q : 0][1]);
                }
              } else {
#pragma unroll
                for (int r = 0; r < NR; ++r) {
                  if (NR * MT == 1 && (kk & 1))
                    mma16816<false>(z2, v, qf[r][kk][0], qf[r][kk][1]);
                  else
                    mma16816<false>(z[r][i], v, qf[r][kk][0], qf[r][kk][1]);
                }
              }
            }
          }
          const uint32_t every = STEP == 32 ? 0xffffffffu : (1u << (STEP & 31)) - 1;
          const bool whole = (valid & every) == every;
          const bool plain = whole && j0 >= lo_all && j0 + STEP - 1 <= hi_all;
#pragma unroll
          for (int r = 0; r < NR; ++r)
#pragma unroll
            for (int i = 0; i < MT; ++i)
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                if (NR * MT == 1 && !E4M3) z[r][i][e] += z2[e];
                z[r][i][e] *= zf[r][e & 1];
              }
          if (!plain) {
#pragma unroll
            for (int r = 0; r < NR; ++r)
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                const int row = max(min(r * 8 + 2 * c4 + e, my_rows - 1), 0);
                const int hi = pos0 + (row0 + row) / G;
                const int lo = p.window > 0 && hi >= p.window ? hi - p.window + 1 : 0;
#pragma unroll
                for (int i = 0; i < MT; ++i)
#pragma unroll
                  for (int h = 0; h < 2; ++h) {
                    const int b = i * 16 + h * 8 + g8;
                    if (j0 + b < lo || j0 + b > hi || !(valid >> b & 1))
                      z[r][i][2 * h + e] = -INFINITY;
                  }
              }
          }
          // ---- running maximum over the tokens (lanes of equal c4 hold them)
          float base[NR][2], fade[NR][2];
          bool grew = false;
#pragma unroll
          for (int r = 0; r < NR; ++r)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              float mx = E4M3 ? -INFINITY : m[r][e];
#pragma unroll
              for (int i = 0; i < MT; ++i) mx = fmaxf(mx, fmaxf(z[r][i][e], z[r][i][2 + e]));
              mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 4));
              mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
              mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
              if (E4M3) mx = fmaxf(m[r][e], mx - F16_POWERS);
              base[r][e] = mx == -INFINITY ? 0.0f : mx;
              fade[r][e] = ex2(m[r][e] - base[r][e]);
              m[r][e] = mx;
              l[r][e] *= fade[r][e];
              grew |= fade[r][e] != 1.0f;
            }
          if (__any_sync(0xffffffffu, grew)) {
#pragma unroll
            for (int r = 0; r < NR; ++r)
#pragma unroll
              for (int d = 0; d < DP / 16; ++d)
#pragma unroll
                for (int e = 0; e < 4; ++e) o[r][d][e] *= fade[r][e & 1];
          }
          // Where `unclean` is looked at, a weight of zero is to mean that the row does not see the
          // token: the least that a seen one has is 2^-100. (Done in every step that is not
          // plain, 16 rows on an e4m3 cache took 144.7 us instead of 140.0.)
          if (!plain && (x.n > 1 || p.window > 0)) {
#pragma unroll
            for (int r = 0; r < NR; ++r)
#pragma unroll
              for (int i = 0; i < MT; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                  const float least = base[r][e & 1] - 100.0f;
                  if (z[r][i][e] < least && z[r][i][e] != -INFINITY) z[r][i][e] = least;
                }
          }
          // ---- weights: summed in fp32, rounded to 16 bits for the product with V, turned so
          // that tokens are the inner dimension. Each is off by 2^-8 (bf16) or 2^-11 (f16) of
          // itself at most, independently of the others. In bf16 that adds up to as much as
          // the output's own rounding where few weights carry a row, to less where many do
          // (relative error against 64 bits 0.0018 to 0.0023, with fp32 weights 0.0017);
          // keeping 16 more bits would take a second product with V.
          uint32_t w[NR][MT][2];
#pragma unroll
          for (int r = 0; r < NR; ++r)
#pragma unroll
            for (int i = 0; i < MT; ++i) {
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                z[r][i][e] = ex2(z[r][i][e] - base[r][e & 1]);
                l[r][e & 1] += z[r][i][e];
              }
              w[r][i][0] = transpose8x8(pack2<E4M3>(z[r][i][0], z[r][i][1]));
              w[r][i][1] = transpose8x8(pack2<E4M3>(z[r][i][2], z[r][i][3]));
            }
          // ---- what weights of zero must not meet: boxes bring whatever lies in the cache
          // past the sequence's end, and stages keep old bytes where a page is missing. Such
          // tokens' values become zeros.
          bool unclean = false;
          if (!plain) {
            if (!whole && p.box > 0) {
              for (int i = lane; i < STEP * C::CPR; i += 32) {
                const int row = i / C::CPR, ch = i % C::CPR;
                if (!(valid >> row & 1))
                  *reinterpret_cast<uint4 *>(stage + TOK * RB + swz<RB, TOK>(tok0 + row, ch)) =
                      make_uint4(0, 0, 0, 0);
              }
              fence_proxy_async_smem();  // before later boxes overwrite these stores
              __syncwarp();
            }
            // A value that is not finite at a token that some rows see and others do not must
            // not reach the others as 0 * inf: such steps (the last few of an item) take the
            // values' finite part through the product and add the rest where it is seen. A
            // sequence's only row sees every token from its window's first on; boxes may
            // bring some before it.
            if (x.n > 1 || p.window > 0) {
              bool bad = false;
              for (int i = lane; i < STEP * C::CPR; i += 32) {
                const uint4 v = *reinterpret_cast<const uint4 *>(
                    stage + TOK * RB + swz<RB, TOK>(tok0 + i / C::CPR, i % C::CPR));
                const uint32_t e[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                  if (E4M3) bad |= __vcmpeq4(e[q] & 0x7f7f7f7fu, 0x7f7f7f7fu) != 0;
                  else bad |= __vcmpeq2(e[q] & 0x7f807f80u, 0x7f807f80u) != 0;
                }
              }
              unclean = __any_sync(0xffffffffu, bad);
            }
          }
          // ---- out [elements, rows] += values . weights
#pragma unroll
          for (int i = 0; i < MT; ++i) {
#pragma unroll
            for (int dd = 0; dd < DP / 16; dd += E4M3 ? 2 : 1) {
              // bf16: quarters (tokens, elements) 0 0 | 0 8 | 8 0 | 8 8; e4m3: the tokens'
              // halves of 16 elements, then of the next 16
              uint32_t v[4];
              ldsm4_t(v, vs + swz<RB, TOK>(
                             tok0 + i * 16 +
                                 (E4M3 ? lane & 15 : (lane & 7) + ((lane >> 4) << 3)),
                             E4M3 ? dd + (lane >> 4) : 2 * dd + ((lane >> 3) & 1)));
              if (unclean) {
#pragma unroll
                for (int q = 0; q < 4; ++q)
                  v[q] &= E4M3 ? ~__vcmpeq4(v[q] & 0x7f7f7f7fu, 0x7f7f7f7fu)
                               : ~__vcmpeq2(v[q] & 0x7f807f80u, 0x7f807f80u);
              }
              if (E4M3) {
#pragma unroll
                for (int q = 0; q < 2; ++q) {  // even elements as rows 0-7, odd as 8-15
                  const uint32_t lo = __byte_perm(v[2 * q], 0, 0x3120);
                  const uint32_t hi = __byte_perm(v[2 * q + 1], 0, 0x3120);
                  const uint32_t a[4] = {e4m3x2_to_f16x2(lo), e4m3x2_to_f16x2(lo >> 16),
                                         e4m3x2_to_f16x2(hi), e4m3x2_to_f16x2(hi >> 16)};
#pragma unroll
                  for (int r = 0; r < NR; ++r)
                    mma16816<true>(o[r][E4M3 ? dd + q : 0], a, w[r][i][0], w[r][i][1]);
                }
              } else {
#pragma unroll
                for (int r = 0; r < NR; ++r)
                  mma16816<false>(o[r][dd], v, w[r][i][0], w[r][i][1]);
              }
            }
          }
          if (unclean) {
#pragma unroll
            for (int i = 0; i < MT; ++i)
#pragma unroll
              for (int h = 0; h < 2; ++h)
#pragma unroll 1
                for (int q = 0; q < 8; ++q) {  // token i * 16 + h * 8 + q
                  float pr[NR][2];
#pragma unroll
                  for (int r = 0; r < NR; ++r)
#pragma unroll
                    for (int e = 0; e < 2; ++e)
                      pr[r][e] = __shfl_sync(0xffffffffu, z[r][i][2 * h + e], q * 4 + c4);
#pragma unroll
                  for (int dd = 0; dd < DP / 16; ++dd)
#pragma unroll
                    for (int f = 0; f < 2; ++f) {
                      const int col = 16 * dd + (E4M3 ? 2 * g8 + f : 8 * f + g8);
                      const uint8_t *at =
                          stage + TOK * RB +
                          swz<RB, TOK>(tok0 + i * 16 + h * 8 + q, col * C::ES >> 4) +
                          (col * C::ES & 15);
                      float val = NAN;
                      bool bad = E4M3 && (*at & 0x7f) == 0x7f;
                      if (!E4M3) {
                        const uint16_t b = *reinterpret_cast<const uint16_t *>(at);
                        bad = (b & 0x7f80) == 0x7f80;
                        val = bf16_to_f32(b);
                      }
                      if (bad) {
#pragma unroll
                        for (int r = 0; r < NR; ++r)
#pragma unroll
                          for (int e = 0; e < 2; ++e)
                            if (pr[r][e] != 0.0f) o[r][dd][2 * f + e] += pr[r][e] * val;
                      }
                    }
                }
          }
        }
      }
      if (t + 1 < c.t1) {  // the stage is free again; the segment's last one after the join
        __syncwarp();
        if (lane == 0) mbar_arrive(&empty[st]);
      }
    }
    ++seg;

    // ---- join the warps in the last stage's memory: row r of warp w at w * MW + r, pairs of
    // 16-byte chunks permuted by the row so that a warp's stores spread over the banks
    const int last_st = (k - 1) % ST;
    float *join = reinterpret_cast<float *>(at_smem + last_st * C::STAGE);
    auto join_at = [&](int row, int col) {
      return join + row * DP + ((col >> 2) ^ ((row & 6))) * 4 + (col & 3);
    };
    named_bar_sync(1, AT_CTHREADS);  // every warp has read the stage
#pragma unroll
    for (int r = 0; r < NR; ++r)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float s = l[r][e];
        s += __shfl_xor_sync(0xffffffffu, s, 4);
        s += __shfl_xor_sync(0xffffffffu, s, 8);
        s += __shfl_xor_sync(0xffffffffu, s, 16);
        const int mine = r * 8 + 2 * c4 + e, row = warp * MW + mine;
        if (g8 == 0) {
          join_ml[row][0] = m[r][e];
          join_ml[row][1] = s;
        }
        if (mine < my_rows) {
#pragma unroll
          for (int d = 0; d < DP / 16; ++d) {
            if (E4M3) {
              *reinterpret_cast<float2 *>(join_at(row, 16 * d + 2 * g8)) =
                  make_float2(o[r][d][e], o[r][d][2 + e]);
            } else {
              *join_at(row, 16 * d + g8) = o[r][d][e];
              *join_at(row, 16 * d + 8 + g8) = o[r][d][2 + e];
            }
          }
        }
      }
    named_bar_sync(1, AT_CTHREADS);

    const long long first = c.item + AT_ITEM_COST;  // the unit of the item's first stage
    const int me = blockIdx.x, c0 = sh.worker_of(first), c1 = sh.worker_of(first + x.kt - 1);
    const ItemOut dst = {x.q0, c.rt * M, c.hk * G, G,
                         p.c.v_scale ? p.c.v_scale[c.hk] : 1.0f};
    const int cols = p.D / 4;
    float *slot = pl.partials + static_cast<size_t>(part_slot(c0, me - c0)) * C::SLOT;
    for (int i = tid; i < n_rows * cols; i += AT_CTHREADS) {
      const int r = i / cols, d = 4 * (i - r * cols);
      float mr = -INFINITY;
#pragma unroll
      for (int g = 0; g < AT_CWARPS / WR; ++g)
        mr = fmaxf(mr, join_ml[g * M + r][0]);
      const float b = mr == -INFINITY ? 0.0f : mr;
      float lr = 0.0f;
      float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
      for (int g = 0; g < AT_CWARPS / WR; ++g) {
        const float f = ex2(join_ml[g * M + r][0] - b);
        const float4 y = *reinterpret_cast<const float4 *>(join_at(g * M + r, d));
        lr += f * join_ml[g * M + r][1];
        v.x += f * y.x;
        v.y += f * y.y;
        v.z += f * y.z;
        v.w += f * y.w;
      }
      if (c0 == c1) {
        dst.put(p, r, d, v, mr, lr);
      } else {
        *reinterpret_cast<float4 *>(slot + r * DP + d) = v;
        if (d == 0)
          *reinterpret_cast<float2 *>(slot + M * DP + 2 * r) = make_float2(mr, lr);
      }
    }
    fence_proxy_async_smem();  // before later boxes overwrite the join's stores
    __syncwarp();
    if (lane == 0) mbar_arrive(&empty[last_st]);
    if (c0 != c1) {
      named_bar_sync(1, AT_CTHREADS);
      if (tid == 0) count_part(pl, me, c0, c1, n_rows, dst, pending, &n_pending);
    }
  }
  __syncwarp();
  named_bar_arrive(3, AT_THREADS);  // no wait of these warps follows: see the copying warps' end
  static_assert(ST * C::STAGE >= 2 * AT_GROUP * M * 8, "ml of a join");
  run_joins<M, DP, AT_CTHREADS>(p, pl, reinterpret_cast<float2 *>(at_smem), pending, &n_pending,
                                &is_last);
}

// CTAs: two per SM by shared memory, one above D = 128.
inline int attn_grid(int DP, int num_sms) { return DP <= 128 ? 2 * num_sms : num_sms; }


// The workspace: counters of items and of groups of workers (zero between calls; the same
// place for every kernel, as calls of any of them may follow each other on one workspace),
// then two partial slots per worker.
inline AttnPlan make_plan(void *ws, const AttnLaunch &a) {
  AttnPlan pl;
  pl.counters = static_cast<int *>(ws);
  pl.group_counters = pl.counters + attn_max_workers(a.num_sms);
  pl.partials = reinterpret_cast<float *>(static_cast<char *>(ws) +
                                          attn_counter_bytes(a.num_sms));
  pl.status = a.status;
  pl.wait_limit_ns = a.wait_limit_ns;
  pl.hold = a.hold;
  return pl;
}

template <bool E4M3, int DP, int NR, int WR>
cudaError_t launch_shape(const AttnParams &p, void *ws, const AttnLaunch &a, cudaStream_t s) {
  using C = AttnCfg<E4M3, DP, NR, WR>;
  auto kernel = attn_decode_kernel<E4M3, DP, NR, WR>;
  const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             static_cast<int>(C::SMEM));
  if (e != cudaSuccess) return e;
  const int grid = attn_grid(DP, a.num_sms);
  return launch_pdl(kernel, dim3(grid), dim3(AT_THREADS), C::SMEM, s, a.kmap, a.vmap, p,
                    make_plan(ws, a));
}

// nr, wr: attn_shape's
template <int DP>
cudaError_t launch_dim(const AttnParams &p, bool e4m3, int nr, int wr, void *ws,
                       const AttnLaunch &a, cudaStream_t s) {
  switch (nr * wr) {
    case 1:
      return e4m3 ? launch_shape<true, DP, 1, 1>(p, ws, a, s)
                  : launch_shape<false, DP, 1, 1>(p, ws, a, s);
    case 2:
      return e4m3 ? launch_shape<true, DP, 2, 1>(p, ws, a, s)
                  : launch_shape<false, DP, 2, 1>(p, ws, a, s);
    case 4:
      return e4m3 ? launch_shape<true, DP, 2, 2>(p, ws, a, s)
                  : launch_shape<false, DP, 2, 2>(p, ws, a, s);
    default:
      return e4m3 ? launch_shape<true, DP, 2, 4>(p, ws, a, s)
                  : launch_shape<false, DP, 2, 4>(p, ws, a, s);
  }
}

}  // namespace
}  // namespace ssd

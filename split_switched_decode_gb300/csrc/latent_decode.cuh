// latent_decode.cuh -- attention of new tokens over a paged cache of latent vectors, on tcgen05
// tensor cores.
//
// Each cached token is one row c_j of R + P elements, key of every head, and its first R
// elements are its value:
//
//     out_r = sum_j p_rj c_j[:R] / sum_j p_rj,   p_rj = 2^(z_rj - m_r),   z = scale log2(e) q.c
//
// A row of the cache is read once for up to MQ rows (new tokens x heads) and carries
// 2 (2R + P) MQ / (R + P) / 2 operations a byte: with 64 rows the copy rate bounds it, with 128
// and more the tensor cores.
//
// Both products have the rows as N. With the rows as M the outputs, 128 x 512 in fp32, would
// fill tensor memory, and a few heads would leave most of it empty:
//
//     S[64 tokens, MQ]  = C . Q^T      A = C, B = Q, both K-major in shared memory
//     O[R, MQ]         += C^T . P      A = C as stored (MN-major), B = P[tokens, MQ] in shared
//                                      memory, rows contiguous; four M blocks of 128 elements
//
// so O takes 4 MQ columns and S MQ. The tokens lie in the lanes of S; its 64 are in 16 lanes
// of each warp's quarter (M = 64), and a thread reads four elements of each 16 x 8 block (two
// tokens, two rows). Two groups of four warps have half of the rows each and share nothing; a
// thread holds the running maximum and its tokens' part of the sum of MQ / 8 rows. The maximum
// is moved only when a row's has grown by 8 or more (weights then stay below 2^8 in bf16, and
// below 2^15 in f16, where they refer to less than the maximum; their rounding, relative 2^-8 or
// 2^-11, is not enlarged): the common stage needs one vote over the
// group and no exchange of maxima. Sums are fp32, of the weights before rounding, added over
// lanes and warps at the segment's end.
//
// A stage is 64 tokens: eight boxes of 8 tokens x the whole row, so any page of whole blocks
// of 8 tokens comes in boxes; a box is laid out as one swizzle group per 64 elements (1 KB
// each), which is the operand layout of both products with strides of a box. Other pages are
// copied in 16-byte loads by four warps into the same layout.
//
// Warps: 8 softmax, 1 each for S, O, the boxes and the boxes of q, 4 that bring the rows of q
// and the stages where boxes do not. E4M3: 8 of those, which widen every stage to f16 on its way
// from global memory through registers (a ring of bytes as they come beside that of the operands
// has no room: with one operand stage, widening, products and softmax took turns, 3.5 us a stage).
//
// E4M3 caches: every e4m3 value is an f16 value; q is scaled by a power of two a row and
// converted to f16, the weights are f16 and refer to F16_POWERS below the maximum.
//
// Division of the work: attn_kernel.cuh's (one kv head). An item that lies in several CTAs leaves
// a part in each (fp32, unscaled, with its maximum and sum), and where those are in a table by row;
// a second kernel joins them: with 64 rows a part is 132 KB, and a long item has a part an SM, which
// its last CTA would read alone.
//
// Measured (without the join): 64 sequences to 16384 tokens, 64 heads, 637 MB: 112 us, 5.7 TB/s;
// one row of 64 heads over 131072 tokens 37 us; 32 x 8 rows of 16 heads over an e4m3 cache 125 us.
#pragma once

#include "attn_tc.cuh"
#include "latent.h"

namespace ssd {
namespace {

// Stages ahead at which boxes are requested into L2, behind the copy of a stage: the ring holds two
// stages, and the one that is on its way (74 KB an SM) is too little for HBM's latency under
// load (64 sequences to 16384 tokens: 124.1 us with one stage, 125.4 with two; three took 11 more than
// two when that was measured, and none 137).
constexpr int LD_AHEAD = 1;
// Units that an item is charged (its q and outputs; the same sequences: 129.4 us at two, 124.1 at
// four, 127.0 at eight), and the smallest share.
constexpr int LD_ITEM_COST = 4, LD_LEAST = 1;

template <int MQ, bool E4M3>
struct LdCfg {
  static constexpr int TOK = 64, DP = LATENT_MAX_R;
  static constexpr int STAGE = TOK * LATENT_MAX_W * 2;
  static constexpr int QBYTES = MQ * LATENT_MAX_W * 2;
  static constexpr int PBYTES = TOK * 128;  // a token's weights in 128 bytes
  static constexpr int QB = MQ == 64 ? 1 : 2, ST = 2;
  static constexpr int NS = 4;  // buffers of scores
  static constexpr int COLS = 8 * MQ;  // O: 4 MQ, then NS S
  static constexpr int GR = MQ / 2;    // rows of a softmax group
  static constexpr int HW = E4M3 ? 8 : 4;  // helping warps
  static constexpr int THREADS = 32 * (12 + HW);
  static constexpr size_t SMEM = ST * STAGE + QB * QBYTES + PBYTES;
  static constexpr int SLOT = MQ * DP;
};

// Shares (attn_kernel.cuh) with divisions in 32 bits where the work has fewer units than 2^31: one
// in 64 bits takes 400 clocks, and a short call waits for several.
struct LdShares {
  long long share_n, share_r;
  bool narrow;
  __device__ __forceinline__ void set(long long total, int workers) {
    narrow = total < 0x7fffffffll;
    if (narrow) {
      const uint32_t t = static_cast<uint32_t>(total), w = workers, n = t / w;
      share_n = n;
      share_r = t - n * w;
    } else {
      share_n = total / workers;
      share_r = total % workers;
    }
  }
  __device__ __forceinline__ int worker_of(long long unit) const {
    const long long longer = share_r * (share_n + 1);
    if (narrow) {
      const uint32_t u = static_cast<uint32_t>(unit), n = static_cast<uint32_t>(share_n);
      return unit < longer ? u / (n + 1)
                           : static_cast<uint32_t>(share_r) +
                                 (u - static_cast<uint32_t>(longer)) / n;
    }
    return static_cast<int>(unit < longer ? unit / (share_n + 1)
                                          : share_r + (unit - longer) / share_n);
  }
};
// begin_range for batches of up to 32 sequences: every warp finds the CTA's range by itself.
template <int TOK, int M, int COST, int LEAST>
__device__ __forceinline__ bool begin_range_small(const AttnParams &p, int H, LdShares &sh,
                                                  Cursor<TOK, M, COST, LEAST> &c) {
  const int lane = threadIdx.x & 31, me = blockIdx.x;
  SeqInfo x = {};
  long long mine = 0;
  if (lane < p.S) {
    x = seq_info<TOK, M>(p, H, lane);
    mine = x.units(1, COST);
  }
  long long incl = mine;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, incl, d);
    if (lane >= d) incl += y;
  }
  const long long total = __shfl_sync(0xffffffffu, incl, 31);
  const long long most = (total + LEAST - 1) / LEAST;
  const int workers = static_cast<int>(most < gridDim.x ? most : gridDim.x);
  if (me >= workers) return false;
  sh.set(total, workers);
  c.cur = me * sh.share_n + min(static_cast<long long>(me), sh.share_r);
  c.end = c.cur + sh.share_n + (me < sh.share_r ? 1 : 0);
  const long long at = incl - mine;  // units before this lane's sequence
  const int from = __ffs(__ballot_sync(0xffffffffu, at <= c.cur && c.cur < incl)) - 1;
  const long long off = c.cur - __shfl_sync(0xffffffffu, at, from);
  c.s = from;
  c.x.q0 = __shfl_sync(0xffffffffu, x.q0, from);
  c.x.n = __shfl_sync(0xffffffffu, x.n, from);
  c.x.len = __shfl_sync(0xffffffffu, x.len, from);
  c.x.begin = __shfl_sync(0xffffffffu, x.begin, from);
  c.x.kt = __shfl_sync(0xffffffffu, x.kt, from);
  c.x.rt = __shfl_sync(0xffffffffu, x.rt, from);
  const int per_item = c.x.kt + COST;
  const long long i = sh.narrow ? static_cast<uint32_t>(off) / static_cast<uint32_t>(per_item)
                                : off / per_item;
  c.hk = 0;
  c.rt = static_cast<int>(i);
  c.item = c.cur - (off - i * per_item);
  return true;
}

struct LatentPlan {
  float2 *ml;  // maxima and sums of parts: [row of the part][begun before or in the range][worker]
  int2 *rows;  // [T * H]: a row's first worker + 65536 * its place in the parts, number of parts
  float *partials;
  unsigned *status;
  uint64_t wait_limit_ns;
  int hold;     // self-test: waits that run out (dec_debug_attn_timeout)
  int q_boxes;  // rows of q in boxes
};

__device__ __forceinline__ void tma_load_2d_to(uint32_t dst, const CUtensorMap *map, uint64_t *bar,
                                               int c0, int c1) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4}], [%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(c0), "r"(c1)
      : "memory");
}

__device__ __forceinline__ void tma_prefetch_4d(const CUtensorMap *map, int c0, int c1, int c2,
                                                int c3) {
  asm volatile("cp.async.bulk.prefetch.tensor.4d.L2.global.tile [%0, {%1, %2, %3, %4}];" ::"l"(
                   reinterpret_cast<uint64_t>(map)),
               "r"(c0), "r"(c1), "r"(c2), "r"(c3)
               : "memory");
}

// 16 lanes x 8 B columns: element (row l / 4 (+ 8), column 8 b + 2 (l % 4) (+ 1)) of block b is
// in v[4 b + 2 (second row) + (second column)] of lane l.
template <int B>
__device__ __forceinline__ void tmem_ld_blocks(uint32_t taddr, float *v) {
  uint32_t r[32];
  if constexpr (B == 1) {
    asm volatile("tcgen05.ld.sync.aligned.16x256b.x1.b32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(taddr)
                 : "memory");
  } else if constexpr (B == 2) {
    asm volatile(
        "tcgen05.ld.sync.aligned.16x256b.x2.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
          "=r"(r[7])
        : "r"(taddr)
        : "memory");
  } else {
    static_assert(B == 4, "blocks");
    asm volatile(
        "tcgen05.ld.sync.aligned.16x256b.x4.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,"
        "%14,%15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
          "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]),
          "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr)
        : "memory");
  }
#pragma unroll
  for (int i = 0; i < 4 * B; ++i) v[i] = __uint_as_float(r[i]);
}
// C consecutive columns of this thread's lane.
template <int C>
__device__ __forceinline__ void tmem_ld_cols(uint32_t taddr, float *v) {
  if constexpr (C == 8) {
    uint32_t r[8];
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]),
                   "=r"(r[6]), "=r"(r[7])
                 : "r"(taddr)
                 : "memory");
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(r[i]);
  } else {
    static_assert(C == 16, "columns");
    tmem_ld16(taddr, v);
  }
}
template <int C>
__device__ __forceinline__ void tmem_st_cols(uint32_t taddr, const uint32_t *r) {
  if constexpr (C == 8)
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(
                     taddr),
                 "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]),
                 "r"(r[7])
                 : "memory");
  else
    tmem_st16(taddr, r);
}
// Whether any of the `n` threads at named barrier `id` says so.
__device__ __forceinline__ bool named_bar_any(int id, int n, bool mine) {
  uint32_t y;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %3, 0;\n\t"
      "barrier.cta.red.or.pred q, %1, %2, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(y)
      : "r"(id), "r"(n), "r"(mine ? 1u : 0u)
      : "memory");
  return y != 0;
}
// Operand descriptor (128-byte swizzle): `leading` and `stride` offsets in bytes.
__device__ __forceinline__ uint64_t sw128_any(uint32_t saddr, uint32_t leading, uint32_t stride) {
  uint64_t d = static_cast<uint64_t>((saddr >> 4) & 0x3FFFu);
  d |= static_cast<uint64_t>(leading >> 4) << 16;
  d |= static_cast<uint64_t>(stride >> 4) << 32;
  d |= static_cast<uint64_t>(1) << 46;
  d |= static_cast<uint64_t>(2) << 61;
  return d;
}

template <int MQ, bool E4M3>
__global__ void __launch_bounds__((LdCfg<MQ, E4M3>::THREADS), 1)
    latent_decode_kernel(const __grid_constant__ CUtensorMap map,
                         const __grid_constant__ CUtensorMap qmap,
                         const __grid_constant__ AttnParams p, const LatentPlan pl,
                         const int width) {
  using C = LdCfg<MQ, E4M3>;
  constexpr int TOK = C::TOK, ST = C::ST, QB = C::QB, NS = C::NS, DP = C::DP;
  constexpr int GR = C::GR, NB = GR / 8, NC = GR / 4;  // of a group: rows, blocks; of a thread: rows
  constexpr int CH = GR < 16 ? GR : 16;  // columns of O at a time
  extern __shared__ __align__(1024) uint8_t ld_smem[];  // ring, q, weights
  __shared__ RangeStart<C::THREADS> start;
  __shared__ __align__(8) uint64_t full[ST], empty[4 * ST], qfull[QB], qempty[QB];
  __shared__ __align__(8) uint64_t s_full[NS], p_full, pv_done[NS], hold, drained[2];
  __shared__ uint64_t stage_valid[ST];  // tokens that exist
  __shared__ float part[4][MQ], by_row[MQ], row_scale[E4M3 ? 4 : 1][MQ];
  __shared__ int row_pos[MQ];
  __shared__ uint32_t tmem_slot;
  __shared__ int abort_flag;
  static_assert(
      fits_shared<sizeof(start) + sizeof(full) + sizeof(empty) + sizeof(qfull) + sizeof(qempty) +
                      sizeof(s_full) + sizeof(pv_done) + 4 * 8 + sizeof(stage_valid) +
                      sizeof(part) + sizeof(by_row) + sizeof(row_scale) + sizeof(row_pos) +
                      2 * sizeof(int),
                  C::SMEM>,
      "all of the above and the dynamic shared memory");
  const int slabs = width >> 6, group_bytes = slabs << 10;
  uint8_t *const ring = ld_smem, *const q_smem = ring + ST * C::STAGE;
  uint8_t *const w_smem = q_smem + QB * C::QBYTES;

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const bool boxes = !E4M3 && p.box > 0;  // or helpers fill the ring
  if (tid == 0) {
    abort_flag = 0;
    for (int i = 0; i < ST; ++i) {
      mbar_init(&full[i], boxes ? 1 : C::HW);
      for (int y = 0; y < 4; ++y) mbar_init(&empty[4 * i + y], 1);
    }
    for (int i = 0; i < QB; ++i) {
      mbar_init(&qfull[i], pl.q_boxes ? 1 : C::HW);
      mbar_init(&qempty[i], 1);
    }
    for (int i = 0; i < NS; ++i) {
      mbar_init(&s_full[i], 1);
      mbar_init(&pv_done[i], 1);
    }
    mbar_init(&p_full, 256);
    mbar_init(&hold, 1);
    mbar_init(&drained[0], 1);
    mbar_init(&drained[1], 1);
    fence_mbar_init();
    if (boxes) prefetch_tensormap(&map);
    if (pl.q_boxes) prefetch_tensormap(&qmap);
  }
  griddep_wait();
  const int H = p.Hq;
  LdShares sh;
  Cursor<TOK, MQ, LD_ITEM_COST, LD_LEAST> c;
  if (p.S <= 32) {
    if (!begin_range_small(p, H, sh, c)) return;
  } else {
    Shares wide;
    if (!begin_range<C::THREADS>(p, H, start, wide, c)) return;
    sh.share_n = wide.share_n;
    sh.share_r = wide.share_r;
    sh.narrow = (wide.share_n + 1) * gridDim.x < 0x7fffffffll;
  }
  if (warp == 8) {
    tmem_alloc(&tmem_slot, C::COLS);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  // after the allocation: a dependent grid's CTA cannot hold the columns this one waits for
  griddep_launch_dependents();
  const uint32_t tmem = tmem_slot, s_tmem = tmem + 4 * MQ;
  auto wait = [&](uint64_t *bar, int phase) {
    return mbar_wait_bounded(bar, phase & 1, pl.status, &abort_flag, pl.wait_limit_ns);
  };
  // For what comes once a segment: the limit times the waits of all `stages` so far (four a
  // stage, each with the limit to itself), as a segment may well take longer than the limit.
  auto wait_stages = [&](uint64_t *bar, int phase, int stages) {
    const uint64_t one = pl.wait_limit_ns;
    const uint64_t limit = one >> 34 == 0 ? one * (4ull * stages + 4) : one;  // below 2^64
    return mbar_wait_bounded(bar, phase & 1, pl.status, &abort_flag, limit);
  };
  // As many barriers in turn as there are S: who waits for stage i knows that i - NS is done.
  auto wait_pv = [&](int i) { wait(&pv_done[i % NS], i / NS); };
  int issued = 0, q_issued = 0;  // boxes: stages, items' q that were begun

  if (warp == 10) {
    // ================================================================ boxes of the cache
    // The pages of 32 blocks of 8 tokens are looked up in one step (four stages), a step ahead;
    // the boxes leave from one thread.
    const uint32_t base = smem_u32(ring);
    int k = 0;
    bool go = boxes;
    while (go && c.next(p, H)) {
      const int32_t *table = p.block_table + static_cast<long long>(c.s) * p.max_pages;
      auto look_up = [&](int from, int &page, int &off) {
        const int t = from + (lane >> 3);
        page = -1;
        off = 0;
        if (t < c.t1) {
          const int j = c.x.begin + t * TOK + ((lane & 7) << 3);
          if (j < c.x.len) {
            const int i = j / p.c.page_size;
            off = j - i * p.c.page_size;
            page = table[i];
          }
        }
      };
      int t = c.t0, page, off, next_page, next_off;
      look_up(t, page, off);
      look_up(t + 4, next_page, next_off);
      while (go && t < c.t1) {
        const uint32_t exist = __ballot_sync(0xffffffffu, page >= 0 && page < p.c.num_pages);
        for (int i = 0; i < 4 && t < c.t1; ++i, ++t) {
          const int at = k + t - c.t0, st = at % ST;
          const uint32_t blocks = exist >> (8 * i) & 255u;
          const int left = c.x.len - c.x.begin - t * TOK;
          uint64_t bits = 0;
#pragma unroll
          for (int b = 0; b < 8; ++b)
            if (blocks >> b & 1) bits |= 255ull << (8 * b);
          if (left < TOK) bits &= (1ull << max(left, 0)) - 1;
          // a quarter of the stage as soon as the last product that reads it is done
#pragma unroll
          for (int y = 0; y < 4; ++y) {
            if (at >= ST)
              go = __all_sync(0xffffffffu, wait(&empty[4 * st + y], at / ST - 1));
            if (!go) break;
            if (y == 0) {
              issued = at + 1;
              if (elect_one()) {
                stage_valid[st] = bits;
                mbar_arrive_expect_tx(&full[st], __popc(blocks) * group_bytes);
              }
            }
#pragma unroll
            for (int b = 2 * y; b < 2 * y + 2; ++b) {
              const int pg = __shfl_sync(0xffffffffu, page, i * 8 + b);
              const int o = __shfl_sync(0xffffffffu, off, i * 8 + b);
              if ((blocks >> b & 1) && elect_one())
                tma_load_4d(base + st * C::STAGE + b * group_bytes, &map, &full[st], 0, o, 0, pg);
              __syncwarp();
            }
          }
          if (!go) break;
          // the boxes LD_AHEAD stages on, toward L2
          const int far = i + LD_AHEAD;
          if (lane >> 3 == (far & 3)) {
            const int pg = far < 4 ? page : next_page;
            if (pg >= 0 && pg < p.c.num_pages) tma_prefetch_4d(&map, 0, far < 4 ? off : next_off, 0, pg);
          }
          __syncwarp();
        }
        page = next_page;
        off = next_off;
        look_up(t + 4, next_page, next_off);
      }
      k += c.t1 - c.t0;
    }
  } else if (warp == 11) {
    // ================================================================ boxes of q
    // Rows past the item's, of other sequences, fill columns that nobody reads.
    int seg = 0, stages = 0;
    bool go = pl.q_boxes;
    while (go && c.next(p, H)) {
      const int qb = seg % QB;
      if (seg >= QB)
        go = __all_sync(0xffffffffu, wait_stages(&qempty[qb], seg / QB - 1, stages));
      stages += c.t1 - c.t0;
      if (!go) break;
      q_issued = seg + 1;
      if (elect_one()) {
        const uint32_t to = smem_u32(q_smem + qb * C::QBYTES);
        mbar_arrive_expect_tx(&qfull[qb], slabs * MQ * 128);
        for (int slab = 0; slab < slabs; ++slab)
          tma_load_2d_to(to + slab * MQ * 128, &qmap, &qfull[qb], slab * 64,
                         c.x.q0 * H + c.rt * MQ);
      }
      __syncwarp();
      ++seg;
    }
  } else if (warp >= 12) {
    // ================================================================ rows of q, stages by hand
    const int hw = warp - 12;
    const bool q_by_hand = !pl.q_boxes;
    const int chunks = width >> 3;  // 16-byte chunks of a row: at most 72
    int k = 0, seg = 0, stages = 0;
    while ((!boxes || q_by_hand) && c.next(p, H)) {
      // q: a warp a row, four rows at a time
      const int qb = seg % QB;
      const int n_rows = min(MQ, c.x.n * H - c.rt * MQ);
      uint8_t *qd = q_smem + qb * C::QBYTES;
      bool waited = seg < QB;
#pragma unroll 1
      for (int r0 = hw; q_by_hand && r0 < MQ; r0 += 4 * C::HW) {
        uint4 v[4][3];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int r = r0 + C::HW * e;
          const int rr = c.rt * MQ + r, tok = rr / H, g = rr - tok * H;
          const uint16_t *src = p.q + (c.x.q0 + tok) * p.q_stride + static_cast<long long>(g) * width;
#pragma unroll
          for (int i = 0; i < 3; ++i) {
            const int ch = lane + 32 * i;
            v[e][i] = make_uint4(0, 0, 0, 0);
            if (r < n_rows && ch < chunks)
              v[e][i] = *reinterpret_cast<const uint4 *>(src + ch * 8);
          }
        }
        if (!waited) {
          wait_stages(&qempty[qb], seg / QB - 1, stages);
          waited = true;
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int r = r0 + C::HW * e;
          if (r >= MQ) break;
          if (E4M3) {
            float mx = 0.0f;
#pragma unroll
            for (int i = 0; i < 3; ++i) {
              const uint32_t u[4] = {v[e][i].x, v[e][i].y, v[e][i].z, v[e][i].w};
#pragma unroll
              for (int d = 0; d < 4; ++d) mx = fmaxf(mx, fmaxf(fabsf(bf16lo(u[d])), fabsf(bf16hi(u[d]))));
            }
#pragma unroll
            for (int d = 16; d > 0; d >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, d));
            const int ex = q_exponent(mx);
            const float f = power_of_two(-ex);
            if (lane == 0) row_scale[seg & 3][r] = power_of_two(ex);
#pragma unroll
            for (int i = 0; i < 3; ++i)
              v[e][i] = make_uint4(pack2<true>(bf16lo(v[e][i].x) * f, bf16hi(v[e][i].x) * f),
                                   pack2<true>(bf16lo(v[e][i].y) * f, bf16hi(v[e][i].y) * f),
                                   pack2<true>(bf16lo(v[e][i].z) * f, bf16hi(v[e][i].z) * f),
                                   pack2<true>(bf16lo(v[e][i].w) * f, bf16hi(v[e][i].w) * f));
          }
#pragma unroll
          for (int i = 0; i < 3; ++i) {
            const int ch = lane + 32 * i;
            if (ch < chunks)
              *reinterpret_cast<uint4 *>(qd + (ch >> 3) * (MQ * 128) + r * 128 +
                                         (((ch & 7) ^ (r & 7)) << 4)) = v[e][i];
          }
        }
      }
      if (q_by_hand) {
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&qfull[qb]);
      }
      ++seg;
      stages += c.t1 - c.t0;
      if (boxes) continue;
      const int32_t *table = p.block_table + static_cast<long long>(c.s) * p.max_pages;
      if constexpr (E4M3) {
        // A warp has eight tokens, one swizzle group; a lane 16 bytes of every 64 of one token.
        // The next stage's bytes are on their way in registers while this one is in use, and
        // those of the one after it are requested into L2.
        const int r = lane >> 2, ch = (lane & 3) * 2;
        auto place = [&](int t) -> long long {  // this lane's token: its element, -1: none
          const int j = c.x.begin + t * TOK + hw * 8 + r;
          if (t >= c.t1 || j >= c.x.len) return -1;
          const int i = j / p.c.page_size, pg = table[i];
          if (pg < 0 || pg >= p.c.num_pages) return -1;
          return pg * p.c.page_stride + (j - i * p.c.page_size) * p.c.token_stride;
        };
        const uint8_t *const bytes = static_cast<const uint8_t *>(p.c.k);
        uint4 v[LATENT_MAX_W / 64];
        auto load = [&](long long at) {
#pragma unroll
          for (int i = 0; i < LATENT_MAX_W / 64; ++i) {
            v[i] = make_uint4(0, 0, 0, 0);
            if (at >= 0 && i < slabs)
              v[i] = *reinterpret_cast<const uint4 *>(bytes + at + i * 64 + ch * 8);
          }
        };
        long long here = place(c.t0), next = place(c.t0 + 1);
        load(here);
        for (int t = c.t0; t < c.t1; ++t, ++k) {
          const int st = k % ST;
          const uint32_t exist = __ballot_sync(0xffffffffu, here >= 0);
          const long long after = place(t + 2);
          if (after >= 0 && (lane & 3) == 0) prefetch_l2_bulk(bytes + after, width);
          if (k >= ST) wait(&empty[4 * st + hw / 2], k / ST - 1);  // this warp's quarter
          uint8_t *d = ring + st * C::STAGE + hw * group_bytes + r * 128;
#pragma unroll
          for (int i = 0; i < LATENT_MAX_W / 64; ++i) {
            if (i >= slabs) break;
            const uint4 y = v[i];
            *reinterpret_cast<uint4 *>(d + i * 1024 + ((ch ^ r) << 4)) =
                make_uint4(e4m3x2_to_f16x2(y.x), e4m3x2_to_f16x2(y.x >> 16),
                           e4m3x2_to_f16x2(y.y), e4m3x2_to_f16x2(y.y >> 16));
            *reinterpret_cast<uint4 *>(d + i * 1024 + (((ch + 1) ^ r) << 4)) =
                make_uint4(e4m3x2_to_f16x2(y.z), e4m3x2_to_f16x2(y.z >> 16),
                           e4m3x2_to_f16x2(y.w), e4m3x2_to_f16x2(y.w >> 16));
          }
          if (lane == 0) {
            uint32_t bits = 0;
#pragma unroll
            for (int i = 0; i < 8; ++i) bits |= (exist >> (4 * i) & 1u) << i;
            reinterpret_cast<volatile uint8_t *>(&stage_valid[st])[hw] =
                static_cast<uint8_t>(bits);
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(&full[st]);
          here = next;
          next = after;
          if (t + 1 < c.t1) load(here);
        }
      } else {
        // 16 tokens a warp, each looked up by itself, in asynchronous copies of 16 bytes: eight lanes
        // a token's 64 elements. The next stage's rows are requested into L2 meanwhile. (Through
        // registers, a few at a time, pages of 13 tokens took 289 us where pages of 32 take 79.)
        auto place = [&](int t) -> long long {  // token `lane` (of the first 16): its element, -1: none
          const int j = c.x.begin + t * TOK + hw * 16 + (lane & 15);
          if (t >= c.t1 || j >= c.x.len) return -1;
          const int i = j / p.c.page_size, pg = table[i];
          if (pg < 0 || pg >= p.c.num_pages) return -1;
          return pg * p.c.page_stride + (j - i * p.c.page_size) * p.c.token_stride;
        };
        const uint16_t *const elements = static_cast<const uint16_t *>(p.c.k);
        long long here = place(c.t0);
        for (int t = c.t0; t < c.t1; ++t, ++k) {
          const int st = k % ST;
          const uint32_t exist = __ballot_sync(0xffffffffu, here >= 0) & 0xffffu;
          if (k >= ST) wait(&empty[4 * st + hw], k / ST - 1);  // this warp's quarter
#pragma unroll 1
          for (int x = 0; x < 4; ++x) {
            const int tok = 4 * x + (lane >> 3), r = tok & 7;
            const long long at = __shfl_sync(0xffffffffu, here, tok);
            const uint16_t *src = elements + (at < 0 ? 0 : at) + (lane & 7) * 8;
            const uint32_t dst = smem_u32(ring + st * C::STAGE + (2 * hw + (tok >> 3)) * group_bytes +
                                          r * 128 + (((lane & 7) ^ r) << 4));
#pragma unroll 1
            for (int slab = 0; slab < slabs; ++slab)
              cp_async16(dst + slab * 1024, src + slab * 64, at >= 0);
          }
          const long long next = place(t + 1);
          if (next >= 0 && lane < 16) prefetch_l2_bulk(elements + next, 2 * width);
          if (lane == 0)
            reinterpret_cast<volatile uint16_t *>(&stage_valid[st])[hw] =
                static_cast<uint16_t>(exist);
          cp_async_wait_all();
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(&full[st]);
          here = next;
        }
      }
    }
  } else if (warp == 8) {
    // ================================================================ S = C . Q^T
    const uint32_t id = (tc_idesc<E4M3>(MQ) & ~(31u << 24)) | (64u >> 4) << 24;
    const uint32_t q_u = smem_u32(q_smem), ring_u = smem_u32(ring);
    int k = 0, seg = 0;
    while (c.next(p, H)) {
      const int qb = seg % QB;
      wait(&qfull[qb], seg / QB);
      for (int t = c.t0; t < c.t1; ++t, ++k) {
        const int st = k % ST;
        wait(&full[st], k / ST);
        if (k >= NS) wait_pv(k - NS);  // its S has been read
        tc_fence_after();
        if (elect_one()) {
          const uint32_t d = s_tmem + (k % NS) * MQ;
          uint64_t a = sw128_any(ring_u + st * C::STAGE, 16, group_bytes);
          uint64_t b = sw128_any(q_u + qb * C::QBYTES, 16, 1024);
#pragma unroll 1
          for (int slab = 0; slab < slabs; ++slab) {
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
              tc_mma(d, a + 2 * kk, b + 2 * kk, id, kk > 0 || slab > 0 ? 1u : 0u);
            a += 1024 >> 4;
            b += (MQ * 128) >> 4;
          }
          tc_commit(&s_full[k % NS]);
          if (t + 1 == c.t1) tc_commit(&qempty[qb]);
        }
        __syncwarp();
      }
      ++seg;
    }
  } else if (warp == 9) {
    // ================================================================ O += C^T . P
    const uint32_t id = tc_idesc<E4M3>(MQ) | (1u << 15) | (1u << 16);
    const uint32_t ring_u = smem_u32(ring);
    const uint64_t b = sw128_any(smem_u32(w_smem), 1024, 1024);
    const int blocks = (p.D + 127) >> 7;
    int k = 0;
    while (c.next(p, H)) {
      for (int t = c.t0; t < c.t1; ++t, ++k) {
        const int st = k % ST;
        wait(&p_full, k);
        tc_fence_after();
        if (elect_one()) {
          const uint32_t acc = t > c.t0 ? 1u : 0u;
          const uint64_t a = sw128_any(ring_u + st * C::STAGE, 1024, group_bytes);
#pragma unroll
          for (int kk = 0; kk < TOK / 16; ++kk) {  // two boxes of tokens
#pragma unroll 1
            for (int blk = 0; blk < blocks; ++blk)
              tc_mma(tmem + blk * MQ, a + ((2 * kk * group_bytes + blk * 2048) >> 4),
                     b + ((kk * 2048) >> 4), id, kk > 0 ? 1u : acc);
            tc_commit(&empty[4 * st + kk]);
          }
          tc_commit(&pv_done[k % NS]);
        }
        __syncwarp();
      }
    }
    if (k > 0) wait_pv(k - 1);  // nothing in flight when the columns are released
  } else {
    // ================================================================ softmax
    constexpr uint32_t INF2 = E4M3 ? 0x7c007c00u : 0x7f807f80u;  // exponents of two values
    const int grp = warp >> 2, w4 = warp & 3, gt = tid & 127, bar = 1 + grp, g0 = grp * GR;
    const uint32_t lanes = static_cast<uint32_t>(w4 * 32) << 16;
    // rows g0 + 8 b + col (+ 1), tokens tok0 (+ 8)
    const int col = 2 * (lane & 3), tok0 = w4 * 16 + (lane >> 2);
    const float scale = p.scale * LOG2E * (p.c.k_scale ? p.c.k_scale[0] : 1.0f);
    int k = 0, seg = 0;
    if (pl.hold) wait(&hold, 0);  // self-test: nobody arrives
    while (c.next(p, H)) {
      const SeqInfo &x = c.x;
      const int n_rows = min(MQ, x.n * H - c.rt * MQ), row0 = c.rt * MQ;
      const int pos0 = x.len - x.n;
      // the last key that a row sees (its token's position); what every row sees
      if (gt < GR) {
        const int r = g0 + gt, tok = (row0 + min(r, n_rows - 1)) / H;
        row_pos[r] = pos0 + tok;
      }
      const int hi_all = pos0 + row0 / H, hi_top = pos0 + (row0 + n_rows - 1) / H;
      const int lo_all = p.window > 0 && hi_top >= p.window ? hi_top - p.window + 1 : 0;
      named_bar_sync(bar, 128);
      float m[NC], l[NC], zf[NC];
#pragma unroll
      for (int i = 0; i < NC; ++i) m[i] = -INFINITY, l[i] = 0.0f, zf[i] = scale;
      for (int t = c.t0; t < c.t1; ++t, ++k) {
        const int st = k % ST;
        wait(&s_full[k % NS], k / NS);
        tc_fence_after();
        float z[4 * NB];
        tmem_ld_blocks<NB>(s_tmem + (k % NS) * MQ + g0 + lanes, z);
        wait(&full[st], k / ST);  // (long since) the copying warps' bits and the values
        const uint64_t valid = stage_valid[st];
        const int j0 = x.begin + t * TOK;
        const bool plain = valid == ~0ull && j0 >= lo_all && j0 + TOK - 1 <= hi_all;
        const bool begins = t == c.t0;
        if (E4M3 && begins) {
#pragma unroll
          for (int i = 0; i < NC; ++i)
            zf[i] = scale * row_scale[seg & 3][g0 + 8 * (i >> 1) + col + (i & 1)];
        }
        tmem_wait_ld();
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
          for (int e = 0; e < 4; ++e) z[4 * b + e] *= zf[2 * b + (e & 1)];
        if (!plain) {
#pragma unroll
          for (int b = 0; b < NB; ++b)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int tok = tok0 + 8 * (e >> 1), j = j0 + tok;
              const int hi = row_pos[g0 + 8 * b + col + (e & 1)];
              const int lo = p.window > 0 && hi >= p.window ? hi - p.window + 1 : 0;
              if (j < lo || j > hi || !(valid >> tok & 1)) z[4 * b + e] = -INFINITY;
            }
        }
        bool grows = false;
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float mx = fmaxf(z[4 * b + e], z[4 * b + 2 + e]);
            if (E4M3) mx -= F16_POWERS;
            grows |= mx - m[2 * b + e] >= TC_LAZY;
          }
        if (named_bar_any(bar, 128, grows || begins)) {
          // move the maxima that grew; the outputs so far are rescaled in tensor memory, after
          // the last product that adds to them
#pragma unroll
          for (int b = 0; b < NB; ++b)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              float mx = fmaxf(z[4 * b + e], z[4 * b + 2 + e]);
#pragma unroll
              for (int d = 4; d < 32; d <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, d));
              if (lane < 4) part[w4][g0 + 8 * b + col + e] = mx;
            }
          named_bar_sync(bar, 128);
#pragma unroll
          for (int b = 0; b < NB; ++b)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const int r = g0 + 8 * b + col + e;
              float mx = fmaxf(fmaxf(part[0][r], part[1][r]), fmaxf(part[2][r], part[3][r]));
              if (E4M3) mx -= F16_POWERS;
              // (each by itself: a row's bits do not depend on what only other rows see)
              const float old = m[2 * b + e], now = mx - old >= TC_LAZY ? mx : old;
              const float fade = ex2(old - (now == -INFINITY ? 0.0f : now));
              m[2 * b + e] = now;
              l[2 * b + e] *= fade;
              if (w4 == 0 && lane < 4) by_row[r] = fade;
            }
          if (!begins) {
            named_bar_sync(bar, 128);
            wait_pv(k - 1);
            tc_fence_after();
#pragma unroll 1
            for (int blk = 0; blk < (p.D + 127) >> 7; ++blk)
#pragma unroll 1
              for (int i = g0; i < g0 + GR; i += CH) {
                float o[CH];
                uint32_t u[CH];
                tmem_ld_cols<CH>(tmem + lanes + blk * MQ + i, o);
                tmem_wait_ld();
#pragma unroll
                for (int e = 0; e < CH; ++e) u[e] = __float_as_uint(o[e] * by_row[i + e]);
                tmem_st_cols<CH>(tmem + lanes + blk * MQ + i, u);
              }
            tmem_wait_st();
          }
        }
        uint32_t w[2 * NB];
#pragma unroll
        for (int b = 0; b < NB; ++b) {
          const float b0 = m[2 * b] == -INFINITY ? 0.0f : m[2 * b];
          const float b1 = m[2 * b + 1] == -INFINITY ? 0.0f : m[2 * b + 1];
          const float y0 = ex2(z[4 * b] - b0), y1 = ex2(z[4 * b + 1] - b1);
          const float y2 = ex2(z[4 * b + 2] - b0), y3 = ex2(z[4 * b + 3] - b1);
          l[2 * b] += y0 + y2;
          l[2 * b + 1] += y1 + y3;
          w[2 * b] = pack2<E4M3>(y0, y1);
          w[2 * b + 1] = pack2<E4M3>(y2, y3);
        }
        if (k > 0) wait_pv(k - 1);  // it reads the weights
        const int r = lane >> 2;
        uint8_t *d = w_smem + tok0 * 128 + (lane & 3) * 4;
#pragma unroll
        for (int b = 0; b < NB; ++b) {
          const int at = ((grp * NB + b) ^ r) << 4;
          *reinterpret_cast<uint32_t *>(d + at) = w[2 * b];
          *reinterpret_cast<uint32_t *>(d + 1024 + at) = w[2 * b + 1];
        }
        if (!plain) {
          // Weights of zero must not meet what is not finite: tokens that do not exist get
          // zeros, and so does what is not finite in a token that some row does not see. (A
          // row that sees it has a score that is not finite either: its weight is NaN, or
          // zero where the score is -infinity.)
          uint8_t *v = ring + st * C::STAGE;
          const int cpr = p.D >> 3;  // chunks of a value
          const int head = min(max(lo_all - j0, 0), TOK), tail = min(max(hi_all + 1 - j0, 0), TOK);
          auto clean = [&](int row) {
            const bool gone = !(valid >> row & 1);
            uint8_t *at = v + (row >> 3) * group_bytes + (row & 7) * 128;
            for (int i = lane; i < cpr; i += 32) {
              uint4 *y = reinterpret_cast<uint4 *>(at + (i >> 3) * 1024 +
                                                   (((i & 7) ^ (row & 7)) << 4));
              if (gone) {
                *y = make_uint4(0, 0, 0, 0);
              } else {
                const uint4 u = *y;
                const uint4 bad = make_uint4(
                    __vcmpeq2(u.x & INF2, INF2), __vcmpeq2(u.y & INF2, INF2),
                    __vcmpeq2(u.z & INF2, INF2), __vcmpeq2(u.w & INF2, INF2));
                if (bad.x | bad.y | bad.z | bad.w)
                  *y = make_uint4(u.x & ~bad.x, u.y & ~bad.y, u.z & ~bad.z, u.w & ~bad.w);
              }
            }
          };
          // tokens that all rows see and that exist need no look
          for (int row = warp; row < TOK; row += 8)
            if (row < head || row >= tail || !(valid >> row & 1)) clean(row);
        }
        fence_proxy_async_smem();  // before the product (and later boxes) touch either
        tc_fence_before();
        mbar_arrive(&p_full);
      }

      // ---- the segment's outputs: sums over lanes and warps, then a thread a latent element
      const int me = blockIdx.x;
      const long long unit = c.item + LD_ITEM_COST;
      const int c0 = sh.worker_of(unit), c1 = sh.worker_of(unit + x.kt - 1);
      const float v_scale = p.c.v_scale ? p.c.v_scale[0] : 1.0f;
      const ItemOut dst = {x.q0, row0, 0, H, v_scale};
      float *slot = pl.partials + static_cast<size_t>(part_slot(c0, me - c0)) * C::SLOT;
      named_bar_sync(bar, 128);  // `part` may still be read
#pragma unroll
      for (int i = 0; i < NC; ++i) {
        float s = l[i];
#pragma unroll
        for (int d = 4; d < 32; d <<= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
        const int r = g0 + 8 * (i >> 1) + col + (i & 1);
        if (lane < 4) {
          part[w4][r] = s;
          if (w4 == 0) by_row[r] = m[i];
        }
      }
      named_bar_sync(bar, 128);
      if (gt < GR && g0 + gt < n_rows) {
        const int r = g0 + gt;
        const float mr = by_row[r];
        const float lr = (part[0][r] + part[1][r]) + (part[2][r] + part[3][r]);
        if (c0 == c1) {
          dst.put_lse(p, r, mr, lr);
          by_row[r] = lr == 0.0f ? 0.0f : v_scale / lr;
        } else {
          pl.ml[(2 * r + (me == c0 ? 1 : 0)) * gridDim.x + me] = make_float2(mr, lr);
        }
        // where the row's parts are
        if (me == c0)
          pl.rows[static_cast<long long>(x.q0) * H + row0 + r] =
              make_int2(c0 | r << 16, c1 - c0 + 1);
      }
      if (k > 0) wait_pv(k - 1);
      tc_fence_after();
      named_bar_sync(bar, 128);
#pragma unroll 1
      for (int d0 = 0; d0 < p.D; d0 += 128) {
        const int dim = d0 + gt;  // past D in a last half block
#pragma unroll 1
        for (int r0 = g0; r0 < min(n_rows, g0 + GR); r0 += CH) {
          float o[CH];
          tmem_ld_cols<CH>(tmem + lanes + (d0 >> 7) * MQ + r0, o);
          tmem_wait_ld();
          if (c0 == c1) {
            // two rows at a time: an even lane has two elements of the first, an odd one of
            // the second
#pragma unroll
            for (int e = 0; e < CH; e += 2) {
              const float f0 = by_row[r0 + e], f1 = by_row[r0 + e + 1];
              // a row that saw nothing: zeros, whatever its columns hold
              const float y0 = f0 == 0.0f ? 0.0f : o[e] * f0;
              const float y1 = f1 == 0.0f ? 0.0f : o[e + 1] * f1;
              const float got = __shfl_xor_sync(0xffffffffu, lane & 1 ? y0 : y1, 1);
              const int r = r0 + e + (lane & 1);
              if (r < n_rows && dim < p.D) {
                const int tok = row_pos[r] - pos0, head = row0 + r - tok * H;
                *reinterpret_cast<uint32_t *>(p.out + (x.q0 + tok) * p.out_stride +
                                              static_cast<long long>(head) * p.D + (dim & ~1)) =
                    lane & 1 ? pack2<false>(got, y1) : pack2<false>(y0, got);
              }
            }
          } else if (dim < p.D) {
#pragma unroll
            for (int e = 0; e < CH; ++e)
              if (r0 + e < n_rows) slot[(r0 + e) * DP + dim] = o[e];
          }
          __syncwarp();  // the next read of tensor memory wants the warp in one place
        }
      }
      tc_fence_before();  // the next segment's products overwrite the columns
      named_bar_sync(bar, 128);
      ++seg;
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  // Every wait of the CTA is over. If one ran out, products and boxes may still be on their way:
  // products end before tensor memory is released, boxes land before the CTA ends.
  if (*static_cast<volatile int *>(&abort_flag)) {
    if (warp == 8 || warp == 9) {
      uint64_t *bar = &drained[warp - 8];
      if (elect_one()) tc_commit(bar);
      __syncwarp();
      mbar_wait_drain(bar, 0, 10000000ull);
    }
    for (int i = issued - 1; i >= 0 && i >= issued - ST; --i)
      mbar_wait_drain(&full[i % ST], (i / ST) & 1, 10000000ull);
    for (int i = q_issued - 1; i >= 0 && i >= q_issued - QB; --i)
      mbar_wait_drain(&qfull[i % QB], (i / QB) & 1, 10000000ull);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
  }
  if (warp == 8) tmem_dealloc(tmem, C::COLS);
}

template <int MQ, bool E4M3>
cudaError_t launch_latent_shape(const AttnParams &p, int width, const LatentLaunch &a,
                                cudaStream_t s) {
  using C = LdCfg<MQ, E4M3>;
  auto kernel = latent_decode_kernel<MQ, E4M3>;
  const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             static_cast<int>(C::SMEM));
  if (e != cudaSuccess) return e;
  LatentPlan pl;
  pl.ml = a.ml;
  pl.rows = static_cast<int2 *>(a.rows);
  pl.partials = a.partials;
  pl.status = a.status;
  pl.wait_limit_ns = a.wait_limit_ns;
  pl.hold = a.hold;
  pl.q_boxes = !E4M3 && a.q_boxes;
  return launch_pdl(kernel, dim3(a.num_sms), dim3(C::THREADS), C::SMEM, s, a.map, a.qmap, p, pl,
                    width);
}

template <bool E4M3>
cudaError_t launch_latent(const AttnParams &p, int width, int rows, const LatentLaunch &a,
                          cudaStream_t s) {
  switch (rows) {
    case 16:
      return launch_latent_shape<16, E4M3>(p, width, a, s);
    case 32:
      return launch_latent_shape<32, E4M3>(p, width, a, s);
    default:
      return launch_latent_shape<64, E4M3>(p, width, a, s);
  }
}

}  // namespace
}  // namespace ssd

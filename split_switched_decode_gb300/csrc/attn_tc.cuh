// attn_tc.cuh -- attention over a paged cache for many rows a kv head (verification rows,
// wide groups) on tcgen05 tensor cores.
//
// (bf16; e4m3 below.) The warps of attn_kernel.cuh take a stage's tokens against 8 rows at a
// time, and above 16 rows these chains of small products, exponentials and shuffles take longer
// than the keys' and values' way from HBM (64 rows, 64 ragged sequences: 406 us where the copy
// takes 160). Here a stage of 64 tokens is two products for up to 128 rows, 512 clocks of the
// tensor core. Up to 64 rows copying bounds it: 32 rows 173 us, 64 rows 179, 6.1 TB/s. With 128
// rows (232 us) twice the exponentials, spilled registers and twice the outputs to join and
// write come before it; heads of 64 (64 rows: 112 us, copy 80) stop at the softmax's chain.
// Division of the work, ring of stages and joins are attn_kernel.cuh's; one CTA an SM has sixteen
// warps (twelve for heads above 128):
//
//   4 or 8  softmax: a thread a TMEM lane; MQ = 32, 64 or 128 rows an item
//   3       TMA boxes into the ring, each every third stage
//   2 + 1   a thread each issues the products below, the scores' in turn
//   2       rows of q into shared memory
//
//     S[rows, 64 tokens] = Q . K^T    A = Q, B = K, both K-major in shared memory (the boxes'
//                                     128-byte swizzle is the operand layout)
//     O[rows, D]        += P . V      A = P from tensor memory, B = V as stored: rows of a
//                                     token, elements contiguous (MN-major)
//
// There are four S, and P (bf16) overwrites its S: scores run up to three stages ahead of the
// softmax, outputs behind it (with two S the way from one stage's weights through its outputs
// to the scores two stages on set the pace). A stage's softmax is a chain of 900 to 1300 clocks
// (wait, tensor memory, maximum, exponentials, tensor memory, arrival) where the copy of a
// stage of heads of 64 takes 600: two groups of four warps take the stages in turn, each
// with a maximum, a sum and outputs of its own (heads above 128: one group, as two outputs
// and the scores exceed tensor memory). M is 128 whatever the rows are: Q stands in shared
// memory 128 / MQ times, and copy g of a row takes the softmax of the g-th part of the
// stage's tokens with weights of zero for the others, again with outputs of its own. All
// are joined at the segment's end. So four warps share the exponentials at any number of
// rows (with one copy and 32 rows a single warp took 2.4 us a stage, twice what its bytes
// take).
//
// The running maximum that weights refer to is moved only when a row's maximum has grown by
// 8 or more (weights then stay below 2^8, and their rounding to bf16, relative 2^-8 as the
// output's own, is not enlarged), so the outputs in tensor memory are rarely rescaled; sums
// are fp32 of the weights before rounding and refer to the same maximum. (On e4m3 caches, whose
// weights are f16, to one smaller by F16_POWERS: attn_kernel.cuh.)
//
// E4M3 caches: the boxes fill a ring of their own, and four warps widen its stages to f16 (every
// e4m3 value is an f16 value) into a short ring of operands; q is scaled by a power of two a
// row and converted to f16, the weights are f16, the rest is the same with one softmax
// group (a second one's registers went to the widening warps). A stage then costs about 0.8
// us of widening, products and softmax in turn: 64 ragged sequences with 64 rows a kv head 225
// to 231 us where the kernel of attn_kernel.cuh takes 437 to 452 (copy: 82).
//
// What is left over the copy: a segment's end (join, stores, the next item's first scores)
// stops the copies for about 3 us, as the ring of six stages is what they need in flight;
// at 64 rows a CTA has four or five ends in its share.
#pragma once

#include <float.h>

#include "attn_kernel.cuh"
#include "tcgen05.cuh"

namespace ssd {
namespace {

constexpr int TC_QTHREADS = 64;
constexpr int TC_NS = 4;  // buffers of scores
constexpr float TC_LAZY = 8.0f;
// An item costs what eight stages do (64 ragged sequences: 64 rows a kv head 179 us, with a
// charge of six 182, of one 200; 128 rows 241, 251 with six, 231 with twelve, at which 32 rows
// and short sequences lose up to 1 us). Work that does not fill the SMs is cut into shares of
// up to 9 units, 5 at least: one that holds only an item's charge does nothing.
constexpr int TC_ITEM_COST = 8, TC_LEAST = 9;

template <int DP, int MQ, bool E4M3>
struct TcCfg {
  static constexpr int TOK = 64, RB = DP * 2, STAGE = 2 * TOK * RB;
  static constexpr int COPIES = 128 / MQ, TS = TOK / COPIES;  // tokens of a copy
  static constexpr int QBYTES = 128 * DP * 2;
  // One CTA an SM: with two, each ring would hold two stages beside Q's copies, and a stage
  // came every 2.2 us where the copy rate gives two in 1.45. E4M3: the stages as they come
  // stand in a ring of their own (RST), their widened form in a short one (ST).
  static constexpr int ST = E4M3 ? (DP == 64 ? 4 : (DP == 128 ? 3 : 1))
                                 : (DP == 64 ? 8 : (DP == 128 ? 6 : 2));
  static constexpr int RST = DP == 64 ? 8 : (DP == 128 ? 6 : 3);
  static constexpr int ES = E4M3 ? 1 : 2, CRB = DP * ES, CSTAGE = 2 * TOK * CRB;  // copied
  static constexpr int CST = E4M3 ? RST : ST;
  // Warps that copy, each every CW-th stage. A wait for a stage's release tells only
  // neighbouring phases apart: stage k - CST, which a warp has seen released when it comes to
  // k + CW, has to be k + CW - 2 CST or later.
  static constexpr int CW = CST < 3 ? 2 : 3;
  static_assert(CW <= CST, "a copying warp must not run two rounds of the ring ahead");
  // Warps that issue the scores, in turn; a stage of the ring belongs to one of them.
  static constexpr int KW = ST % 2 == 0 ? 2 : 1;
  static constexpr int QB = DP == 64 ? 2 : 1;
  static constexpr size_t SMEM = QB * QBYTES + ST * STAGE + (E4M3 ? RST * CSTAGE : 0);
  // softmax warpgroups, which take the stages in turn, each with outputs of its own
  static constexpr int GROUPS = DP <= 128 && !E4M3 ? 2 : 1;
  static constexpr int SW = 4 * GROUPS, PARTS = GROUPS * COPIES;
  static constexpr int THREADS = 32 * (SW + 8 + (E4M3 ? 4 : 0));
  static constexpr int COLS = 512;  // all: the groups' O, then TC_NS S of 64 columns
  static_assert(GROUPS * DP + TC_NS * 64 <= COLS, "tensor memory");
  static constexpr int SLOT = MQ * DP + 2 * MQ;
};

// D[tmem] (+)= A[tmem] * B[smem], bf16, fp32 accumulate; one thread issues.
__device__ __forceinline__ void tc_mma_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t bdesc,
                                          uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, float *v) {
  uint32_t r[32];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,"
      "%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]),
        "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]),
        "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]),
        "=r"(r[31])
      : "r"(taddr)
      : "memory");
#pragma unroll
  for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
}
// Two fp32 operations in one instruction: a * b + c, a + b.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("{\n\t.reg .b64 x, y, z;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\t"
      "mov.b64 z, {%6, %7};\n\tfma.rn.f32x2 x, x, y, z;\n\tmov.b64 {%0, %1}, x;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 d;
  asm("{\n\t.reg .b64 x, y;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\t"
      "add.rn.f32x2 x, x, y;\n\tmov.b64 {%0, %1}, x;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}
__device__ __forceinline__ uint32_t tmem_ld1(uint32_t taddr) {
  uint32_t r;
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x1.b32 {%0}, [%1];" : "=r"(r) : "r"(taddr)
               : "memory");
  return r;
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t *r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,"
      "%14,%15,%16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
      "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]),
      "r"(r[15])
      : "memory");
}
__device__ __forceinline__ void tmem_wait_st() {
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}
// Descriptor of an operand whose M or N dimension is contiguous, in slabs of 64 elements (128
// bytes, swizzled) x K rows: 8 rows of K are 1024 bytes (stride offset), the next 64 elements
// `slab_bytes` on (leading offset).
__device__ __forceinline__ uint64_t sw128_mn_desc(uint32_t saddr, uint32_t slab_bytes) {
  uint64_t d = static_cast<uint64_t>((saddr >> 4) & 0x3FFFu);
  d |= static_cast<uint64_t>(slab_bytes >> 4) << 16;
  d |= static_cast<uint64_t>(1024 >> 4) << 32;
  d |= static_cast<uint64_t>(1) << 46;
  d |= static_cast<uint64_t>(2) << 61;
  return d;
}

// Instruction descriptor: f16 or bf16 operands, 128 rows, n columns.
template <bool F16>
__device__ __forceinline__ uint32_t tc_idesc(int n) {
  return F16 ? idesc_bf16(n) & ~(1u << 7 | 1u << 10) : idesc_bf16(n);
}
template <bool F16>
__device__ __forceinline__ float to_f32(uint32_t bits) {
  return F16 ? __half2float(__ushort_as_half(static_cast<uint16_t>(bits)))
             : bf16_to_f32(static_cast<uint16_t>(bits));
}
// Eight bf16 elements of a row of q, `lanes` neighbouring lanes a row, as f16: divided by a power
// of two (q_exponent), which goes to `scale`.
__device__ __forceinline__ uint4 q_to_f16(uint4 v, int lanes, float *scale) {
  float mx = fmaxf(fmaxf(fmaxf(fabsf(bf16lo(v.x)), fabsf(bf16hi(v.x))),
                         fmaxf(fabsf(bf16lo(v.y)), fabsf(bf16hi(v.y)))),
                   fmaxf(fmaxf(fabsf(bf16lo(v.z)), fabsf(bf16hi(v.z))),
                         fmaxf(fabsf(bf16lo(v.w)), fabsf(bf16hi(v.w)))));
  for (int d = 1; d < lanes; d <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, d));
  const int e = q_exponent(mx);
  const float f = power_of_two(-e);
  if (scale) *scale = power_of_two(e);
  return make_uint4(pack2<true>(bf16lo(v.x) * f, bf16hi(v.x) * f),
                    pack2<true>(bf16lo(v.y) * f, bf16hi(v.y) * f),
                    pack2<true>(bf16lo(v.z) * f, bf16hi(v.z) * f),
                    pack2<true>(bf16lo(v.w) * f, bf16hi(v.w) * f));
}

template <int DP, int MQ, bool E4M3>
__global__ void __launch_bounds__((TcCfg<DP, MQ, E4M3>::THREADS), 1)
    attn_tc_kernel(const __grid_constant__ CUtensorMap kmap,
                   const __grid_constant__ CUtensorMap vmap,
                   const __grid_constant__ AttnParams p, const AttnPlan pl) {
  using C = TcCfg<DP, MQ, E4M3>;
  constexpr int TOK = C::TOK, RB = C::RB, ST = C::ST, TS = C::TS, GROUPS = C::GROUPS, SW = C::SW;
  extern __shared__ __align__(1024) uint8_t at_smem[];  // q, then the ring
  __shared__ RangeStart<C::THREADS> start;
  __shared__ __align__(8) uint64_t full[ST], empty[ST], qfull[C::QB], qempty[C::QB];
  __shared__ __align__(8) uint64_t s_full[TC_NS], p_full[TC_NS];
  __shared__ __align__(8) uint64_t pv_done[TC_NS], clean[GROUPS], stored[2], drained[3];
  __shared__ uint64_t stage_valid[ST];  // tokens of the stage that exist
  __shared__ __align__(8) uint64_t raw_full[C::RST], raw_empty[C::RST];  // E4M3
  __shared__ uint64_t raw_valid[C::RST];
  __shared__ float row_scale[2][MQ];  // E4M3: what q's rows were divided by
  __shared__ PendingJoin pending[2];
  __shared__ uint32_t tmem_slot;
  __shared__ int abort_flag, n_pending, is_last, keep_first[TC_NS];
  __shared__ float join_ml[GROUPS * 128][2];
  __shared__ uint8_t row_tok[MQ];  // a row's token, from the item's first
  static_assert(
      fits_shared<sizeof(start) + sizeof(full) + sizeof(empty) + sizeof(qfull) + sizeof(qempty) +
                      sizeof(s_full) + sizeof(p_full) + sizeof(pv_done) + sizeof(clean) +
                      sizeof(stored) + sizeof(drained) + sizeof(stage_valid) +
                      (E4M3 ? sizeof(raw_full) + sizeof(raw_empty) + sizeof(raw_valid) +
                                  sizeof(row_scale)
                            : 0) +
                      sizeof(pending) + 4 * sizeof(int) + sizeof(keep_first) + sizeof(join_ml) +
                      sizeof(row_tok),
                  C::SMEM>,
      "all of the above and the dynamic shared memory");
  uint8_t *ring = at_smem + C::QB * C::QBYTES;
  // what the copying warps fill: the ring itself, or (E4M3) the one that is widened into it
  uint8_t *copied = E4M3 ? ring + ST * C::STAGE : ring;
  uint64_t *const copy_full = E4M3 ? raw_full : full, *const copy_empty = E4M3 ? raw_empty : empty;
  uint64_t *const copy_valid = E4M3 ? raw_valid : stage_valid;

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (tid == 0) {
    abort_flag = 0;
    n_pending = 0;
    for (int i = 0; i < ST; ++i) {
      mbar_init(&full[i], E4M3 ? 4 : 1);
      mbar_init(&empty[i], 1);
    }
    for (int i = 0; E4M3 && i < C::RST; ++i) {
      mbar_init(&raw_full[i], 1);
      mbar_init(&raw_empty[i], 4);
    }
    for (int i = 0; i < C::QB; ++i) {
      mbar_init(&qfull[i], TC_QTHREADS);
      mbar_init(&qempty[i], C::KW);
    }
    for (int i = 0; i < TC_NS; ++i) {
      mbar_init(&s_full[i], 1);
      mbar_init(&p_full[i], 128);
      mbar_init(&pv_done[i], 1);
      keep_first[i] = 0;
    }
    for (int i = 0; i < GROUPS; ++i) mbar_init(&clean[i], 128);
    for (int i = 0; i < 3; ++i) mbar_init(&drained[i], 1);
    mbar_init(&stored[0], GROUPS * 128);
    mbar_init(&stored[1], GROUPS * 128);
    fence_mbar_init();
    prefetch_tensormap(&kmap);
    prefetch_tensormap(&vmap);
  }
  griddep_wait();
  const int G = p.Hq / p.Hkv;
  Shares sh;
  Cursor<TOK, MQ, TC_ITEM_COST, TC_LEAST> c;
  if (!begin_range<C::THREADS>(p, G, start, sh, c)) return;
  if (warp == SW + 4) {
    tmem_alloc(&tmem_slot, C::COLS);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  // after the allocation: a dependent grid's CTA cannot hold the columns this one waits for
  griddep_launch_dependents();
  const uint32_t tmem = tmem_slot, o_tmem = tmem, s_tmem = tmem + GROUPS * DP;
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
  // Outputs of stage i added. As many barriers in turn as there are S: who waits for stage i
  // knows that i - TC_NS is done (the scores of i were issued after it), and a wait tells
  // only neighbouring phases apart.
  int issued = 0;  // a copying warp's stages: one past its last
  auto wait_pv = [&](int i) { wait(&pv_done[i % TC_NS], i / TC_NS); };

  if (warp >= SW && warp < SW + 3) {
    // ================================================================ K and V boxes
    // The pages of 32 blocks of `box` tokens are looked up in one step, a step ahead, and the
    // boxes leave from one thread with uniform operands. (With half of the tokens of every
    // stage a warp, a look-up and a box a lane each time, the warps took 0.75 us a stage,
    // however few bytes it had.)
    constexpr int CST = C::CST, CRB = C::CRB, ROW = CRB == 64 ? 64 : 128, SLABS = CRB / ROW;
    const int lg = 31 - __clz(p.box), nb = TOK >> lg, per = 32 / nb;  // blocks, stages a step
    int k = 0;
    bool go = warp - SW < C::CW;  // until a time-out: no box into a stage that may be in use
    while (go && c.next(p, G)) {
      const int32_t *table = p.block_table + static_cast<long long>(c.s) * p.max_pages;
      // lane: block lane % nb of the (lane / nb)-th of this warp's stages from `from` on: its
      // page and the block's place in it
      auto look_up = [&](int from, int &page, int &off) {
        const int t = from + lane / nb * C::CW;
        page = -1;
        off = 0;
        if (t < c.t1) {
          const int j = c.x.begin + t * TOK + ((lane & (nb - 1)) << lg);
          if (j < c.x.len) {
            const int i = j / p.c.page_size;
            off = j - i * p.c.page_size;
            page = table[i];
          }
        }
      };
      int t = c.t0 + (warp - SW + C::CW - k % C::CW) % C::CW;
      int page, off, next_page, next_off;
      look_up(t, page, off);
      look_up(t + C::CW * per, next_page, next_off);
      while (go && t < c.t1) {
        const uint32_t exist = __ballot_sync(0xffffffffu, page >= 0 && page < p.c.num_pages);
        for (int i = 0; i < per && t < c.t1; ++i, t += C::CW) {
          const int at = k + t - c.t0, st = at % CST;
          const uint32_t all = (1u << nb) - 1, blocks = exist >> (i * nb) & all;
          const int left = c.x.len - c.x.begin - t * TOK;
          uint64_t bits = ~0ull;  // the tokens that exist
          if (blocks != all || left < TOK) {
            bits = 0;
#pragma unroll 1
            for (int b = 0; b < nb; ++b)
              if (blocks >> b & 1) bits |= (~0ull >> (64 - p.box)) << (b << lg);
            if (left < TOK) bits &= (1ull << left) - 1;
          }
          if (at >= CST) {
            go = __all_sync(0xffffffffu, wait(&copy_empty[st], at / CST - 1));
            if (!go) break;
          }
          issued = at + 1;
          if (elect_one()) {
            copy_valid[st] = bits;
            mbar_arrive_expect_tx(&copy_full[st], __popc(blocks) * p.box * 2 * CRB);
          }
          const uint32_t dst = smem_u32(copied + st * C::CSTAGE);
#pragma unroll 1
          for (int b = 0; b < nb; ++b) {
            const int pg = __shfl_sync(0xffffffffu, page, i * nb + b);
            const int o = __shfl_sync(0xffffffffu, off, i * nb + b);
            if ((blocks >> b & 1) && elect_one()) {
#pragma unroll
              for (int slab = 0; slab < SLABS; ++slab) {
                const uint32_t to = dst + slab * (TOK * 128) + (b << lg) * ROW;
                tma_load_4d(to, &kmap, &copy_full[st], slab * (128 / C::ES), o, c.hk, pg);
                tma_load_4d(to + TOK * CRB, &vmap, &copy_full[st], slab * (128 / C::ES), o, c.hk,
                            pg);
              }
            }
            __syncwarp();
          }
        }
        page = next_page;
        off = next_off;
        look_up(t + C::CW * per, next_page, next_off);
      }
      k += c.t1 - c.t0;
    }
  } else if (E4M3 && warp >= SW + 8) {
    // ================================================================ e4m3 -> f16
    constexpr int CRB = C::CRB, CH = DP / 16, N = 2 * TOK * CH;  // 16-byte chunks
    const int at = tid - (SW + 8) * 32;
    int k = 0;
    while (c.next(p, G)) {
      for (int t = c.t0; t < c.t1; ++t, ++k) {
        const int rs = k % C::RST, st = k % ST;
        wait(&raw_full[rs], k / C::RST);
        if (k >= ST) wait(&empty[st], k / ST - 1);
        const uint8_t *from = copied + rs * C::CSTAGE;
        uint8_t *to = ring + st * C::STAGE;
#pragma unroll 4
        for (int i = at; i < N; i += 128) {
          const int val = i / (N / 2), row = i / CH % TOK, ch = i % CH;
          const uint4 v = *reinterpret_cast<const uint4 *>(from + val * (TOK * CRB) +
                                                           swz<CRB, TOK>(row, ch));
          uint8_t *d = to + val * (TOK * RB);
          *reinterpret_cast<uint4 *>(d + swz<RB, TOK>(row, 2 * ch)) =
              make_uint4(e4m3x2_to_f16x2(v.x), e4m3x2_to_f16x2(v.x >> 16),
                         e4m3x2_to_f16x2(v.y), e4m3x2_to_f16x2(v.y >> 16));
          *reinterpret_cast<uint4 *>(d + swz<RB, TOK>(row, 2 * ch + 1)) =
              make_uint4(e4m3x2_to_f16x2(v.z), e4m3x2_to_f16x2(v.z >> 16),
                         e4m3x2_to_f16x2(v.w), e4m3x2_to_f16x2(v.w >> 16));
        }
        if (at == 0) stage_valid[st] = raw_valid[rs];
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&full[st]);
          mbar_arrive(&raw_empty[rs]);
        }
      }
    }
  } else if (warp >= SW + 6) {
    // ================================================================ rows of q
    // A thread has one 16-byte column of the head and every PER_PASS-th row.
    constexpr int CH = DP / 8, PER_PASS = TC_QTHREADS / CH;
    const int at = tid - (SW + 6) * 32, ch = at % CH;
    int seg = 0, stages = 0;
    decltype(c) last = c;  // the segment before this one
    // Its part, if it is one of several, is stored: the last warp counts it. (Two barriers in
    // turn: the softmax can be one segment ahead of this warp, whose rows of q it needs for a
    // second.) E4M3: both warps wait, as the softmax may then still read row_scale.
    auto count = [&](int done) {
      wait_stages(&stored[done & 1], done >> 1, stages);
      const long long unit = last.item + TC_ITEM_COST;
      const int c0 = sh.worker_of(unit), c1 = sh.worker_of(unit + last.x.kt - 1);
      if (c0 != c1 && lane == 0 && warp == SW + 7)
        count_part(pl, blockIdx.x, c0, c1, min(MQ, last.x.n * G - last.rt * MQ),
                   {last.x.q0, last.rt * MQ, last.hk * G, G,
                    p.c.v_scale ? p.c.v_scale[last.hk] : 1.0f},
                   pending, &n_pending);
    };
    while (c.next(p, G)) {
      const int qb = seg % C::QB;
      stages += c.t1 - c.t0;
      const int n_rows = min(MQ, c.x.n * G - c.rt * MQ);
      uint8_t *qd = at_smem + qb * C::QBYTES;
      const uint16_t *head = p.q + static_cast<long long>(c.hk * G) * p.D + ch * 8;
      constexpr int AHEAD = MQ / PER_PASS < 16 ? MQ / PER_PASS : 16;
      for (int r0 = at / CH; r0 < MQ; r0 += AHEAD * PER_PASS) {
        uint4 v[AHEAD];
#pragma unroll
        for (int e = 0; e < AHEAD; ++e) {
          const int r = r0 + e * PER_PASS;
          v[e] = make_uint4(0, 0, 0, 0);  // past the rows and past D
          if (r < n_rows && ch * 8 < p.D) {
            const int rr = c.rt * MQ + r, tok = rr / G, g = rr - tok * G;
            v[e] = *reinterpret_cast<const uint4 *>(head + (c.x.q0 + tok) * p.q_stride + g * p.D);
          }
        }
        // (the first rows are on their way while the last segment's products read the buffer)
        if (r0 < PER_PASS && seg >= C::QB) wait_stages(&qempty[qb], seg / C::QB - 1, stages);
#pragma unroll
        for (int e = 0; e < AHEAD; ++e) {
          const int r = r0 + e * PER_PASS;
          if (r < MQ) {
            if (E4M3) v[e] = q_to_f16(v[e], CH, ch == 0 ? &row_scale[seg & 1][r] : nullptr);
#pragma unroll
            for (int copy = 0; copy < C::COPIES; ++copy)
              *reinterpret_cast<uint4 *>(qd + swz<DP * 2, 128>(copy * MQ + r, ch)) = v[e];
          }
        }
      }
      fence_proxy_async_smem();
      mbar_arrive(&qfull[qb]);
      if ((E4M3 || warp == SW + 7) && seg > 0) count(seg - 1);
      last = c;
      ++seg;
    }
    if ((E4M3 || warp == SW + 7) && seg > 0) count(seg - 1);
  } else if (warp >= SW && warp < SW + 5) {
    // ================================================================ products
    // S = Q . K^T, every second stage a warp (one warp took 0.45 us a stage of heads of 64)
    const int qk = warp - SW - 3;
    const uint32_t id_s = tc_idesc<E4M3>(TOK), q_u = smem_u32(at_smem), ring_u = smem_u32(ring);
    int k = 0, seg = 0;
    while (qk < C::KW && c.next(p, G)) {
      const int qb = seg % C::QB;
      wait(&qfull[qb], seg / C::QB);
      // of this warp, or before t0
      const int last = c.t1 - 1 - ((k + c.t1 - c.t0 - 1 - qk) & (C::KW - 1));
      for (int t = c.t0; t < c.t1; ++t, ++k) {
        if ((k & (C::KW - 1)) != qk) continue;
        const int st = k % ST;
        wait(&full[st], k / ST);
        if (k >= TC_NS) wait_pv(k - TC_NS);  // its S held that product's weights
        tc_fence_after();
        if (elect_one()) {
          // 16 elements a product: 32 bytes of a 128-byte slab; whole slabs, then the rest
          const uint32_t d_tmem = s_tmem + (k % TC_NS) * 64;
          uint64_t a = sw128_desc(q_u + qb * C::QBYTES);
          uint64_t b = sw128_desc(ring_u + st * C::STAGE);
          uint32_t acc = 0;
#pragma unroll 1
          for (int slab = p.D >> 6; slab > 0; --slab) {
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
              tc_mma(d_tmem, a + 2 * kk, b + 2 * kk, id_s, kk > 0 ? 1u : acc);
            acc = 1;
            a += 128 * 128 / 16;
            b += TOK * 128 / 16;
          }
#pragma unroll 1
          for (int kk = (p.D & 63) >> 4; kk > 0; --kk) {
            tc_mma(d_tmem, a, b, id_s, acc);
            acc = 1;
            a += 2;
            b += 2;
          }
          tc_commit(&s_full[k % TC_NS]);
          if (t == last) tc_commit(&qempty[qb]);
        }
        __syncwarp();
      }
      if (last < c.t0 && lane == 0) mbar_arrive(&qempty[qb]);
      ++seg;
    }
  } else if (warp == SW + 5) {
    // O += P . V
    const uint32_t id_o = tc_idesc<E4M3>(p.D) | (1u << 16), ring_u = smem_u32(ring);
    int k = 0;
    while (c.next(p, G)) {
      for (int t = c.t0; t < c.t1; ++t, ++k) {
        const int st = k % ST, sb = k % TC_NS;
        wait(&p_full[sb], k / TC_NS);
        tc_fence_after();
        const bool keep = *static_cast<volatile int *>(&keep_first[sb]) != 0;
        const uint32_t acc = t >= c.t0 + GROUPS || keep ? 1u : 0u;
        const uint32_t to = o_tmem + k % GROUPS * DP;
        const uint64_t v = sw128_mn_desc(ring_u + st * C::STAGE + TOK * RB, TOK * 128);
        if (elect_one()) {
#pragma unroll
          for (int kk = 0; kk < TOK / 16; ++kk)  // 16 tokens: 2048 bytes of V, 8 columns of P
            tc_mma_ts(to, s_tmem + sb * 64 + kk * 8, v + (2048 >> 4) * kk, id_o,
                      kk > 0 ? 1u : acc);
          // a segment's (each group's) last stage is released after its join
          if (t + GROUPS < c.t1) tc_commit(&empty[st]);
          tc_commit(&pv_done[sb]);
        }
        __syncwarp();
      }
    }
    if (k > 0) wait_pv(k - 1);  // nothing in flight when the columns are released
  } else {
    // ================================================================ softmax, a thread a lane
    const int grp = warp >> 2, gt = tid & 127;
    const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t my_o = o_tmem + grp * DP + lanes;
    const int copy = gt / MQ, r = gt % MQ, first_tok = copy * TS;
    constexpr uint32_t INF2 = E4M3 ? 0x7c007c00u : 0x7f807f80u;  // exponents of two values
    int k = 0, cleans = 0, segs = 0;
    if (pl.hold) wait(&stored[0], 0);  // self-test: nobody but these warps, later, arrives here
    while (c.next(p, G)) {
      const SeqInfo &x = c.x;
      const int n_rows = min(MQ, x.n * G - c.rt * MQ), row0 = c.rt * MQ;
      // what this row sees, and what every row of the item sees
      const int pos0 = x.len - x.n;
      const int hi = pos0 + (row0 + min(r, n_rows - 1)) / G;
      const int lo = p.window > 0 && hi >= p.window ? hi - p.window + 1 : 0;
      const int hi_all = pos0 + row0 / G, hi_top = pos0 + (row0 + n_rows - 1) / G;
      const int lo_all = p.window > 0 && hi_top >= p.window ? hi_top - p.window + 1 : 0;
      float zf = p.scale * LOG2E * (p.c.k_scale ? p.c.k_scale[c.hk] : 1.0f);
      float m = -INFINITY, l = 0.0f;  // m: the maximum that weights refer to
      for (int t = c.t0; t < c.t1; ++t, ++k) {
        if (k % GROUPS != grp) continue;
        const int st = k % ST, sb = k % TC_NS;
        const uint32_t s_at = s_tmem + sb * 64 + lanes;
        wait(&s_full[sb], k / TC_NS);
        tc_fence_after();
        const bool begins = t < c.t0 + GROUPS;
        if (E4M3 && begins) zf *= row_scale[segs & 1][r];
        float z[TS];
        if (TS == 16) tmem_ld16(s_at + first_tok, z);
        else
#pragma unroll
          for (int i = 0; i < TS; i += 32) tmem_ld32(s_at + first_tok + i, z + i);
        wait(&full[st], k / ST);  // (long since) the copying warps' bits and the values
        const uint64_t valid = stage_valid[st];
        const int j0 = x.begin + t * TOK;
        const bool plain = valid == ~0ull && j0 >= lo_all && j0 + TOK - 1 <= hi_all;
        tmem_wait_ld();
        if (!plain) {
          const uint64_t mine = valid >> first_tok;
          const int from = lo - j0 - first_tok, to = hi - j0 - first_tok;
#pragma unroll
          for (int i = 0; i < TS; ++i) {
            z[i] *= zf;
            if (i < from || i > to || !(mine >> i & 1)) z[i] = -INFINITY;
          }
        }
        // the largest score; where every token counts, of the unscaled ones
        float part[4] = {z[0], z[1], z[2], z[3]};  // short chains
        const bool least = plain && zf < 0.0f;
        if (least) {
#pragma unroll
          for (int i = 4; i < TS; ++i) part[i & 3] = fminf(part[i & 3], z[i]);
        } else {
#pragma unroll
          for (int i = 4; i < TS; ++i) part[i & 3] = fmaxf(part[i & 3], z[i]);
        }
        float mx = least ? fminf(fminf(part[0], part[1]), fminf(part[2], part[3]))
                         : fmaxf(fmaxf(part[0], part[1]), fmaxf(part[2], part[3]));
        if (plain) mx *= zf;
        if (E4M3) mx -= F16_POWERS;
        if (begins) {
          m = mx;
        } else if (__any_sync(0xffffffffu, mx - m >= TC_LAZY)) {
          // move every row's maximum: the outputs so far are rescaled in tensor memory,
          // after the last product that adds to them
          const float m_new = fmaxf(m, mx);
          const float fade = ex2(m - (m_new == -INFINITY ? 0.0f : m_new));
          m = m_new;
          l *= fade;
          wait_pv(k - GROUPS);
          tc_fence_after();
          for (int d = 0; d < p.D; d += 16) {
            float o[16];
            uint32_t u[16];
            tmem_ld16(my_o + d, o);
            tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 16; ++e) u[e] = __float_as_uint(o[e] * fade);
            tmem_st16(my_o + d, u);
          }
          tmem_wait_st();
        }
        const float base = m == -INFINITY ? 0.0f : m, by = plain ? zf : 1.0f;
        uint32_t w[TS / 2];
        float2 sum[2] = {make_float2(0.0f, 0.0f), make_float2(0.0f, 0.0f)};
#pragma unroll
        for (int i = 0; i < TS / 2; ++i) {
          float2 y = fma2(make_float2(z[2 * i], z[2 * i + 1]), make_float2(by, by),
                          make_float2(-base, -base));
          y.x = ex2(y.x);
          y.y = ex2(y.y);
          sum[i & 1] = add2(sum[i & 1], y);
          w[i] = pack2<E4M3>(y.x, y.y);
        }
        sum[0] = add2(sum[0], sum[1]);
        l += sum[0].x + sum[0].y;
        // the weights of this copy's tokens, zeros for the others'
#pragma unroll
        for (int b = 0; b < 32; b += 16) {
          uint32_t u[16];
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            u[e] = 0u;
#pragma unroll
            for (int g = 0; g < C::COPIES; ++g) {
              const int i = b + e - g * (TS / 2);
              if (i >= 0 && i < TS / 2 && (C::COPIES == 1 || copy == g)) u[e] = w[i];
            }
          }
          tmem_st16(s_at + b, u);
        }
        tmem_wait_st();
        int keep = 0;
        if (!plain) {
          // Weights of zero must not meet what is not finite. Tokens that do not exist (boxes
          // bring what lies past the end) get values of zero. Where a value of a token that
          // some row does not see is not finite, the stage's values go through the product
          // without what is not finite in them, and that is added where it is seen.
          uint8_t *v = ring + st * C::STAGE + TOK * RB;
          bool bad = false;
          constexpr int CH = RB / 16;
          const int head = min(max(lo_all - j0, 0), TOK), tail = min(max(hi_all + 1 - j0, 0), TOK);
          auto look = [&](int row0, int row1) {
            for (int i = row0 * CH + lane; i < row1 * CH; i += 32) {
              const int row = i / CH;
              uint4 *at = reinterpret_cast<uint4 *>(v + swz<RB, TOK>(row, i % CH));
              if (!(valid >> row & 1)) {
                *at = make_uint4(0, 0, 0, 0);
              } else if (row < head || row >= tail) {
                const uint4 y = *at;
                bad |= (__vcmpeq2(y.x & INF2, INF2) |
                        __vcmpeq2(y.y & INF2, INF2) |
                        __vcmpeq2(y.z & INF2, INF2) |
                        __vcmpeq2(y.w & INF2, INF2)) != 0;
              }
            }
          };
          // rows that all see and that exist need no look: only a missing page makes holes there
          const bool holes = tail > head &&
                             (~(valid >> head) & (~0ull >> (64 - (tail - head)))) != 0;
          if (holes) {
            look(0, TOK);
          } else {
            look(0, min(head, tail));
            look(tail, TOK);
          }
          __syncwarp();
          if (__any_sync(0xffffffffu, bad)) {
            if (!begins) wait_pv(k - GROUPS);
            tc_fence_after();
            for (int d = 0; d < p.D; d += 16) {
              float o[16];
              uint32_t u[16];
              tmem_ld16(my_o + d, o);
              tmem_wait_ld();
#pragma unroll
              for (int e = 0; e < 16; ++e) o[e] = begins ? 0.0f : o[e];
              for (int i = 0; i < TOK; ++i) {
                const uint32_t pw2 = tmem_ld1(s_at + i / 2);
                tmem_wait_ld();
                float pr = to_f32<E4M3>(i & 1 ? pw2 >> 16 : pw2 & 0xffffu);
                // seen, in this copy? (a weight of zero does not tell: one far below the row's
                // maximum is zero too, and is taken as the smallest number)
                const int at = i - first_tok;
                if (at >= 0 && at < TS && at >= lo - j0 - first_tok && at <= hi - j0 - first_tok &&
                    (valid >> i & 1)) {
                  if (pr == 0.0f) pr = FLT_MIN;
#pragma unroll
                  for (int e = 0; e < 16; ++e) {
                    const uint16_t y = *reinterpret_cast<const uint16_t *>(
                        v + swz<RB, TOK>(i, (d + e) >> 3) + ((d + e) & 7) * 2);
                    if ((y & INF2) == (INF2 & 0xffffu)) o[e] += pr * to_f32<E4M3>(y);
                  }
                }
                __syncwarp();  // what reads and writes tensor memory next wants the warp in one place
              }
#pragma unroll
              for (int e = 0; e < 16; ++e) u[e] = __float_as_uint(o[e]);
              tmem_st16(my_o + d, u);
            }
            tmem_wait_st();
            // every row has read the values (not a CTA barrier: this depends on data, and
            // after a time-out the warps may see different bytes)
            mbar_arrive(&clean[grp]);
            wait(&clean[grp], cleans++);
            for (int i = gt; i < TOK * (RB / 16); i += 128) {
              uint4 *at = reinterpret_cast<uint4 *>(
                  v + swz<RB, TOK>(i / (RB / 16), i % (RB / 16)));
              uint4 y = *at;
              y.x &= ~__vcmpeq2(y.x & INF2, INF2);
              y.y &= ~__vcmpeq2(y.y & INF2, INF2);
              y.z &= ~__vcmpeq2(y.z & INF2, INF2);
              y.w &= ~__vcmpeq2(y.w & INF2, INF2);
              *at = y;
            }
            keep = 1;  // the segment's first outputs add to these
          }
          fence_proxy_async_smem();  // before the product (and later boxes) touch the values
        }
        if (gt == 0) keep_first[sb] = keep;
        tc_fence_before();
        mbar_arrive(&p_full[sb]);
      }

      // ---- the segment's outputs: the copies joined in the memory of each group's last stage,
      // half of the columns at a time (a row of DP / 2 floats a lane, 16-byte chunks permuted
      // by the row). In a segment of one stage one group has none.
      auto last_of = [&](int g) { return k - 1 - ((k - 1 - g) & (GROUPS - 1)); };  // or -1
      const int my_last = last_of(grp), me = blockIdx.x;
      const bool has = my_last >= k - (c.t1 - c.t0);
      const long long unit = c.item + TC_ITEM_COST;
      const int c0 = sh.worker_of(unit), c1 = sh.worker_of(unit + x.kt - 1);
      const ItemOut dst = {x.q0, row0, c.hk * G, G, p.c.v_scale ? p.c.v_scale[c.hk] : 1.0f};
      float *slot = pl.partials + static_cast<size_t>(part_slot(c0, me - c0)) * C::SLOT;
      float *join[GROUPS];
#pragma unroll
      for (int g = 0; g < GROUPS; ++g)
        join[g] = reinterpret_cast<float *>(ring + max(last_of(g), 0) % ST * C::STAGE);
      constexpr int HALF = DP / 2;
      auto join_at = [&](int g, int row, int chunk) {
        return reinterpret_cast<float4 *>(join[g] + row * HALF + ((chunk ^ (row & 7)) << 2));
      };
      join_ml[tid][0] = m;
      join_ml[tid][1] = l;
      named_bar_sync(1, GROUPS * 128);
      // a row's thread: the copies' factors (with the division, where the item ends here), and
      // the row's lse or (m, l). What is not to be read at all (a group without a stage: its
      // memory holds anything; a finished row that saw nothing: zeros) has the factor -0; a
      // factor that has become zero is +0, so that what is not finite in that part is not lost.
      float factor[C::PARTS];
      if (tid < n_rows) {
        float mr = -INFINITY, lr = 0.0f;
#pragma unroll
        for (int g = 0; g < C::PARTS; ++g) mr = fmaxf(mr, join_ml[g * MQ + tid][0]);
        const float b = mr == -INFINITY ? 0.0f : mr;
#pragma unroll
        for (int g = 0; g < C::PARTS; ++g) {
          factor[g] = ex2(join_ml[g * MQ + tid][0] - b);
          lr += factor[g] * join_ml[g * MQ + tid][1];
        }
        const int rr = row0 + tid, tok = rr / G;
        row_tok[tid] = static_cast<uint8_t>(tok - row0 / G);
        if (c0 == c1) {
          dst.put_lse(p, tid, mr, lr);
          const float inv = lr == 0.0f ? 0.0f : dst.v_scale / lr;
#pragma unroll
          for (int g = 0; g < C::PARTS; ++g) factor[g] *= inv;
        } else {
          *reinterpret_cast<float2 *>(slot + MQ * DP + 2 * tid) = make_float2(mr, lr);
        }
#pragma unroll
        for (int g = 0; g < C::PARTS; ++g) {
          const bool none = last_of(g / C::COPIES) < k - (c.t1 - c.t0) || (c0 == c1 && lr == 0.0f);
          join_ml[g * MQ + tid][0] = none ? -0.0f : (factor[g] == 0.0f ? 0.0f : factor[g]);
        }
      }
      if (has) wait_pv(my_last);
      tc_fence_after();
#pragma unroll 1
      for (int half = 0; half < 2; ++half) {
        const int d0 = half * HALF, width = min(HALF, p.D - d0);  // a multiple of 16, or none
        if (width <= 0) break;
        if (has) {  // past D: columns that hold nothing, which nobody reads
          constexpr int CHUNK = HALF < 64 ? HALF : 64;
#pragma unroll 1
          for (int d = 0; d < HALF; d += CHUNK) {
            float o[CHUNK];
#pragma unroll
            for (int e = 0; e < CHUNK; e += 32) tmem_ld32(my_o + d0 + d + e, o + e);
            tmem_wait_ld();
            if (r < n_rows) {
#pragma unroll
              for (int e = 0; e < CHUNK; e += 4)
                *join_at(grp, gt, (d + e) >> 2) = make_float4(o[e], o[e + 1], o[e + 2], o[e + 3]);
            }
            __syncwarp();  // (as above)
          }
        }
        tc_fence_before();  // the next segment's products overwrite the columns
        named_bar_sync(1, GROUPS * 128);
        const int cols = width / 4;
        auto store = [&](int row, int d) {
          const int col = d0 + 4 * d;
          float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
          for (int g = 0; g < C::PARTS; ++g) {
            const float f = join_ml[g * MQ + row][0];
            const float4 y = *join_at(g / C::COPIES, g % C::COPIES * MQ + row, d);
            if (__float_as_uint(f) != 0x80000000u) {
              v.x += f * y.x;
              v.y += f * y.y;
              v.z += f * y.z;
              v.w += f * y.w;
            }
          }
          if (c0 == c1) {
            uint2 u;
            u.x = pack2<false>(v.x, v.y);
            u.y = pack2<false>(v.z, v.w);
            const int tok = row0 / G + row_tok[row];
            *reinterpret_cast<uint2 *>(p.out + (x.q0 + tok) * p.out_stride +
                                       static_cast<long long>(c.hk * G + row0 + row - tok * G) *
                                           p.D + col) = u;
          } else {
            *reinterpret_cast<float4 *>(slot + row * DP + col) = v;
          }
        };
        if (width == HALF) {  // no division at run time
#pragma unroll 4
          for (int i = tid; i < n_rows * (HALF / 4); i += GROUPS * 128)
            store(i / (HALF / 4), i % (HALF / 4));
        } else {
          for (int i = tid; i < n_rows * cols; i += GROUPS * 128) store(i / cols, i % cols);
        }
        fence_proxy_async_smem();  // before later boxes overwrite the join's stores
        named_bar_sync(1, GROUPS * 128);
      }
      if (gt == 0 && has) mbar_arrive(&empty[my_last % ST]);
      // a split item's part is stored: the last warp counts it, off the softmax's way
      mbar_arrive(&stored[segs++ & 1]);
    }
  }
  static_assert(ST * C::STAGE >= 2 * AT_GROUP * MQ * 8, "ml of a join");
  run_joins<MQ, DP, C::THREADS>(p, pl, reinterpret_cast<float2 *>(ring), pending, &n_pending,
                                &is_last);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  // Every wait of the CTA is over. If one ran out, products and boxes may still be on their way:
  // products end before tensor memory is released, boxes land before the CTA ends.
  if (*static_cast<volatile int *>(&abort_flag)) {
    if (warp >= SW + 3 && warp < SW + 6) {
      uint64_t *bar = &drained[warp - SW - 3];
      if (elect_one()) tc_commit(bar);
      __syncwarp();
      mbar_wait_drain(bar, 0, 10000000ull);
    }
    for (int i = issued - 1; i >= 0 && i >= issued - C::CST; i -= C::CW)
      mbar_wait_drain(&copy_full[i % C::CST], (i / C::CST) & 1, 10000000ull);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
  }
  if (warp == SW + 4) tmem_dealloc(tmem, C::COLS);
}

template <bool E4M3, int DP, int MQ>
cudaError_t launch_tc_shape(const AttnParams &p, void *ws, const AttnLaunch &a, cudaStream_t s) {
  using C = TcCfg<DP, MQ, E4M3>;
  auto kernel = attn_tc_kernel<DP, MQ, E4M3>;
  const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             static_cast<int>(C::SMEM));
  if (e != cudaSuccess) return e;
  const int grid = a.num_sms;
  return launch_pdl(kernel, dim3(grid), dim3(C::THREADS), C::SMEM, s, a.kmap, a.vmap, p,
                    make_plan(ws, a));
}

template <bool E4M3, int DP>
cudaError_t launch_tc_dim(const AttnParams &p, int rows, void *ws, const AttnLaunch &a,
                          cudaStream_t s) {
  if constexpr (tc_min_rows(E4M3, DP) < 32)
    if (rows == 32) return launch_tc_shape<E4M3, DP, 32>(p, ws, a, s);
  if constexpr (tc_min_rows(E4M3, DP) < 64)
    if (rows == 64) return launch_tc_shape<E4M3, DP, 64>(p, ws, a, s);
  return launch_tc_shape<E4M3, DP, 128>(p, ws, a, s);
}

// rows: tc_rows
template <bool E4M3>
cudaError_t launch_tc(const AttnParams &p, int padded, int rows, void *ws, const AttnLaunch &a,
                      cudaStream_t s) {
  switch (padded) {
    case 64:
      return launch_tc_dim<E4M3, 64>(p, rows, ws, a, s);
    case 128:
      return launch_tc_dim<E4M3, 128>(p, rows, ws, a, s);
    default:
      return launch_tc_dim<E4M3, 256>(p, rows, ws, a, s);
  }
}

}  // namespace
}  // namespace ssd

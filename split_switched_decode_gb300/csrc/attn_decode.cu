// attn_decode.cu -- attention of new tokens over a paged key-value cache.
//
// For a kv head and the rows r = (new token i, head g of the group) that read it,
//
//     out_r = sum_j p_rj v_j / sum_j p_rj,   p_rj = 2^(z_rj - m_r),   z = scale log2(e) q.k
//
// in one pass over the keys with a running maximum m and sum l. The keys and values are
// read once from HBM and carry 2 G multiply-adds a byte (G rows), so the copy rate bounds
// it; the work is cut so that every SM streams the same number of tokens:
//
//   - An item is one (sequence, kv head, tile of 16 rows). Its keys are cut into tiles of
//     TK tokens. All tiles of all items, in order, are divided evenly among the CTAs; a CTA
//     works through its range segment by segment (a segment is its part of one item).
//   - Inside a segment the CTA's warps take tiles in turn, each with its own ring of
//     shared-memory stages filled by 16-byte asynchronous copies (the warp's lanes look up
//     the pages of the tile's tokens), its own m and l and its own output accumulators in
//     registers: no barrier between warps until the segment ends.
//   - Both products run on mma.sync m16n8k16 with the rows as M: at 16 rows a tile of
//     tokens needs a fifth of the legacy tensor rate at the full copy rate, scores and
//     weights stay in registers, and the weights' accumulator layout is the next product's
//     operand layout.
//   - At the end of a segment the warps' (m, l, out) are joined through shared memory. An
//     item that lies in one CTA is finished there; otherwise each CTA stores its fp32
//     partial in the workspace, and the last to arrive at the item's counter adds them in
//     CTA order: the result depends on the lengths only.
//
// e4m3 caches are widened to f16 in registers (every e4m3 value is an f16 value); q is
// scaled by a power of two per row so that its largest element is in [1, 2) and converted
// to f16: exact but for elements 2^-14 below the row's largest. The key scale joins the
// score's factor, the value scale the last division.
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "attn.h"
#include "common.cuh"

namespace ssd {
namespace {

constexpr int AT_WARPS = 4;
constexpr int AT_THREADS = 32 * AT_WARPS;
constexpr int AT_M = 16;      // rows of an item
constexpr int AT_STAGES = 2;  // ring stages per warp
constexpr float LOG2E = 1.4426950408889634f, LN2 = 0.6931471805599453f;

template <bool E4M3, int DP>
struct AttnCfg {
  static constexpr int ES = E4M3 ? 1 : 2;              // bytes of a cache element
  static constexpr int RB = DP * ES;                   // bytes of a token's row in a stage
  static constexpr int TK = RB >= 256 ? 16 : 32;       // tokens of a tile
  static constexpr int CPR = RB / 16;                  // 16-byte chunks of a row
  static constexpr int STAGE = 2 * TK * RB;            // K then V
  static constexpr int OLD = DP + 8;                   // floats of a row of the join buffer
  static constexpr int RING = AT_WARPS * AT_STAGES * STAGE;
  static constexpr int QB = AT_M * DP * 2;
  static constexpr int JOIN = AT_WARPS * AT_M * OLD * 4;
  static constexpr size_t SMEM = RING + QB + JOIN;
  static constexpr bool QREG = DP <= 128;              // q fragments kept in registers
  // one partial result: AT_M rows of DP outputs, then m and l of the rows
  static constexpr int SLOT = AT_M * DP + 2 * AT_M;
};

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
__device__ __forceinline__ void cp_async_commit() {
  asm volatile("cp.async.commit_group;" ::: "memory");
}
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
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
// Shared-memory byte offset of 16-byte chunk `ch` of row `row` (rows of RB bytes): eight
// consecutive rows' equal chunks fall into different 16-byte bank groups.
template <int RB>
__device__ __forceinline__ uint32_t swz(int row, int ch) {
  return row * RB + ((ch ^ (RB >= 128 ? row & 7 : (row >> 1) & 3)) << 4);
}

// One sequence's rows and keys.
struct SeqInfo {
  int q0, n;       // first row, rows
  int len, begin;  // keys [begin, len) that some row can see
  int kt;          // tiles of keys (at least 1: an empty row still has to be written)
  int rt;          // row tiles
  __device__ __forceinline__ long long tiles(int Hkv) const {
    return static_cast<long long>(Hkv) * rt * kt;
  }
};

template <int TK>
__device__ __forceinline__ SeqInfo seq_info(const AttnParams &p, int G, int s) {
  SeqInfo x;
  x.q0 = s;
  x.n = 1;
  if (p.q_start) {
    x.q0 = min(max(p.q_start[s], 0), p.T);
    x.n = max(0, min(max(p.q_start[s + 1], 0), p.T) - x.q0);
  }
  // what the table holds, and no token number of a tile's end passes 2^31
  const long long cap =
      min(static_cast<long long>(p.max_pages) * p.c.page_size, 0x7fffff00ll);
  x.len = static_cast<int>(min(static_cast<long long>(max(p.seq_len[s], 0)), cap));
  const int pos = x.len - x.n;  // the first row's
  x.begin = p.window > 0 && pos >= p.window ? pos - p.window + 1 : 0;
  x.kt = x.len > x.begin ? (x.len - x.begin - 1) / TK + 1 : 1;
  x.rt = (x.n * G + AT_M - 1) / AT_M;
  return x;
}

struct AttnPlan {
  int grid;       // CTAs, the most workers
  int min_tiles;  // tiles a worker takes at least
  float *partials;
  int *counters;
};

template <bool E4M3, int DP>
__global__ void __launch_bounds__(AT_THREADS) attn_decode_kernel(const AttnParams p,
                                                                 const AttnPlan pl) {
  using C = AttnCfg<E4M3, DP>;
  constexpr int TK = C::TK, RB = C::RB, NT = TK / 8;
  extern __shared__ __align__(128) uint8_t at_smem[];
  __shared__ long long warp_sum[AT_WARPS];
  __shared__ int start_seq;
  __shared__ long long start_off;
  __shared__ float q_exp[AT_M];                  // e4m3: the power of two taken out of q
  __shared__ float join_ml[AT_WARPS][AT_M][2];   // m, l of each warp
  __shared__ int is_last;
  __shared__ uint32_t stage_valid[AT_WARPS][AT_STAGES];
  uint8_t *q_smem = at_smem + C::RING;
  float *join = reinterpret_cast<float *>(at_smem + C::RING + C::QB);

  griddep_wait();
  griddep_launch_dependents();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int G = p.Hq / p.Hkv;

  // ---- this CTA's share of all tiles: one pass over the sequences
  const int per = (p.S + AT_THREADS - 1) / AT_THREADS;
  const int s_lo = min(tid * per, p.S), s_hi = min(s_lo + per, p.S);
  long long mine = 0;
  for (int s = s_lo; s < s_hi; ++s) mine += seq_info<TK>(p, G, s).tiles(p.Hkv);
  long long incl = mine;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, incl, d);
    if (lane >= d) incl += y;
  }
  if (lane == 31) warp_sum[warp] = incl;
  __syncthreads();
  long long total = 0, before = 0;
#pragma unroll
  for (int w = 0; w < AT_WARPS; ++w) {
    if (w < warp) before += warp_sum[w];
    total += warp_sum[w];
  }
  const long long most = (total + pl.min_tiles - 1) / pl.min_tiles;
  const int workers = static_cast<int>(most < gridDim.x ? most : gridDim.x);
  const int me = blockIdx.x;
  if (me >= workers) return;
  // worker c takes share_n tiles, one more for the first share_r workers
  const long long share_n = total / workers, share_r = total % workers;
  auto worker_of = [&](long long tile) {
    const long long longer = share_r * (share_n + 1);
    return static_cast<int>(tile < longer ? tile / (share_n + 1)
                                          : share_r + (tile - longer) / share_n);
  };
  long long cur = me * share_n + min(static_cast<long long>(me), share_r);
  const long long end = cur + share_n + (me < share_r ? 1 : 0);
  {
    long long at = before + incl - mine;  // tiles before this thread's sequences
    if (at <= cur && cur < at + mine) {
      for (int s = s_lo; s < s_hi; ++s) {
        const long long n = seq_info<TK>(p, G, s).tiles(p.Hkv);
        if (cur < at + n) {
          start_seq = s;
          start_off = cur - at;
          break;
        }
        at += n;
      }
    }
  }
  __syncthreads();
  int s = start_seq;
  SeqInfo x = seq_info<TK>(p, G, s);
  const long long per_head = static_cast<long long>(x.rt) * x.kt;
  int hk = static_cast<int>(start_off / per_head);
  int rt = static_cast<int>((start_off - hk * per_head) / x.kt);
  int t0 = static_cast<int>(start_off - hk * per_head - static_cast<long long>(rt) * x.kt);

  uint8_t *ring = at_smem + warp * AT_STAGES * C::STAGE;
  const uint32_t ring_u = smem_u32(ring), q_u = smem_u32(q_smem);

  while (cur < end) {
    // ---- one segment: tiles [t0, t1) of item (s, hk, rt)
    const long long left = end - cur;
    const int t1 = static_cast<int>(left < x.kt - t0 ? t0 + left : x.kt);
    const int n_rows = min(AT_M, x.n * G - rt * AT_M);
    const int mine_t = t1 - t0 > warp ? (t1 - t0 - warp - 1) / AT_WARPS + 1 : 0;
    const int32_t *table = p.block_table + static_cast<long long>(s) * p.max_pages;
    const char *kbase = static_cast<const char *>(p.c.k);
    const char *vbase = static_cast<const char *>(p.c.v);

    // token of this lane in this warp's i-th tile
    auto token_of = [&](int i) {
      return x.begin + (t0 + warp + i * AT_WARPS) * TK + lane % TK;
    };
    auto page_of = [&](int i) {
      const int j = token_of(i);
      return i < mine_t && j < x.len ? table[j / p.c.page_size] : -1;
    };
    int page = page_of(0);
    auto issue = [&](int i) {  // fill stage i % AT_STAGES with this warp's i-th tile
      if (i < mine_t) {
        const int st = i % AT_STAGES;
        const bool ok = page >= 0 && page < p.c.num_pages;
        long long off = -1;
        if (ok)
          off = (page * p.c.page_stride + hk * p.c.head_stride +
                 token_of(i) % p.c.page_size * p.c.token_stride) * C::ES;
        const uint32_t valid = __ballot_sync(0xffffffffu, ok);
        if (lane == 0) stage_valid[warp][st] = valid;
        const uint32_t dst = ring_u + st * C::STAGE;
#pragma unroll
        for (int c = 0; c < TK * C::CPR / 32; ++c) {
          const int row = (c * 32 + lane) / C::CPR, ch = (c * 32 + lane) % C::CPR;
          const long long o = __shfl_sync(0xffffffffu, off, row);
          const bool in = o >= 0 && ch * 16 < p.D * C::ES;
          const long long at = in ? o + ch * 16 : 0;
          const uint32_t d = dst + swz<RB>(row, ch);
          cp_async16(d, kbase + at, in);
          cp_async16(d + TK * RB, vbase + at, in);
        }
        page = page_of(i + 1);
      }
      cp_async_commit();
    };
#pragma unroll
    for (int i = 0; i < AT_STAGES - 1; ++i) issue(i);

    // ---- the item's rows of q, zeros past them and past D
    __syncthreads();  // the last segment's readers of q and of the join buffer are done
    for (int c = tid; c < AT_M * DP / 8; c += AT_THREADS) {
      const int r = c / (DP / 8), ch = c % (DP / 8);
      uint4 v = make_uint4(0, 0, 0, 0);
      if (r < n_rows && ch * 8 < p.D) {
        const int rr = rt * AT_M + r, i = rr / G, g = rr - i * G;
        v = *reinterpret_cast<const uint4 *>(p.q + (x.q0 + i) * p.q_stride +
                                             static_cast<long long>(hk * G + g) * p.D + ch * 8);
      }
      *reinterpret_cast<uint4 *>(q_smem + swz<DP * 2>(r, ch)) = v;
    }
    __syncthreads();
    if (E4M3) {
      // a warp per 4 rows: largest magnitude, power of two, f16 in the order in which the
      // widened keys come out of their registers (d = 4c + e of each 16 -> 2c + e for
      // e < 2, 8 + 2c + e - 2 above)
      for (int r = warp * 4; r < warp * 4 + 4; ++r) {
        constexpr int PER = DP / 32;
        float v[PER];
        float mx = 0.0f;
#pragma unroll
        for (int k = 0; k < PER; ++k) {
          const int d = lane + 32 * k;
          v[k] = bf16_to_f32(*reinterpret_cast<const uint16_t *>(
              q_smem + swz<DP * 2>(r, d >> 3) + (d & 7) * 2));
          mx = fmaxf(mx, fabsf(v[k]));
        }
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, d));
        int e = static_cast<int>(__float_as_uint(mx) >> 23) - 127;
        if (mx == 0.0f || e > 127) e = 0;  // zeros, infinities: as they are
        if (e < -126) e = -126;
        const float f = e == 127 ? 0.5f * __uint_as_float(1u << 23)
                                 : __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
        __syncwarp();
#pragma unroll
        for (int k = 0; k < PER; ++k) {
          const int d = lane + 32 * k, c4 = (d & 15) >> 2, el = d & 3;
          const int to = (d & ~15) + (el < 2 ? 2 * c4 + el : 8 + 2 * c4 + el - 2);
          *reinterpret_cast<__half *>(q_smem + swz<DP * 2>(r, to >> 3) + (to & 7) * 2) =
              __float2half_rn(v[k] * f);
        }
        if (lane == 0) q_exp[r] = __uint_as_float(static_cast<uint32_t>(e + 127) << 23);
      }
      __syncthreads();
    }
    uint32_t qf[C::QREG ? DP / 16 : 1][4];
    if (C::QREG) {
#pragma unroll
      for (int kk = 0; kk < DP / 16; ++kk)
        ldsm4(qf[kk], q_u + swz<DP * 2>(lane & 15, 2 * kk + (lane >> 4)));
    }

    // ---- this thread's two rows: what they see, and their score factor
    const int ra = lane >> 2;
    float zf[2];
    int lo[2], hi[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int r = min(ra + 8 * h, n_rows - 1);  // rows past the last: as the last
      hi[h] = x.len - x.n + (rt * AT_M + r) / G;
      lo[h] = p.window > 0 && hi[h] >= p.window ? hi[h] - p.window + 1 : 0;
      zf[h] = p.scale * LOG2E * (p.c.k_scale ? p.c.k_scale[hk] : 1.0f);
      if (E4M3) zf[h] *= q_exp[ra + 8 * h];
    }
    // what every row of the item sees: [lo_all, hi_all]
    const int hi_all = x.len - x.n + rt * AT_M / G;
    const int hi_top = x.len - x.n + (rt * AT_M + n_rows - 1) / G;
    const int lo_all = p.window > 0 && hi_top >= p.window ? hi_top - p.window + 1 : 0;

    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.0f, 0.0f};
    float o[DP / 8][4];
#pragma unroll
    for (int i = 0; i < DP / 8; ++i)
#pragma unroll
      for (int k = 0; k < 4; ++k) o[i][k] = 0.0f;

    for (int i = 0; i < mine_t; ++i) {
      issue(i + AT_STAGES - 1);
      cp_async_wait<AT_STAGES - 1>();
      __syncwarp();
      const int st = i % AT_STAGES;
      const uint32_t ks = ring_u + st * C::STAGE, vs = ks + TK * RB;
      const uint32_t valid = stage_valid[warp][st];
      const int j0 = x.begin + (t0 + warp + i * AT_WARPS) * TK;

      // ---- scores [16 rows, TK tokens]
      float z[NT][4];
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int k = 0; k < 4; ++k) z[n][k] = 0.0f;
#pragma unroll
      for (int kk = 0; kk < DP / 16; kk += E4M3 ? 2 : 1) {
        uint32_t qa[4], qb[4];
        if (!C::QREG) {
          ldsm4(qa, q_u + swz<DP * 2>(lane & 15, 2 * kk + (lane >> 4)));
          if (E4M3) ldsm4(qb, q_u + swz<DP * 2>(lane & 15, 2 * kk + 2 + (lane >> 4)));
        }
        const uint32_t(&a0)[4] = C::QREG ? qf[C::QREG ? kk : 0] : qa;
        const uint32_t(&a1)[4] = C::QREG ? qf[C::QREG && E4M3 ? kk + 1 : 0] : qb;
#pragma unroll
        for (int tb = 0; tb < TK / 16; ++tb) {
          uint32_t r[4];
          if (E4M3) {
            ldsm4(r, ks + swz<RB>(tb * 16 + (lane & 15), kk + (lane >> 4)));
#pragma unroll
            for (int q = 0; q < 4; ++q) {  // token half q & 1, k step q >> 1
              const uint32_t b0 = e4m3x2_to_f16x2(r[q]), b1 = e4m3x2_to_f16x2(r[q] >> 16);
              mma16816<true>(z[2 * tb + (q & 1)], q < 2 ? a0 : a1, b0, b1);
            }
          } else {
            ldsm4(r, ks + swz<RB>(tb * 16 + (lane & 7) + ((lane >> 4) << 3),
                                  2 * kk + ((lane >> 3) & 1)));
            mma16816<false>(z[2 * tb], a0, r[0], r[1]);
            mma16816<false>(z[2 * tb + 1], a0, r[2], r[3]);
          }
        }
      }
      // ---- running maximum
      const uint32_t full = TK == 32 ? 0xffffffffu : (1u << (TK & 31)) - 1;
      const bool plain = (valid & full) == full && j0 >= lo_all && j0 + TK - 1 <= hi_all;
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          z[n][k] *= zf[k >> 1];
          if (!plain) {
            const int b = n * 8 + 2 * (lane & 3) + (k & 1), j = j0 + b;
            if (j < lo[k >> 1] || j > hi[k >> 1] || !(valid >> b & 1)) z[n][k] = -INFINITY;
          }
        }
      float base[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float mx = m[h];
#pragma unroll
        for (int n = 0; n < NT; ++n) mx = fmaxf(mx, fmaxf(z[n][2 * h], z[n][2 * h + 1]));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
        base[h] = mx == -INFINITY ? 0.0f : mx;
        const float a = ex2(m[h] - base[h]);
        m[h] = mx;
        l[h] *= a;
        if (__any_sync(0xffffffffu, a != 1.0f)) {
#pragma unroll
          for (int d = 0; d < DP / 8; ++d) {
            o[d][2 * h] *= a;
            o[d][2 * h + 1] *= a;
          }
        }
      }
      // ---- weights: summed in fp32, rounded to 16 bits for the product with V (relative
      // error 2^-9 bf16, 2^-12 f16 for each, far below the output's own rounding once summed)
      uint32_t w[NT][2];
#pragma unroll
      for (int n = 0; n < NT; ++n) {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          z[n][k] = ex2(z[n][k] - base[k >> 1]);
          l[k >> 1] += z[n][k];
        }
        w[n][0] = pack2<E4M3>(z[n][0], z[n][1]);
        w[n][1] = pack2<E4M3>(z[n][2], z[n][3]);
      }
      // ---- a value that is not finite at a token that some rows do not see must not reach
      // them as 0 * inf: such tiles (the last few of an item) take the values' finite part
      // through the product and add the rest where it is seen. A sequence's only row sees
      // every token that is loaded.
      bool unclean = false;
      if (x.n > 1 && !plain) {
        bool bad = false;
        for (int c = lane; c < TK * C::CPR; c += 32) {
          const uint4 v = *reinterpret_cast<const uint4 *>(ring + st * C::STAGE + TK * RB + c * 16);
          const uint32_t e[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            if (E4M3) bad |= __vcmpeq4(e[k] & 0x7f7f7f7fu, 0x7f7f7f7fu) != 0;
            else bad |= __vcmpeq2(e[k] & 0x7f807f80u, 0x7f807f80u) != 0;
          }
        }
        unclean = __any_sync(0xffffffffu, bad);
      }
      // ---- out += weights . values
      auto finite = [&](uint32_t v) {
        return E4M3 ? v & ~__vcmpeq4(v & 0x7f7f7f7fu, 0x7f7f7f7fu)
                    : v & ~__vcmpeq2(v & 0x7f807f80u, 0x7f807f80u);
      };
#pragma unroll
      for (int tb = 0; tb < TK / 16; ++tb) {
        const uint32_t a[4] = {w[2 * tb][0], w[2 * tb][1], w[2 * tb + 1][0], w[2 * tb + 1][1]};
#pragma unroll
        for (int dd = 0; dd < DP / 16; dd += E4M3 ? 2 : 1) {
          uint32_t r[4];
          ldsm4_t(r, vs + swz<RB>(tb * 16 + (lane & 15), (E4M3 ? dd : 2 * dd) + (lane >> 4)));
          if (unclean) {
#pragma unroll
            for (int k = 0; k < 4; ++k) r[k] = finite(r[k]);
          }
          if (E4M3) {
#pragma unroll
            for (int q = 0; q < 2; ++q) {
              const uint32_t x0 = __byte_perm(r[2 * q], 0, 0x3120);
              const uint32_t x1 = __byte_perm(r[2 * q + 1], 0, 0x3120);
              mma16816<true>(o[2 * (dd + q)], a, e4m3x2_to_f16x2(x0), e4m3x2_to_f16x2(x1));
              mma16816<true>(o[2 * (dd + q) + 1], a, e4m3x2_to_f16x2(x0 >> 16),
                             e4m3x2_to_f16x2(x1 >> 16));
            }
          } else {
            mma16816<false>(o[2 * dd], a, r[0], r[1]);
            mma16816<false>(o[2 * dd + 1], a, r[2], r[3]);
          }
        }
      }
      if (unclean) {
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int e = 0; e < 2; ++e)
            for (int c = 0; c < 4; ++c) {
              const int from = (lane & ~3) | c, row = n * 8 + 2 * c + e;
              const float pa = __shfl_sync(0xffffffffu, z[n][e], from);
              const float pb = __shfl_sync(0xffffffffu, z[n][2 + e], from);
              const uint8_t *v = ring + st * C::STAGE + TK * RB;
#pragma unroll
              for (int d = 0; d < DP / 8; ++d)
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                  const int col = E4M3 ? 16 * (d >> 1) + 4 * (lane & 3) + 2 * k + (d & 1)
                                       : 8 * d + 2 * (lane & 3) + k;
                  const int byte = col * C::ES;
                  const uint8_t *at = v + swz<RB>(row, byte >> 4) + (byte & 15);
                  float val;
                  bool bad;
                  if (E4M3) {
                    bad = (*at & 0x7f) == 0x7f;
                    val = NAN;
                  } else {
                    const uint16_t b = *reinterpret_cast<const uint16_t *>(at);
                    bad = (b & 0x7f80) == 0x7f80;
                    val = bf16_to_f32(b);
                  }
                  if (bad && pa != 0.0f) o[d][k] += pa * val;
                  if (bad && pb != 0.0f) o[d][2 + k] += pb * val;
                }
            }
      }
      __syncwarp();  // the stage is free again
    }
    cp_async_wait<0>();

    // ---- join the warps
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      l[h] += __shfl_xor_sync(0xffffffffu, l[h], 1);
      l[h] += __shfl_xor_sync(0xffffffffu, l[h], 2);
      const int r = ra + 8 * h;
      if ((lane & 3) == 0) {
        join_ml[warp][r][0] = m[h];
        join_ml[warp][r][1] = l[h];
      }
      if (r < n_rows) {
        float *row = join + (warp * AT_M + r) * C::OLD;
        if (E4M3) {
#pragma unroll
          for (int d = 0; d < DP / 16; ++d)
            *reinterpret_cast<float4 *>(row + 16 * d + 4 * (lane & 3)) =
                make_float4(o[2 * d][2 * h], o[2 * d + 1][2 * h], o[2 * d][2 * h + 1],
                            o[2 * d + 1][2 * h + 1]);
        } else {
#pragma unroll
          for (int d = 0; d < DP / 8; ++d)
            *reinterpret_cast<float2 *>(row + 8 * d + 2 * (lane & 3)) =
                make_float2(o[d][2 * h], o[d][2 * h + 1]);
        }
      }
    }
    __syncthreads();

    const long long item0 = cur - t0;  // the item's tiles are [item0, item0 + kt)
    const int c0 = worker_of(item0), c1 = worker_of(item0 + x.kt - 1);
    const float v_scale = p.c.v_scale ? p.c.v_scale[hk] : 1.0f;
    auto row_out = [&](int r, int d, float4 v, float mr, float lr) {
      const int rr = rt * AT_M + r, i = rr / G, g = rr - i * G;
      // nothing seen: l = 0
      const float inv = lr == 0.0f ? 0.0f : v_scale / lr;
      if (lr == 0.0f) v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      uint2 u;
      u.x = pack2<false>(v.x * inv, v.y * inv);
      u.y = pack2<false>(v.z * inv, v.w * inv);
      const long long row = x.q0 + i, head = hk * G + g;
      *reinterpret_cast<uint2 *>(p.out + row * p.out_stride + head * p.D + d) = u;
      if (p.lse && d == 0)
        p.lse[row * p.Hq + head] = lr == 0.0f ? -INFINITY : (mr + log2f(lr)) * LN2;
    };
    const int cols = p.D / 4;
    float *slot = pl.partials + static_cast<size_t>(2 * me + (me == c0 ? 1 : 0)) * C::SLOT;
    for (int c = tid; c < n_rows * cols; c += AT_THREADS) {
      const int r = c / cols, d = 4 * (c - r * cols);
      float mr = -INFINITY;
#pragma unroll
      for (int w = 0; w < AT_WARPS; ++w) mr = fmaxf(mr, join_ml[w][r][0]);
      const float b = mr == -INFINITY ? 0.0f : mr;
      float lr = 0.0f;
      float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
      for (int w = 0; w < AT_WARPS; ++w) {
        const float f = ex2(join_ml[w][r][0] - b);
        const float4 y = *reinterpret_cast<const float4 *>(join + (w * AT_M + r) * C::OLD + d);
        lr += f * join_ml[w][r][1];
        v.x += f * y.x;
        v.y += f * y.y;
        v.z += f * y.z;
        v.w += f * y.w;
      }
      if (c0 == c1) {
        row_out(r, d, v, mr, lr);
      } else {
        *reinterpret_cast<float4 *>(slot + r * DP + d) = v;
        if (d == 0) {
          slot[AT_M * DP + 2 * r] = mr;
          slot[AT_M * DP + 2 * r + 1] = lr;
        }
      }
    }
    // ---- join the CTAs of a split item: the last to arrive
    if (c0 != c1) {
      __syncthreads();
      if (tid == 0)
        is_last = atom_add_acq_rel_gpu(pl.counters + c0, 1) == c1 - c0;
      __syncthreads();
      if (is_last) {
        if (tid == 0) pl.counters[c0] = 0;
        auto part = [&](int c) {
          return pl.partials + static_cast<size_t>(2 * c + (c == c0 ? 1 : 0)) * C::SLOT;
        };
        for (int c = tid; c < n_rows * cols; c += AT_THREADS) {
          const int r = c / cols, d = 4 * (c - r * cols);
          float mr = -INFINITY;
          for (int k = c0; k <= c1; ++k) mr = fmaxf(mr, __ldcg(part(k) + AT_M * DP + 2 * r));
          const float b = mr == -INFINITY ? 0.0f : mr;
          float lr = 0.0f;
          float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
          for (int k = c0; k <= c1; ++k) {
            const float *q = part(k);
            const float f = ex2(__ldcg(q + AT_M * DP + 2 * r) - b);
            const float4 y = __ldcg(reinterpret_cast<const float4 *>(q + r * DP + d));
            lr += f * __ldcg(q + AT_M * DP + 2 * r + 1);
            v.x += f * y.x;
            v.y += f * y.y;
            v.z += f * y.z;
            v.w += f * y.w;
          }
          row_out(r, d, v, mr, lr);
        }
      }
    }

    // ---- the next item
    cur += t1 - t0;
    t0 = 0;
    if (cur < end && ++rt == x.rt) {
      rt = 0;
      if (++hk == p.Hkv) {
        hk = 0;
        do x = seq_info<TK>(p, G, ++s);
        while (x.rt == 0);
      }
    }
  }
}

int padded_dim(int D) { return D <= 64 ? 64 : (D <= 128 ? 128 : 256); }

// CTAs per SM by shared memory: 2 up to D = 128, 1 above.
int attn_grid(int D, int num_sms) { return padded_dim(D) <= 128 ? 2 * num_sms : num_sms; }

template <bool E4M3, int DP>
cudaError_t launch(const AttnParams &p, const AttnPlan &pl, cudaStream_t s) {
  using C = AttnCfg<E4M3, DP>;
  auto kernel = attn_decode_kernel<E4M3, DP>;
  const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             static_cast<int>(C::SMEM));
  if (e != cudaSuccess) return e;
  return launch_pdl(kernel, dim3(pl.grid), dim3(AT_THREADS), C::SMEM, s, p, pl);
}

}  // namespace

// Counters (one per worker, zero between calls), then two partial slots per worker.
size_t attn_workspace_bytes(int, int, int, int, int D, int num_sms) {
  const int dp = padded_dim(D), grid = attn_grid(D, num_sms);
  const size_t counters = (static_cast<size_t>(grid) * sizeof(int) + 255) / 256 * 256;
  return counters + static_cast<size_t>(2) * grid * (AT_M * dp + 2 * AT_M) * sizeof(float);
}

cudaError_t launch_attn_decode(const AttnParams &p, bool e4m3, void *ws, int num_sms,
                               cudaStream_t s) {
  AttnPlan pl;
  pl.grid = attn_grid(p.D, num_sms);
  pl.min_tiles = AT_WARPS;
  pl.counters = static_cast<int *>(ws);
  const size_t counters = (static_cast<size_t>(pl.grid) * sizeof(int) + 255) / 256 * 256;
  pl.partials = reinterpret_cast<float *>(static_cast<char *>(ws) + counters);
  switch (padded_dim(p.D)) {
    case 64:
      return e4m3 ? launch<true, 64>(p, pl, s) : launch<false, 64>(p, pl, s);
    case 128:
      return e4m3 ? launch<true, 128>(p, pl, s) : launch<false, 128>(p, pl, s);
    default:
      return e4m3 ? launch<true, 256>(p, pl, s) : launch<false, 256>(p, pl, s);
  }
}

}  // namespace ssd

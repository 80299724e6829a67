// latent_prompt.cu -- causal attention of whole prompts in the expanded form of latent attention,
// on tcgen05 tensor cores: keys of N elements a head and P rotary ones that all heads share,
// values of V elements a head.
//
//     z_ij = scale log2(e) (q_i[:N] . k_j + q_i[N:] . r_j),  out_i = sum_j 2^(z_ij - m_i) v_j / sum
//
// 2 (N + P + V) operations a pair of row and key where a tile's keys come from L2: the tensor cores
// bound it, 1280 clocks for 128 x 128 pairs of 192 + 128 elements at their nominal rate, where 2^x
// of the pairs takes 512 to 1024. A CTA takes 256 rows of one head as two tiles, and while the
// scores of one are made weights by its four warps (a thread a row), the tensor core works on the
// other's: with S0, S1, O0, O1 tensor memory is full (128 columns each), weights overwrite
// their scores as bf16 and are the next product's A from there:
//
//     S[128 rows, 128 keys] = Q . [K | R]^T   A = Q, B = K, K-major in shared memory
//     O[128 rows, V]       += P . V           A = P in tensor memory, B = V as stored (MN-major)
//
// in the order PV0(j) S0(j+1) PV1(j) S1(j+1). Products of a thread run in order, so the scores
// of j + 1 may overwrite the weights of j, and their arrival tells the softmax that O is whole.
// Keys and values stream through a ring of eight slabs (128 tokens x 64 elements, 16 KB): K(j),
// V(j), K(j+1), ...; V's two slabs are products of 64 columns each, as they need not be
// neighbours.
//
// The running maximum is moved only when it has grown by 8 or more (attn_tc.cuh); sums are
// fp32 of the weights before rounding to bf16 (off by 2^-8 of themselves).
//
// What is not finite in values: in tiles that some row does not see whole, two warps take it
// out of shared memory and note the tokens; rows that see such a token add it from global
// memory themselves. Elsewhere the products carry it.
//
// Blocks of rows are handed out by the grid's order, the last of a sequence (with the most
// keys) first, heads next to each other.
#include <float.h>

#include "attn_tc.cuh"
#include "latent.h"
#include "tma3.cuh"

namespace ssd {
namespace {

constexpr int PR_THREADS = 384;  // 8 softmax warps, boxes, products, 2 that look at values
constexpr int PR_SLOTS = 8, PR_SLAB = 128 * 128, PR_ROWS = 256, PR_VB = 4;
constexpr int PR_MAX_Q = 3;  // slabs of q and k
constexpr size_t PR_SMEM = (2 * PR_MAX_Q + PR_SLOTS) * static_cast<size_t>(PR_SLAB);

struct PromptBlock {
  int q0, n, k0, len, row0;  // the sequence's rows and keys, the block's first row
};

struct PromptSearch {
  int warp_sum[PR_THREADS / 32];
  int seq, block;
};
__device__ __forceinline__ int2 clamped_range(const int32_t *start, int s, int most) {
  const int a = min(max(start[s], 0), most), b = min(max(start[s + 1], 0), most);
  return make_int2(a, max(b - a, 0));
}
// The blk-th block of rows of all sequences; false: there are fewer.
__device__ __forceinline__ bool find_block(const LatentPromptParams &p, int blk,
                                           PromptSearch &f, PromptBlock &b) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int per = (p.S + PR_THREADS - 1) / PR_THREADS;
  const int lo = min(tid * per, p.S), hi = min(lo + per, p.S);
  auto blocks = [&](int s) {
    return (clamped_range(p.q_start, s, p.T).y + PR_ROWS - 1) / PR_ROWS;
  };
  int mine = 0;
  for (int s = lo; s < hi; ++s) mine += blocks(s);
  int incl = mine;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, incl, d);
    if (lane >= d) incl += y;
  }
  if (lane == 31) f.warp_sum[warp] = incl;
  __syncthreads();
  int before = 0, total = 0;
#pragma unroll
  for (int w = 0; w < PR_THREADS / 32; ++w) {
    if (w < warp) before += f.warp_sum[w];
    total += f.warp_sum[w];
  }
  if (blk >= total) return false;
  int at = before + incl - mine;
  if (at <= blk && blk < at + mine) {
    for (int s = lo; s < hi; ++s) {
      const int n = blocks(s);
      if (blk < at + n) {
        f.seq = s;
        f.block = n - 1 - (blk - at);
        break;
      }
      at += n;
    }
  }
  __syncthreads();
  const int2 q = clamped_range(p.q_start, f.seq, p.T), k = clamped_range(p.k_start, f.seq, p.Tk);
  b.q0 = q.x;
  b.n = q.y;
  b.k0 = k.x;
  b.len = k.y;
  b.row0 = f.block * PR_ROWS;
  return true;
}

__global__ void __launch_bounds__(PR_THREADS, 1)
    latent_prompt_kernel(const __grid_constant__ CUtensorMap qmap,
                         const __grid_constant__ CUtensorMap kmap,
                         const __grid_constant__ CUtensorMap rmap,
                         const __grid_constant__ CUtensorMap vmap,
                         const __grid_constant__ LatentPromptParams p, const uint16_t *values,
                         const long long v_stride, const long long v_head) {
  extern __shared__ __align__(1024) uint8_t pr_smem[];  // Q0, Q1, the ring
  __shared__ PromptSearch search;
  __shared__ __align__(8) uint64_t qfull[2], full[PR_SLOTS], empty[PR_SLOTS], v_ready[PR_VB];
  __shared__ __align__(8) uint64_t s_full[2], p_full[2], o_full[2], drained;
  __shared__ uint32_t bad[PR_VB][4];  // tokens with values that are not finite
  __shared__ uint32_t tmem_slot;
  __shared__ int abort_flag, keep_first[2];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (tid == 0) {
    abort_flag = 0;
    for (int i = 0; i < PR_SLOTS; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 1);
    }
    for (int i = 0; i < PR_VB; ++i) mbar_init(&v_ready[i], 2);
    for (int g = 0; g < 2; ++g) {
      mbar_init(&qfull[g], 1);
      mbar_init(&s_full[g], 1);
      mbar_init(&p_full[g], 128);
      mbar_init(&o_full[g], 1);
      keep_first[g] = 0;
    }
    mbar_init(&drained, 1);
    fence_mbar_init();
    prefetch_tensormap(&qmap);
    prefetch_tensormap(&kmap);
    if (p.P > 0) prefetch_tensormap(&rmap);
    prefetch_tensormap(&vmap);
  }
  griddep_wait();
  const int h = blockIdx.x % p.H;
  PromptBlock b;
  if (!find_block(p, blockIdx.x / p.H, search, b)) return;
  if (warp == 9) {
    tmem_alloc(&tmem_slot, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  // after the allocation: a dependent grid's CTA cannot hold the columns this one waits for
  griddep_launch_dependents();
  const uint32_t tmem = tmem_slot;  // S0, S1, O0, O1
  const int kn = (p.N + p.P) >> 6, vn = p.V >> 6, step = kn + vn;
  // position of row i is shift + i; tiles of 128 keys that some row of a group sees
  const int shift = b.len - b.n;
  auto rows_of = [&](int g) { return min(128, b.n - b.row0 - 128 * g); };
  auto tiles_of = [&](int g) {
    const int rows = rows_of(g);
    return rows > 0 ? (max(shift + b.row0 + 128 * g + rows, 0) + 127) >> 7 : 0;
  };
  const int nt0 = tiles_of(0), nt1 = tiles_of(1), nt = max(nt0, nt1);
  // whether some row of the group does not see the whole tile
  auto partial = [&](int g, int j) {
    return j < (g ? nt1 : nt0) && j * 128 + 127 > shift + b.row0 + 128 * g;
  };
  auto wait = [&](uint64_t *bar, int phase) {
    return mbar_wait_bounded(bar, phase & 1, p.status, &abort_flag, p.wait_limit_ns);
  };
  uint8_t *const ring = pr_smem + 2 * PR_MAX_Q * PR_SLAB;
  int issued = 0;

  if (warp == 8) {
    // ================================================================ boxes
    bool go = true;
    if (elect_one()) {
      for (int g = 0; g < 2; ++g) {
        if ((g ? nt1 : nt0) == 0) continue;
        mbar_arrive_expect_tx(&qfull[g], kn * PR_SLAB);
        for (int i = 0; i < kn; ++i)
          tma_load_3d(smem_u32(pr_smem + (g * PR_MAX_Q + i) * PR_SLAB), &qmap, &qfull[g], i * 64, h,
                      b.q0 + b.row0 + 128 * g);
      }
    }
    __syncwarp();
    for (int i = 0; go && i < nt * step; ++i) {
      const int slot = i % PR_SLOTS, j = i / step, x = i - j * step, tok = b.k0 + j * 128;
      if (i >= PR_SLOTS) go = __all_sync(0xffffffffu, wait(&empty[slot], i / PR_SLOTS - 1));
      if (!go) break;
      issued = i + 1;
      if (elect_one()) {
        const uint32_t to = smem_u32(ring + slot * PR_SLAB);
        mbar_arrive_expect_tx(&full[slot], PR_SLAB);
        if (x * 64 < p.N) tma_load_3d(to, &kmap, &full[slot], x * 64, h, tok);
        else if (x < kn) tma_load_3d(to, &rmap, &full[slot], x * 64 - p.N, 0, tok);
        else tma_load_3d(to, &vmap, &full[slot], (x - kn) * 64, h, tok);
      }
      __syncwarp();
    }
  } else if (warp == 9) {
    // ================================================================ products
    const uint32_t id_s = idesc_bf16(128), id_o = idesc_bf16(64) | (1u << 16);
    const uint32_t ring_u = smem_u32(ring), q_u = smem_u32(pr_smem);
    auto scores = [&](int g, int j, bool last) {
      for (int i = 0; i < kn; ++i) {
        const int at = j * step + i;
        wait(&full[at % PR_SLOTS], at / PR_SLOTS);
      }
      tc_fence_after();
      if (elect_one()) {
#pragma unroll 1
        for (int i = 0; i < kn; ++i) {
          const int slot = (j * step + i) % PR_SLOTS;
          const uint64_t a = sw128_desc(q_u + (g * PR_MAX_Q + i) * PR_SLAB);
          const uint64_t k = sw128_desc(ring_u + slot * PR_SLAB);
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            tc_mma(tmem + g * 128, a + 2 * kk, k + 2 * kk, id_s, i > 0 || kk > 0 ? 1u : 0u);
          if (last) tc_commit(&empty[slot]);
        }
        tc_commit(&s_full[g]);
      }
      __syncwarp();
    };
    auto outputs = [&](int g, int j, bool last) {
      wait(&p_full[g], j);
      wait(&v_ready[j % PR_VB], j / PR_VB);
      tc_fence_after();
      const uint32_t acc = j > 0 || *static_cast<volatile int *>(&keep_first[g]) != 0 ? 1u : 0u;
      if (elect_one()) {
#pragma unroll 1
        for (int i = 0; i < vn; ++i) {
          const int slot = (j * step + kn + i) % PR_SLOTS;
          const uint64_t v = sw128_mn_desc(ring_u + slot * PR_SLAB, PR_SLAB);
#pragma unroll
          for (int kk = 0; kk < 8; ++kk)
            tc_mma_ts(tmem + 256 + g * 128 + i * 64, tmem + g * 128 + kk * 8,
                      v + (2048 >> 4) * kk, id_o, kk > 0 ? 1u : acc);
          if (last) tc_commit(&empty[slot]);
        }
        if (j + 1 == (g ? nt1 : nt0)) tc_commit(&o_full[g]);
      }
      __syncwarp();
    };
    if (nt0 > 0) {
      wait(&qfull[0], 0);
      scores(0, 0, nt1 == 0);
    }
    if (nt1 > 0) {
      wait(&qfull[1], 0);
      scores(1, 0, true);
    }
    for (int j = 0; j < nt; ++j) {
      if (j < nt0) outputs(0, j, j >= nt1);
      if (j + 1 < nt0) scores(0, j + 1, j + 1 >= nt1);
      if (j < nt1) outputs(1, j, true);
      if (j + 1 < nt1) scores(1, j + 1, true);
    }
  } else if (warp >= 10) {
    // ================================================================ values
    const int w = warp - 10;
    for (int j = 0; j < nt; ++j) {
      // Every slab in turn, the keys' too: a wait tells only neighbouring phases apart, and a slot
      // whose last slab has not landed would pass for one that holds the next (values that landed
      // before the first keys let these warps run ahead of the products, which then never
      // saw v_ready's phase).
      for (int at = j * step; at < (j + 1) * step; ++at) wait(&full[at % PR_SLOTS], at / PR_SLOTS);
      if (partial(0, j) || partial(1, j)) {
        // 64 tokens a warp, four rows of eight chunks a step
#pragma unroll 1
        for (int half = 0; half < 2; ++half) {
          uint32_t seen = 0;
          for (int i = 0; i < vn; ++i) {
            uint8_t *slab = ring + (j * step + kn + i) % PR_SLOTS * PR_SLAB;
#pragma unroll 4
            for (int x = 0; x < 8; ++x) {
              const int tok = w * 64 + half * 32 + x * 4 + (lane >> 3);
              uint4 *at = reinterpret_cast<uint4 *>(slab + tok * 128 + ((lane & 7) << 4));
              const uint4 u = *at;
              constexpr uint32_t INF2 = 0x7f807f80u;
              const uint4 no = make_uint4(__vcmpeq2(u.x & INF2, INF2), __vcmpeq2(u.y & INF2, INF2),
                                          __vcmpeq2(u.z & INF2, INF2), __vcmpeq2(u.w & INF2, INF2));
              const bool any = (no.x | no.y | no.z | no.w) != 0;
              if (any) *at = make_uint4(u.x & ~no.x, u.y & ~no.y, u.z & ~no.z, u.w & ~no.w);
              const uint32_t vote = __ballot_sync(0xffffffffu, any);
#pragma unroll
              for (int r = 0; r < 4; ++r)
                if (vote >> (8 * r) & 255u) seen |= 1u << (x * 4 + r);
            }
          }
          if (lane == 0) bad[j % PR_VB][2 * w + half] = seen;
        }
        fence_proxy_async_smem();
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&v_ready[j % PR_VB]);
    }
  } else {
    // ================================================================ softmax, a thread a row
    const int g = warp >> 2, r = tid & 127;
    const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t s_at = tmem + g * 128 + lanes, o_at = tmem + 256 + g * 128 + lanes;
    const int mine = g ? nt1 : nt0, row = b.row0 + 128 * g + r, pos = shift + row;
    const float zf = p.scale * LOG2E;
    float m = -INFINITY, l = 0.0f;
    for (int j = 0; j < mine; ++j) {
      wait(&s_full[g], j);
      tc_fence_after();
      const bool whole = !partial(g, j);
      const int to = pos - j * 128;  // the last key seen, in the tile
      const bool least = zf < 0.0f;
      float best[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) best[i] = least ? INFINITY : -INFINITY;
#pragma unroll
      for (int c0 = 0; c0 < 128; c0 += 32) {
        float z[32];
        tmem_ld32(s_at + c0, z);
        tmem_wait_ld();
        if (!whole) {
#pragma unroll
          for (int i = 0; i < 32; ++i)
            if (c0 + i > to) z[i] = least ? INFINITY : -INFINITY;
        }
        if (least) {
#pragma unroll
          for (int i = 0; i < 32; ++i) best[i & 3] = fminf(best[i & 3], z[i]);
        } else {
#pragma unroll
          for (int i = 0; i < 32; ++i) best[i & 3] = fmaxf(best[i & 3], z[i]);
        }
      }
      float mx = least ? fminf(fminf(best[0], best[1]), fminf(best[2], best[3]))
                       : fmaxf(fmaxf(best[0], best[1]), fmaxf(best[2], best[3]));
      mx = to < 0 ? -INFINITY : mx * zf;
      if (j == 0) {
        m = mx;
      } else if (__any_sync(0xffffffffu, mx - m >= TC_LAZY)) {
        const float now = mx - m >= TC_LAZY ? mx : m;
        const float fade = ex2(m - (now == -INFINITY ? 0.0f : now));
        m = now;
        l *= fade;
#pragma unroll 1
        for (int d = 0; d < p.V; d += 16) {
          float o[16];
          uint32_t u[16];
          tmem_ld16(o_at + d, o);
          tmem_wait_ld();
#pragma unroll
          for (int e = 0; e < 16; ++e) u[e] = __float_as_uint(o[e] * fade);
          tmem_st16(o_at + d, u);
        }
        tmem_wait_st();
      }
      const float base = m == -INFINITY ? 0.0f : m;
      float2 sum[2] = {make_float2(0.0f, 0.0f), make_float2(0.0f, 0.0f)};
#pragma unroll
      for (int c0 = 0; c0 < 128; c0 += 32) {
        float z[32];
        uint32_t u[16];
        tmem_ld32(s_at + c0, z);
        tmem_wait_ld();
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          float2 y = fma2(make_float2(z[2 * i], z[2 * i + 1]), make_float2(zf, zf),
                          make_float2(-base, -base));
          y.x = ex2(y.x);
          y.y = ex2(y.y);
          if (!whole) {
            if (c0 + 2 * i > to) y.x = 0.0f;
            if (c0 + 2 * i + 1 > to) y.y = 0.0f;
          }
          sum[i & 1] = add2(sum[i & 1], y);
          u[i] = pack2<false>(y.x, y.y);
        }
        tmem_st16(s_at + c0 / 2, u);
      }
      sum[0] = add2(sum[0], sum[1]);
      l += sum[0].x + sum[0].y;
      tmem_wait_st();
      int keep = 0;
      if (partial(0, j) || partial(1, j)) {
        wait(&v_ready[j % PR_VB], j / PR_VB);
        const volatile uint32_t *from = bad[j % PR_VB];
        const uint32_t words[4] = {from[0], from[1], from[2], from[3]};
        if (words[0] | words[1] | words[2] | words[3]) {
          // values that were taken out: added where they are seen (a weight of zero is taken
          // as the smallest number)
          keep = 1;
#pragma unroll 1
          for (int d = 0; d < p.V; d += 16) {
            float o[16];
            uint32_t u[16];
            tmem_ld16(o_at + d, o);
            tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 16; ++e) o[e] = j == 0 ? 0.0f : o[e];
#pragma unroll 1
            for (int t = 0; t < 128; ++t) {
              if (!(words[t >> 5] >> (t & 31) & 1) || j * 128 + t >= b.len) continue;
              const uint32_t two = tmem_ld1(s_at + t / 2);
              tmem_wait_ld();
              float w = bf16_to_f32(static_cast<uint16_t>(t & 1 ? two >> 16 : two & 0xffffu));
              if (t > to) continue;
              if (w == 0.0f) w = FLT_MIN;
              const uint16_t *v = values + (b.k0 + j * 128 + t) * v_stride + h * v_head + d;
#pragma unroll
              for (int e = 0; e < 16; ++e)
                if ((v[e] & 0x7f80u) == 0x7f80u) o[e] += w * bf16_to_f32(v[e]);
            }
#pragma unroll
            for (int e = 0; e < 16; ++e) u[e] = __float_as_uint(o[e]);
            tmem_st16(o_at + d, u);
          }
          tmem_wait_st();
        }
      }
      if (r == 0) keep_first[g] = keep;
      tc_fence_before();
      mbar_arrive(&p_full[g]);
    }
    if (mine > 0) wait(&o_full[g], 0);
    tc_fence_after();
    const bool stored = r < rows_of(g);
    if (stored && p.lse)
      p.lse[static_cast<long long>(b.q0 + row) * p.H + h] =
          l == 0.0f ? -INFINITY : (m + log2f(l)) * LN2;
    const float inv = l == 0.0f ? 0.0f : 1.0f / l;
    uint16_t *out = p.out + (b.q0 + row) * p.out_stride + static_cast<long long>(h) * p.V;
#pragma unroll 1
    for (int d = 0; d < p.V; d += 32) {
      float o[32];
      if (mine > 0) {
        tmem_ld32(o_at + d, o);
        tmem_wait_ld();
      }
      if (!stored) continue;
#pragma unroll
      for (int e = 0; e < 32; e += 8) {
        float y[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i] = l == 0.0f ? 0.0f : o[e + i] * inv;
        *reinterpret_cast<uint4 *>(out + d + e) =
            make_uint4(pack2<false>(y[0], y[1]), pack2<false>(y[2], y[3]),
                       pack2<false>(y[4], y[5]), pack2<false>(y[6], y[7]));
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (*static_cast<volatile int *>(&abort_flag)) {
    // a wait ran out: products end before tensor memory is released, boxes land before the
    // CTA ends
    if (warp == 9) {
      if (elect_one()) tc_commit(&drained);
      __syncwarp();
      mbar_wait_drain(&drained, 0, 10000000ull);
    }
    if (warp == 8) {
      for (int g = 0; g < 2; ++g)
        if ((g ? nt1 : nt0) > 0) mbar_wait_drain(&qfull[g], 0, 10000000ull);
      for (int i = issued - 1; i >= 0 && i >= issued - PR_SLOTS; --i)
        mbar_wait_drain(&full[i % PR_SLOTS], (i / PR_SLOTS) & 1, 10000000ull);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
  }
  if (warp == 9) tmem_dealloc(tmem, 512);
}

}  // namespace

cudaError_t launch_latent_prompt(const LatentPromptParams &p, const uint16_t *q,
                                 long long q_stride, const uint16_t *k, long long k_stride,
                                 long long k_head, const uint16_t *k_rope, long long r_stride,
                                 const uint16_t *v, long long v_stride, long long v_head,
                                 int num_sms, cudaStream_t s) {
  (void)num_sms;
  CUtensorMap qm, km, rm = {}, vm;
  const int D = p.N + p.P;
  // strides of dimensions of one are never used, but have to be valid
  if (p.H == 1) k_head = p.N, v_head = p.V;
  if (p.Tk == 1) k_stride = k_head * p.H, v_stride = v_head * p.H, r_stride = p.P;
  if (p.T == 1) q_stride = static_cast<long long>(p.H) * D;
  const long long qd[3] = {D, p.H, p.T}, qs[2] = {D, q_stride};
  const long long kd[3] = {p.N, p.H, p.Tk}, ks[2] = {k_head, k_stride};
  const long long rd[3] = {p.P, 1, p.Tk}, rs[2] = {p.P, r_stride};
  const long long vd[3] = {p.V, p.H, p.Tk}, vs[2] = {v_head, v_stride};
  const int box[3] = {64, 1, 128};
  if (!host_map(&qm, q, 2, 3, qd, qs, box, true) || !host_map(&km, k, 2, 3, kd, ks, box, true) ||
      (p.P > 0 && !host_map(&rm, k_rope, 2, 3, rd, rs, box, true)) ||
      !host_map(&vm, v, 2, 3, vd, vs, box, true))
    return cudaErrorInvalidValue;
  const cudaError_t e = cudaFuncSetAttribute(
      latent_prompt_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(PR_SMEM));
  if (e != cudaSuccess) return e;
  // as many blocks of rows as there can be: a part of one a sequence
  const long long blocks = p.T / PR_ROWS + p.S;
  return launch_pdl(latent_prompt_kernel, dim3(static_cast<unsigned>(blocks * p.H)),
                    dim3(PR_THREADS), PR_SMEM, s, qm, km, rm, vm, p, v, v_stride, v_head);
}

}  // namespace ssd

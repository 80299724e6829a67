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
// The tensor core holds a few products ahead of their execution, so what the issuing thread does
// between two lots has to stay below 300 clocks: it waits alone, for whole tiles, with the shape
// known at compile time.
//
// Keys and values stream through a ring of eight slabs (128 tokens x 64 elements, 16 KB): K(j),
// V(j), K(j+1), ... The two slabs of a V tile are one product of 128 columns where they are
// neighbours, two of 64 where the ring's end is between them.
//
// A thread's 128 scores come 64 at a time. The first half's maximum decides whether the running
// maximum moves (by 8 or more; attn_tc.cuh), its weights are stored and their product starts;
// the second half refers to the same maximum unless it exceeds it by 16 or more: larger weights
// cost no bits, as their rounding is relative (2^-8, to bf16) and sums are fp32, and stay far
// below what overflows. Only then O is rescaled once more, behind the first half's product. (With a
// pass for the maximum of all 128 first, the way from scores to weights took 1800 clocks
// instead of 1150, longer than the other group's products.)
//
// What is not finite in values: in tiles that some row does not see whole, two warps take it
// out of shared memory and note the tokens; rows that see such a token add it from global
// memory themselves. Elsewhere the products carry it.
//
// Blocks of rows are handed out by the grid's order, the last of a sequence (with the most
// keys) first, heads next to each other.
//
// While there are fewer blocks of 256 rows than SMs, a CTA takes 128 (SPLIT): the two groups have
// the same rows, one the even tiles of keys and the other the odd ones, each with its own maximum,
// sum and outputs, which join at the end from tensor memory, where every warp reaches its lanes of
// both. A row's way through its keys is half as long. Each tile of keys then serves 128 rows
// instead of 256, so copies bound it sooner: keys and values have rings of two tiles of their own,
// as keys leave a tile long before its values do (with one ring 8192 tokens of two heads took 95 us
// instead of 57). us, 128 / 256 rows a CTA: 777 tokens, 16 heads 12.5 / 17.4; 2048, 16 28.3 / 37.3;
// 512, 32 11.2 / 14.3; 8192, 2 55 / 111; 128 rows behind 4096 tokens, 16 heads 33 / 54; with more
// blocks than SMs 4096, 64 393 (with one ring) / 260.
//
// Measured: 4096 tokens, 64 heads of 128 + 64 and 128 elements 257 to 263 us at the highest clock, 1337
// to 1308 TFLOP/s of the pairs seen (241 us without loads of keys and values past the first two
// tiles), 276 after seconds of load, when the power limit has lowered the clock by some 6 %; 777
// tokens, 16 heads 12.3 us.
#include <float.h>

#include "attn_tc.cuh"
#include "latent.h"
#include "tma3.cuh"

namespace ssd {
namespace {

constexpr int PR_THREADS = 384;  // 8 softmax warps, boxes, products, 2 that look at values
constexpr int PR_SLAB = 128 * 128;
constexpr int PR_MAX_Q = 3;  // slabs of q and k
// Barriers of tiles, taken in turn: as many as there are tiles in the ring (two slabs each at least),
// so that the last use of one is over when it is armed again.
constexpr int PR_TB = 4;
constexpr float PR_LATE = 16.0f;  // growth in the second half that moves the maximum

template <bool SPLIT>
struct PrCfg {
  static constexpr int ROWS = SPLIT ? 128 : 256;  // of a block
  static constexpr int QS = SPLIT ? 1 : 2;        // tiles of q
  // Slabs of the ring, or of two rings of two tiles each.
  static constexpr int SLOTS = SPLIT ? 10 : 8;
  static constexpr size_t SMEM = (QS * PR_MAX_Q + SLOTS) * static_cast<size_t>(PR_SLAB);
};

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
template <int ROWS>
__device__ __forceinline__ bool find_block(const LatentPromptParams &p, int blk,
                                           PromptSearch &f, PromptBlock &b) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int per = (p.S + PR_THREADS - 1) / PR_THREADS;
  const int lo = min(tid * per, p.S), hi = min(lo + per, p.S);
  auto blocks = [&](int s) {
    return (clamped_range(p.q_start, s, p.T).y + ROWS - 1) / ROWS;
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
  b.row0 = f.block * ROWS;
  return true;
}

// Of three numbers in one instruction; NaN as in fmaxf.
__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
__device__ __forceinline__ float min3(float a, float b, float c) {
  float d;
  asm("min.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

template <int KN, int VN, bool SPLIT>  // slabs of a key tile, of a value tile
__global__ void __launch_bounds__(PR_THREADS, 1)
    latent_prompt_kernel(const __grid_constant__ CUtensorMap qmap,
                         const __grid_constant__ CUtensorMap kmap,
                         const __grid_constant__ CUtensorMap rmap,
                         const __grid_constant__ CUtensorMap vmap,
                         const __grid_constant__ LatentPromptParams p, const uint16_t *values,
                         const long long v_stride, const long long v_head) {
  using C = PrCfg<SPLIT>;
  extern __shared__ __align__(1024) uint8_t pr_smem[];  // q, the ring
  __shared__ PromptSearch search;
  __shared__ __align__(8) uint64_t k_full[PR_TB], k_empty[PR_TB], v_full[PR_TB], v_empty[PR_TB];
  __shared__ __align__(8) uint64_t v_ready[PR_TB], qfull[2], s_full[2], p_half[2], p_full[2], h_done[2];
  __shared__ __align__(8) uint64_t o_full[2], drained;
  __shared__ uint32_t bad[PR_TB][4];  // tokens with values that are not finite
  __shared__ uint32_t tmem_slot;
  __shared__ int abort_flag;
  __shared__ float2 half_ml[SPLIT ? 2 : 1][SPLIT ? 128 : 1];  // a group's maximum and sum of a row
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (tid == 0) {
    abort_flag = 0;
    for (int i = 0; i < PR_TB; ++i) {
      mbar_init(&k_full[i], 1);
      mbar_init(&k_empty[i], 1);
      mbar_init(&v_full[i], 1);
      mbar_init(&v_empty[i], 1);
      mbar_init(&v_ready[i], 2);
    }
    for (int g = 0; g < 2; ++g) {
      mbar_init(&qfull[g], 1);
      mbar_init(&s_full[g], p.hold ? 2 : 1);  // self-test: one arrival too many is waited for
      mbar_init(&p_half[g], 128);
      mbar_init(&p_full[g], 128);
      mbar_init(&h_done[g], 1);
      mbar_init(&o_full[g], 1);
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
  if (!find_block<C::ROWS>(p, blockIdx.x / p.H, search, b)) return;
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
  constexpr int STEP = KN + VN;
  // position of row i is shift + i; tiles of 128 keys that some row of a group sees
  const int shift = b.len - b.n;
  auto first_of = [&](int g) { return b.row0 + (SPLIT ? 0 : 128 * g); };  // a group's first row
  auto rows_of = [&](int g) { return min(128, b.n - first_of(g)); };
  auto tiles_of = [&](int g) {
    const int rows = rows_of(g);
    return rows > 0 ? (max(shift + first_of(g) + rows, 0) + 127) >> 7 : 0;
  };
  // A group's tiles, and the CTA's; a group's i-th.
  const int both = tiles_of(0);
  const int nt0 = SPLIT ? (both + 1) >> 1 : both, nt1 = SPLIT ? both >> 1 : tiles_of(1);
  const int nt = SPLIT ? both : max(nt0, nt1);
  auto tile = [&](int g, int i) { return SPLIT ? 2 * i + g : i; };
  // whether some row of the group does not see the whole tile
  auto partial = [&](int g, int j) {
    return (SPLIT || j < (g ? nt1 : nt0)) && j * 128 + 127 > shift + first_of(g);
  };
  auto wait = [&](uint64_t *bar, int phase) {
    return mbar_wait_bounded(bar, phase & 1, p.status, &abort_flag, p.wait_limit_ns);
  };
  uint8_t *const ring = pr_smem + C::QS * PR_MAX_Q * PR_SLAB;
  // the slot of slab x of tile j: keys, then values
  auto slot_of = [&](int j, int x) {
    if (SPLIT) return x < KN ? (j & 1) * KN + x : 2 * KN + (j & 1) * VN + x - KN;
    return static_cast<int>(static_cast<uint32_t>(j * STEP + x) % C::SLOTS);
  };
  int k_issued = 0, v_issued = 0;  // tiles that were begun

  if (warp == 8) {
    // ================================================================ boxes
    bool go = true;
    auto queries = [&](int g) {
      if ((g ? nt1 : nt0) > 0 && elect_one()) {
        mbar_arrive_expect_tx(&qfull[g], KN * PR_SLAB);
        for (int i = 0; i < KN; ++i)
          tma_load_3d(smem_u32(pr_smem + (g * PR_MAX_Q + i) * PR_SLAB), &qmap, &qfull[g], i * 64, h,
                      b.q0 + b.row0 + 128 * g);
      }
      __syncwarp();
    };
    auto box = [&](int j, int x, uint32_t to) {  // slab x of tile j
      const int tok = b.k0 + j * 128;
      uint64_t *const bar = x < KN ? &k_full[j % PR_TB] : &v_full[j % PR_TB];
      if (x == 0) mbar_arrive_expect_tx(bar, KN * PR_SLAB);
      if (x == KN) mbar_arrive_expect_tx(bar, VN * PR_SLAB);
      if (x * 64 < p.N) tma_load_3d(to, &kmap, bar, x * 64, h, tok);
      else if (x < KN) tma_load_3d(to, &rmap, bar, x * 64 - p.N, 0, tok);
      else tma_load_3d(to, &vmap, bar, (x - KN) * 64, h, tok);
    };
    queries(0);
    if constexpr (SPLIT) {
      auto part = [&](int j, int from, int end) {  // keys or values of tile j
        if (go && j >= 2 && j < nt) {
          uint64_t *const bar = from < KN ? &k_empty[(j - 2) % PR_TB] : &v_empty[(j - 2) % PR_TB];
          go = __all_sync(0xffffffffu, wait(bar, (j - 2) / PR_TB));
        }
        if (go && j < nt) {
          (from < KN ? k_issued : v_issued) = j + 1;
          if (elect_one())
            for (int x = from; x < end; ++x) box(j, x, smem_u32(ring + slot_of(j, x) * PR_SLAB));
          __syncwarp();
        }
      };
      // in the order in which slots become free: keys leave a tile before its values do
      part(0, 0, KN);
      part(0, KN, STEP);
      part(1, 0, KN);
      part(1, KN, STEP);
      part(2, 0, KN);
      part(3, 0, KN);
#pragma unroll 1
      for (int j = 2; go && j < nt; ++j) {
        part(j, KN, STEP);
        part(j + 2, 0, KN);
      }
    } else {
      for (int i = 0, j = 0; go && j < nt; ++j) {
#pragma unroll 1
        for (int x = 0; x < STEP; ++x, ++i) {
          if (i >= C::SLOTS) {  // what held the slot: a slab of tile j2's keys or values
            const int j2 = (i - C::SLOTS) / STEP, x2 = i - C::SLOTS - j2 * STEP;
            uint64_t *const bar = x2 < KN ? &k_empty[j2 % PR_TB] : &v_empty[j2 % PR_TB];
            go = __all_sync(0xffffffffu, wait(bar, j2 / PR_TB));
            if (!go) break;
          }
          (x < KN ? k_issued : v_issued) = j + 1;
          if (elect_one()) box(j, x, smem_u32(ring + i % C::SLOTS * PR_SLAB));
          __syncwarp();
          if (i == KN - 1) queries(1);  // behind the first keys, with which the first rows begin
        }
      }
    }
  } else if (warp == 9) {
    // ================================================================ products
    if (elect_one()) {
      const uint32_t id_s = idesc_bf16(128), id_o = idesc_bf16(64 * VN) | (1u << 16);
      const uint32_t id_o64 = idesc_bf16(64) | (1u << 16);
      const uint64_t ring_k = sw128_desc(smem_u32(ring));
      const uint64_t ring_v = sw128_mn_desc(smem_u32(ring), PR_SLAB);
      // `last`: no other rows need the tile
      auto scores = [&](int g, int n, bool last) {
        const int j = tile(g, n);
        const uint64_t q = sw128_desc(smem_u32(pr_smem) + (SPLIT ? 0 : g * PR_MAX_Q * PR_SLAB));
        if (SPLIT || g == 0 || j >= nt0) wait(&k_full[j % PR_TB], j / PR_TB);
        tc_fence_after();
#pragma unroll
        for (int i = 0; i < KN; ++i) {
          const uint64_t a = q + i * (PR_SLAB >> 4);
          const uint64_t k = ring_k + static_cast<uint32_t>(slot_of(j, i)) * (PR_SLAB >> 4);
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            tc_mma(tmem + g * 128, a + 2 * kk, k + 2 * kk, id_s, i > 0 || kk > 0 ? 1u : 0u);
        }
        tc_commit(&s_full[g]);
        if (SPLIT || last) tc_commit(&k_empty[j % PR_TB]);
      };
      auto outputs = [&](int g, int n, bool last) {
        const int j = tile(g, n);
        const uint32_t slot = slot_of(j, KN);
        const uint64_t v = ring_v + slot * (PR_SLAB >> 4);
        const bool split = !SPLIT && VN == 2 && slot == C::SLOTS - 1;  // the second slab is slot 0
        const uint32_t o = tmem + 256 + g * 128, w = tmem + g * 128;
        if (SPLIT || g == 0 || j >= nt0) wait(&v_ready[j % PR_TB], j / PR_TB);
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          wait(half ? &p_full[g] : &p_half[g], n);
          tc_fence_after();
          const uint32_t acc = half || n > 0 ? 1u : 0u;
          if (!split) {
#pragma unroll
            for (int kk = 4 * half; kk < 4 * half + 4; ++kk)
              tc_mma_ts(o, w + kk * 8, v + (2048 >> 4) * kk, id_o, (kk & 3) > 0 ? 1u : acc);
          } else {
#pragma unroll
            for (int kk = 4 * half; kk < 4 * half + 4; ++kk) {
              tc_mma_ts(o, w + kk * 8, v + (2048 >> 4) * kk, id_o64, (kk & 3) > 0 ? 1u : acc);
              tc_mma_ts(o + 64, w + kk * 8, ring_v + (2048 >> 4) * kk, id_o64,
                        (kk & 3) > 0 ? 1u : acc);
            }
          }
          if (half == 0) tc_commit(&h_done[g]);
        }
        if (SPLIT || last) tc_commit(&v_empty[j % PR_TB]);
        if (n + 1 == (g ? nt1 : nt0)) tc_commit(&o_full[g]);
      };
      if constexpr (SPLIT) {
        // S0 S1, then PV0 S0 PV1 S1 of every step, in one copy of either: jumping back over two
        // copies takes 400 clocks (2048 tokens, 16 heads 29.8 us, 28.3 with one). Where blocks of 256
        // rows fill the SMs one copy gains nothing (4096 tokens, 64 heads: 264 us against 261).
#pragma unroll 1
        for (int i = -2; i < 2 * nt0; ++i) {
          const int g = i & 1, n = i >> 1, mine = g ? nt1 : nt0;
          if (n >= 0 && n < mine) outputs(g, n, true);
          if (i == -2 && nt0 > 0) wait(&qfull[0], 0);
          if (n + 1 < mine) scores(g, n + 1, true);
        }
      } else {
        if (nt0 > 0) {
          wait(&qfull[0], 0);
          scores(0, 0, nt1 == 0);
        }
        if (nt1 > 0) {
          wait(&qfull[1], 0);
          scores(1, 0, true);
        }
#pragma unroll 1
        for (int j = 0; j < nt; ++j) {
          if (j < nt0) outputs(0, j, j >= nt1);
          if (j + 1 < nt0) scores(0, j + 1, j + 1 >= nt1);
          if (j < nt1) outputs(1, j, true);
          if (j + 1 < nt1) scores(1, j + 1, true);
        }
      }
    }
    __syncwarp();
  } else if (warp >= 10) {
    // ================================================================ values
    const int w = warp - 10;
    for (int j = 0; j < nt; ++j) {
      // Every tile in turn: a wait tells only neighbouring phases apart. (These warps once waited
      // for slots in which keys stood before, without waiting for the keys; values that landed
      // first let them run ahead, and the products never saw v_ready's phase.)
      wait(&v_full[j % PR_TB], j / PR_TB);
      if (partial(0, j) || partial(1, j)) {
        // 64 tokens a warp, four rows of eight chunks a step. An exponent of all ones is the only
        // one that carries into the sign's place: nothing but a look where all are finite.
        uint32_t carry = 0;
#pragma unroll
        for (int i = 0; i < VN; ++i) {
          const uint8_t *from = ring + slot_of(j, KN + i) * PR_SLAB + w * (64 * 128);
#pragma unroll 8
          for (int x = 0; x < 16; ++x) {
            const uint4 u = *reinterpret_cast<const uint4 *>(from + x * 512 + lane * 16);
            carry |= ((u.x & 0x7f807f80u) + 0x00800080u) | ((u.y & 0x7f807f80u) + 0x00800080u) |
                     ((u.z & 0x7f807f80u) + 0x00800080u) | ((u.w & 0x7f807f80u) + 0x00800080u);
          }
        }
        uint32_t seen[2] = {0, 0};
        if (__any_sync(0xffffffffu, carry & 0x80008000u)) {
#pragma unroll 1
          for (int i = 0; i < VN; ++i) {
            uint8_t *slab = ring + slot_of(j, KN + i) * PR_SLAB + w * (64 * 128);
#pragma unroll 1
            for (int x = 0; x < 16; ++x) {
              uint4 *at = reinterpret_cast<uint4 *>(slab + x * 512 + lane * 16);
              const uint4 u = *at;
              constexpr uint32_t INF2 = 0x7f807f80u;
              const uint4 no = make_uint4(__vcmpeq2(u.x & INF2, INF2), __vcmpeq2(u.y & INF2, INF2),
                                          __vcmpeq2(u.z & INF2, INF2), __vcmpeq2(u.w & INF2, INF2));
              const bool any = (no.x | no.y | no.z | no.w) != 0;
              if (any) *at = make_uint4(u.x & ~no.x, u.y & ~no.y, u.z & ~no.z, u.w & ~no.w);
              const uint32_t vote = __ballot_sync(0xffffffffu, any);
              for (int r = 0; r < 4; ++r)
                if (vote >> (8 * r) & 255u) seen[x >> 3] |= 1u << ((x & 7) * 4 + r);
            }
          }
          fence_proxy_async_smem();
        }
        if (lane == 0) {
          bad[j % PR_TB][2 * w] = seen[0];
          bad[j % PR_TB][2 * w + 1] = seen[1];
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&v_ready[j % PR_TB]);
    }
  } else {
    // ================================================================ softmax, a thread a row
    const int g = warp >> 2, r = tid & 127;
    const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t s_at = tmem + g * 128 + lanes, o_at = tmem + 256 + g * 128 + lanes;
    const int mine = g ? nt1 : nt0, row = first_of(g) + r, pos = shift + row;
    // (a scale of zero as one that no score shows: keys not seen stay at -infinity)
    const float zf = p.scale == 0.0f ? FLT_MIN : p.scale * LOG2E;
    const bool least = zf < 0.0f;
    float m = -INFINITY, l = 0.0f;
    float z[2][32];
    float2 sum[2];
    for (int n = 0; n < mine; ++n) {
      const int j = tile(g, n);
      wait(&s_full[g], n);
      tc_fence_after();
      const bool whole = !partial(g, j);
      const int to = pos - j * 128;  // the last key seen, in the tile
      // in a tile that some row does not see whole: tokens whose values were taken out
      const volatile uint32_t *words = bad[j % PR_TB];
      bool taken = false;
      if (partial(0, j) || partial(1, j)) {
        wait(&v_ready[j % PR_TB], j / PR_TB);
        taken = (words[0] | words[1] | words[2] | words[3]) != 0;
      }
      // The largest of scores 64 half .. 64 half + 63, which are in z; those not seen are taken out.
      auto largest = [&](int half) {
        if (!whole) {
#pragma unroll
          for (int i = 0; i < 64; ++i)
            if (64 * half + i > to) z[i >> 5][i & 31] = least ? INFINITY : -INFINITY;
        }
        float best[4] = {z[0][0], z[0][1], z[0][2], z[0][3]};
        if (least) {
#pragma unroll
          for (int i = 4; i < 64; i += 2)
            best[i >> 1 & 3] = min3(best[i >> 1 & 3], z[i >> 5][i & 31], z[i >> 5][(i & 31) + 1]);
        } else {
#pragma unroll
          for (int i = 4; i < 64; i += 2)
            best[i >> 1 & 3] = max3(best[i >> 1 & 3], z[i >> 5][i & 31], z[i >> 5][(i & 31) + 1]);
        }
        const float mx = least ? fminf(fminf(best[0], best[1]), fminf(best[2], best[3]))
                               : fmaxf(fmaxf(best[0], best[1]), fmaxf(best[2], best[3]));
        return to < 64 * half ? -INFINITY : mx * zf;
      };
      // Moves the maximum of rows that grew by `by`, their sums and outputs with it.
      auto move = [&](float mx, float by) {
        const float now = mx - m >= by ? mx : m;
        const float fade = ex2(m - (now == -INFINITY ? 0.0f : now));
        m = now;
        l *= fade;
        sum[0] = make_float2(sum[0].x * fade, sum[0].y * fade);
        sum[1] = make_float2(sum[1].x * fade, sum[1].y * fade);
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
      };
      sum[0] = sum[1] = make_float2(0.0f, 0.0f);
      tmem_ld32(s_at, z[0]);
      tmem_ld32(s_at + 32, z[1]);
      tmem_wait_ld();
      float mx = largest(0);
      if (n == 0) m = mx;
      else if (__any_sync(0xffffffffu, mx - m >= TC_LAZY)) move(mx, TC_LAZY);
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        if (c == 2) {
          tmem_wait_ld();
          mx = largest(1);
          if (__any_sync(0xffffffffu, mx - m >= PR_LATE)) {
            wait(&h_done[g], n);
            tc_fence_after();
            move(mx, PR_LATE);
          }
        }
        float *const x = z[c & 1];
        const float base = m == -INFINITY ? 0.0f : m;
        uint32_t u[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          float2 y = fma2(make_float2(x[2 * i], x[2 * i + 1]), make_float2(zf, zf),
                          make_float2(-base, -base));
          y.x = ex2(y.x);
          y.y = ex2(y.y);
          sum[i & 1] = add2(sum[i & 1], y);
          u[i] = pack2<false>(y.x, y.y);
        }
        tmem_st16(s_at + 16 * c, u);  // over scores that have been read
        if (c < 2) tmem_ld32(s_at + 64 + 32 * c, x);
        if (c == 1) {  // the first half of the keys: their products begin
          tmem_wait_st();
          tc_fence_before();
          mbar_arrive(&p_half[g]);
        }
      }
      sum[0] = add2(sum[0], sum[1]);
      l += sum[0].x + sum[0].y;
      tmem_wait_st();
      if (taken) {
        // values that were taken out: added where they are seen (a weight of zero is taken as
        // the smallest number), between the two products
        wait(&h_done[g], n);
        tc_fence_after();
#pragma unroll 1
        for (int d = 0; d < p.V; d += 16) {
          float o[16];
          uint32_t u[16];
          tmem_ld16(o_at + d, o);
          tmem_wait_ld();
#pragma unroll 1
          for (int t = 0; t < 128; ++t) {
            if ((words[t >> 5] >> (t & 31) & 1) && j * 128 + t < b.len) {
              const uint32_t two = tmem_ld1(s_at + t / 2);
              tmem_wait_ld();
              if (t <= to) {  // rows differ here
                float w = bf16_to_f32(static_cast<uint16_t>(t & 1 ? two >> 16 : two & 0xffffu));
                if (w == 0.0f) w = FLT_MIN;
                const uint16_t *v = values + (b.k0 + j * 128 + t) * v_stride + h * v_head + d;
#pragma unroll
                for (int e = 0; e < 16; ++e)
                  if ((v[e] & 0x7f80u) == 0x7f80u) o[e] += w * bf16_to_f32(v[e]);
              }
            }
            __syncwarp();  // what reads and writes tensor memory next wants the warp in one place
          }
#pragma unroll
          for (int e = 0; e < 16; ++e) u[e] = __float_as_uint(o[e]);
          tmem_st16(o_at + d, u);
        }
        tmem_wait_st();
      }
      tc_fence_before();
      mbar_arrive(&p_full[g]);
    }
    // what the row's two groups (or its one) hold, as factors of the outputs in tensor memory
    float f0 = 1.0f, f1 = 0.0f;
    if constexpr (SPLIT) {
      half_ml[g][r] = make_float2(m, l);
      named_bar_sync(1, 256);
      const float2 x = half_ml[0][r], y = half_ml[1][r];
      m = fmaxf(x.x, y.x);
      const float base = m == -INFINITY ? 0.0f : m;
      f0 = ex2(x.x - base);
      f1 = ex2(y.x - base);
      l = f0 * x.y + f1 * y.y;
      if (nt0 > 0) wait(&o_full[0], 0);
      if (nt1 > 0) wait(&o_full[1], 0);
    } else if (mine > 0) {
      wait(&o_full[g], 0);
    }
    tc_fence_after();
    const bool stored = r < rows_of(g);
    if (stored && p.lse && (!SPLIT || g == 0))
      p.lse[static_cast<long long>(b.q0 + row) * p.H + h] =
          l == 0.0f ? -INFINITY : (m + log2f(l)) * LN2;
    const float inv = l == 0.0f ? 0.0f : 1.0f / l;
    uint16_t *out = p.out + (b.q0 + row) * p.out_stride + static_cast<long long>(h) * p.V;
    // (of one tile of rows each group writes every other 32 elements)
#pragma unroll 1
    for (int d = SPLIT ? 32 * g : 0; d < p.V; d += SPLIT ? 64 : 32) {
      float o[32];
      if (SPLIT ? nt0 > 0 : mine > 0) {
        tmem_ld32((SPLIT ? tmem + 256 + lanes : o_at) + d, o);
        tmem_wait_ld();
      }
      if (SPLIT && nt1 > 0) {
        float o1[32];
        tmem_ld32(tmem + 384 + lanes + d, o1);
        tmem_wait_ld();
#pragma unroll
        for (int e = 0; e < 32; ++e) o[e] = f0 * o[e] + f1 * o1[e];
      }
      if (stored) {
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
      __syncwarp();  // (as above)
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
      for (int g = 0; g < C::QS; ++g)
        if ((g ? nt1 : nt0) > 0) mbar_wait_drain(&qfull[g], 0, 10000000ull);
      // (a tile of which only some slabs were requested never completes: short waits)
      for (int j = k_issued - 1; j >= 0 && j >= k_issued - PR_TB; --j)
        mbar_wait_drain(&k_full[j % PR_TB], (j / PR_TB) & 1, 5000000ull);
      for (int j = v_issued - 1; j >= 0 && j >= v_issued - PR_TB; --j)
        mbar_wait_drain(&v_full[j % PR_TB], (j / PR_TB) & 1, 5000000ull);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
  }
  if (warp == 9) tmem_dealloc(tmem, 512);
}

template <bool SPLIT>
cudaError_t launch_widths(const LatentPromptParams &p, cudaStream_t s, const CUtensorMap &qm,
                          const CUtensorMap &km, const CUtensorMap &rm, const CUtensorMap &vm,
                          const uint16_t *v, long long v_stride, long long v_head) {
  using C = PrCfg<SPLIT>;
  void (*kernel)(CUtensorMap, CUtensorMap, CUtensorMap, CUtensorMap, LatentPromptParams,
                 const uint16_t *, long long, long long) = nullptr;
  switch ((p.N + p.P) / 64 * 2 + p.V / 64 - 1) {
    case 2: kernel = latent_prompt_kernel<1, 1, SPLIT>; break;
    case 3: kernel = latent_prompt_kernel<1, 2, SPLIT>; break;
    case 4: kernel = latent_prompt_kernel<2, 1, SPLIT>; break;
    case 5: kernel = latent_prompt_kernel<2, 2, SPLIT>; break;
    case 6: kernel = latent_prompt_kernel<3, 1, SPLIT>; break;
    default: kernel = latent_prompt_kernel<3, 2, SPLIT>; break;
  }
  const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             static_cast<int>(C::SMEM));
  if (e != cudaSuccess) return e;
  const long long blocks = p.T / C::ROWS + static_cast<long long>(p.S);
  return launch_pdl(kernel, dim3(static_cast<unsigned>(blocks * p.H)), dim3(PR_THREADS), C::SMEM, s,
                    qm, km, rm, vm, p, v, v_stride, v_head);
}

}  // namespace

cudaError_t launch_latent_prompt(const LatentPromptParams &p, const uint16_t *q,
                                 long long q_stride, const uint16_t *k, long long k_stride,
                                 long long k_head, const uint16_t *k_rope, long long r_stride,
                                 const uint16_t *v, long long v_stride, long long v_head,
                                 int num_sms, cudaStream_t s) {
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
  if (!host_map(&qm, q, 3, qd, qs, box) || !host_map(&km, k, 3, kd, ks, box) ||
      (p.P > 0 && !host_map(&rm, k_rope, 3, rd, rs, box)) ||
      !host_map(&vm, v, 3, vd, vs, box))
    return cudaErrorInvalidValue;
  // as many blocks of rows as there can be: a part of one a sequence
  const long long blocks = (p.T / PrCfg<false>::ROWS + static_cast<long long>(p.S)) * p.H;
  // (both sides are at the top)
  auto launch = blocks < num_sms ? launch_widths<true> : launch_widths<false>;
  return launch(p, s, qm, km, rm, vm, v, v_stride, v_head);
}

}  // namespace ssd

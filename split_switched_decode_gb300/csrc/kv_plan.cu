// kv_plan.cu -- block tables and slot maps of a paged key-value cache from request lengths.
#include "attn.h"
#include "common.cuh"

namespace ssd {
namespace {

constexpr int KP_THREADS = 1024;
constexpr int KP_CLUSTER = 8;
constexpr int KP_CLUSTER_TOKENS = 4096;  // rows from which a cluster is launched
// Dynamic shared memory of a launch without the opt-in: 48 KB, less what the kernel has
// statically (256 bytes of warps' sums) with room to spare.
constexpr size_t KP_SMEM_DEFAULT = 47 * 1024;

__device__ __forceinline__ int pages_of(int tokens, int page_size) {
  return tokens / page_size + (tokens % page_size != 0);
}

// Exclusive sum over the CTA's threads, *total the whole sum. Three barriers.
__device__ long long cta_exclusive_sum(long long v, long long *total) {
  __shared__ long long warp_sum[32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  long long x = v;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, x, d);
    if (lane >= d) x += y;
  }
  if (lane == 31) warp_sum[warp] = x;
  __syncthreads();
  if (warp == 0) {
    long long w = lane < static_cast<int>(blockDim.x >> 5) ? warp_sum[lane] : 0;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const long long y = __shfl_up_sync(0xffffffffu, w, d);
      if (lane >= d) w += y;
    }
    warp_sum[lane] = w;
  }
  __syncthreads();
  const long long before = warp > 0 ? warp_sum[warp - 1] : 0;
  *total = warp_sum[(blockDim.x >> 5) - 1];
  __syncthreads();
  return before + x - v;
}

// Largest i in [0, n) with first[i] <= x (first[0] <= x, ascending).
__device__ __forceinline__ int last_at_most(const int *first, int n, int x) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (first[mid] <= x) lo = mid;
    else hi = mid;
  }
  return lo;
}

// Two sums over the sequences (rows, then new pages) into shared memory, then every new page
// and every row finds its sequence by bisection. What it reads and writes would take 0.1 us
// for 65 thousand rows: the launch and the dependent steps (lengths, two sums, bisection,
// page, store) bound a decode step's call. One CTA does it all, or with many rows a cluster
// of 8, each with the sums of all sequences and an eighth of the rows, which it walks 1024 at
// a time: eight such chains in a row for 65 thousand rows, while the other SMs idle (the
// cluster's barrier is what allows outputs in place of inputs). Everything that may be overwritten is
// read before the (cluster's) barrier and the first output is written after it, so seq_len
// may be kv_len and free_used part of summary. Measured in a graph: 64 sequences 4.0 us,
// 512 prompts with 65 thousand rows 12.4 us (one CTA: 70).
template <bool CLUSTER>
__global__ void __launch_bounds__(KP_THREADS) kv_plan_kernel(const KvPlanParams p) {
  extern __shared__ int kp_smem[];
  int *row0 = kp_smem;            // [S] first row of the sequence
  int *rank0 = row0 + p.S;        // [S] rank of its first new page
  int *held = rank0 + p.S;        // [S] pages it holds
  int *kv0 = held + p.S;          // [S] tokens in the cache
  griddep_wait();
  griddep_launch_dependents();
  const int tid = threadIdx.x;
  int used = p.free_used ? *p.free_used : 0;
  used = used < 0 ? 0 : (used > p.num_free ? p.num_free : used);
  long long rows = 0, fresh = 0, wanted = 0;  // sums so far
  for (int base = 0; base < p.S; base += KP_THREADS) {
    const int s = base + tid;
    int kv = 0, nw = 0;
    if (s < p.S) {
      kv = max(p.kv_len[s], 0);
      nw = p.new_len ? max(p.new_len[s], 0) : 1;
    }
    long long sum;
    const long long first = rows + cta_exclusive_sum(nw, &sum);
    const long long cap = p.max_tokens;
    const int r0 = static_cast<int>(first < cap ? first : cap);
    const int r1 = static_cast<int>(first + nw < cap ? first + nw : cap);
    rows += sum;
    const int len = static_cast<int>(min(static_cast<long long>(kv) + (r1 - r0), 0x7fffffffll));
    const int have = pages_of(kv, p.page_size), need = pages_of(len, p.page_size);
    const int have_t = min(have, p.max_pages), need_t = min(need, p.max_pages);
    // new pages that the table has room for, and in the upper half those beyond it: both sums
    // are at most the rows, below 2^31
    const int beyond = (need - have) - (need_t - have_t);
    const long long f0 =
        fresh + (cta_exclusive_sum((static_cast<long long>(beyond) << 32) | (need_t - have_t),
                                   &sum) & 0xffffffffll);
    fresh += sum & 0xffffffffll;
    wanted += (sum & 0xffffffffll) + (sum >> 32);
    if (s < p.S) {
      row0[s] = r0;
      rank0[s] = static_cast<int>(min(f0, 0x7fffffffll));
      held[s] = have_t;
      kv0[s] = kv;
    }
  }
  if (CLUSTER) cluster_sync_all();
  else __syncthreads();
  const int first = blockIdx.x * KP_THREADS + tid, step = gridDim.x * KP_THREADS;
  const int T = static_cast<int>(min(rows, static_cast<long long>(p.max_tokens)));
  const int F = static_cast<int>(min(fresh, 0x7fffffffll));
  auto row_end = [&](int s) { return s + 1 < p.S ? row0[s + 1] : T; };
  // the page of rank r in the free list, -1 past its end
  auto page_at = [&](long long r) {
    return used + r < p.num_free ? p.free_pages[used + r] : -1;
  };
  for (int s = first; s < p.S; s += step) {
    p.q_start[s] = row0[s];
    p.seq_len[s] = static_cast<int>(
        min(static_cast<long long>(kv0[s]) + (row_end(s) - row0[s]), 0x7fffffffll));
  }
  for (int f = first; f < F; f += step) {
    const int s = last_at_most(rank0, p.S, f);
    p.block_table[static_cast<long long>(s) * p.max_pages + held[s] + (f - rank0[s])] =
        page_at(f);
  }
  for (int t = first; t < p.max_tokens; t += step) {
    int pos = 0, slot = -1;
    if (t < T) {
      const int s = last_at_most(row0, p.S, t);
      pos = static_cast<int>(min(static_cast<long long>(kv0[s]) + (t - row0[s]), 0x7fffffffll));
      const int i = pos / p.page_size, o = pos % p.page_size;
      if (i < p.max_pages) {
        const int page =
            i < held[s] ? p.block_table[static_cast<long long>(s) * p.max_pages + i]
                        : page_at(static_cast<long long>(rank0[s]) + (i - held[s]));
        const long long at = static_cast<long long>(page) * p.page_size + o;
        if (page >= 0 && at <= 0x7fffffffll) slot = static_cast<int>(at);
      }
    }
    p.positions[t] = pos;
    p.slots[t] = slot;
  }
  if (first == 0) {
    const long long after = min(used + fresh, static_cast<long long>(p.num_free));
    p.q_start[p.S] = T;
    p.summary[0] = T;
    p.summary[1] = static_cast<int>(after);
    p.summary[2] = static_cast<int>(min(rows - T, 0x7fffffffll));
    p.summary[3] = static_cast<int>(min(wanted - (after - used), 0x7fffffffll));
  }
}

}  // namespace

cudaError_t launch_kv_plan(const KvPlanParams &p, cudaStream_t s) {
  const size_t smem = static_cast<size_t>(4) * p.S * sizeof(int);
  const bool cluster = p.max_tokens > KP_CLUSTER_TOKENS;
  auto kernel = cluster ? kv_plan_kernel<true> : kv_plan_kernel<false>;
  if (smem > KP_SMEM_DEFAULT) {
    const cudaError_t e = cudaFuncSetAttribute(
        kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
    if (e != cudaSuccess) return e;
  }
  if (cluster)
    return launch_pdl_cluster(kernel, dim3(KP_CLUSTER), dim3(KP_THREADS), smem, s, KP_CLUSTER, p);
  return launch_pdl(kernel, dim3(1), dim3(KP_THREADS), smem, s, p);
}

}  // namespace ssd

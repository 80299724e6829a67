// latent_project.cu -- one matrix a head: y[t, h, :] = W[h] x[t, h, :], the way of queries into
// the latent space and of latent outputs back to a head's elements, on tcgen05 tensor cores.
//
// Few rows: every weight is used once a row, so reading the weights bounds it; many rows: each
// element of x and y is read or written once (K N / (K + N) operations a byte, 102 for 128 and
// 512, below what the tensor cores need), so the copy rate bounds that too. Rows are the M of
// the products at any count: BM = 64 rows x BN = 64 columns a tile while the rows fill one tile,
// so that a decode step's products come to several tiles an SM (64 heads of 128 x 512: 512
// tiles of 16 KB), 128 x 64 while the widest tiles would leave SMs idle, and 128 x 256 above, which
// read x and W from L2 0.5 + 1 times for each byte of y (launch_latent_project has what each
// measured; 4096 rows of 64 heads, 128 to 512, 60.6 us, 5.7 TB/s). Tiles go around the CTAs that
// stay; loads of the next tile and the stores of the last overlap the products through a ring of
// k-blocks of 64 and two accumulators.
//
// Warps: 4 write tiles out (TMEM, bf16, shared memory, one TMA box of their rows each 64
// columns; boxes leave out what lies past the tensor), one brings boxes, one issues products.
#include "attn_tc.cuh"
#include "latent.h"
#include "tma3.cuh"

namespace ssd {
namespace {

constexpr int LP_THREADS = 192;

template <int BM, int BN>
struct LpCfg {
  static constexpr int STAGE = (BM + BN) * 128;
  static constexpr int OUT = BM * BN * 2;
  static constexpr int MAX_ST = BN == 64 ? 8 : 3;
  static constexpr int COLS = 2 * BN;
  static constexpr int ROWS = BM / 4;  // rows of a warp
};

template <int BM, int BN>
__global__ void __launch_bounds__(LP_THREADS)
    latent_project_kernel(const __grid_constant__ CUtensorMap xmap,
                          const __grid_constant__ CUtensorMap wmap,
                          const __grid_constant__ CUtensorMap ymap, const LatentProjectParams p) {
  using C = LpCfg<BM, BN>;
  extern __shared__ __align__(1024) uint8_t lp_smem[];  // outputs, then the ring
  __shared__ __align__(8) uint64_t full[C::MAX_ST], empty[C::MAX_ST], done[2], freed[2], drained;
  __shared__ uint32_t tmem_slot;
  __shared__ int abort_flag;
  uint8_t *const ring = lp_smem + C::OUT;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, ST = p.stages;
  if (tid == 0) {
    abort_flag = 0;
    for (int i = 0; i < ST; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&done[i], p.hold ? 2 : 1);  // self-test: one arrival too many is waited for
      mbar_init(&freed[i], 4);
    }
    mbar_init(&drained, 1);
    fence_mbar_init();
    prefetch_tensormap(&xmap);
    prefetch_tensormap(&wmap);
    prefetch_tensormap(&ymap);
  }
  griddep_wait();
  if (warp == 5) {
    tmem_alloc(&tmem_slot, C::COLS);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  // after the allocation: a dependent grid's CTA cannot hold the columns this one waits for
  griddep_launch_dependents();
  const uint32_t tmem = tmem_slot;
  auto wait = [&](uint64_t *bar, int phase) {
    return mbar_wait_bounded(bar, phase & 1, p.status, &abort_flag, p.wait_limit_ns);
  };
  // item: head, row tile, column tile (the fastest, so that neighbours share rows of x)
  auto place = [&](long long item, int &h, int &t0, int &n0) {
    const int i = static_cast<int>(item / p.nb);
    n0 = static_cast<int>(item - static_cast<long long>(i) * p.nb) * BN;
    h = i / p.tb;
    t0 = (i - h * p.tb) * BM;
  };
  int issued = 0;
  if (warp == 4) {
    int k = 0;
    bool go = true;
    for (long long item = blockIdx.x; go && item < p.items; item += gridDim.x) {
      int h, t0, n0;
      place(item, h, t0, n0);
      for (int b = 0; b < p.kb; ++b, ++k) {
        const int st = k % ST;
        if (k >= ST) go = __all_sync(0xffffffffu, wait(&empty[st], k / ST - 1));
        if (!go) break;
        issued = k + 1;
        if (elect_one()) {
          const uint32_t to = smem_u32(ring + st * C::STAGE);
          mbar_arrive_expect_tx(&full[st], C::STAGE);
          tma_load_3d(to, &xmap, &full[st], b * 64, h, t0);
          tma_load_3d(to + BM * 128, &wmap, &full[st], b * 64, n0, h);
        }
        __syncwarp();
      }
    }
  } else if (warp == 5) {
    const uint32_t id = (idesc_bf16(BN) & ~(31u << 24)) | static_cast<uint32_t>(BM >> 4) << 24;
    int k = 0, i = 0;
    for (long long item = blockIdx.x; item < p.items; item += gridDim.x, ++i) {
      const int buf = i & 1;
      if (i >= 2) wait(&freed[buf], (i >> 1) - 1);
      for (int b = 0; b < p.kb; ++b, ++k) {
        const int st = k % ST;
        wait(&full[st], k / ST);
        tc_fence_after();
        if (elect_one()) {
          const uint32_t at = smem_u32(ring + st * C::STAGE);
          const uint64_t a = sw128_desc(at), w = sw128_desc(at + BM * 128);
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            tc_mma(tmem + buf * BN, a + 2 * kk, w + 2 * kk, id, b > 0 || kk > 0 ? 1u : 0u);
          tc_commit(&empty[st]);
          if (b + 1 == p.kb) tc_commit(&done[buf]);
        }
        __syncwarp();
      }
    }
  } else {
    // rows 16 w + lane (BM = 64: 16 lanes of a warp's quarter) or 32 w + lane
    uint8_t *const out = lp_smem + warp * (C::ROWS * BN * 2);
    const uint32_t lanes = static_cast<uint32_t>(warp * 32) << 16;
    int i = 0;
    for (long long item = blockIdx.x; item < p.items; item += gridDim.x, ++i) {
      int h, t0, n0;
      place(item, h, t0, n0);
      const int buf = i & 1;
      if (i > 0) {
        if (lane == 0) bulk_wait_read();  // the last tile's boxes
        __syncwarp();
      }
      wait(&done[buf], i >> 1);
      tc_fence_after();
#pragma unroll
      for (int c0 = 0; c0 < BN; c0 += 32) {
        float v[32];
        tmem_ld32(tmem + buf * BN + lanes + c0, v);
        tmem_wait_ld();
        if (lane < C::ROWS) {
          uint8_t *d = out + (c0 >> 6) * (C::ROWS * 128) + lane * 128;
#pragma unroll
          for (int e = 0; e < 32; e += 8)
            *reinterpret_cast<uint4 *>(d + (((((c0 & 63) + e) >> 3) ^ (lane & 7)) << 4)) =
                make_uint4(pack2<false>(v[e], v[e + 1]), pack2<false>(v[e + 2], v[e + 3]),
                           pack2<false>(v[e + 4], v[e + 5]), pack2<false>(v[e + 6], v[e + 7]));
        }
      }
      tc_fence_before();
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(&freed[buf]);
        const int row = t0 + warp * C::ROWS;
        for (int c = 0; c < BN && row < p.T && n0 + c < p.N; c += 64)
          tma_store_3d(&ymap, smem_u32(out + (c >> 6) * (C::ROWS * 128)), n0 + c, h, row);
        bulk_commit_group();
      }
      __syncwarp();
    }
    if (lane == 0) bulk_wait_all();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (*static_cast<volatile int *>(&abort_flag)) {
    // a wait ran out: products end before tensor memory is released, boxes land before the
    // CTA ends
    if (warp == 5) {
      if (elect_one()) tc_commit(&drained);
      __syncwarp();
      mbar_wait_drain(&drained, 0, 10000000ull);
    }
    for (int i = issued - 1; i >= 0 && i >= issued - ST; --i)
      mbar_wait_drain(&full[i % ST], (i / ST) & 1, 10000000ull);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
  }
  if (warp == 5) tmem_dealloc(tmem, C::COLS);
}

template <int BM, int BN>
cudaError_t launch_shape(LatentProjectParams p, const uint16_t *x, long long x_stride,
                         long long x_head, const uint16_t *w, uint16_t *y, long long y_stride,
                         long long y_head, int num_sms, cudaStream_t s) {
  using C = LpCfg<BM, BN>;
  p.kb = (p.K + 63) / 64;
  p.nb = (p.N + BN - 1) / BN;
  p.tb = (p.T + BM - 1) / BM;
  p.items = static_cast<long long>(p.H) * p.tb * p.nb;
  p.stages = p.kb < C::MAX_ST && BN == 64 ? p.kb : C::MAX_ST;
  CUtensorMap xm, wm, ym;
  const long long xd[3] = {p.K, p.H, p.T}, xs[2] = {x_head, x_stride};
  const long long wd[3] = {p.K, p.N, p.H}, wst[2] = {p.K, static_cast<long long>(p.N) * p.K};
  const long long yd[3] = {p.N, p.H, p.T}, ys[2] = {y_head, y_stride};
  const int xb[3] = {64, 1, BM}, wb[3] = {64, BN, 1}, yb[3] = {64, 1, C::ROWS};
  if (!host_map(&xm, x, 3, xd, xs, xb) || !host_map(&wm, w, 3, wd, wst, wb) ||
      !host_map(&ym, y, 3, yd, ys, yb))
    return cudaErrorInvalidValue;
  auto kernel = latent_project_kernel<BM, BN>;
  const size_t smem = C::OUT + static_cast<size_t>(p.stages) * C::STAGE;
  const cudaError_t e = cudaFuncSetAttribute(
      kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
      static_cast<int>(C::OUT + C::MAX_ST * C::STAGE));
  if (e != cudaSuccess) return e;
  // CTAs an SM: by shared memory, and by tensor memory, which a CTA would otherwise wait for
  int ctas = static_cast<int>(227 * 1024 / (smem + 2048));
  if (ctas > 512 / C::COLS) ctas = 512 / C::COLS;
  const long long grid = static_cast<long long>(ctas) * num_sms;
  return launch_pdl(kernel, dim3(static_cast<unsigned>(p.items < grid ? p.items : grid)),
                    dim3(LP_THREADS), smem, s, xm, wm, ym, p);
}

}  // namespace

cudaError_t launch_latent_project(const uint16_t *x, long long x_stride, long long x_head,
                                  const uint16_t *w, uint16_t *y, long long y_stride,
                                  long long y_head, int T, int H, int K, int N, int num_sms,
                                  unsigned *status, uint64_t wait_limit_ns, bool hold,
                                  cudaStream_t s) {
  LatentProjectParams p = {};
  p.hold = hold;
  p.T = T;
  p.H = H;
  p.K = K;
  p.N = N;
  p.status = status;
  p.wait_limit_ns = wait_limit_ns;
  // strides of dimensions of one are never used, but have to be valid
  if (H == 1) x_head = K, y_head = N;
  if (T == 1) x_stride = x_head * H, y_stride = y_head * H;
  // us, with inputs that take turns from memory, tiles of 64 x 64 / 128 x 64 / 128 x 256 (heads x
  // K to N):
  //      1 row,  64 x 128 to 512    4.9 /  5.9 /  5.5      64 rows, 64 x 512 to 128    6.2 /  6.4 /  7.8
  //    128 rows, 16 x 128 to 512    4.1 /  4.2 /  5.7     128 rows, 64 x 512 to 128    8.5 /  7.1 /  8.6
  //    512 rows, 16 x 128 to 512    6.0 /  5.6 /  6.3     512 rows, 64 x 512 to 128   21.1 / 15.1 / 14.1
  //    512 rows, 64 x 128 to 512   13.9 / 12.2 / 13.2    4096 rows, 64 x 128 to 512   83.6 / 74.7 / 60.6
  // (512 rows of 64 heads into the latent space are on the slower side of the rule.)
  const long long wide = static_cast<long long>(H) * ((T + 127) / 128) * ((N + 255) / 256);
  auto launch = T <= 64 ? launch_shape<64, 64>
                        : (wide < num_sms ? launch_shape<128, 64> : launch_shape<128, 256>);
  return launch(p, x, x_stride, x_head, w, y, y_stride, y_head, num_sms, s);
}

}  // namespace ssd

// latent_decode.cu -- host side of the latent attention kernel (latent_decode.cuh): rows of an
// item, workspace and tensor maps; and the kernel for bf16 caches.
#include "latent_decode.cuh"

namespace ssd {
namespace {

// Rows of an item, from those of an average sequence (what the host knows). More columns than rows
// cost operands, fewer read the tokens again. us, items of 16 / 32 / 64 rows:
//                                          bf16                    e4m3
//   64 sequences to 8192, 8 heads      61.9 /  63.9 / 67.7    56.0 /  66.0 / 71.7
//                         16           63.2 /  65.0 / 68.5    56.4 /  66.5 / 72.6
//                         32          100.3 /  67.3 / 70.7    95.7 /  67.9 / 76.1
//                         64          180.9 / 109.2 / 77.6   177.3 / 115.6 / 83.1
//   one of 777 tokens, 16               9.3 /   9.8 / 11.0    10.5 /  11.7 / 14.4
//   one of 131072, 16                  34.3 /  35.0 / 37.7    31.4 /  35.4 / 40.3
//                  32                  46.7 /  36.5 / 39.3    47.9 /  36.3 / 41.3
int latent_rows(int S, int T, int H) {
  const long long rows = static_cast<long long>((T + S - 1) / S) * H;
  return rows <= 16 ? 16 : (rows <= 32 ? 32 : 64);
}
size_t table_bytes(int T, int H) {
  return (static_cast<size_t>(T) * H * sizeof(int2) + 255) / 256 * 256;
}
size_t ml_bytes(int rows, int num_sms) {
  return (2 * static_cast<size_t>(rows) * num_sms * sizeof(float2) + 255) / 256 * 256;
}

}  // namespace

size_t latent_workspace_bytes(int S, int T, int H, int num_sms) {
  const size_t M = latent_rows(S, T, H);
  return table_bytes(T, H) + ml_bytes(static_cast<int>(M), num_sms) +
         2 * static_cast<size_t>(num_sms) * M * LATENT_MAX_R * sizeof(float);
}

cudaError_t launch_latent_decode(const AttnParams &params, int width, bool e4m3, void *ws,
                                 int num_sms, unsigned *status, uint64_t wait_limit_ns, bool hold,
                                 cudaStream_t s) {
  AttnParams p = params;
  LatentLaunch a = {};
  a.num_sms = num_sms;
  a.rows = ws;
  const int rows = latent_rows(p.S, p.T, p.Hq);
  char *const at = static_cast<char *>(ws) + table_bytes(p.T, p.Hq);
  a.ml = reinterpret_cast<float2 *>(at);
  a.partials = reinterpret_cast<float *>(at + ml_bytes(rows, num_sms));
  a.status = status;
  a.wait_limit_ns = wait_limit_ns;
  a.hold = hold;
  p.box = 0;
  // boxes of 8 tokens of a page; strides of zero (a broadcast cache) or an encoder that
  // refuses: copies by hand
  if (!e4m3 && p.c.page_size % 8 == 0 && p.c.page_stride > 0 && p.c.token_stride > 0) {
    const long long dims[4] = {64, p.c.page_size, width / 64, p.c.num_pages};
    const long long strides[3] = {p.c.token_stride, 64, p.c.page_stride};
    const int box[4] = {64, 8, width / 64, 1};
    if (host_map(&a.map, p.c.k, 4, dims, strides, box)) p.box = 8;
  }
  // rows of q without gaps between tokens: boxes of an item's rows (for e4m3 caches they are
  // converted on the way)
  if (!e4m3 && (p.T == 1 || p.q_stride == static_cast<long long>(p.Hq) * width)) {
    const long long dims[2] = {width, static_cast<long long>(p.T) * p.Hq};
    const long long strides[1] = {width};
    const int box[2] = {64, rows};
    a.q_boxes = host_map(&a.qmap, p.q, 2, dims, strides, box);
  }
  const cudaError_t e = e4m3 ? launch_latent_e4m3(p, width, rows, a, s)
                             : launch_latent<false>(p, width, rows, a, s);
  return e != cudaSuccess ? e : launch_latent_join(p, rows, a, s);
}

}  // namespace ssd

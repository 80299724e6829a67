// attn_d128.cu -- the attention kernel for heads of 65 to 128 elements.
#include "attn_kernel.cuh"

namespace ssd {

cudaError_t launch_attn_d128(const AttnParams &p, bool e4m3, int nr, int wr, void *ws,
                           const AttnLaunch &a, cudaStream_t s) {
  return launch_dim<128>(p, e4m3, nr, wr, ws, a, s);
}

}  // namespace ssd

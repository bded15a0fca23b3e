// The E4M3-cache instances of the paged attention kernel.
#include "paged_attention_mma.cuh"

namespace moe {
namespace attn {
cudaError_t launch_e4m3(const Params& p, int dim, int nt, unsigned blocks, cudaStream_t s) {
  if (dim <= 64) {
    if (nt == 1) return launch_mma<64, 1, true>(p, blocks, s);
    return launch_mma<64, 2, true>(p, blocks, s);
  }
  if (dim <= 128) {
    if (nt == 1) return launch_mma<128, 1, true>(p, blocks, s);
    return launch_mma<128, 2, true>(p, blocks, s);
  }
  if (nt == 1) return launch_mma<256, 1, true>(p, blocks, s);
  return launch_mma<256, 2, true>(p, blocks, s);
}
}  // namespace attn
}  // namespace moe

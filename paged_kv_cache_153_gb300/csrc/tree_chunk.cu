// Attention of prompt chunks to the first tokens and a window, 16-bit caches.
#include "tree.cuh"

namespace pkv {
TreeLauncher chunk_launcher(int q_dtype, int head_dim, int q_tiles) {
  return q_dtype == PKV_F16 ? pick_chunk<F16>(head_dim, q_tiles) : pick_chunk<BF16>(head_dim, q_tiles);
}
}  // namespace pkv

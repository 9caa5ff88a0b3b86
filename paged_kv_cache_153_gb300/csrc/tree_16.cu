// Attention of drafted tokens, 16-bit caches.
#include "tree.cuh"

namespace pkv {
TreeLauncher tree_launcher_16(int q_dtype, int head_dim, int q_tiles) {
  return q_dtype == PKV_F16 ? pick_tree<F16, F16>(head_dim, q_tiles) : pick_tree<BF16, BF16>(head_dim, q_tiles);
}
}  // namespace pkv

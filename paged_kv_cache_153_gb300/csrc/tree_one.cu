// Attention of drafted tokens with one query head per KV head: fp16 and FP8 caches, whose
// weights are two fp16 parts.
#include "tree.cuh"

namespace pkv {
TreeLauncher tree_launcher_one(int kv_kind, int head_dim, int q_tiles) {
  return kv_kind == 0   ? pick_tree<F16, F16, true>(head_dim, q_tiles)
         : kv_kind == 3 ? pick_tree<F16, E5M2, true>(head_dim, q_tiles)
                        : pick_tree<F16, E4M3, true>(head_dim, q_tiles);
}
}  // namespace pkv

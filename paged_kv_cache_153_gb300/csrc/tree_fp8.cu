// Attention of drafted tokens, FP8 caches (q and out in fp16 or bf16, products in fp16).
#include "tree.cuh"

namespace pkv {
TreeLauncher tree_launcher_fp8(int kv_kind, int head_dim, int q_tiles) {
  return kv_kind == 3 ? pick_tree<F16, E5M2>(head_dim, q_tiles) : pick_tree<F16, E4M3>(head_dim, q_tiles);
}
}  // namespace pkv

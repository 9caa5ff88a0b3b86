// Decode variants over the first and the last tokens of a context, FP8 caches (q and out in fp16 or bf16).
#include "decode_launch.cuh"

namespace pkv {
DecodeLauncher decode_launcher_window_fp8(int kv_kind, int q_dtype, int head_dim, int group) {
  const bool e5m2 = kv_kind == 3;
  if (q_dtype == PKV_F16)
    return e5m2 ? pick_dim_group<F16, E5M2, kWindow>(head_dim, group)
                : pick_dim_group<F16, E4M3, kWindow>(head_dim, group);
  if (q_dtype == PKV_BF16)
    return e5m2 ? pick_dim_group<BF16, E5M2, kWindow>(head_dim, group)
                : pick_dim_group<BF16, E4M3, kWindow>(head_dim, group);
  return nullptr;
}
}  // namespace pkv

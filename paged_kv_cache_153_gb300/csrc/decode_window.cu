// Decode variants over the first and the last tokens of a context, 16-bit caches.
#include "decode_launch.cuh"

namespace pkv {
DecodeLauncher decode_launcher_window_16(int q_dtype, int head_dim, int group) {
  if (q_dtype == PKV_F16) return pick_dim_group<F16, F16, kWindow>(head_dim, group);
  if (q_dtype == PKV_BF16) return pick_dim_group<BF16, BF16, kWindow>(head_dim, group);
  return nullptr;
}
}  // namespace pkv

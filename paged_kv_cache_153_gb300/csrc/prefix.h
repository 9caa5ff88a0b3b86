// Shared between the prefix kernel, its merge and the entry point.
#pragma once

#include <cuda.h>
#include <stdint.h>

#include "decode_launch.cuh"

namespace pkv {

constexpr int kMaxPrefixGroups = 1024;   // groups whose geometry a thread block keeps in shared memory
constexpr int kPrefixUnitRows = 256;     // query rows of one unit of work: two tiles of 128

// one group's share of the work; cost counts (unit, 128-key tile) pairs
struct PrefixGroup {
  int64_t cost;                  // of all groups before it
  int32_t start;                 // its first sequence
  int32_t rows;                  // sequences x query heads per KV head
  int32_t blocks;                // whole blocks shared (0: none of its sequences is that long)
  int32_t owner;                 // first sequence that covers them: the table they are read through
};

struct PrefixParams {
  CUtensorMap tmap_k;            // [NB * Hkv * 16 rows, D] 16-bit, [16 x 64] boxes, 128B swizzle
  CUtensorMap tmap_v;
  CUtensorMap tmap_q;            // [B, Hq, D] 16-bit, boxes of [128 / G, G, 64], 128B swizzle
  const int32_t* block_tables;
  const int32_t* context_lens;
  const int32_t* group_starts;   // [num_groups + 1]
  const int32_t* prefix_lens;    // [num_groups]
  PrefixGroup* groups;           // workspace: [num_groups + 1], for the merge
  float* ml;                     // workspace: [rows, 2] (m, l) and
  float* o;                      // [rows, D] o of the pieces
  int32_t* err;
  unsigned long long wait_limit_ns;   // limit of each pipeline wait
  int64_t num_blocks;
  int batch, num_groups, n_q_heads, n_kv_heads, max_blocks_per_seq;
  int max_nblk;                  // ceil(max_context_len / 16)
  int q_tiles;                   // row tiles in shared memory: 2, or 1 where no unit has more than 128 rows
  float qk_scale_log2;
};

// Piece of unit u's rows in range r of the cost axis: rows
// [piece_row(...), + unit rows) of ml and o.  Successive pieces differ in the
// unit or in the range, so they never overlap.
__host__ __device__ inline int64_t piece_row(int64_t group_start, int n_q_heads, int g, int rows, int unit_in_head,
                                             int64_t range) {
  return group_start * n_q_heads + static_cast<int64_t>(g) * rows +
         static_cast<int64_t>(unit_in_head) * kPrefixUnitRows + range * kPrefixUnitRows;
}

// dynamic shared memory of the prefix kernel
size_t prefix_smem_bytes(int head_dim, int num_groups);
// the prefix kernel's attributes on the current device, once for each device
pkv_status prepare_prefix(int group, int head_dim, pkv_dtype dtype);
// ranges: the grid of the prefix kernel
pkv_status launch_prefix(PrefixParams& p, int ranges, int group, int head_dim, pkv_dtype dtype, cudaStream_t stream);
pkv_status launch_prefix_merge(const PrefixParams& p, int ranges, const DecodeParams& rest, int rest_grid, int group,
                               int head_dim, pkv_dtype dtype, cudaStream_t stream);

}  // namespace pkv

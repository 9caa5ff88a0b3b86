// Shared between the kernels of the drafted tokens' attention and the entry points.
#pragma once

#include <cuda.h>
#include <stdint.h>

#include "host_util.h"

namespace pkv {

constexpr int kTreeMaxBatch = 1024;      // sequences whose geometry a thread block keeps in shared memory
constexpr int kTreeMaxWords = 4;         // 64-bit words of a token's mask
constexpr int kTreeRows = 128;           // query rows of a tile
constexpr int kTreeKeys = 128;           // keys of a K / V tile

// one sequence's place on the cost axis
struct TreeSeq {
  int64_t cost;                  // of all sequences before it
  int32_t start, n;              // its drafted tokens: first, count (0: none, or not to be attended)
  int32_t ctx;                   // cached tokens, the drafted ones among them
  int32_t pad;
};

struct TreeParams {
  CUtensorMap tmap_k;            // 16-bit caches: [NB Hkv 2, D / 64, 8, 64], boxes of a block's rows
  CUtensorMap tmap_v;            // (FP8: tmap_k alone, [NB Hkv 16, D] bytes, boxes of 16 rows, D-byte swizzle)
  CUtensorMap tmap_q;            // [T, Hq, D], boxes of [q_box tokens, G, 64]
                                 // (FP8: q's parts, [3 or 5 T, Hq, D] bytes, boxes of [q_box tokens, G, D])
  const void* q;                 // FP8 caches
  uint8_t* parts;                // workspace: q's parts
  float* part_scale;             // [T, Hq], below 0: the row needs the E5M2 parts
  const uint8_t* v_codes;
  const float* k_scale;
  const float* v_scale;
  const void* v_cache;           // any: rows with infinities or NaN are read again
  const int32_t* block_tables;
  const int32_t* context_lens;
  const int32_t* cu_nodes;
  const uint32_t* mask;          // [T, 2 mask_words]
  void* out;
  TreeSeq* seqs;                 // workspace: [batch + 1], for the merge
  float* ml;                     // workspace: [rows, 2] (m, l) and
  float* o;                      // [rows, D] o of the pieces
  int32_t* err;
  unsigned long long wait_limit_ns;
  int64_t num_blocks, num_tokens;
  int batch, n_q_heads, n_kv_heads, group_shift, max_blocks_per_seq;
  int setup_cost;                // of a unit, in half tiles
  int mask_words, max_nodes;     // (chunks: max_nodes is the longest query)
  int window, num_sinks;         // chunks
  int q_box;                     // tokens of a Q box
  int q_bf16;                    // type of q and out: bf16 (else fp16)
  float qk_scale_log2;
};

// kv_kind: 0 = q's 16-bit type, 1 = E4M3, 3 = E5M2; q_tiles: row tiles of a unit
using TreeLauncher = pkv_status (*)(TreeParams&, int ranges, cudaStream_t);
TreeLauncher tree_launcher_16(int q_dtype, int head_dim, int q_tiles);
TreeLauncher tree_launcher_fp8(int kv_kind, int head_dim, int q_tiles);
// one query head per KV head, products in fp16 (fp16 and FP8 caches)
TreeLauncher tree_launcher_one(int kv_kind, int head_dim, int q_tiles);
// prompt chunks with a window, 16-bit caches; `ranges` is the units of the longest one
TreeLauncher chunk_launcher(int q_dtype, int head_dim, int q_tiles);

}  // namespace pkv

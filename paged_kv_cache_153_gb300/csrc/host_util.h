// Host-side helpers shared by the C-ABI translation units.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <utility>

#include "../../include/pkv.h"

namespace pkv {

// Limit of each pipeline wait of a kernel: kWaitLimitNs (1 s), or (for tests of
// the timeout paths) PKV_WAIT_LIMIT_NS nanoseconds.
unsigned long long wait_limit_ns();

// Record a failed CUDA runtime call (name + error) for pkv_last_error() and
// clear the runtime's last-error state so it cannot leak into a later call.
// Returns true when `e` is an error.
bool cuda_failed(cudaError_t e, const char* what);

// Tiled TMA view of a KV cache [rows, head_dim] (rows = num_blocks * H_kv * 16)
// with a [16 rows x 128 bytes] box and the 128-byte swizzle.  Returns false
// (with the reason kept for pkv_last_error) on failure.
// Launch with programmatic stream serialisation allowed (the kernel must call
// pdl_wait_and_release() before it touches global memory).
template <typename... KArgs, typename... Args>
cudaError_t launch_pdl(void (*kern)(KArgs...), dim3 grid, dim3 block, size_t smem, cudaStream_t stream,
                       Args&&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, std::forward<Args>(args)...);
}

bool encode_cache_tmap(CUtensorMap* map, const void* base, int64_t rows, int head_dim, int elt_bytes);

// Tiled TMA view of queries [tokens, n_q_heads, head_dim] (16-bit) with boxes of
// [box_tokens, group heads, 64 elements] and the 128-byte swizzle.
bool encode_query_tmap(CUtensorMap* map, const void* base, int64_t tokens, int n_q_heads, int head_dim, int group,
                       int box_tokens);

// Tiled TMA view of a 16-bit KV cache as [2 slabs, head_dim / 64, 8 rows, 64
// elements] (a slab: the 16 rows of a block and head) with boxes of one slab,
// which land as 8-row atoms of the 128-byte swizzle, the halves of a row side by
// side.
bool encode_block_tmap(CUtensorMap* map, const void* base, int64_t slabs, int head_dim);

// Tiled TMA view of an FP8 cache [rows, head_dim] with boxes of 16 rows and a
// swizzle of a row's bytes (64 or 128).
bool encode_code_tmap(CUtensorMap* map, const void* base, int64_t rows, int head_dim);

// encode_query_tmap over one-byte elements: boxes of [box_tokens, group heads,
// head_dim] and a swizzle of a row's bytes.
bool encode_parts_tmap(CUtensorMap* map, const void* base, int64_t tokens, int n_q_heads, int head_dim, int group,
                       int box_tokens);

// SMs of the current device (0, with the reason kept, when it cannot be asked)
int sm_count();

// The append of the INT8 decode step (append_int8.cu): slots from the block
// table, re-quantising append, early release of the decode launch that
// follows (which waits for it before reading the cache).
pkv_status launch_append_int8_step(const void* k_new, const void* v_new, uint8_t* k_cache, uint8_t* v_cache,
                                   float* slab_params, const int32_t* block_tables, const int32_t* context_lens,
                                   int batch, int max_blocks_per_seq, int64_t num_blocks, int num_kv_heads,
                                   int head_dim, pkv_dtype in_dtype, int64_t* slots_out, int32_t* err_flag,
                                   cudaStream_t stream);

}  // namespace pkv

// C-ABI entry points of the drafted tokens' attention and of the windowed prompt
// chunks: argument checks, workspace and dispatch.
#include "tree.cuh"

#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>

#include "pkv_common.cuh"

namespace pkv {
namespace {

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
size_t round256(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }

// Workspace, from a 256-byte boundary on: the sequences' geometry | [rows, 2]
// fp32 (m, l) | [rows, D] fp32 o, stored 32 bytes at a time | (FP8 caches) [5, T, Hq,
// D] codes of q's parts (bf16 q: three of them) and [T, Hq] fp32 scales.
struct TreeWs {
  size_t seqs, ml, o, parts, part_scale, total;
};

// A call whose bound allows no tokens attends none: what is left of it is the report of
// the sequences that have some, or do not fit (the bounds are checked as anywhere else).
__global__ void __launch_bounds__(256) no_tokens_kernel(const __grid_constant__ TreeParams p) {
  pdl_wait_and_release();
  for (int b = threadIdx.x; b < p.batch; b += 256) tree_sequence<1>(p, b, p.err);
}

pkv_status report_tokens(const int32_t* cu, const int32_t* context_lens, int64_t num_tokens, int batch,
                         int max_blocks_per_seq, int32_t* err_flag, void* stream) {
  if (err_flag == nullptr) return PKV_OK;
  if (!cu || !context_lens) return PKV_ERR_INVALID_ARG;
  TreeParams p{};
  p.cu_nodes = cu;
  p.context_lens = context_lens;
  p.num_tokens = num_tokens;
  p.batch = batch;
  p.max_blocks_per_seq = max_blocks_per_seq;
  p.n_kv_heads = 1;
  p.err = err_flag;
  return cuda_failed(launch_pdl(no_tokens_kernel, dim3(1), dim3(256), 0, static_cast<cudaStream_t>(stream), p),
                     "no_tokens_kernel launch")
             ? PKV_ERR_CUDA
             : PKV_OK;
}

// row tiles of a unit: two where a sequence may have more than one tile of rows
int tree_q_tiles(int max_nodes, int group) { return max_nodes * group > kTreeRows ? 2 : 1; }

bool tree_ws(int batch, int64_t num_tokens, int n_q_heads, int n_kv_heads, int head_dim, int max_nodes, int num_sms,
             TreeWs* w) {
  if (batch < 0 || num_tokens < 0 || num_tokens > INT32_MAX || n_q_heads <= 0 || n_kv_heads <= 0 ||
      n_q_heads % n_kv_heads || n_q_heads / n_kv_heads > 8 || head_dim <= 0 || max_nodes < 0 ||
      max_nodes > 64 * kTreeMaxWords || num_sms <= 0)
    return false;
  const size_t rows = static_cast<size_t>(num_tokens) * n_q_heads +
                      static_cast<size_t>(kTreeRows) * tree_q_tiles(max_nodes, n_q_heads / n_kv_heads) * num_sms;
  size_t at = 0;
  auto take = [&](size_t n) {
    const size_t here = at;
    at += round256(n);
    return here;
  };
  w->seqs = take((static_cast<size_t>(batch) + 1) * sizeof(TreeSeq));
  w->ml = take(rows * 2 * sizeof(float));
  w->o = take(rows * head_dim * sizeof(float));
  w->parts = take(static_cast<size_t>(num_tokens) * n_q_heads * head_dim * 5);
  w->part_scale = take(static_cast<size_t>(num_tokens) * n_q_heads * sizeof(float));
  w->total = at + 256;
  return true;
}

pkv_status tree_common(int kv_kind, const void* q, const void* k_cache, const void* v_cache, const float* k_scale,
                       const float* v_scale, const int32_t* block_tables, const int32_t* context_lens,
                       const int32_t* cu_nodes, const uint64_t* tree_mask, int mask_words, int max_nodes,
                       int64_t num_tokens, int batch, int n_q_heads, int n_kv_heads, int head_dim, int block_size,
                       int max_blocks_per_seq, int64_t num_blocks, int max_context_len, float scale, void* out,
                       pkv_dtype dtype, void* workspace, size_t workspace_bytes, int32_t* err_flag, void* stream) {
  if (batch < 0 || num_tokens < 0 || n_q_heads <= 0 || n_kv_heads <= 0 || n_q_heads % n_kv_heads ||
      max_blocks_per_seq <= 0 || num_blocks < 0 || max_context_len < 0 || max_nodes < 0 || mask_words <= 0 ||
      max_nodes > 64ll * mask_words || !std::isfinite(scale) || scale <= 0.f)
    return PKV_ERR_INVALID_ARG;
  if (dtype != PKV_F16 && dtype != PKV_BF16) return PKV_ERR_INVALID_ARG;
  if (block_size != kBlockSize || (head_dim != 64 && head_dim != 128)) return PKV_ERR_UNSUPPORTED;
  const int group = n_q_heads / n_kv_heads;
  if (group != 1 && group != 2 && group != 4 && group != 8) return PKV_ERR_UNSUPPORTED;
  if (mask_words > kTreeMaxWords || batch > kTreeMaxBatch || n_kv_heads > 65535) return PKV_ERR_UNSUPPORTED;
  if (num_tokens > INT32_MAX / 5 || num_tokens * n_q_heads > INT32_MAX || num_blocks * n_kv_heads > INT32_MAX / kBlockSize)
    return PKV_ERR_UNSUPPORTED;                      // (32-bit TMA row coordinates)
  if (batch == 0 || num_tokens == 0) return PKV_OK;
  if (max_nodes == 0)
    return report_tokens(cu_nodes, context_lens, num_tokens, batch, max_blocks_per_seq, err_flag, stream);
  if (!q || !k_cache || !v_cache || !block_tables || !context_lens || !cu_nodes || !tree_mask || !out || !workspace)
    return PKV_ERR_INVALID_ARG;
  if (kv_kind != 0 && (!k_scale || !v_scale)) return PKV_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(k_cache) || !aligned16(v_cache) || !aligned16(out) || !aligned16(workspace))
    return PKV_ERR_INVALID_ARG;
  if (num_blocks == 0) return PKV_ERR_INVALID_ARG;
  const int num_sms = sm_count();
  if (num_sms <= 0) return PKV_ERR_CUDA;
  TreeWs w;
  if (!tree_ws(batch, num_tokens, n_q_heads, n_kv_heads, head_dim, max_nodes, num_sms, &w)) return PKV_ERR_INVALID_ARG;
  if (workspace_bytes < w.total) return PKV_ERR_WORKSPACE;

  const int q_tiles = tree_q_tiles(max_nodes, group);
  char* ws = reinterpret_cast<char*>(round256(reinterpret_cast<uintptr_t>(workspace)));
  TreeParams p{};
  p.group_shift = group == 8 ? 3 : group == 4 ? 2 : group - 1;
  p.q_box = std::min(kTreeRows / group, max_nodes);
  if (kv_kind == 0 ? !encode_query_tmap(&p.tmap_q, q, num_tokens, n_q_heads, head_dim, group, p.q_box) ||
                         !encode_block_tmap(&p.tmap_k, k_cache, num_blocks * n_kv_heads, head_dim) ||
                         !encode_block_tmap(&p.tmap_v, v_cache, num_blocks * n_kv_heads, head_dim)
                   : !encode_code_tmap(&p.tmap_k, k_cache, num_blocks * n_kv_heads * kBlockSize, head_dim) ||
                         !encode_parts_tmap(&p.tmap_q, ws + w.parts, (dtype == PKV_BF16 ? 3 : 5) * num_tokens, n_q_heads, head_dim, group,
                                            p.q_box))
    return PKV_ERR_CUDA;
  p.parts = reinterpret_cast<uint8_t*>(ws + w.parts);
  p.part_scale = reinterpret_cast<float*>(ws + w.part_scale);
  p.q = q;
  p.v_codes = static_cast<const uint8_t*>(v_cache);
  p.k_scale = k_scale;
  p.v_scale = v_scale;
  p.v_cache = v_cache;
  p.block_tables = block_tables;
  p.context_lens = context_lens;
  p.cu_nodes = cu_nodes;
  p.mask = reinterpret_cast<const uint32_t*>(tree_mask);
  p.out = out;
  p.seqs = reinterpret_cast<TreeSeq*>(ws + w.seqs);
  p.ml = reinterpret_cast<float*>(ws + w.ml);
  p.o = reinterpret_cast<float*>(ws + w.o);
  p.err = err_flag;
  p.wait_limit_ns = wait_limit_ns();
  p.num_blocks = num_blocks;
  p.num_tokens = num_tokens;
  p.batch = batch;
  p.n_q_heads = n_q_heads;
  p.n_kv_heads = n_kv_heads;
  p.max_blocks_per_seq = max_blocks_per_seq;
  p.mask_words = mask_words;
  p.max_nodes = max_nodes;
  p.q_bf16 = dtype == PKV_BF16;
  p.qk_scale_log2 = scale * kLog2e;
  // a range per SM, but no more than there can be key tiles
  const int64_t units = static_cast<int64_t>(batch) * n_kv_heads *
                        ((max_nodes * group + kTreeRows * q_tiles - 1) / (kTreeRows * q_tiles));
  const int64_t tiles = std::max<int64_t>(1, (static_cast<int64_t>(max_context_len) + kTreeKeys - 1) / kTreeKeys);
  const int ranges = static_cast<int>(std::min<int64_t>(num_sms, units * tiles));
  const TreeLauncher launch = group == 1 && (kv_kind != 0 || dtype == PKV_F16)
                                  ? tree_launcher_one(kv_kind, head_dim, q_tiles)
                              : kv_kind == 0 ? tree_launcher_16(dtype, head_dim, q_tiles)
                                             : tree_launcher_fp8(kv_kind, head_dim, q_tiles);
  return launch(p, ranges, static_cast<cudaStream_t>(stream));
}

}  // namespace
}  // namespace pkv

using namespace pkv;

extern "C" size_t pkv_tree_workspace_bytes(int batch, int64_t num_tokens, int num_q_heads, int num_kv_heads,
                                           int head_dim, int max_nodes) {
  const int num_sms = sm_count();
  TreeWs w;
  if (num_sms <= 0 || !tree_ws(batch, num_tokens, num_q_heads, num_kv_heads, head_dim, max_nodes, num_sms, &w))
    return 0;
  return w.total;
}

extern "C" pkv_status pkv_paged_tree_attention(
    const void* q, const void* k_cache, const void* v_cache, const int32_t* block_tables, const int32_t* context_lens,
    const int32_t* cu_nodes, const uint64_t* tree_mask, int mask_words, int max_nodes, int64_t num_tokens, int batch,
    int num_q_heads, int num_kv_heads, int head_dim, int block_size, int max_blocks_per_seq, int64_t num_blocks,
    int max_context_len, float scale, void* out, pkv_dtype dtype, void* workspace, size_t workspace_bytes,
    int32_t* err_flag, void* stream) {
  return tree_common(0, q, k_cache, v_cache, nullptr, nullptr, block_tables, context_lens, cu_nodes, tree_mask,
                     mask_words, max_nodes, num_tokens, batch, num_q_heads, num_kv_heads, head_dim, block_size,
                     max_blocks_per_seq, num_blocks, max_context_len, scale, out, dtype, workspace, workspace_bytes,
                     err_flag, stream);
}

extern "C" pkv_status pkv_paged_tree_attention_fp8(
    const void* q, const uint8_t* k_cache, const uint8_t* v_cache, const float* k_scale, const float* v_scale,
    const int32_t* block_tables, const int32_t* context_lens, const int32_t* cu_nodes, const uint64_t* tree_mask,
    int mask_words, int max_nodes, int64_t num_tokens, int batch, int num_q_heads, int num_kv_heads, int head_dim,
    int block_size, int max_blocks_per_seq, int64_t num_blocks, int max_context_len, float scale, void* out,
    pkv_dtype q_dtype, void* workspace, size_t workspace_bytes, int32_t* err_flag, void* stream) {
  return tree_common(1, q, k_cache, v_cache, k_scale, v_scale, block_tables, context_lens, cu_nodes, tree_mask,
                     mask_words, max_nodes, num_tokens, batch, num_q_heads, num_kv_heads, head_dim, block_size,
                     max_blocks_per_seq, num_blocks, max_context_len, scale, out, q_dtype, workspace, workspace_bytes,
                     err_flag, stream);
}

extern "C" pkv_status pkv_paged_tree_attention_e5m2(
    const void* q, const uint8_t* k_cache, const uint8_t* v_cache, const float* k_scale, const float* v_scale,
    const int32_t* block_tables, const int32_t* context_lens, const int32_t* cu_nodes, const uint64_t* tree_mask,
    int mask_words, int max_nodes, int64_t num_tokens, int batch, int num_q_heads, int num_kv_heads, int head_dim,
    int block_size, int max_blocks_per_seq, int64_t num_blocks, int max_context_len, float scale, void* out,
    pkv_dtype q_dtype, void* workspace, size_t workspace_bytes, int32_t* err_flag, void* stream) {
  return tree_common(3, q, k_cache, v_cache, k_scale, v_scale, block_tables, context_lens, cu_nodes, tree_mask,
                     mask_words, max_nodes, num_tokens, batch, num_q_heads, num_kv_heads, head_dim, block_size,
                     max_blocks_per_seq, num_blocks, max_context_len, scale, out, q_dtype, workspace, workspace_bytes,
                     err_flag, stream);
}

extern "C" pkv_status pkv_paged_prefill_attention_window(
    const void* q, const void* k_cache, const void* v_cache, const int32_t* block_tables, const int32_t* context_lens,
    const int32_t* cu_seqlens, int64_t num_tokens, int batch, int num_q_heads, int num_kv_heads, int head_dim,
    int block_size, int max_blocks_per_seq, int64_t num_blocks, int max_query_len, int window, int num_sinks,
    float scale, void* out, pkv_dtype dtype, int32_t* err_flag, void* stream) {
  if (batch < 0 || num_tokens < 0 || num_q_heads <= 0 || num_kv_heads <= 0 || num_q_heads % num_kv_heads ||
      max_blocks_per_seq <= 0 || num_blocks < 0 || max_query_len < 0 || window <= 0 || num_sinks < 0 ||
      !std::isfinite(scale) || scale <= 0.f)
    return PKV_ERR_INVALID_ARG;
  if (dtype != PKV_F16 && dtype != PKV_BF16) return PKV_ERR_INVALID_ARG;
  if (block_size != kBlockSize || (head_dim != 64 && head_dim != 128)) return PKV_ERR_UNSUPPORTED;
  const int group = num_q_heads / num_kv_heads;
  if (group != 1 && group != 2 && group != 4 && group != 8) return PKV_ERR_UNSUPPORTED;
  if (batch > 65535 || num_kv_heads > 65535 || num_tokens > INT32_MAX / group ||
      num_blocks * num_kv_heads > INT32_MAX / kBlockSize)
    return PKV_ERR_UNSUPPORTED;
  if (batch == 0 || num_tokens == 0) return PKV_OK;
  if (max_query_len == 0)
    return report_tokens(cu_seqlens, context_lens, num_tokens, batch, max_blocks_per_seq, err_flag, stream);
  if (!q || !k_cache || !v_cache || !block_tables || !context_lens || !cu_seqlens || !out || num_blocks == 0)
    return PKV_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(k_cache) || !aligned16(v_cache) || !aligned16(out)) return PKV_ERR_INVALID_ARG;
  const int64_t longest = std::min<int64_t>(max_query_len, num_tokens);
  // Units of 256 rows read K and V half as often (four prompts of 2048 tokens 459 us, 476
  // with units of 128); while units of 128 leave SMs idle, they are done sooner (300
  // tokens of 8 heads 13.2 us, 11.8 with 128).
  const int64_t units128 = (num_tokens * group + kTreeRows - 1) / kTreeRows * num_kv_heads;
  const int q_tiles = longest * group > kTreeRows && units128 > sm_count() ? 2 : 1;
  TreeParams p{};
  p.group_shift = group == 8 ? 3 : group == 4 ? 2 : group - 1;
  p.q_box = static_cast<int>(std::min<int64_t>(kTreeRows / group, longest));
  if (!encode_query_tmap(&p.tmap_q, q, num_tokens, num_q_heads, head_dim, group, p.q_box) ||
      !encode_block_tmap(&p.tmap_k, k_cache, num_blocks * num_kv_heads, head_dim) ||
      !encode_block_tmap(&p.tmap_v, v_cache, num_blocks * num_kv_heads, head_dim))
    return PKV_ERR_CUDA;
  p.v_cache = v_cache;
  p.block_tables = block_tables;
  p.context_lens = context_lens;
  p.cu_nodes = cu_seqlens;
  p.out = out;
  p.err = err_flag;
  p.wait_limit_ns = wait_limit_ns();
  p.num_blocks = num_blocks;
  p.num_tokens = num_tokens;
  p.batch = batch;
  p.n_q_heads = num_q_heads;
  p.n_kv_heads = num_kv_heads;
  p.max_blocks_per_seq = max_blocks_per_seq;
  p.max_nodes = static_cast<int>(longest);
  p.window = window;
  p.num_sinks = num_sinks;
  p.q_bf16 = dtype == PKV_BF16;
  p.qk_scale_log2 = scale * kLog2e;
  const int64_t units = (longest * group + kTreeRows * q_tiles - 1) / (kTreeRows * q_tiles);
  return chunk_launcher(dtype, head_dim, q_tiles)(p, static_cast<int>(units), static_cast<cudaStream_t>(stream));
}

// Drafted tokens of a speculative step (sm_103a): what each of them sees, and
// the move of the accepted ones' cached rows.
//
// The n drafted tokens of a sequence are nodes of a forest: token i hangs on
// token parent[i] < i, or (-1) on the context's last token.  They are cached
// behind the context in that order, token i at position base + i, with
// base = context_len - n.
//
// Plan.  Token i sees itself and its ancestors, and its rotary position is base
// plus its number of ancestors.  One thread block per sequence, one thread per
// token, by pointer jumping: in each round
//     seen[i] |= seen[up[i]],  up[i] = up[up[i]]
// so that after r rounds seen[i] holds the 2^r nearest ones; a round is two
// barriers, and a forest of depth d takes log2 d of them (256 sequences of 100
// to 256 tokens: 4.1 us; all of it is latency: two loads that wait for each
// other, the rounds, the stores).
//
// Commit.  An accepted path is a strictly ascending list a_0 < a_1 < ..., so
// a_k >= k: row base + a_k moves to base + k in every head.  A thread owns 16
// bytes of the rows of one head of K or V and takes them in order: row k is
// written only after the rows up to k have been read, and nothing behind k is
// read from where k is written (a_j >= j > k).  So it can move in place, eight
// loads ahead of their stores.  (64 sequences, 32 layers of 8 heads in one cache:
// 64 to 86 MB of rows move, by the paths; 16 to 19 us with inputs taken in turn, 21 to
// 24 with nothing of them in L2, about half of the copy rate: 2048 thread blocks, each
// with a chain of lengths, lists and tables ahead of the few rows that it moves.)
#include <cuda_runtime.h>

#include <algorithm>

#include "host_util.h"
#include "pkv_common.cuh"

namespace pkv {

constexpr int kPlanWords = 4;                    // 64-bit words of a visibility row at most
constexpr int kMaxNodes = 64 * kPlanWords;

template <int W>
__global__ void __launch_bounds__(64 * W)
    tree_plan_kernel(const int32_t* __restrict__ parents, const int32_t* __restrict__ cu_nodes,
                     const int32_t* __restrict__ block_tables, const int32_t* __restrict__ context_lens,
                     int64_t num_tokens, int max_blocks, int64_t num_blocks, uint64_t* __restrict__ mask,
                     int32_t* __restrict__ positions, int64_t* __restrict__ slots, int32_t* err) {
  __shared__ uint64_t seen[W][64 * W];
  __shared__ int up[64 * W];
  pdl_wait_and_release();   // (writes nothing that a kernel reads before its wait)
  const int b = blockIdx.x, i = threadIdx.x;
  const int64_t t0 = cu_nodes[b], t1 = cu_nodes[b + 1];
  const int ctx = context_lens[b];
  if (t0 < 0 || t1 < t0 || t1 > num_tokens) {
    if (i == 0) record_error(err, PKV_ERR_OOB);
    return;
  }
  const int64_t n = t1 - t0;
  if (n > 64 * W || ctx < n) {
    // no plan for these tokens: they see nothing and have no place
    if (i == 0) record_error(err, PKV_ERR_OOB);
    for (int64_t t = t0 + i; t < t1; t += 64 * W) {
      for (int w = 0; w < W; ++w) mask[t * W + w] = 0;
      if (positions) positions[t] = -1;
      if (slots) slots[t] = -1;
    }
    return;
  }
  const bool live = i < n;
  const int base = ctx - static_cast<int>(n);
  int parent = -1;
  int64_t slot = -1;
  if (live) {
    parent = parents[t0 + i];
    if (slots) {
      const int p = base + i, logical = p / kBlockSize;
      const int32_t id = logical < max_blocks ? block_tables[static_cast<int64_t>(b) * max_blocks + logical] : -1;
      if (id < 0 || id >= num_blocks)
        record_error(err, PKV_ERR_OOB);
      else
        slot = static_cast<int64_t>(id) * kBlockSize + p % kBlockSize;
    }
    if (parent < -1 || parent >= i) {
      record_error(err, PKV_ERR_OOB);
      parent = -1;
    }
  }
  uint64_t m[W];
#pragma unroll
  for (int w = 0; w < W; ++w) m[w] = (i >> 6) == w ? 1ull << (i & 63) : 0;
  int next = parent;
  while (true) {
#pragma unroll
    for (int w = 0; w < W; ++w) seen[w][i] = m[w];
    up[i] = next;
    if (!__syncthreads_or(next >= 0)) break;
    if (next >= 0) {
#pragma unroll
      for (int w = 0; w < W; ++w) m[w] |= seen[w][next];
      next = up[next];
    }
    __syncthreads();
  }
  if (!live) return;
  int count = 0;
#pragma unroll
  for (int w = 0; w < W; ++w) {
    mask[(t0 + i) * W + w] = m[w];
    count += __popcll(m[w]);
  }
  if (positions) positions[t0 + i] = base + count - 1;
  if (slots) slots[t0 + i] = slot;
}

constexpr int kCommitThreads = 256;
constexpr int kMaxAccept = 1024;
constexpr int kCommitBatch = 8;                  // rows whose loads are issued together

__global__ void __launch_bounds__(kCommitThreads)
    tree_commit_kernel(uint4* __restrict__ k_cache, uint4* __restrict__ v_cache,
                       const int32_t* __restrict__ block_tables, const int32_t* __restrict__ context_lens,
                       const int32_t* __restrict__ cu_nodes, const int32_t* __restrict__ accepted, int max_accept,
                       int max_blocks, int64_t num_blocks, int heads, int chunks, int32_t* __restrict__ new_lens,
                       int32_t* err) {
  __shared__ int64_t from[kMaxAccept], to[kMaxAccept];   // rows of head 0, in 16-byte chunks
  __shared__ int count_s, moves_s, bad_s;
  pdl_wait();   // (writes the cache: no early release of the next launch)
  const int b = blockIdx.y, tid = threadIdx.x;
  const int32_t* list = accepted + static_cast<int64_t>(b) * max_accept;
  const int ctx = context_lens[b];
  const int64_t n = static_cast<int64_t>(cu_nodes[b + 1]) - cu_nodes[b];
  if (tid == 0) {
    count_s = max_accept;
    moves_s = 0;
    bad_s = (cu_nodes[b] < 0 || n < 0 || ctx < n || (ctx + kBlockSize - 1ll) / kBlockSize > max_blocks) ? 1 : 0;
  }
  __syncthreads();
  for (int k = tid; k < max_accept; k += kCommitThreads)
    if (list[k] < 0) atomicMin(&count_s, k);
  __syncthreads();
  const int count = count_s;
  if (bad_s == 0) {
    const int base = ctx - static_cast<int>(n);
    const int32_t* row = block_tables + static_cast<int64_t>(b) * max_blocks;
    auto chunk_of = [&](int pos) -> int64_t {      // -1: no such block
      const int32_t id = row[pos / kBlockSize];
      if (id < 0 || id >= num_blocks) return -1;
      return (static_cast<int64_t>(id) * heads * kBlockSize + pos % kBlockSize) * chunks;
    };
    for (int k = tid; k < count; k += kCommitThreads) {
      const int a = list[k];
      if (a >= n || (k > 0 && a <= list[k - 1])) {
        bad_s = 1;
      } else if (a != k) {
        from[k] = chunk_of(base + a);
        to[k] = chunk_of(base + k);
        if (from[k] < 0 || to[k] < 0) bad_s = 1;
        atomicMax(&moves_s, count - k);            // (ascending: from the first that moves on, all do)
      }
    }
  }
  __syncthreads();
  if (bad_s != 0) {
    if (tid == 0) record_error(err, PKV_ERR_OOB);
    return;
  }
  if (blockIdx.x == 0 && tid == 0 && new_lens != nullptr) new_lens[b] = ctx - static_cast<int>(n) + count;
  const int64_t x = static_cast<int64_t>(blockIdx.x) * kCommitThreads + tid;
  const int64_t per_cache = static_cast<int64_t>(heads) * chunks;
  if (x >= 2 * per_cache) return;
  const int64_t y = x >= per_cache ? x - per_cache : x;
  uint4* cache = (x >= per_cache ? v_cache : k_cache) + (y / chunks) * kBlockSize * chunks + y % chunks;
  for (int k0 = count - moves_s; k0 < count; k0 += kCommitBatch) {
    uint4 v[kCommitBatch];
#pragma unroll
    for (int j = 0; j < kCommitBatch; ++j)
      if (k0 + j < count) v[j] = cache[from[k0 + j]];
#pragma unroll
    for (int j = 0; j < kCommitBatch; ++j)
      if (k0 + j < count) cache[to[k0 + j]] = v[j];
  }
}

}  // namespace pkv

using namespace pkv;

extern "C" pkv_status pkv_tree_plan(const int32_t* parents, const int32_t* cu_nodes, const int32_t* block_tables,
                                    const int32_t* context_lens, int batch, int64_t num_tokens, int mask_words,
                                    int block_size, int max_blocks_per_seq, int64_t num_blocks, uint64_t* tree_mask,
                                    int32_t* positions, int64_t* slot_mapping, int32_t* err_flag, void* stream) {
  if (batch < 0 || num_tokens < 0 || mask_words <= 0 || num_blocks < 0) return PKV_ERR_INVALID_ARG;
  if (slot_mapping != nullptr && max_blocks_per_seq <= 0) return PKV_ERR_INVALID_ARG;
  if (block_size != kBlockSize || mask_words > kPlanWords) return PKV_ERR_UNSUPPORTED;
  if (batch == 0 || num_tokens == 0) return PKV_OK;
  if (!parents || !cu_nodes || !context_lens || !tree_mask || (slot_mapping != nullptr && !block_tables))
    return PKV_ERR_INVALID_ARG;
  auto kern = mask_words == 1   ? tree_plan_kernel<1>
              : mask_words == 2 ? tree_plan_kernel<2>
              : mask_words == 3 ? tree_plan_kernel<3>
                                : tree_plan_kernel<4>;
  const cudaError_t e =
      launch_pdl(kern, dim3(static_cast<unsigned>(batch)), dim3(64 * static_cast<unsigned>(mask_words)), 0,
                 static_cast<cudaStream_t>(stream), parents, cu_nodes, block_tables, context_lens, num_tokens,
                 max_blocks_per_seq, num_blocks, tree_mask, positions, slot_mapping, err_flag);
  return cuda_failed(e, "tree_plan_kernel launch") ? PKV_ERR_CUDA : PKV_OK;
}

extern "C" pkv_status pkv_tree_commit(void* k_cache, void* v_cache, const int32_t* block_tables,
                                      const int32_t* context_lens, const int32_t* cu_nodes, const int32_t* accepted,
                                      int max_accept, int batch, int num_kv_heads, int head_dim, int block_size,
                                      int max_blocks_per_seq, int64_t num_blocks, int elt_bytes, int32_t* new_lens,
                                      int32_t* err_flag, void* stream) {
  if (batch < 0 || max_accept < 0 || num_kv_heads <= 0 || num_blocks < 0 || max_blocks_per_seq <= 0)
    return PKV_ERR_INVALID_ARG;
  if (elt_bytes != 1 && elt_bytes != 2) return PKV_ERR_INVALID_ARG;
  if (block_size != kBlockSize || (head_dim != 64 && head_dim != 128)) return PKV_ERR_UNSUPPORTED;
  if (max_accept > kMaxAccept || batch > 65535) return PKV_ERR_UNSUPPORTED;
  if (batch == 0) return PKV_OK;
  if (!k_cache || !v_cache || !block_tables || !context_lens || !cu_nodes || (max_accept > 0 && !accepted))
    return PKV_ERR_INVALID_ARG;
  // (several thread blocks read a sequence's length, one writes its new one)
  if (new_lens != nullptr && new_lens < context_lens + batch && context_lens < new_lens + batch)
    return PKV_ERR_INVALID_ARG;
  if ((reinterpret_cast<uintptr_t>(k_cache) | reinterpret_cast<uintptr_t>(v_cache)) & 15u) return PKV_ERR_INVALID_ARG;
  const int chunks = head_dim * elt_bytes / 16;
  const int64_t grid = (2ll * num_kv_heads * chunks + kCommitThreads - 1) / kCommitThreads;
  if (grid > INT32_MAX) return PKV_ERR_UNSUPPORTED;
  const cudaError_t e =
      launch_pdl(tree_commit_kernel, dim3(static_cast<unsigned>(grid), static_cast<unsigned>(batch)),
                 dim3(kCommitThreads), 0, static_cast<cudaStream_t>(stream), static_cast<uint4*>(k_cache),
                 static_cast<uint4*>(v_cache), block_tables, context_lens, cu_nodes, accepted, max_accept,
                 max_blocks_per_seq, num_blocks, num_kv_heads, chunks, new_lens, err_flag);
  return cuda_failed(e, "tree_commit_kernel launch") ? PKV_ERR_CUDA : PKV_OK;
}

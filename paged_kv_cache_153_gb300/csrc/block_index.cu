// Block index of block-sparse decode (sm_103a): bounds of the cached keys per
// (block, KV head), scores of a step's queries against them, and the choice of
// the blocks to attend to.
//
// Bounds.  lo[d] = min_r K[r][d], hi[d] = max_r K[r][d] over the rows r of a
// block that hold tokens.  Minima and maxima are exact in the key's own type
// (an FP8 code's value is exact in fp16 and bf16), so nothing is rounded.
// Scores.  For any key of the block <q, K> <= sum_d max(q_d lo_d, q_d hi_d) =
// <q+, hi> + <q-, lo> with q+ = max(q, 0), q- = min(q, 0): an upper bound of
// the block's logits, as one product of length 2 D per query head, taken on
// the tensor cores with 16 blocks as M, the group's query heads (padded to 8)
// as N and fp32 sums.  A block's score is the maximum over the group, so that
// a KV head's query heads share one list and each listed block is read once.
// Selection.  The first and last blocks of the context always, then the
// highest scores, ties to the lowest index, in ascending order.
//
// All three are bound by memory (or by latency, for a few sequences): a key
// slab, a bounds row and a score are each read once.  Early start, as in the
// decode kernel: before they wait for the previous kernel they read lengths,
// tables and (bounds) the cache, which no kernel that releases early writes
// after its release (a fused step releases once its new rows are fenced).
// They let the next kernel launch as soon as their own wait is over: what they
// write (bounds, scores, lists) no kernel of this library reads before its own.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>

#include "host_util.h"
#include "pkv_common.cuh"

namespace pkv {

// ---------------------------------------------------------------------------
// packed minima and maxima of two 16-bit values; a NaN on either side stays
// ---------------------------------------------------------------------------
__device__ __forceinline__ uint32_t min2(uint32_t a, uint32_t b, F16) {
  uint32_t r;
  asm("min.NaN.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b, F16) {
  uint32_t r;
  asm("max.NaN.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t min2(uint32_t a, uint32_t b, BF16) {
  uint32_t r;
  asm("min.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b, BF16) {
  uint32_t r;
  asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// 16 bytes of a cache row -> packed 16-bit pairs (NP of them), exactly
template <typename KV>
struct RowChunk {
  static constexpr int kPairs = KV::kBytes == 2 ? 4 : 8;
  using type = std::conditional_t<KV::kBytes == 2, KV, F16>;   // element type of the pairs
  static __device__ __forceinline__ void unpack(const uint4& v, uint32_t* w) {
    const uint32_t x[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (KV::kBytes == 2) {
        w[i] = x[i];
      } else if constexpr (std::is_same<KV, E5M2>::value) {
        w[2 * i] = e5m2x2_to_f16x2(x[i]);
        w[2 * i + 1] = __byte_perm(x[i], 0u, 0x3424u);
      } else {
        asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, lo;\n\t"
            "cvt.rn.f16x2.e4m3x2 %1, hi;\n\t}"
            : "=r"(w[2 * i]), "=r"(w[2 * i + 1])
            : "r"(x[i]));
      }
    }
  }
};

// ---------------------------------------------------------------------------
// Two ways to deal a call's units (slabs, or tiles of blocks) to warps.
//   by sequence   the launch has max_units warps per sequence, and those past
//                 a sequence's own units leave at once: no set-up, but with
//                 mixed lengths most warps may be such.
//   flat          a grid that fills the GPU once; every thread block scans the
//                 sequences' unit counts into shared memory and each warp
//                 takes an equal run of consecutive units.
// Flat is taken when the launch by sequence would be more than kFlatWaves
// times the resident warps.  On GB300: bounds of 32 contexts of 2048..32768
// tokens (E4M3, 389 MB) 60.3 us flat, 111 by sequence; scores of 64 contexts of
// 1024..32768 (141 MB) 26.2 against 27.6, but with two of 131072 among 62 of
// 1000 (83 MB) 16.0 against 70.4; one step's bounds of 64 sequences stay by
// sequence (1.8 us).
// ---------------------------------------------------------------------------
constexpr int kFlatWaves = 2;
constexpr int kFlatMaxBatch = 900;               // whose counts fit in shared memory beside the stages

// cum[b] = units of the sequences before b, cum[batch] = all (whole block; ends synchronised)
template <int THREADS, typename F>
__device__ __forceinline__ void scan_units(int batch, int* cum, int* warp_sum, F&& units_of) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  int carry = 0;
  for (int b0 = 0; b0 < batch; b0 += THREADS) {
    const int b = b0 + tid;
    const int own = b < batch ? units_of(b) : 0;
    int x = own;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int u = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += u;
    }
    if (lane == 31) warp_sum[warp] = x;
    __syncthreads();
    int before = carry;
    for (int w = 0; w < THREADS / 32; ++w) {
      if (w < warp) before += warp_sum[w];
      carry += warp_sum[w];
    }
    if (b < batch) cum[b] = before + x - own;
    __syncthreads();
  }
  if (tid == 0) cum[batch] = carry;
  __syncthreads();
}

// the sequence that holds unit u: the last b with cum[b] <= u
__device__ __forceinline__ int unit_sequence(const int* cum, int batch, int u) {
  int lo = 0, hi = batch - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (cum[mid] <= u) lo = mid; else hi = mid - 1;
  }
  return lo;
}

struct BoundsParams {
  const unsigned char* k_cache;  // [NB, Hkv, 16, D]
  unsigned char* bounds;         // [NB, Hkv, 2, D] 16-bit
  const int32_t* block_tables;
  const int32_t* context_lens;
  const int32_t* new_lens;       // null: the whole context
  int32_t* err;
  int64_t num_blocks;
  int batch, n_kv_heads, max_blocks_per_seq;
  int max_touched;               // touched blocks of a sequence, at most
};

constexpr int kBoundsWarps = 8;

// the context of sequence b, how many of its tokens are new, and its touched
// blocks [first, last) (errors reported when report)
struct Touched {
  int ctx, first, last;
};
__device__ __forceinline__ Touched touched_blocks(const BoundsParams& p, int b, bool report) {
  int ctx = p.context_lens[b];
  int fresh = p.new_lens != nullptr ? p.new_lens[b] : INT32_MAX;
  const int64_t room = static_cast<int64_t>(p.max_blocks_per_seq) * kBlockSize;
  bool bad = ctx < 0 || ctx > room;
  ctx = static_cast<int>(min(static_cast<int64_t>(max(ctx, 0)), room));
  if (p.new_lens == nullptr) fresh = ctx;
  bad |= fresh < 0 || fresh > ctx;
  fresh = min(max(fresh, 0), ctx);
  Touched t;
  t.ctx = ctx;
  t.first = (ctx - fresh) / kBlockSize;
  t.last = fresh == 0 ? t.first : (ctx - 1) / kBlockSize + 1;
  if (t.last - t.first > p.max_touched) {   // more new tokens than max_new_len
    bad = true;
    t.last = t.first + p.max_touched;
  }
  if (bad && report) record_error(p.err, PKV_ERR_OOB);
  return t;
}

// One warp per (block, KV head) slab: a lane loads every (32 / LPR)-th row's
// 16-byte chunk, all of them at once, so a warp has a whole slab in flight (in
// the flat form kSlabs of them); the lanes of one chunk then meet by shuffles.
// Heads are the fastest index: consecutive slabs of a cache block.
template <typename KV, int D>
struct BoundsSlab {
  using C = RowChunk<KV>;
  using T = typename C::type;
  static constexpr int kRow = D * KV::kBytes;
  static constexpr int kLPR = kRow / 16;                  // lanes per row
  static constexpr int kRows = 32 / kLPR;                 // rows per load
  static constexpr int kLoads = kBlockSize / kRows;
  static constexpr int NP = C::kPairs;
  uint4 v[kLoads];

  __device__ __forceinline__ void load(const unsigned char* slab, int rows, int lane) {
    const unsigned char* src = slab + (lane % kLPR) * 16;
#pragma unroll
    for (int l = 0; l < kLoads; ++l) {
      // (a row past the context is replaced by row 0, which holds a token; from
      // L2, where a fused step that released this launch early has its new rows)
      const int r = l * kRows + lane / kLPR;
      v[l] = __ldcg(reinterpret_cast<const uint4*>(src + (r < rows ? r : 0) * kRow));
    }
  }
  template <typename OT>
  __device__ __forceinline__ void store(unsigned char* bounds, int lane, OT) {
    uint32_t lo[NP], hi[NP];
    C::unpack(v[0], lo);
#pragma unroll
    for (int x = 0; x < NP; ++x) hi[x] = lo[x];
#pragma unroll
    for (int l = 1; l < kLoads; ++l) {
      uint32_t w[NP];
      C::unpack(v[l], w);
#pragma unroll
      for (int x = 0; x < NP; ++x) {
        lo[x] = min2(lo[x], w[x], T{});
        hi[x] = max2(hi[x], w[x], T{});
      }
    }
    // Lanes that differ in `kLPR` hold the same columns.  The first exchange
    // also splits the work: the lower lanes go on with the minima, the upper
    // ones with the maxima.
    const bool up = (lane & kLPR) != 0;
#pragma unroll
    for (int x = 0; x < NP; ++x) {
      const uint32_t other = __shfl_xor_sync(0xffffffffu, up ? lo[x] : hi[x], kLPR);
      lo[x] = up ? max2(hi[x], other, T{}) : min2(lo[x], other, T{});
    }
#pragma unroll
    for (int m = 2 * kLPR; m < 32; m <<= 1)
#pragma unroll
      for (int x = 0; x < NP; ++x) {
        const uint32_t other = __shfl_xor_sync(0xffffffffu, lo[x], m);
        lo[x] = up ? max2(lo[x], other, T{}) : min2(lo[x], other, T{});
      }
    if (lane < 2 * kLPR) {
      unsigned char* dst = bounds + (up ? D * 2 : 0) + (lane % kLPR) * NP * 4;
#pragma unroll
      for (int x = 0; x < NP; x += 4) {
        uint32_t o[4];
#pragma unroll
        for (int y = 0; y < 4; ++y) {
          o[y] = lo[x + y];
          if constexpr (!std::is_same<T, OT>::value) {
            const float2 f = unpack2(o[y], T{});
            o[y] = pack2(f.x, f.y, OT{});
          }
        }
        *reinterpret_cast<uint4*>(dst + x * 4) = make_uint4(o[0], o[1], o[2], o[3]);
      }
    }
  }
};

template <typename KV, typename OT, int D>
__global__ void __launch_bounds__(kBoundsWarps * 32) block_bounds_kernel(const __grid_constant__ BoundsParams p) {
  using S = BoundsSlab<KV, D>;
  const int lane = threadIdx.x & 31;
  const int item = blockIdx.x * kBoundsWarps + static_cast<int>(threadIdx.x >> 5);
  if (item >= p.max_touched * p.n_kv_heads) {
    pdl_wait_and_release();
    return;
  }
  const int g = item % p.n_kv_heads, step = item / p.n_kv_heads;
  bool waited = false;
  for (int b = blockIdx.y; b < p.batch; b += gridDim.y) {
    const Touched t = touched_blocks(p, b, item == 0 && lane == 0);
    const int i = t.first + step;
    if (i >= t.last) continue;
    const int32_t id = p.block_tables[static_cast<int64_t>(b) * p.max_blocks_per_seq + i];
    if (id < 0 || id >= p.num_blocks) {
      if (g == 0 && lane == 0) record_error(p.err, PKV_ERR_OOB);
      continue;
    }
    const int64_t slab = static_cast<int64_t>(id) * p.n_kv_heads + g;
    S s;
    s.load(p.k_cache + slab * kBlockSize * S::kRow, min(kBlockSize, t.ctx - i * kBlockSize), lane);
    if (!waited) pdl_wait_and_release();
    waited = true;
    s.store(p.bounds + slab * 4 * D, lane, OT{});
  }
  if (!waited) pdl_wait_and_release();
}

template <typename KV, typename OT, int D>
__global__ void __launch_bounds__(kBoundsWarps * 32, 3) block_bounds_flat_kernel(const __grid_constant__ BoundsParams p) {
  using S = BoundsSlab<KV, D>;
  constexpr int kSlabs = 8 / S::kLoads;            // slabs in flight per warp: 4 KiB
  extern __shared__ int cum[];                     // [batch + 1] touched blocks
  __shared__ int warp_sum[kBoundsWarps];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  scan_units<kBoundsWarps * 32>(p.batch, cum, warp_sum, [&](int b) {
    const Touched t = touched_blocks(p, b, blockIdx.x == 0);
    return t.last - t.first;
  });
  const int64_t total = static_cast<int64_t>(cum[p.batch]) * p.n_kv_heads;
  const int64_t warps = static_cast<int64_t>(gridDim.x) * kBoundsWarps;
  const int64_t w = static_cast<int64_t>(blockIdx.x) * kBoundsWarps + warp;
  const int64_t end = (w + 1) * total / warps;
  bool waited = false;
  // 32 slabs at a time: each lane finds one, then the warp reduces them in turn
  for (int64_t s0 = w * total / warps; s0 < end; s0 += 32) {
    int64_t slab = -1;
    int rows = 0;
    if (s0 + lane < end) {
      const int blk = static_cast<int>((s0 + lane) / p.n_kv_heads), g = static_cast<int>((s0 + lane) % p.n_kv_heads);
      const int b = unit_sequence(cum, p.batch, blk);
      const Touched t = touched_blocks(p, b, false);
      const int i = t.first + (blk - cum[b]);
      const int32_t id = p.block_tables[static_cast<int64_t>(b) * p.max_blocks_per_seq + i];
      if (id >= 0 && id < p.num_blocks) {
        slab = static_cast<int64_t>(id) * p.n_kv_heads + g;
        rows = min(kBlockSize, t.ctx - i * kBlockSize);
      } else {
        record_error(p.err, PKV_ERR_OOB);
      }
    }
    const int n = static_cast<int>(min(static_cast<int64_t>(32), end - s0));
    for (int k = 0; k < n; k += kSlabs) {
      S s[kSlabs];
      int64_t at[kSlabs];
#pragma unroll
      for (int u = 0; u < kSlabs; ++u) {
        at[u] = __shfl_sync(0xffffffffu, slab, (k + u) & 31);
        const int r = __shfl_sync(0xffffffffu, rows, (k + u) & 31);
        if (k + u >= n) at[u] = -1;
        if (at[u] >= 0) s[u].load(p.k_cache + at[u] * kBlockSize * S::kRow, r, lane);
      }
      if (!waited) pdl_wait_and_release();
      waited = true;
#pragma unroll
      for (int u = 0; u < kSlabs; ++u)
        if (at[u] >= 0) s[u].store(p.bounds + at[u] * 4 * D, lane, OT{});
    }
  }
  if (!waited) pdl_wait_and_release();
}

struct ScoreParams {
  const unsigned char* q;        // [B, Hq, D]
  const unsigned char* bounds;   // [NB, Hkv, 2, D]
  const int32_t* block_tables;
  const int32_t* context_lens;
  const float* k_scale;          // [Hkv], or null
  float* scores;                 // [B, Hkv, max_blocks_per_seq]
  int32_t* err;
  unsigned long long wait_limit_ns;   // limit of each pipeline wait (flat form)
  int64_t num_blocks;
  int batch, n_q_heads, n_kv_heads, max_blocks_per_seq;
  int max_nblk;                  // ceil(max_context_len / 16), at most max_blocks_per_seq
  float scale;
};

constexpr int kScoreWarps = 4;

__device__ __forceinline__ void mma_16816(float* c, const uint32_t* a, uint32_t b0, uint32_t b1, BF16) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_16816(float* c, const uint32_t* a, uint32_t b0, uint32_t b1, F16) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// blocks of sequence b that are scored (errors reported when report)
__device__ __forceinline__ int scored_blocks(const ScoreParams& p, int b, bool report) {
  const int ctx = p.context_lens[b];
  const int nblk = ctx <= 0 ? 0 : static_cast<int>((static_cast<int64_t>(ctx) + kBlockSize - 1) / kBlockSize);
  if (report && (ctx < 0 || nblk > p.max_nblk)) record_error(p.err, PKV_ERR_OOB);
  return min(nblk, p.max_nblk);
}

// The product of one warp: 16 blocks of one (sequence, KV head).  Lane (r, c) =
// (lane / 4, lane % 4) holds rows r and r + 8 of the 16 and, of each row, the
// 16-byte chunks c, c + 4, ...: these are already the A fragments of two
// k-steps each, the product's k order being free (element 4 u + e of chunk
// 4 m + c is k = 2 c + e % 2 + 8 (e / 2) of step 2 m + u).  B takes q in the
// same order: min(q, 0) against lo, max(q, 0) against hi.  a(h, m): chunk
// 4 m + c of row r + 8 h (lo, then hi); q(m): chunk 4 m + c of head r.  Returns
// the two rows' maxima over the group's heads in s.
template <typename QT, int D, int G, typename FA, typename FQ>
__device__ __forceinline__ void score_product(int lane, FA&& a, FQ&& q, float* s) {
  constexpr int kChunks = D / 32;                   // 16-byte chunks of one bound per lane
  const int r4 = lane >> 2, q4 = lane & 3;
  float acc[2][4] = {};
#pragma unroll
  for (int m = 0; m < kChunks; ++m) {
    const uint4 qv = q(m);
    const uint32_t w[4] = {qv.x, qv.y, qv.z, qv.w};
#pragma unroll
    for (int part = 0; part < 2; ++part) {        // lo, then hi
      uint32_t bq[4];
#pragma unroll
      for (int e = 0; e < 4; ++e)
        bq[e] = r4 >= G ? 0u : part == 0 ? min2(w[e], 0u, QT{}) : max2(w[e], 0u, QT{});
      const uint4 x = a(0, part * kChunks + m), y = a(1, part * kChunks + m);
      const uint32_t a0[4] = {x.x, y.x, x.y, y.y}, a1[4] = {x.z, y.z, x.w, y.w};
      mma_16816(acc[part], a0, bq[0], bq[1], QT{});
      mma_16816(acc[part], a1, bq[2], bq[3], QT{});
    }
  }
  // columns 2 q4, 2 q4 + 1 are heads; the maximum over the group's G
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const float s0 = acc[0][2 * h] + acc[1][2 * h], s1 = acc[0][2 * h + 1] + acc[1][2 * h + 1];
    float x = 2 * q4 < G ? s0 : -INFINITY;
    if (2 * q4 + 1 < G) x = max_nan(x, s1);
    x = max_nan(x, __shfl_xor_sync(0xffffffffu, x, 1));
    s[h] = max_nan(x, __shfl_xor_sync(0xffffffffu, x, 2));
  }
}

// By sequence: a warp's rows straight from global memory, all in flight.
template <typename QT, int D, int G>
__global__ void __launch_bounds__(kScoreWarps * 32) block_scores_kernel(const __grid_constant__ ScoreParams p) {
  constexpr int kChunks = D / 32;
  const int lane = threadIdx.x & 31, r4 = lane >> 2, q4 = lane & 3;
  const int item = blockIdx.x * kScoreWarps + static_cast<int>(threadIdx.x >> 5);
  const int g = item % p.n_kv_heads, i0 = item / p.n_kv_heads * 16;
  bool waited = false;
  for (int b = blockIdx.y; b < p.batch; b += gridDim.y) {
    const int nblk = scored_blocks(p, b, item == 0 && lane == 0);
    if (i0 >= nblk) continue;
    // rows r4 and r4 + 8 (a row behind the context, or of a bad id, is not read)
    const int32_t* row = p.block_tables + static_cast<int64_t>(b) * p.max_blocks_per_seq;
    uint4 a[2][2 * kChunks];
    int32_t ids[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) ids[h] = i0 + r4 + 8 * h < nblk ? row[i0 + r4 + 8 * h] : -1;
    if (!waited) pdl_wait_and_release();   // (the bounds may be the previous kernel's)
    waited = true;
    bool live[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int i = i0 + r4 + 8 * h;
      const int32_t id = ids[h];
      live[h] = id >= 0 && id < p.num_blocks;
      if (i < nblk && !live[h] && q4 == 0 && g == 0) record_error(p.err, PKV_ERR_OOB);
      const unsigned char* src =
          p.bounds + ((live[h] ? static_cast<int64_t>(id) : 0) * p.n_kv_heads + g) * 2 * D * 2 + q4 * 16;
#pragma unroll
      for (int m = 0; m < 2 * kChunks; ++m)
        a[h][m] = live[h] ? *reinterpret_cast<const uint4*>(src + m * 64) : make_uint4(0, 0, 0, 0);
    }
    const unsigned char* qrow =
        p.q + ((static_cast<int64_t>(b) * p.n_q_heads) + g * G + (r4 < G ? r4 : 0)) * D * 2 + q4 * 16;
    float s[2];
    score_product<QT, D, G>(
        lane, [&](int h, int m) { return a[h][m]; },
        [&](int m) { return *reinterpret_cast<const uint4*>(qrow + m * 64); }, s);
    const float sc = p.scale * (p.k_scale ? p.k_scale[g] : 1.f);
    float* out = p.scores + (static_cast<int64_t>(b) * p.n_kv_heads + g) * p.max_blocks_per_seq + i0;
#pragma unroll
    for (int h = 0; h < 2; ++h)
      if (q4 == 0 && i0 + r4 + 8 * h < nblk) out[r4 + 8 * h] = live[h] ? s[h] * sc : -INFINITY;
  }
  if (!waited) pdl_wait_and_release();
}

// Flat: a persistent thread block takes units of `tile` blocks and up to
// kScoreHeads KV heads; one warp copies a unit's bounds into a ring of stages
// -- one 1-D bulk copy of up to 4 KiB per block, its heads being contiguous --
// with the unit's queries behind them, and 8 warps take its (16 blocks, head)
// products from there.  The bulk copies set the pace: a thread block gets one
// about every 185 clocks, which at 4 KiB each is this SM's share of HBM (half the
// heads per unit, 2 KiB, took twice as long, with 8 warps or 12).  Rows lie 64
// bytes past a multiple of 128 apart, so a quarter warp's 16-byte loads touch
// every bank once.
constexpr int kScoreConsumers = 8;
constexpr int kScoreThreads = (kScoreConsumers + 1) * 32;
constexpr int kScoreStages = 3;
constexpr int kScoreMaxTile = 128;
constexpr int kScoreStageBytes = 73 * 1024;       // three of them, and the counts, fit one SM

template <int D>
constexpr int kScoreHeads = 4096 / (4 * D);

struct ScoreUnit {
  int b, i0, g0, n;              // n blocks from i0 on of sequence b; n < 0: no more units
  uint32_t live[kScoreMaxTile / 32];
};

template <int D>
struct ScoreLayout {
  int heads, tile, row, q_off, stage;   // heads of a unit at most; bytes
  __host__ __device__ ScoreLayout(int n_kv_heads, int group) {
    heads = n_kv_heads < kScoreHeads<D> ? n_kv_heads : kScoreHeads<D>;
    while (16 * (heads * 4 * D + 64) + heads * group * D * 2 > kScoreStageBytes) heads = (heads + 1) / 2;
    row = heads * 4 * D + 64;
    const int q = heads * group * D * 2;
    tile = (kScoreStageBytes - q) / row / 16 * 16;
    tile = tile > kScoreMaxTile ? kScoreMaxTile : tile;
    q_off = tile * row;
    stage = (q_off + q + 127) / 128 * 128;
  }
  __host__ __device__ size_t bytes(int batch) const {
    return 128 + static_cast<size_t>(kScoreStages) * (stage + sizeof(ScoreUnit)) + 16 * kScoreStages +
           (2 * static_cast<size_t>(batch) + 1) * sizeof(int);
  }
};

template <typename QT, int D, int G>
__global__ void __launch_bounds__(kScoreThreads, 1) block_scores_flat_kernel(const __grid_constant__ ScoreParams p) {
  extern __shared__ unsigned char score_smem[];
  __shared__ int warp_sum[kScoreThreads / 32];
  const ScoreLayout<D> lay(p.n_kv_heads, G);
  unsigned char* ring = score_smem + ((128 - (smem_u32(score_smem) & 127)) & 127);
  ScoreUnit* units = reinterpret_cast<ScoreUnit*>(ring + static_cast<size_t>(kScoreStages) * lay.stage);
  uint64_t* full = reinterpret_cast<uint64_t*>(units + kScoreStages);
  uint64_t* empty = full + kScoreStages;
  int* cum = reinterpret_cast<int*>(empty + kScoreStages);   // [batch + 1] tiles
  int* scored = cum + p.batch + 1;                           // [batch] blocks
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (tid == 0) {
    for (int s = 0; s < kScoreStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], kScoreConsumers);
    }
    fence_mbar_init();
  }
  scan_units<kScoreThreads>(p.batch, cum, warp_sum, [&](int b) {
    scored[b] = scored_blocks(p, b, blockIdx.x == 0);
    return (scored[b] + lay.tile - 1) / lay.tile;
  });
  const int chunks = (p.n_kv_heads + lay.heads - 1) / lay.heads;
  const int64_t total = static_cast<int64_t>(cum[p.batch]) * chunks;

  if (warp == kScoreConsumers) {
    // ---- producer: stage s of unit k is its (k % stages)-th.  The next unit's
    // table entries are loaded before this one's stage is waited for and filled. ----
    const uint64_t pol = policy_evict_first();
    struct Next {
      int b, i0, g0, n;
      int32_t ids[kScoreMaxTile / 32];
    };
    auto fetch = [&](int64_t u) {
      Next x;
      x.n = -1;
      x.b = x.i0 = x.g0 = 0;
      if (u < total) {
        const int64_t t = u / chunks;
        x.g0 = static_cast<int>(u - t * chunks) * lay.heads;
        x.b = unit_sequence(cum, p.batch, static_cast<int>(t));
        x.i0 = (static_cast<int>(t) - cum[x.b]) * lay.tile;
        x.n = min(lay.tile, scored[x.b] - x.i0);
      }
      const int32_t* row = p.block_tables + static_cast<int64_t>(x.b) * p.max_blocks_per_seq + x.i0;
#pragma unroll
      for (int k = 0; k < kScoreMaxTile / 32; ++k) x.ids[k] = 32 * k + lane < x.n ? row[32 * k + lane] : -1;
      return x;
    };
    uint32_t k = 0;
    bool ok = true;
    Next cur = fetch(blockIdx.x);
    pdl_wait_and_release();   // (the bounds may be the previous kernel's)
    for (int64_t u = blockIdx.x; ok; u += gridDim.x, ++k) {
      const int s = k % kScoreStages;
      const Next nxt = fetch(u + gridDim.x);
      ok = k < kScoreStages || mbar_poll(&empty[s], (k / kScoreStages - 1) & 1, p.err, p.wait_limit_ns);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      ScoreUnit d;
      d.b = cur.b, d.i0 = cur.i0, d.g0 = cur.g0, d.n = cur.n;
      int n_live = 0;
#pragma unroll
      for (int x = 0; x < kScoreMaxTile / 32; ++x) {
        const bool live = cur.ids[x] >= 0 && cur.ids[x] < p.num_blocks;
        if (32 * x + lane < cur.n && !live) record_error(p.err, PKV_ERR_OOB);
        if (!live) cur.ids[x] = -1;
        d.live[x] = __ballot_sync(0xffffffffu, live);
        n_live += __popc(d.live[x]);
      }
      if (lane == 0) units[s] = d;
      if (d.n < 0) {
        if (lane == 0) mbar_arrive(&full[s]);
        break;
      }
      const int heads = min(lay.heads, p.n_kv_heads - d.g0);
      unsigned char* dst = ring + static_cast<size_t>(s) * lay.stage;
      if (lane == 0) {
        mbar_arrive_expect_tx(&full[s], (n_live * 4 * D + G * D * 2) * heads);
        bulk_g2s(dst + lay.q_off, p.q + (static_cast<int64_t>(d.b) * p.n_q_heads + d.g0 * G) * D * 2, heads * G * D * 2,
                 &full[s], pol);
      }
      __syncwarp();
#pragma unroll
      for (int x = 0; x < kScoreMaxTile / 32; ++x)
        if (cur.ids[x] >= 0)
          bulk_g2s(dst + (32 * x + lane) * lay.row,
                   p.bounds + (static_cast<int64_t>(cur.ids[x]) * p.n_kv_heads + d.g0) * 4 * D, heads * 4 * D, &full[s],
                   pol);
      __syncwarp();
      cur = nxt;
    }
    // The last units' copies land before the block's memory goes (bounded, with
    // the full limit): a consumer's wait for them may have run out.  Unit k is
    // the end marker, in a stage whose unit before was consumed, or the one
    // whose stage never came free.
    const unsigned long long deadline = global_ns() + kWaitLimitNs;
    for (uint32_t j = k < kScoreStages ? 0 : k - kScoreStages + (ok ? 1 : 0); j < k; ++j)
      mbar_wait_until(&full[j % kScoreStages], (j / kScoreStages) & 1, deadline);
    return;
  }
  // ---- consumers ----
  pdl_wait();
  const int r4 = lane >> 2, q4 = lane & 3;
  for (uint32_t k = 0;; ++k) {
    const int s = k % kScoreStages;
    if (!__all_sync(0xffffffffu, mbar_poll(&full[s], (k / kScoreStages) & 1, p.err, p.wait_limit_ns))) return;
    const ScoreUnit& d = units[s];
    const int n = d.n, b = d.b, i0 = d.i0, g0 = d.g0;
    if (n < 0) return;
    const int heads = min(lay.heads, p.n_kv_heads - g0);
    const unsigned char* src = ring + static_cast<size_t>(s) * lay.stage;
    for (int job = warp; job < heads * ((n + 15) / 16); job += kScoreConsumers) {
      const int h = job % heads, row0 = job / heads * 16;
      const unsigned char* arow = src + (row0 + r4) * lay.row + h * 4 * D + q4 * 16;
      const unsigned char* qrow = src + lay.q_off + (h * G + (r4 < G ? r4 : 0)) * D * 2 + q4 * 16;
      float sc2[2];
      score_product<QT, D, G>(
          lane, [&](int x, int m) { return *reinterpret_cast<const uint4*>(arow + 8 * x * lay.row + m * 64); },
          [&](int m) { return *reinterpret_cast<const uint4*>(qrow + m * 64); }, sc2);
      const float sc = p.scale * (p.k_scale ? p.k_scale[g0 + h] : 1.f);
      float* out = p.scores + (static_cast<int64_t>(b) * p.n_kv_heads + g0 + h) * p.max_blocks_per_seq + i0;
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const int i = row0 + r4 + 8 * x;   // (rows that were not copied hold older data: their sums are not used)
        if (q4 == 0 && i < n) out[i] = (d.live[i >> 5] >> (i & 31)) & 1u ? sc2[x] * sc : -INFINITY;
      }
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(&empty[s]);
  }
}

// the most that a flat launch asks for
constexpr int kFlatMaxSmem = 128 + kScoreStages * (kScoreStageBytes + static_cast<int>(sizeof(ScoreUnit))) +
                             16 * kScoreStages + (2 * kFlatMaxBatch + 1) * static_cast<int>(sizeof(int));
static_assert(kFlatMaxSmem + 64 <= 227 * 1024, "stages and counts fit one SM");

struct SelectParams {
  const float* scores;           // [B, Hkv, max_blocks_per_seq]
  const int32_t* context_lens;
  int32_t* selected;             // [B, Hkv, budget]
  int32_t* err;
  int n_kv_heads, max_blocks_per_seq, num_first, num_last, budget;
};

constexpr int kSelBits = 11;                        // histogram bits per pass
constexpr int kSelBins = 1 << kSelBits;

// order-preserving key of a score: -0 and +0 alike, every NaN above +inf
__device__ __forceinline__ uint32_t score_key(float s) {
  if (s != s) return 0xffffffffu;
  const uint32_t u = __float_as_uint(s + 0.f);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// One thread block per (sequence, KV head), its candidates' keys in shared
// memory (beyond 8192 of them, chunks of 8192 are read again in each step).
//   1. smallest and largest key: the candidates' spread is far below 32 bits,
//      so a histogram over it separates them at once;
//   2. with at least a candidate per thread and at most 256 to keep, a histogram
//      of the 512 threads' own maxima: the K-th highest of them is a lower bound
//      of the K-th highest candidate.  The candidates from it on, seldom many
//      more than K, are listed in order (of up to 8192), and if there are at
//      most 256 of them, each is ranked among them and the K highest are the
//      answer (11.3 to 10.3 us in the batch below);
//   else, among what is left:
//   3. 2048 bins over the bracket; the bin of the K-th highest candidate
//      becomes the bracket, until it holds at most 64 (or one key only);
//   4. the bracket's candidates are ranked among themselves: the K-th one's
//      key and index are the threshold (for one key shared by more than 64,
//      the index is found by counting them in order);
//   5. what lies above the threshold becomes a bit per candidate; a scan over
//      the words' bit counts gives each word its place in the list.
// Bound by instructions and barriers, not by the 5.6 MB of scores, and by a second
// wave (at 40 registers, 456 thread blocks fit the GPU): 512 pairs of
// 512 to 8192 blocks take 10.3 us (by steps 3 to 5 alone, before step 2: 14.1 with
// the keys in registers and every pass unrolled, which missed the instruction
// cache; 15.3 reading the scores again in each pass; 18 with 256 threads or 1024).
constexpr int kSelThreads = 512;
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kSelChunk = 8192;
constexpr int kSelRank = 64;
constexpr int kSelShort = 256;
static_assert(kSelRank <= kSelShort && kSelShort <= kSelThreads, "a thread per listed candidate");
static_assert(kSelChunk / 32 <= kSelThreads, "a thread per word of a chunk's bits");

__global__ void __launch_bounds__(kSelThreads) select_blocks_kernel(const __grid_constant__ SelectParams p) {
  extern __shared__ uint32_t keys[];                     // [min(max_blocks_per_seq, kSelChunk)]
  __shared__ uint32_t bins[kSelBins];
  __shared__ uint32_t red[2][kSelWarps];
  __shared__ uint32_t pick[3];
  __shared__ uint64_t listed[kSelShort];
  __shared__ uint32_t n_listed;
  __shared__ uint32_t bits[kSelChunk / 32];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t full = 0xffffffffu;
  const int64_t unit = blockIdx.x;
  const int b = static_cast<int>(unit / p.n_kv_heads);
  for (int x = tid; x < kSelBins; x += kSelThreads) bins[x] = 0;
  if (tid == 0) n_listed = 0;
  const int ctx = p.context_lens[b];
  pdl_wait_and_release();
  int n = ctx <= 0 ? 0 : static_cast<int>((static_cast<int64_t>(ctx) + kBlockSize - 1) / kBlockSize);
  if (ctx < 0 || n > p.max_blocks_per_seq) {
    if (tid == 0) record_error(p.err, PKV_ERR_OOB);
    n = min(n, p.max_blocks_per_seq);
  }
  int32_t* out = p.selected + unit * p.budget;
  if (n <= p.budget) {
    for (int i = tid; i < p.budget; i += kSelThreads) out[i] = i < n ? i : -1;
    return;
  }
  const int c0 = p.num_first, c1 = n - p.num_last;       // candidates [c0, c1)
  const float* scores = p.scores + unit * p.max_blocks_per_seq + c0;
  const uint32_t room = static_cast<uint32_t>(p.budget - p.num_first - p.num_last);
  uint32_t need = room;
  for (int i = tid; i < p.num_first; i += kSelThreads) out[i] = i;
  for (int i = tid; i < p.num_last; i += kSelThreads) out[p.budget - p.num_last + i] = c1 + i;
  if (need == 0) return;

  const int cand = c1 - c0;
  // f(key, candidate) over this thread's candidates; a thread reads only the
  // keys that it stored itself (in the pass over the scores, below)
  auto each = [&](auto&& f) {
    for (int from = 0; from < cand; from += kSelChunk) {
      const int m = min(kSelChunk, cand - from);
      if (cand > kSelChunk)
        for (int i = tid; i < m; i += kSelThreads) keys[i] = score_key(scores[from + i]);
#pragma unroll 8
      for (int i = tid; i < m; i += kSelThreads) f(keys[i], from + i);
    }
  };
  // inclusive sum over the threads before and including this one
  auto scan = [&](uint32_t own) {
    uint32_t incl = own;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t u = __shfl_up_sync(full, incl, o);
      if (lane >= o) incl += u;
    }
    if (lane == 31) red[0][warp] = incl;
    __syncthreads();
    return incl + __reduce_add_sync(full, lane < warp ? red[0][lane % kSelWarps] : 0u);
  };
  // the bin that holds the k-th highest of what was counted: pick = its index,
  // the rank within it and its count (ends synchronised)
  auto find_bin = [&](uint32_t k) {
    constexpr int kPer = kSelBins / kSelThreads;           // thread t owns the t-th group of bins from the top
    uint32_t sum = 0;
#pragma unroll
    for (int x = 0; x < kPer; ++x) sum += bins[kSelBins - 1 - (tid * kPer + x)];
    uint32_t before = scan(sum) - sum;
    if (before < k && k <= before + sum) {
      int x = 0;
      uint32_t c;
      while (k > before + (c = bins[kSelBins - 1 - (tid * kPer + x)])) {
        before += c;
        ++x;
      }
      pick[0] = static_cast<uint32_t>(kSelBins - 1 - (tid * kPer + x));
      pick[1] = k - before;
      pick[2] = c;
    }
    __syncthreads();
  };

  uint32_t lo = full, hi = 0u, own_max = 0u;
#pragma unroll 8
  for (int i = tid; i < cand; i += kSelThreads) {
    const uint32_t k = score_key(scores[i]);
    if (i < kSelChunk) keys[i] = k;
    lo = min(lo, k);
    own_max = max(own_max, k);
  }
  lo = __reduce_min_sync(full, lo);
  hi = __reduce_max_sync(full, own_max);
  if (lane == 0) {
    red[0][warp] = lo;
    red[1][warp] = hi;
  }
  __syncthreads();
  lo = __reduce_min_sync(full, red[0][lane % kSelWarps]);
  hi = __reduce_max_sync(full, red[1][lane % kSelWarps]);
  __syncthreads();

  // bracket: keys [base, base + span]; everything above it is kept, and of its
  // candidates (`inside` of them, once counted) the `need` highest
  uint32_t base = lo, span = hi - lo, inside = static_cast<uint32_t>(cand);
  auto shift_of = [&]() { return span == 0 ? 0 : max(0, 32 - __clz(span) - kSelBits); };
  auto clear_bins = [&]() {
    for (int x = tid; x < kSelBins; x += kSelThreads) bins[x] = 0;
    __syncthreads();
  };
  int32_t* dst = out + p.num_first;
  bool dirty = false;
  if (need <= kSelShort && cand >= kSelThreads) {
    const int shift = shift_of();
    atomicAdd(&bins[(own_max - base) >> shift], 1u);       // (every thread has candidates here)
    __syncthreads();
    find_bin(need);
    base += pick[0] << shift;
    span = hi - base;
    dirty = true;
  }
  if (dirty && cand <= kSelChunk) {
    // the candidates from base on, in order
#pragma unroll 4
    for (int i0 = warp * 32; i0 < cand; i0 += kSelThreads) {
      const int i = i0 + lane;
      const uint32_t mask = __ballot_sync(full, i < cand && keys[i] >= base);
      if (lane == 0) bits[i0 >> 5] = mask;
    }
    __syncthreads();
    uint32_t mask = 32 * tid < cand ? bits[tid] : 0u;
    const uint32_t own = __popc(mask);
    const uint32_t upto = scan(own);
    if (tid == kSelThreads - 1) pick[0] = upto;
    for (uint32_t at = upto - own; mask != 0 && at < kSelShort; ++at) {
      const uint32_t i = 32 * tid + __ffs(mask) - 1;
      // (higher key first, then lower index: one 64-bit order)
      listed[at] = (static_cast<uint64_t>(keys[i]) << 32) | (full - i);
      mask &= mask - 1;
    }
    __syncthreads();
    const int m = static_cast<int>(pick[0]);
    if (m <= kSelShort) {
      uint32_t above = 0;
      const uint64_t mine = tid < m ? listed[tid] : 0u;
      if (warp * 32 < m) {
#pragma unroll 8
        for (int x = 0; x < m; ++x) above += listed[x] > mine;
      }
      const bool keep = tid < m && above < need;
      const uint32_t kept = __ballot_sync(full, keep);
      if (lane == 0) red[1][warp] = __popc(kept);
      __syncthreads();
      const uint32_t before = __reduce_add_sync(full, lane < warp ? red[1][lane % kSelWarps] : 0u);
      const uint32_t at = before + __popc(kept & ((1u << lane) - 1));
      if (keep && at < room) dst[at] = c0 + static_cast<int>(full - static_cast<uint32_t>(mine));
      return;
    }
  }
  while (inside > kSelRank && span > 0) {
    const int shift = shift_of();
    if (dirty) clear_bins();
    dirty = true;
    each([&](uint32_t k, int) {
      if (k >= base && k - base <= span) atomicAdd(&bins[(k - base) >> shift], 1u);
    });
    __syncthreads();
    find_bin(need);
    base += pick[0] << shift;
    span = min((1u << shift) - 1, hi - base);
    need = pick[1];
    inside = pick[2];
  }

  // threshold: key t_key, and for that key candidates up to t_index
  uint32_t t_key = base;
  int t_index = cand;
  if (need < inside) {
    if (inside <= kSelRank) {
      each([&](uint32_t k, int i) {
        // (higher key first, then lower index: one 64-bit order)
        if (k >= base && k - base <= span) {
          const uint32_t at = atomicAdd(&n_listed, 1u);
          if (at < kSelRank) listed[at] = (static_cast<uint64_t>(k) << 32) | (full - static_cast<uint32_t>(i));
        }
      });
      __syncthreads();
      if (tid < static_cast<int>(inside)) {
        const uint64_t mine = listed[tid];
        uint32_t above = 0;
        for (uint32_t x = 0; x < inside; ++x) above += listed[x] > mine;
        if (above == need - 1) {
          pick[0] = static_cast<uint32_t>(mine >> 32);
          pick[1] = full - static_cast<uint32_t>(mine);
        }
      }
      __syncthreads();
      t_key = pick[0];
      t_index = static_cast<int>(pick[1]);
    } else {
      // one key, many candidates: the need-th of them in index order
      uint32_t seen = 0;
      for (int from = 0; from < cand; from += kSelThreads) {
        const int i = from + tid;
        const bool same = i < cand && score_key(scores[i]) == base;
        const uint32_t m = __ballot_sync(full, same);
        __syncthreads();
        if (lane == 0) red[0][warp] = __popc(m);
        __syncthreads();
        const uint32_t w = red[0][lane % kSelWarps];
        const uint32_t prior = seen + __reduce_add_sync(full, lane < warp ? w : 0u);
        seen += __reduce_add_sync(full, lane < kSelWarps ? w : 0u);
        if (same && prior + __popc(m & ((1u << lane) - 1)) == need - 1) pick[0] = static_cast<uint32_t>(i);
      }
      __syncthreads();
      t_index = static_cast<int>(pick[0]);
    }
  }

  uint32_t done = 0;                                       // kept in earlier chunks
  for (int from = 0; from < cand; from += kSelChunk) {
    const int m = min(kSelChunk, cand - from), words = (m + 31) / 32;
    if (cand > kSelChunk)
      for (int i = tid; i < m; i += kSelThreads) keys[i] = score_key(scores[from + i]);
    // (whole warps: word i / 32 holds the 32 candidates that a warp looks at together)
#pragma unroll 8
    for (int i0 = warp * 32; i0 < m; i0 += kSelThreads) {
      const int i = i0 + lane;
      const uint32_t k = i < m ? keys[i] : 0u;             // (0 is no score's key)
      const uint32_t mask = __ballot_sync(full, k > t_key || (k == t_key && from + i <= t_index));
      if (lane == 0) bits[i0 >> 5] = mask;
    }
    __syncthreads();
    uint32_t mask = tid < words ? bits[tid] : 0u;
    const uint32_t own = __popc(mask);
    const uint32_t upto = scan(own);
    for (uint32_t at = done + upto - own; mask != 0 && at < room; ++at) {
      dst[at] = c0 + from + 32 * tid + __ffs(mask) - 1;
      mask &= mask - 1;
    }
    if (from + kSelChunk < cand) {
      if (tid == kSelThreads - 1) pick[0] = upto;
      __syncthreads();
      done += pick[0];
      __syncthreads();
    }
  }
}

namespace {

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

constexpr int kMaxGridYZ = 65535;

// Thread blocks of the flat form (0: by sequence), for `items` warps of work at
// most: 24 warps per SM, with 4 to 8 KiB each in flight.  (Its unit counts are
// 32-bit: by sequence beyond.)
bool flat_grid(int64_t items, int warps_per_block, int batch, int* blocks) {
  int dev = 0, sms = 0;
  if (cuda_failed(cudaGetDevice(&dev), "cudaGetDevice") ||
      cuda_failed(cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev), "cudaDeviceGetAttribute"))
    return false;
  const int resident = sms * 24 / warps_per_block;
  *blocks = (items > static_cast<int64_t>(kFlatWaves) * resident * warps_per_block && items <= INT32_MAX &&
             batch <= kFlatMaxBatch)
                ? resident
                : 0;
  return true;
}

template <typename P>
pkv_status launch_flat(void (*kern)(P), int threads, int blocks, const P& p, size_t smem, cudaStream_t stream,
                       const char* what) {
  // (the same limit each time: another thread's call may come between this and the launch)
  if (smem > 32 * 1024 &&
      cuda_failed(cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kFlatMaxSmem),
                  "cudaFuncSetAttribute"))
    return PKV_ERR_CUDA;
  return cuda_failed(launch_pdl(kern, dim3(static_cast<unsigned>(blocks)), dim3(static_cast<unsigned>(threads)), smem,
                                stream, p),
                     what)
             ? PKV_ERR_CUDA
             : PKV_OK;
}

template <typename KV, typename OT>
pkv_status launch_bounds(const BoundsParams& p, int head_dim, cudaStream_t stream) {
  const int64_t items = static_cast<int64_t>(p.max_touched) * p.n_kv_heads;
  int resident = 0;
  if (!flat_grid(items * p.batch, kBoundsWarps, p.batch, &resident)) return PKV_ERR_CUDA;
  if (resident > 0) {
    auto kern = head_dim == 64 ? block_bounds_flat_kernel<KV, OT, 64> : block_bounds_flat_kernel<KV, OT, 128>;
    return launch_flat(kern, kBoundsWarps * 32, resident, p, (static_cast<size_t>(p.batch) + 1) * sizeof(int), stream,
                       "block_bounds_flat_kernel launch");
  }
  auto kern = head_dim == 64 ? block_bounds_kernel<KV, OT, 64> : block_bounds_kernel<KV, OT, 128>;
  const dim3 grid(static_cast<unsigned>((items + kBoundsWarps - 1) / kBoundsWarps),
                  static_cast<unsigned>(std::min(p.batch, kMaxGridYZ)));
  return cuda_failed(launch_pdl(kern, grid, dim3(kBoundsWarps * 32), 0, stream, p), "block_bounds_kernel launch")
             ? PKV_ERR_CUDA
             : PKV_OK;
}

// kv: 0 = 16-bit (dtype), 1 = E4M3, 2 = E5M2 (bounds in dtype)
pkv_status bounds_common(int kv, const void* k_cache, const int32_t* block_tables, const int32_t* context_lens,
                         const int32_t* new_lens, int max_new_len, int batch, int num_kv_heads, int head_dim,
                         int block_size, int max_blocks_per_seq, int64_t num_blocks, void* bounds, pkv_dtype dtype,
                         int32_t* err_flag, void* stream) {
  if (batch < 0 || num_kv_heads <= 0 || max_blocks_per_seq <= 0 || num_blocks < 0 || max_new_len < 0)
    return PKV_ERR_INVALID_ARG;
  if (dtype != PKV_F16 && dtype != PKV_BF16) return PKV_ERR_INVALID_ARG;
  if (block_size != kBlockSize || (head_dim != 64 && head_dim != 128)) return PKV_ERR_UNSUPPORTED;
  if (batch == 0 || max_new_len == 0) return PKV_OK;
  if (!k_cache || !block_tables || !context_lens || !bounds) return PKV_ERR_INVALID_ARG;
  if (!aligned16(k_cache) || !aligned16(bounds)) return PKV_ERR_INVALID_ARG;
  // n tokens that end anywhere in a block touch at most this many blocks
  // (a whole context starts at its first block's first row)
  const int64_t touched = new_lens == nullptr ? (static_cast<int64_t>(max_new_len) + kBlockSize - 1) / kBlockSize
                                              : (static_cast<int64_t>(max_new_len) + kBlockSize - 2) / kBlockSize + 1;
  const int64_t max_touched = std::min<int64_t>(touched, max_blocks_per_seq);
  if (max_touched * num_kv_heads > INT32_MAX - 32) return PKV_ERR_UNSUPPORTED;
  BoundsParams p{};
  p.k_cache = static_cast<const unsigned char*>(k_cache);
  p.bounds = static_cast<unsigned char*>(bounds);
  p.block_tables = block_tables;
  p.context_lens = context_lens;
  p.new_lens = new_lens;
  p.err = err_flag;
  p.num_blocks = num_blocks;
  p.batch = batch;
  p.n_kv_heads = num_kv_heads;
  p.max_blocks_per_seq = max_blocks_per_seq;
  p.max_touched = static_cast<int>(max_touched);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (dtype == PKV_F16)
    return kv == 0 ? launch_bounds<F16, F16>(p, head_dim, s)
         : kv == 1 ? launch_bounds<E4M3, F16>(p, head_dim, s)
                   : launch_bounds<E5M2, F16>(p, head_dim, s);
  return kv == 0 ? launch_bounds<BF16, BF16>(p, head_dim, s)
       : kv == 1 ? launch_bounds<E4M3, BF16>(p, head_dim, s)
                 : launch_bounds<E5M2, BF16>(p, head_dim, s);
}

template <typename QT, int D>
pkv_status launch_scores(const ScoreParams& p, int group, cudaStream_t stream) {
  const int64_t items = static_cast<int64_t>((p.max_nblk + 15) / 16) * p.n_kv_heads;
  int resident = 0;
  if (!flat_grid(items * p.batch, kScoreWarps, p.batch, &resident)) return PKV_ERR_CUDA;
  if (resident > 0) {
    auto kern = group == 1   ? block_scores_flat_kernel<QT, D, 1>
                : group == 2 ? block_scores_flat_kernel<QT, D, 2>
                : group == 4 ? block_scores_flat_kernel<QT, D, 4>
                             : block_scores_flat_kernel<QT, D, 8>;
    // (one thread block per SM)
    return launch_flat(kern, kScoreThreads, resident * kScoreWarps / 24, p,
                       ScoreLayout<D>(p.n_kv_heads, group).bytes(p.batch), stream, "block_scores_flat_kernel launch");
  }
  auto kern = group == 1   ? block_scores_kernel<QT, D, 1>
              : group == 2 ? block_scores_kernel<QT, D, 2>
              : group == 4 ? block_scores_kernel<QT, D, 4>
                           : block_scores_kernel<QT, D, 8>;
  const dim3 grid(static_cast<unsigned>((items + kScoreWarps - 1) / kScoreWarps),
                  static_cast<unsigned>(std::min(p.batch, kMaxGridYZ)));
  return cuda_failed(launch_pdl(kern, grid, dim3(kScoreWarps * 32), 0, stream, p), "block_scores_kernel launch")
             ? PKV_ERR_CUDA
             : PKV_OK;
}

}  // namespace
}  // namespace pkv

using namespace pkv;

extern "C" pkv_status pkv_kv_block_bounds(const void* k_cache, const int32_t* block_tables,
                                          const int32_t* context_lens, const int32_t* new_lens, int max_new_len,
                                          int batch, int num_kv_heads, int head_dim, int block_size,
                                          int max_blocks_per_seq, int64_t num_blocks, void* bounds, pkv_dtype dtype,
                                          int32_t* err_flag, void* stream) {
  return bounds_common(0, k_cache, block_tables, context_lens, new_lens, max_new_len, batch, num_kv_heads, head_dim,
                       block_size, max_blocks_per_seq, num_blocks, bounds, dtype, err_flag, stream);
}

extern "C" pkv_status pkv_kv_block_bounds_fp8(const uint8_t* k_cache, const int32_t* block_tables,
                                              const int32_t* context_lens, const int32_t* new_lens, int max_new_len,
                                              int batch, int num_kv_heads, int head_dim, int block_size,
                                              int max_blocks_per_seq, int64_t num_blocks, void* bounds,
                                              pkv_dtype bounds_dtype, int32_t* err_flag, void* stream) {
  return bounds_common(1, k_cache, block_tables, context_lens, new_lens, max_new_len, batch, num_kv_heads, head_dim,
                       block_size, max_blocks_per_seq, num_blocks, bounds, bounds_dtype, err_flag, stream);
}

extern "C" pkv_status pkv_kv_block_bounds_e5m2(const uint8_t* k_cache, const int32_t* block_tables,
                                               const int32_t* context_lens, const int32_t* new_lens, int max_new_len,
                                               int batch, int num_kv_heads, int head_dim, int block_size,
                                               int max_blocks_per_seq, int64_t num_blocks, void* bounds,
                                               pkv_dtype bounds_dtype, int32_t* err_flag, void* stream) {
  return bounds_common(2, k_cache, block_tables, context_lens, new_lens, max_new_len, batch, num_kv_heads, head_dim,
                       block_size, max_blocks_per_seq, num_blocks, bounds, bounds_dtype, err_flag, stream);
}

extern "C" pkv_status pkv_block_scores(const void* q, const void* bounds, const int32_t* block_tables,
                                       const int32_t* context_lens, const float* k_scale, int batch, int num_q_heads,
                                       int num_kv_heads, int head_dim, int block_size, int max_blocks_per_seq,
                                       int64_t num_blocks, int max_context_len, float scale, float* scores,
                                       pkv_dtype dtype, int32_t* err_flag, void* stream) {
  if (batch < 0 || num_q_heads <= 0 || num_kv_heads <= 0 || max_blocks_per_seq <= 0 || num_blocks < 0 ||
      max_context_len < 0 || !std::isfinite(scale) || scale < 0.f)
    return PKV_ERR_INVALID_ARG;
  if (dtype != PKV_F16 && dtype != PKV_BF16) return PKV_ERR_INVALID_ARG;
  if (num_q_heads % num_kv_heads) return PKV_ERR_INVALID_ARG;
  if (block_size != kBlockSize || (head_dim != 64 && head_dim != 128)) return PKV_ERR_UNSUPPORTED;
  const int group = num_q_heads / num_kv_heads;
  if (group != 1 && group != 2 && group != 4 && group != 8) return PKV_ERR_UNSUPPORTED;
  if ((static_cast<int64_t>(max_blocks_per_seq) + 15) / 16 * num_kv_heads > INT32_MAX) return PKV_ERR_UNSUPPORTED;
  if (batch == 0 || max_context_len == 0) return PKV_OK;
  if (!q || !bounds || !block_tables || !context_lens || !scores) return PKV_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(bounds)) return PKV_ERR_INVALID_ARG;
  ScoreParams p{};
  p.q = static_cast<const unsigned char*>(q);
  p.bounds = static_cast<const unsigned char*>(bounds);
  p.block_tables = block_tables;
  p.context_lens = context_lens;
  p.k_scale = k_scale;
  p.scores = scores;
  p.err = err_flag;
  p.wait_limit_ns = wait_limit_ns();
  p.num_blocks = num_blocks;
  p.batch = batch;
  p.n_q_heads = num_q_heads;
  p.n_kv_heads = num_kv_heads;
  p.max_blocks_per_seq = max_blocks_per_seq;
  p.max_nblk = static_cast<int>(
      std::min<int64_t>((static_cast<int64_t>(max_context_len) + kBlockSize - 1) / kBlockSize, max_blocks_per_seq));
  p.scale = scale;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (dtype == PKV_F16)
    return head_dim == 64 ? launch_scores<F16, 64>(p, group, s) : launch_scores<F16, 128>(p, group, s);
  return head_dim == 64 ? launch_scores<BF16, 64>(p, group, s) : launch_scores<BF16, 128>(p, group, s);
}

extern "C" pkv_status pkv_select_blocks(const float* scores, const int32_t* context_lens, int batch,
                                        int num_kv_heads, int block_size, int max_blocks_per_seq, int num_first,
                                        int num_last, int budget, int32_t* selected, int32_t* err_flag,
                                        void* stream) {
  if (batch < 0 || num_kv_heads <= 0 || max_blocks_per_seq <= 0 || num_first < 0 || num_last < 0 || budget <= 0 ||
      static_cast<int64_t>(num_first) + num_last > budget)
    return PKV_ERR_INVALID_ARG;
  if (block_size != kBlockSize) return PKV_ERR_UNSUPPORTED;
  if (batch == 0) return PKV_OK;
  if (!scores || !context_lens || !selected) return PKV_ERR_INVALID_ARG;
  const int64_t units = static_cast<int64_t>(batch) * num_kv_heads;
  if (units > INT32_MAX) return PKV_ERR_UNSUPPORTED;
  SelectParams p{scores, context_lens, selected, err_flag, num_kv_heads, max_blocks_per_seq, num_first, num_last,
                 budget};
  const size_t smem = sizeof(uint32_t) * std::min(max_blocks_per_seq, kSelChunk);
  const cudaError_t e = launch_pdl(select_blocks_kernel, dim3(static_cast<unsigned>(units)), dim3(kSelThreads), smem,
                                   static_cast<cudaStream_t>(stream), p);
  return cuda_failed(e, "select_blocks_kernel launch") ? PKV_ERR_CUDA : PKV_OK;
}

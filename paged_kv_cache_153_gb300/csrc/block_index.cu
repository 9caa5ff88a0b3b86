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
// slab, a bounds row and a score are each read once.
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

struct BoundsParams {
  const unsigned char* k_cache;  // [NB, Hkv, 16, D]
  unsigned char* bounds;         // [NB, Hkv, 2, D] 16-bit
  const int32_t* block_tables;
  const int32_t* context_lens;
  const int32_t* new_lens;       // null: the whole context
  int32_t* err;
  int64_t num_blocks;
  int batch, n_kv_heads, max_blocks_per_seq;
  int items;                     // (touched blocks per sequence at most) x KV heads
};

constexpr int kBoundsWarps = 8;

// One warp per (block, KV head) slab: a lane loads every (32 / LPR)-th row's
// 16-byte chunk, all of them at once, so a warp has its whole slab in flight;
// the lanes of one chunk then meet by shuffles.  Heads are the fastest index:
// a thread block reads a cache block's consecutive slabs.
template <typename KV, typename OT, int D>
__global__ void __launch_bounds__(kBoundsWarps * 32) block_bounds_kernel(const __grid_constant__ BoundsParams p) {
  using C = RowChunk<KV>;
  using T = typename C::type;
  constexpr int kRow = D * KV::kBytes;
  constexpr int kLPR = kRow / 16;                  // lanes per row
  constexpr int kRows = 32 / kLPR;                 // rows per load
  constexpr int kLoads = kBlockSize / kRows;
  constexpr int NP = C::kPairs;
  const int lane = threadIdx.x & 31;
  const int item = blockIdx.x * kBoundsWarps + static_cast<int>(threadIdx.x >> 5);
  pdl_wait();   // (writes the bounds: no early release of the next launch)
  if (item >= p.items) return;
  const int g = item % p.n_kv_heads, step = item / p.n_kv_heads;
  for (int b = blockIdx.y; b < p.batch; b += gridDim.y) {
    int ctx = p.context_lens[b];
    if (ctx < 0 || ctx > static_cast<int64_t>(p.max_blocks_per_seq) * kBlockSize) {
      if (item == 0 && lane == 0) record_error(p.err, PKV_ERR_OOB);
      ctx = ctx < 0 ? 0 : p.max_blocks_per_seq * kBlockSize;
    }
    int fresh = ctx;
    if (p.new_lens != nullptr) {
      fresh = p.new_lens[b];
      if (fresh < 0 || fresh > ctx) {
        if (item == 0 && lane == 0) record_error(p.err, PKV_ERR_OOB);
        fresh = fresh < 0 ? 0 : ctx;
      }
    }
    const int first = (ctx - fresh) / kBlockSize, last = (ctx + kBlockSize - 1) / kBlockSize;
    if (item == 0 && lane == 0 && fresh > 0 && last - first > p.items / p.n_kv_heads)
      record_error(p.err, PKV_ERR_OOB);   // more new tokens than max_new_len
    const int i = first + step;
    if (fresh == 0 || i >= last) continue;
    const int32_t id = p.block_tables[static_cast<int64_t>(b) * p.max_blocks_per_seq + i];
    if (id < 0 || id >= p.num_blocks) {
      if (g == 0 && lane == 0) record_error(p.err, PKV_ERR_OOB);
      continue;
    }
    const int rows = min(kBlockSize, ctx - i * kBlockSize);
    const int64_t slab = static_cast<int64_t>(id) * p.n_kv_heads + g;
    const unsigned char* src = p.k_cache + slab * kBlockSize * kRow + (lane % kLPR) * 16;
    uint4 v[kLoads];
#pragma unroll
    for (int l = 0; l < kLoads; ++l) {
      // (a row past the context is replaced by row 0, which holds a token)
      const int r = l * kRows + lane / kLPR;
      v[l] = *reinterpret_cast<const uint4*>(src + (r < rows ? r : 0) * kRow);
    }
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
#pragma unroll
    for (int m = kLPR; m < 32; m <<= 1)
#pragma unroll
      for (int x = 0; x < NP; ++x) {
        lo[x] = min2(lo[x], __shfl_xor_sync(0xffffffffu, lo[x], m), T{});
        hi[x] = max2(hi[x], __shfl_xor_sync(0xffffffffu, hi[x], m), T{});
      }
    if (lane < 2 * kLPR) {
      const bool up = lane >= kLPR;
      unsigned char* dst = p.bounds + (slab * 2 + (up ? 1 : 0)) * D * 2 + (lane % kLPR) * NP * 4;
#pragma unroll
      for (int x = 0; x < NP; x += 4) {
        uint32_t o[4];
#pragma unroll
        for (int y = 0; y < 4; ++y) {
          o[y] = up ? hi[x + y] : lo[x + y];
          if constexpr (!std::is_same<T, OT>::value) {
            const float2 f = unpack2(o[y], T{});
            o[y] = pack2(f.x, f.y, OT{});
          }
        }
        *reinterpret_cast<uint4*>(dst + x * 4) = make_uint4(o[0], o[1], o[2], o[3]);
      }
    }
  }
}

struct ScoreParams {
  const unsigned char* q;        // [B, Hq, D]
  const unsigned char* bounds;   // [NB, Hkv, 2, D]
  const int32_t* block_tables;
  const int32_t* context_lens;
  const float* k_scale;          // [Hkv], or null
  float* scores;                 // [B, Hkv, max_blocks_per_seq]
  int32_t* err;
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

// One warp per (sequence, KV head, 16 blocks).  Lane (r, c) = (lane / 4,
// lane % 4) holds rows r and r + 8 of the 16 and, of each row, the 16-byte
// chunks c, c + 4, ...: straight from global memory, all in flight, and
// already the A fragments of two k-steps each, the product's k order being
// free (element 4 u + e of chunk 4 m + c is k = 2 c + e % 2 + 8 (e / 2) of
// step 2 m + u).  B takes q in the same order: min(q, 0) against lo,
// max(q, 0) against hi.
template <typename QT, int D, int G>
__global__ void __launch_bounds__(kScoreWarps * 32) block_scores_kernel(const __grid_constant__ ScoreParams p) {
  constexpr int kChunks = D / 32;                   // 16-byte chunks of one bound per lane
  const int lane = threadIdx.x & 31, r4 = lane >> 2, q4 = lane & 3;
  const int tile = blockIdx.x * kScoreWarps + static_cast<int>(threadIdx.x >> 5);
  const int g = blockIdx.y;
  pdl_wait();   // (writes the scores: no early release of the next launch)
  for (int b = blockIdx.z; b < p.batch; b += gridDim.z) {
    const int ctx = p.context_lens[b];
    int nblk = ctx <= 0 ? 0 : static_cast<int>((static_cast<int64_t>(ctx) + kBlockSize - 1) / kBlockSize);
    if (ctx < 0 || nblk > p.max_nblk) {
      if (tile == 0 && g == 0 && lane == 0) record_error(p.err, PKV_ERR_OOB);
      nblk = min(nblk, p.max_nblk);
    }
    const int i0 = tile * 16;
    if (i0 >= nblk) continue;
    // rows r4 and r4 + 8 (a row behind the context, or of a bad id, is not read)
    const int32_t* row = p.block_tables + static_cast<int64_t>(b) * p.max_blocks_per_seq;
    uint4 a[2][2 * kChunks];
    bool live[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int i = i0 + r4 + 8 * h;
      const int32_t id = i < nblk ? row[i] : -1;
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
    float acc[2][4] = {};
#pragma unroll
    for (int m = 0; m < kChunks; ++m) {
      const uint4 qv = *reinterpret_cast<const uint4*>(qrow + m * 64);
      const uint32_t w[4] = {qv.x, qv.y, qv.z, qv.w};
#pragma unroll
      for (int part = 0; part < 2; ++part) {        // lo, then hi
        uint32_t bq[4];
#pragma unroll
        for (int e = 0; e < 4; ++e)
          bq[e] = r4 >= G ? 0u : part == 0 ? min2(w[e], 0u, QT{}) : max2(w[e], 0u, QT{});
        const uint4 &x = a[0][part * kChunks + m], &y = a[1][part * kChunks + m];
        const uint32_t a0[4] = {x.x, y.x, x.y, y.y}, a1[4] = {x.z, y.z, x.w, y.w};
        mma_16816(acc[part], a0, bq[0], bq[1], QT{});
        mma_16816(acc[part], a1, bq[2], bq[3], QT{});
      }
    }
    // columns 2 q4, 2 q4 + 1 are heads; the maximum over the group's G
    const float sc = p.scale * (p.k_scale ? p.k_scale[g] : 1.f);
    float* out = p.scores + (static_cast<int64_t>(b) * p.n_kv_heads + g) * p.max_blocks_per_seq + i0;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const float s0 = acc[0][2 * h] + acc[1][2 * h], s1 = acc[0][2 * h + 1] + acc[1][2 * h + 1];
      float s = 2 * q4 < G ? s0 : -INFINITY;
      if (2 * q4 + 1 < G) s = max_nan(s, s1);
      s = max_nan(s, __shfl_xor_sync(0xffffffffu, s, 1));
      s = max_nan(s, __shfl_xor_sync(0xffffffffu, s, 2));
      if (q4 == 0 && i0 + r4 + 8 * h < nblk) out[r4 + 8 * h] = live[h] ? s * sc : -INFINITY;
    }
  }
}

struct SelectParams {
  const float* scores;           // [B, Hkv, max_blocks_per_seq]
  const int32_t* context_lens;
  int32_t* selected;             // [B, Hkv, budget]
  int32_t* err;
  int n_kv_heads, max_blocks_per_seq, num_first, num_last, budget;
};

constexpr int kSelThreads = 512;
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kSelBits = 11;                        // histogram bits per pass
constexpr int kSelBins = 1 << kSelBits;

// order-preserving key of a score: -0 and +0 alike, every NaN above +inf
__device__ __forceinline__ uint32_t score_key(float s) {
  if (s != s) return 0xffffffffu;
  const uint32_t u = __float_as_uint(s + 0.f);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// One thread block per (sequence, KV head).  The threshold of the K-th highest
// candidate is found by a radix search over the keys between the candidates'
// smallest and largest (their spread is far below the full 32 bits, so the
// first histogram already separates them): each pass counts the keys of the
// current bracket in 2048 bins and narrows it to the bin that holds the K-th.
// Then every warp walks its share of the indices twice, once to count what it
// keeps and once, after a scan over the warps, to write it.  Scores are read
// again in each pass: 32 KiB of a 131072-token context stay in L1.
__global__ void __launch_bounds__(kSelThreads) select_blocks_kernel(const __grid_constant__ SelectParams p) {
  __shared__ uint32_t bins[kSelBins];
  __shared__ uint32_t red[2][kSelWarps];
  __shared__ uint32_t pick[3];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int64_t unit = blockIdx.x;
  const int b = static_cast<int>(unit / p.n_kv_heads);
  pdl_wait();   // (writes the lists: no early release of the next launch)
  const int ctx = p.context_lens[b];
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
  const float* scores = p.scores + unit * p.max_blocks_per_seq;
  const int c0 = p.num_first, c1 = n - p.num_last;       // candidates [c0, c1)
  uint32_t need = static_cast<uint32_t>(p.budget - p.num_first - p.num_last);
  for (int i = tid; i < p.num_first; i += kSelThreads) out[i] = i;
  for (int i = tid; i < p.num_last; i += kSelThreads) out[p.budget - p.num_last + i] = c1 + i;
  if (need == 0) return;
  // smallest and largest candidate key
  uint32_t lo = 0xffffffffu, hi = 0u;
  for (int i = c0 + tid; i < c1; i += kSelThreads) {
    const uint32_t k = score_key(scores[i]);
    lo = min(lo, k);
    hi = max(hi, k);
  }
  lo = __reduce_min_sync(0xffffffffu, lo);
  hi = __reduce_max_sync(0xffffffffu, hi);
  if (lane == 0) {
    red[0][warp] = lo;
    red[1][warp] = hi;
  }
  __syncthreads();
  for (int w = 0; w < kSelWarps; ++w) {
    lo = min(lo, red[0][w]);
    hi = max(hi, red[1][w]);
  }
  // bracket [base, base + 2^shift): the need-th highest candidate lies in it,
  // and everything above it is kept
  uint32_t base = lo;
  int shift = hi == lo ? 0 : 32 - __clz(hi - lo);
  while (shift > 0) {
    const int bits = min(shift, kSelBits);
    const uint32_t span = shift == 32 ? 0xffffffffu : (1u << shift) - 1;   // last offset of the bracket
    shift -= bits;
    __syncthreads();
    for (int x = tid; x < kSelBins; x += kSelThreads) bins[x] = 0;
    __syncthreads();
    for (int i = c0 + tid; i < c1; i += kSelThreads) {
      const uint32_t k = score_key(scores[i]);
      if (k >= base && k - base <= span) atomicAdd(&bins[(k - base) >> shift], 1u);
    }
    __syncthreads();
    // thread t owns bins [4 t', 4 t' + 4) from the top: t' = threads - 1 - t
    constexpr int kPer = kSelBins / kSelThreads;
    uint32_t cnt[kPer], sum = 0;
#pragma unroll
    for (int x = 0; x < kPer; ++x) {
      cnt[x] = bins[kSelBins - 1 - (tid * kPer + x)];
      sum += cnt[x];
    }
    uint32_t incl = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t u = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += u;
    }
    if (lane == 31) red[0][warp] = incl;
    __syncthreads();
    uint32_t before = incl - sum;                          // candidates above this thread's bins
    for (int w = 0; w < warp; ++w) before += red[0][w];
    if (before < need && need <= before + sum) {
#pragma unroll
      for (int x = 0; x < kPer; ++x) {
        if (before < need && need <= before + cnt[x]) {
          pick[0] = static_cast<uint32_t>(kSelBins - 1 - (tid * kPer + x));
          pick[1] = need - before;
          pick[2] = cnt[x];
          before += cnt[x];
          break;
        }
        before += cnt[x];
      }
    }
    __syncthreads();
    base += pick[0] << shift;
    need = pick[1];
    if (need == pick[2]) break;                            // the whole bin is kept
  }
  const uint32_t span = shift == 32 ? 0xffffffffu : (1u << shift) - 1;
  // keep keys above the bracket, and of the bracket the `need` lowest indices
  const int per = ((c1 - c0 + kSelWarps - 1) / kSelWarps + 31) & ~31;
  const int w0 = c0 + warp * per, w1 = min(c1, w0 + per);
  uint32_t above = 0, inside = 0;
  for (int i = w0 + lane; i < w1; i += 32) {
    const uint32_t k = score_key(scores[i]);
    above += k >= base && k - base > span;
    inside += k >= base && k - base <= span;
  }
  above = __reduce_add_sync(0xffffffffu, above);
  inside = __reduce_add_sync(0xffffffffu, inside);
  __syncthreads();
  if (lane == 0) {
    red[0][warp] = above;
    red[1][warp] = inside;
  }
  __syncthreads();
  uint32_t seen = 0, at = 0;                               // bracket keys, kept keys before this warp
  for (int w = 0; w < warp; ++w) {
    const uint32_t in = red[1][w], left = need > seen ? need - seen : 0u;
    at += red[0][w] + min(in, left);
    seen += in;
  }
  int32_t* dst = out + p.num_first;
  const uint32_t below_me = (1u << lane) - 1;
  for (int i0 = w0; i0 < w1; i0 += 32) {
    const int i = i0 + lane;
    const uint32_t k = i < w1 ? score_key(scores[i]) : 0u;
    const bool valid = i < w1 && k >= base;
    const bool in = valid && k - base <= span;
    const uint32_t in_mask = __ballot_sync(0xffffffffu, in);
    const bool keep = valid && (!in || seen + __popc(in_mask & below_me) < need);
    const uint32_t keep_mask = __ballot_sync(0xffffffffu, keep);
    if (keep) dst[at + __popc(keep_mask & below_me)] = i;
    at += __popc(keep_mask);
    seen += __popc(in_mask);
  }
}

namespace {

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

constexpr int kMaxGridYZ = 65535;

template <typename KV, typename OT>
pkv_status launch_bounds(const BoundsParams& p, int head_dim, cudaStream_t stream) {
  auto kern = head_dim == 64 ? block_bounds_kernel<KV, OT, 64> : block_bounds_kernel<KV, OT, 128>;
  const dim3 grid(static_cast<unsigned>((p.items + kBoundsWarps - 1) / kBoundsWarps),
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
  const int64_t items = std::min<int64_t>(touched, max_blocks_per_seq) * num_kv_heads;
  if (items > INT32_MAX) return PKV_ERR_UNSUPPORTED;
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
  p.items = static_cast<int>(items);
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
  auto kern = group == 1   ? block_scores_kernel<QT, D, 1>
              : group == 2 ? block_scores_kernel<QT, D, 2>
              : group == 4 ? block_scores_kernel<QT, D, 4>
                           : block_scores_kernel<QT, D, 8>;
  const int tiles = (p.max_nblk + 15) / 16;
  const dim3 grid(static_cast<unsigned>((tiles + kScoreWarps - 1) / kScoreWarps), static_cast<unsigned>(p.n_kv_heads),
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
  if (num_kv_heads > kMaxGridYZ) return PKV_ERR_UNSUPPORTED;
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
  const cudaError_t e = launch_pdl(select_blocks_kernel, dim3(static_cast<unsigned>(units)), dim3(kSelThreads), 0,
                                   static_cast<cudaStream_t>(stream), p);
  return cuda_failed(e, "select_blocks_kernel launch") ? PKV_ERR_CUDA : PKV_OK;
}

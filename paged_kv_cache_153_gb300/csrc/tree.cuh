// Attention of drafted tokens over the paged cache (sm_103a).
//
// What is computed.  The n drafted tokens of a sequence are its last n cached
// ones; token i sees every token before them and those of the n that its mask
// names (its ancestors and itself, or any other set):
//   out[i, h] = sum_j p_j V_j,  p = softmax of scale <q[i, h], K_j> over the j
//   with j < base, or bit j - base of mask[i] set,   base = ctx - n.
//
// Work.  The n G query rows of a KV head (G query heads per KV head) are one
// matrix against its keys: a unit is up to 128 q_tiles of them.  Its cost is
// that of its 128-key tiles and of its set-up, and the units' costs lie on one
// axis, cut into equal ranges, one per thread block (one per SM).  A unit that one
// range holds is written out there; otherwise each range that meets it leaves
// one fp32 state (m, l, o) per row, and the merge joins them:
//   out = sum_r 2^(m_r - M) o_r / sum_r 2^(m_r - M) l_r.
//
// What bounds it.  A tile is 64 KiB of 16-bit K and V (32 KiB of FP8) for 128
// rows: an SM's share of the memory bandwidth brings it in about 2800 clocks
// (1400), the two products of one row tile take 1024 (1536 with bf16's second
// part of P).  So up to 128 rows the reads bound it, and up to 256 rows both do.
//
// Tiles.  K and V of a block are 16 rows of D elements, contiguous: one TMA box
// [64 elements, 8 rows, D / 64 halves, 2] takes all of it into 8-row atoms of
// the 128-byte swizzle, the halves of the row next to each other, so that a tile
// is eight requests instead of the 32 of [16 x 128 B] boxes (16-row boxes move
// about 25 bytes a clock).  As an operand, 8-key groups are D / 64 KiB apart and
// the halves of a row 1 KiB, in K (K-major) and V (MN-major) alike.
// Per operation, one row tile against one key tile:
//   S = Q K^T     into one of the S / P buffers in TMEM (three, or two where the
//                 outputs of two row tiles with head_dim 128 take the rest)
//   softmax       8 warps, two threads per row: 64 columns each, the row's
//                 maximum exchanged through shared memory; P overwrites S.  bf16
//                 P is two bf16 parts (p truncated, the rounded remainder: exact
//                 to 2^-16, where one rounding, 2^-9, would be as large as the
//                 output's own); fp16 P (2^-12) is rounded once, and l sums the
//                 rounded values.  The row reference moves only when a tile's
//                 maximum exceeds it by more than 2^8; only then is O rescaled.
//   O += P V      P from TMEM.
// Key tiles go from the last to the first: the ones with drafted tokens need a
// look at their rows, which then overlaps the first loads.
//
// Masked places.  Scores of keys that a row does not see become -inf, whatever K
// holds.  But 0 times an infinity or a NaN of V is a NaN, so a row of V behind the
// context is cleared in shared memory, and an element of a drafted token's V that
// is not finite is set to 0 there and the token remembered: at the end every row
// that sees it adds the element itself (an infinity or a NaN whatever the weight).
//
// FP8 caches.  Codes are staged by 1-D copies and converted to fp16 tiles by four
// warps (every E4M3 and E5M2 value is a half); q is fp16 (bf16 q converted in
// place: exact in fp16's normal range).  The products then run in fp16.
//
// Warps 0-7: softmax; 8: producer; 9: TMEM owner and Q K^T issuer; 10: P V
// issuer; 11-14: rows of V with drafted tokens, or the conversions.  Waits are
// bounded as in the other kernels.
#pragma once

#include <cuda_runtime.h>

#include <algorithm>
#include <mutex>

#include "decode.cuh"
#include "pkv_common.cuh"
#include "tcgen05.cuh"
#include "tree.h"

namespace pkv {

constexpr int kTThreads = 480;
constexpr int kTSoftmax = 256;
constexpr int kTXform = 4;                        // warps 11-14
constexpr int kTTileBlocks = kTreeKeys / kBlockSize;
constexpr float kTRescaleLog2 = 8.f;
constexpr int kTBadSlots = 4;                     // pieces whose remembered tokens live at once

// cost of a unit's set-up (Q, the first tile's latency, its outputs) and of a key
// tile against one row tile or two, in half tiles
constexpr int kTUnitCost = 3;
__host__ __device__ constexpr int tree_tile_cost(int rows) { return rows > kTreeRows ? 3 : 2; }

template <int D, bool FP8, int NQ>
struct TreeSmem {
  static constexpr int kTile = kTreeKeys * D * 2;                  // a Q, K or V tile
  static constexpr int kStage = kTile / 2;                         // FP8: a staged tile of codes
  static constexpr int kKStages = FP8 ? 1 : 2;
  static constexpr int kVStages = FP8 ? 3 - NQ : 4 - NQ;
  static constexpr int kCodeStages = FP8 ? 4 : 0;
  static constexpr int kQ = 0;
  static constexpr int kK = NQ * kTile;
  static constexpr int kV = kK + kKStages * kTile;
  static constexpr int kCodes = kV + kVStages * kTile;
  static constexpr int kBar = kCodes + kCodeStages * kStage;       // 512 bytes
  static constexpr int kBad = kBar + 512;                          // uint32 [slots][warps][8]
  static constexpr int kRed = kBad + kTBadSlots * kTXform * 32;    // float [3][2][128]
  static constexpr int kSeqs = kRed + 3 * 2 * kTreeRows * 4;       // TreeSeq [batch + 1]
  static __host__ __device__ constexpr size_t bytes(int batch) {
    return 1024 + kSeqs + sizeof(TreeSeq) * (static_cast<size_t>(batch) + 1);
  }
  // S / P buffers, and the outputs behind them
  static constexpr int kSBufs = (512 - NQ * D) / 128 < 3 ? (512 - NQ * D) / 128 : 3;
  static constexpr int kOCol = kSBufs * kTreeKeys;
  // 8-key groups of a K / V tile and the 64-element halves of a row
  static constexpr int kGroup = 1024 * (D / 64);
  static constexpr int kHalf = 1024;
  static constexpr int kHalfQ = kTreeRows * 128;
};
static_assert(TreeSmem<128, false, 2>::bytes(kTreeMaxBatch) <= 232448, "16-bit tiles");
static_assert(TreeSmem<128, true, 1>::bytes(kTreeMaxBatch) <= 232448, "FP8 tiles");

// a piece of a range: key tiles [t0, t1) of one unit
struct TreeSeg {
  int64_t next;                  // cost position behind it
  int64_t row;                   // first row of its states
  int b, g, unit, rows, t0, t1, kt;
};

// units of a sequence's rows, key tiles of its context, cost of one unit
template <int NQ>
__device__ __forceinline__ int tree_units(int rows) { return (rows + kTreeRows * NQ - 1) / (kTreeRows * NQ); }
__device__ __forceinline__ int tree_tiles(int ctx) { return ctx / kTreeKeys + (ctx % kTreeKeys != 0); }
__device__ __forceinline__ int64_t tree_unit_cost(int rows, int kt) {
  return kTUnitCost + static_cast<int64_t>(kt) * tree_tile_cost(rows);
}
// first tile at or behind position x of its unit's cost
__device__ __forceinline__ int tree_tile_at(int64_t x, int rows, int kt) {
  if (x <= kTUnitCost) return 0;
  const int w = tree_tile_cost(rows);
  return static_cast<int>(min(static_cast<int64_t>(kt), div_nonneg(x - kTUnitCost + w - 1, w)));
}
// States of unit u's rows in range r lie at rows [tree_piece_row(...), + unit
// rows) of ml and o.  Successive pieces differ in the unit or in the range, so
// they never overlap.
__device__ __forceinline__ int64_t tree_piece_row(int64_t start, int n_q_heads, int g, int rows, int64_t first_row,
                                                  int64_t range, int unit_rows) {
  return start * n_q_heads + static_cast<int64_t>(g) * rows + first_row + range * unit_rows;
}

template <int NQ>
__device__ __forceinline__ TreeSeg tree_segment(const TreeSeq* seqs, int batch, int shift, int n_q_heads, int64_t pos,
                                                int64_t end, int64_t range) {
  int lo = 0, hi = batch - 1;    // the last sequence that starts at or before pos (a non-empty one)
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (seqs[mid].cost <= pos) lo = mid; else hi = mid - 1;
  }
  const TreeSeq sq = seqs[lo];
  const int rows = sq.n << shift, units = tree_units<NQ>(rows), kt = tree_tiles(sq.ctx);
  const int64_t cost = tree_unit_cost(rows, kt), rem = pos - sq.cost;
  const int64_t u = div_nonneg(rem, cost), off = rem - u * cost;
  TreeSeg s;
  s.b = lo;
  s.g = static_cast<int>(u) / units;
  s.unit = static_cast<int>(u) - s.g * units;
  s.kt = kt;
  s.t0 = tree_tile_at(off, rows, kt);
  s.t1 = tree_tile_at(off + (end - pos), rows, kt);
  s.next = pos + min(cost - off, end - pos);
  s.rows = min(kTreeRows * NQ, rows - s.unit * kTreeRows * NQ);
  s.row = tree_piece_row(sq.start, n_q_heads, s.g, rows, static_cast<int64_t>(s.unit) * kTreeRows * NQ, range,
                         kTreeRows * NQ);
  return s;
}

// a position in a ring of N stages
template <int N>
struct Ring {
  uint32_t s = 0, ph = 0;
  __device__ __forceinline__ void next() {
    if (++s == N) {
      s = 0;
      ph ^= 1u;
    }
  }
};

// one box of a block's rows
__device__ __forceinline__ void tma_load_4d(void* dst, const CUtensorMap* map, int w, uint64_t* bar, uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint [%0], [%1, {%2, "
      "%2, %2, %3}], [%4], %5;" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(0), "r"(w), "r"(smem_u32(bar)), "l"(policy)
      : "memory");
}

// bits o .. o + 31 of a mask row of `words` 32-bit words, those below 0 set (the
// context) and those from n on clear
__device__ __forceinline__ uint32_t tree_bits(const uint32_t* row, int words, int n, int o) {
  if (o <= -32) return 0xffffffffu;
  if (o >= n) return 0u;
  const int at = max(o, 0) >> 5;
  const uint32_t lo = at < words ? row[at] : 0u, hi = at + 1 < words ? row[at + 1] : 0u;
  uint32_t m = o >= 0 ? __funnelshift_r(lo, hi, o & 31) : (lo << -o) | ((1u << -o) - 1u);
  if (n - o < 32) m &= (1u << (n - o)) - 1u;
  return m;
}

// two 16-bit elements that are not finite as they are, the others 0
template <typename MT>
__device__ __forceinline__ uint32_t nonfinite2(uint32_t w) {
  constexpr uint32_t e = std::is_same<MT, BF16>::value ? 0x7f80u : 0x7c00u;
  uint32_t keep = 0;
  if ((w & e) == e) keep |= 0xffffu;
  if (((w >> 16) & e) == e) keep |= 0xffff0000u;
  return w & keep;
}

// MT: 16-bit type of the products; KV: the cache's (MT, or an FP8 format)
template <typename MT, typename KV, int D, int NQ>
__global__ void __launch_bounds__(kTThreads, 1) tree_kernel(const __grid_constant__ TreeParams p) {
  constexpr bool kFp8 = KV::kBytes == 1;
  using L = TreeSmem<D, kFp8, NQ>;
  constexpr bool kSplit = std::is_same<MT, BF16>::value;
  constexpr int NB = L::kSBufs;
  extern __shared__ unsigned char tsm_raw[];
  unsigned char* sm = tsm_raw + ((1024 - (smem_u32(tsm_raw) & 1023)) & 1023);
  uint64_t* k_full = reinterpret_cast<uint64_t*>(sm + L::kBar);   // [kKStages] K tile landed (FP8: converted)
  uint64_t* k_empty = k_full + L::kKStages;        // its Q K^T done
  uint64_t* v_full = k_empty + L::kKStages;        // [kVStages] V tile landed (16-bit)
  uint64_t* v_ready = v_full + L::kVStages;        // its rows looked at, or converted
  uint64_t* v_empty = v_ready + L::kVStages;       // its P V done
  uint64_t* c_full = v_empty + L::kVStages;        // [kCodeStages] codes landed
  uint64_t* c_empty = c_full + L::kCodeStages;     // converted
  uint64_t* s_full = c_empty + L::kCodeStages;     // [NB] scores ready
  uint64_t* p_full = s_full + NB;                  // [NB] P written, O rescaled
  uint64_t* pv_done = p_full + NB;                 // [NB] P V done
  uint64_t* q_full = pv_done + NB;                 // Q of a piece landed
  uint64_t* q_ready = q_full + 1;                  // and converted
  uint64_t* q_empty = q_ready + 1;                 // its Q K^T done
  uint64_t* mma_idle = q_empty + 1;                // [2] an issuer's MMAs done
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(mma_idle + 2);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  static_assert((2 * 2 + 3 * 3 + 2 * 5 + 3 * 3 + 5 + 1) * 8 <= 512, "barrier block overflows");
  uint32_t* bad = reinterpret_cast<uint32_t*>(sm + L::kBad);
  float* red = reinterpret_cast<float*>(sm + L::kRed);
  TreeSeq* seqs = reinterpret_cast<TreeSeq*>(sm + L::kSeqs);

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int shift = p.group_shift;
  if (warp == 9) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_slot)),
                 "r"(512)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  if (tid == 8 * 32) {
    *abort_flag = 0;
    for (int s = 0; s < L::kKStages; ++s) {
      mbar_init(&k_full[s], kFp8 ? kTXform : 1);
      mbar_init(&k_empty[s], 1);
    }
    for (int s = 0; s < L::kVStages; ++s) {
      mbar_init(&v_full[s], 1);
      mbar_init(&v_ready[s], kTXform);
      mbar_init(&v_empty[s], 1);
    }
    for (int s = 0; s < L::kCodeStages; ++s) {
      mbar_init(&c_full[s], 1);
      mbar_init(&c_empty[s], kTXform);
    }
    for (int s = 0; s < NB; ++s) {
      mbar_init(&s_full[s], 1);
      mbar_init(&p_full[s], kTSoftmax);
      mbar_init(&pv_done[s], 1);
    }
    mbar_init(q_full, 1);
    mbar_init(q_ready, kTXform);
    mbar_init(q_empty, 1);
    mbar_init(&mma_idle[0], 1);
    mbar_init(&mma_idle[1], 1);
    fence_mbar_init();
  }
  // Until the waits below this kernel reads lengths, offsets and (in the producer)
  // tables only, which no kernel that releases early writes.

  // ---- the sequences: drafted tokens, context, cost ----
  for (int b = tid; b < p.batch; b += kTThreads) {
    const int64_t t0 = p.cu_nodes[b], t1 = p.cu_nodes[b + 1];
    const int ctx = p.context_lens[b];
    TreeSeq sq{0, 0, 0, 0, 0};
    const int64_t n = t1 - t0;
    if (t0 < 0 || n < 0 || t1 > p.num_tokens || n > p.max_nodes || ctx < n ||
        ctx > static_cast<int64_t>(p.max_blocks_per_seq) * kBlockSize) {
      record_error(p.err, PKV_ERR_OOB);
    } else if (n > 0) {
      const int rows = static_cast<int>(n) << shift;
      sq.start = static_cast<int>(t0);
      sq.n = static_cast<int>(n);
      sq.ctx = ctx;
      sq.cost = p.n_kv_heads * tree_units<NQ>(rows) * tree_unit_cost(rows, tree_tiles(ctx));
    }
    seqs[b] = sq;
  }
  __syncthreads();
  if (warp == 0) {   // exclusive prefix of the costs
    int64_t carry = 0;
    for (int b0 = 0; b0 < p.batch; b0 += 32) {
      const int b = b0 + lane;
      const int64_t mine = b < p.batch ? seqs[b].cost : 0;
      int64_t x = mine;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int64_t u = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += u;
      }
      if (b < p.batch) seqs[b].cost = carry + x - mine;
      carry += __shfl_sync(0xffffffffu, x, 31);
    }
    if (lane == 0) seqs[p.batch] = TreeSeq{carry, 0, 0, 0, 0};
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (blockIdx.x == 0) {
    pdl_wait();
    for (int b = tid; b <= p.batch; b += kTThreads) p.seqs[b] = seqs[b];
  }
  const uint32_t tmem = *tmem_slot;
  const int64_t V = seqs[p.batch].cost, R = gridDim.x, range = blockIdx.x;
  const int64_t first = div_nonneg(range * V, R), end = div_nonneg((range + 1) * V, R);
  auto segment = [&](int64_t pos) {
    return tree_segment<NQ>(seqs, p.batch, shift, p.n_q_heads, pos, end, range);
  };

  if (warp < 8) {
    // ============================ softmax / epilogue ============================
    const int r = tid & (kTreeRows - 1), half = tid >> 7, quarter = warp & 3;
    const int pair_bar = 2 + quarter;                // named barrier of warps w and w + 4 (one row each)
    const uint32_t lane_base = static_cast<uint32_t>(quarter * 32) << 16;
    Ring<NB> sr;                                     // S / P buffer of the next operation
    uint32_t slot = 0;                               // of remembered tokens
    bool ok = true;
    int flip = 0;                                    // slot of the row exchange
    pdl_wait();
    for (int64_t pos = first; pos < end && ok;) {
      const TreeSeg sg = segment(pos);
      pos = sg.next;
      if (sg.t0 >= sg.t1) continue;
      const TreeSeq sq = seqs[sg.b];
      const int base = sq.ctx - sq.n;
      const int nq = NQ == 2 && sg.rows > kTreeRows ? 2 : 1;
      const float scale_log2 = p.qk_scale_log2 * (kFp8 ? p.k_scale[sg.g] : 1.f);
      float m_ref[NQ], l_run[NQ];
#pragma unroll
      for (int c = 0; c < NQ; ++c) m_ref[c] = -INFINITY, l_run[c] = 0.f;
      Ring<NB> last[NQ];                             // buffer of a row tile's previous operation
      for (int t = sg.t1 - 1; t >= sg.t0 && ok; --t) {
#pragma unroll
        for (int c = 0; c < NQ; ++c) {
          if (c >= nq || !ok) break;
          const int row = c * kTreeRows + r;         // of the unit
          const bool live = c * kTreeRows + quarter * 32 < sg.rows;   // any row of this warp
          const bool tail = (t + 1) * kTreeKeys > base;
          uint32_t see[2] = {0xffffffffu, 0xffffffffu};
          if (tail && live) {
            const int node = min((sg.unit * kTreeRows * NQ + row) >> shift, sq.n - 1);
            const uint32_t* words = p.mask + (static_cast<int64_t>(sq.start) + node) * (2 * p.mask_words);
            const int o = t * kTreeKeys + 64 * half - base;
            see[0] = tree_bits(words, 2 * p.mask_words, sq.n, o);
            see[1] = tree_bits(words, 2 * p.mask_words, sq.n, o + 32);
          }
          const uint32_t ts = tmem + lane_base + sr.s * kTreeKeys + 64 * half;
          const uint32_t to = tmem + lane_base + L::kOCol + c * D;
          ok = __all_sync(0xffffffffu, mbar_wait(&s_full[sr.s], sr.ph, p.err, p.wait_limit_ns) && !*abort_flag);
          tc_fence_after();
          float v[64];
          float mx = -INFINITY;
          if (ok && live) {
            tmem_ld64(ts, v);
            if (tail && __any_sync(0xffffffffu, (see[0] & see[1]) != 0xffffffffu)) {
#pragma unroll
              for (int i = 0; i < 64; ++i) v[i] = (see[i >> 5] >> (i & 31)) & 1u ? v[i] : -INFINITY;
            }
            mx = max64(v);
            red[(flip * 2 + half) * kTreeRows + r] = mx;
          }
          // (a failed wait on either side ends both warps of the pair here)
          if (named_bar_red_or(pair_bar, 64, !ok)) {
            ok = false;
            break;
          }
          if (live) {
            mx = fmaxf(mx, red[(flip * 2 + (1 - half)) * kTreeRows + r]);
            flip ^= 1;
            const float m_tile = mx * scale_log2;
            float alpha = 1.f;
            if (m_tile > m_ref[c] + kTRescaleLog2) {
              alpha = ex2_approx(m_ref[c] - m_tile);
              m_ref[c] = m_tile;
            }
            bool waited = true;
            if (t < sg.t1 - 1 && __any_sync(0xffffffffu, alpha != 1.f)) {
              // O may be touched once the row tile's previous P V has completed
              waited = __all_sync(0xffffffffu, mbar_wait(&pv_done[last[c].s], last[c].ph, p.err, p.wait_limit_ns));
              tc_fence_after();
              if (waited) {
#pragma unroll 1
                for (int x = half * (D / 2); x < (half + 1) * (D / 2); x += 16) {
                  float o[16];
                  tmem_ld16(to + x, o);
#pragma unroll
                  for (int i = 0; i < 16; ++i) o[i] *= alpha;
                  tmem_st16(to + x, o);
                }
              }
            }
            const float nref = (m_ref[c] == -INFINITY) ? 0.f : -m_ref[c];
            const uint64_t scale2 = f32x2(scale_log2, scale_log2), nref2 = f32x2(nref, nref);
            uint64_t acc[4] = {0ull, 0ull, 0ull, 0ull};
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              uint32_t pk[32];
#pragma unroll
              for (int i = 0; i < 32; i += 2) {
                const float2 x = f32x2_split(fma_f32x2(f32x2(v[32 * h + i], v[32 * h + i + 1]), scale2, nref2));
                const float e0 = ex2_approx(x.x), e1 = ex2_approx(x.y);
                uint64_t e01 = f32x2(e0, e1);
                if constexpr (kSplit) {
                  const uint32_t b0 = __float_as_uint(e0), b1 = __float_as_uint(e1);
                  pk[i / 2] = __byte_perm(b0, b1, 0x7632);
                  const float2 lo = f32x2_split(
                      sub_f32x2(e01, f32x2(__uint_as_float(b0 & 0xffff0000u), __uint_as_float(b1 & 0xffff0000u))));
                  pk[16 + i / 2] = pack2(lo.x, lo.y, MT{});
                } else {
                  pk[i / 2] = pack2(e0, e1, MT{});
                  const float2 hi = unpack2(pk[i / 2], MT{});
                  e01 = f32x2(hi.x, hi.y);           // (l sums what is multiplied)
                }
                acc[(i / 2) & 3] = add_f32x2(acc[(i / 2) & 3], e01);
              }
              if constexpr (kSplit)
                tmem_st32u(ts + 32 * h, pk);
              else
                tmem_st16u(ts + 32 * h, pk);
            }
            const float2 s0 = f32x2_split(add_f32x2(add_f32x2(acc[0], acc[1]), add_f32x2(acc[2], acc[3])));
            tmem_wait_st();
            l_run[c] = l_run[c] * alpha + (s0.x + s0.y);
            if (!waited) *abort_flag = 1;            // (the next exchange stops both warps)
          }
          tc_fence_before();
          mbar_arrive(&p_full[sr.s]);
          last[c] = sr;
          sr.next();
        }
      }
      if (!ok) break;
      // the piece's outputs or states, once the last P V is done
      const Ring<NB> fin = last[nq - 1];
      ok = __all_sync(0xffffffffu, mbar_wait(&pv_done[fin.s], fin.ph, p.err, p.wait_limit_ns) && !*abort_flag);
#pragma unroll
      for (int c = 0; c < NQ; ++c) red[((2 * c) * 2 + half) * kTreeRows + r] = l_run[c];
      if (named_bar_red_or(pair_bar, 64, !ok)) {
        ok = false;
        break;
      }
      tc_fence_after();
      // drafted tokens of this piece with elements of V that are not finite
      const uint32_t mine = bad[(slot % kTBadSlots) * (kTXform * 8) + lane];
      const bool any_bad = __any_sync(0xffffffffu, mine != 0u);
      ++slot;
      const bool direct = sg.t0 == 0 && sg.t1 == sg.kt;
      const float v_scale = kFp8 ? p.v_scale[sg.g] : 1.f;
#pragma unroll
      for (int c = 0; c < NQ; ++c) {
        if (c >= nq) break;
        const int row0 = c * kTreeRows + quarter * 32, n_rows = sg.rows - row0;
        if (n_rows <= 0) continue;
        const int row = row0 + lane;
        const int unit_row = sg.unit * kTreeRows * NQ + row;           // of the sequence's rows
        const int node = min(unit_row >> shift, sq.n - 1), head = (sg.g << shift) + (unit_row & ((1 << shift) - 1));
        const float l = l_run[c] + red[((2 * c) * 2 + (1 - half)) * kTreeRows + r];
        const float weight = direct ? (l > 0.f ? v_scale / l : 0.f) : v_scale;
#pragma unroll 1
        for (int x = half * (D / 2); x < (half + 1) * (D / 2); x += 32) {
          float o[32];
          tmem_ld32(tmem + lane_base + L::kOCol + c * D + x, o);
#pragma unroll
          for (int i = 0; i < 32; ++i) o[i] *= weight;
          if (any_bad) {
            // (rare) every row adds what it sees of them
            for (int w = 0; w < 8; ++w) {
              uint32_t bits = 0;
#pragma unroll
              for (int k = 0; k < kTXform; ++k) bits |= __shfl_sync(0xffffffffu, mine, 8 * k + w);
              if (w >= 2 * p.mask_words) break;
              bits &= p.mask[(static_cast<int64_t>(sq.start) + node) * (2 * p.mask_words) + w];
              for (; bits != 0u; bits &= bits - 1u) {
                const int at = base + 32 * w + __ffs(bits) - 1;
                const int id = p.block_tables[static_cast<int64_t>(sg.b) * p.max_blocks_per_seq + at / kBlockSize];
                if (id < 0 || id >= p.num_blocks) continue;
                const int64_t e = ((static_cast<int64_t>(id) * p.n_kv_heads + sg.g) * kBlockSize + at % kBlockSize) * D;
#pragma unroll
                for (int i = 0; i < 32; i += 8) {
                  float f[8];
                  load8(static_cast<const unsigned char*>(p.v_cache) + (e + x + i) * KV::kBytes, f, KV{});
#pragma unroll
                  for (int k = 0; k < 8; ++k)
                    if (!isfinite(f[k])) o[i + k] += f[k];
                }
              }
            }
            __syncwarp();
          }
          if (direct) {
            if (row < sg.rows) {
              auto* dst = reinterpret_cast<uint4*>(
                  static_cast<uint16_t*>(p.out) +
                  ((static_cast<int64_t>(sq.start) + node) * p.n_q_heads + head) * D + x);
              const bool bf16 = kFp8 ? p.q_bf16 != 0 : kSplit;
#pragma unroll
              for (int i = 0; i < 32; i += 8)
                dst[i / 8] = bf16 ? make_uint4(pack2(o[i], o[i + 1], BF16{}), pack2(o[i + 2], o[i + 3], BF16{}),
                                               pack2(o[i + 4], o[i + 5], BF16{}), pack2(o[i + 6], o[i + 7], BF16{}))
                                  : make_uint4(pack2(o[i], o[i + 1], F16{}), pack2(o[i + 2], o[i + 3], F16{}),
                                               pack2(o[i + 4], o[i + 5], F16{}), pack2(o[i + 6], o[i + 7], F16{}));
            }
          } else {
            store_rows32<D>(p.o + (sg.row + row0) * D + x, o, n_rows, lane);
          }
        }
        if (!direct && half == 0 && lane < n_rows)
          *reinterpret_cast<float2*>(p.ml + (sg.row + row) * 2) = make_float2(m_ref[c], l);
      }
      // (the partner's sums have been read before the next piece's first maxima overwrite them)
      named_bar_sync(pair_bar, 64);
    }
    if (!ok) *abort_flag = 1;
  } else if (warp == 8) {
    // ============================ producer ============================
    Ring<L::kKStages> kr;
    Ring<L::kVStages> vr;
    Ring<(kFp8 ? L::kCodeStages : 1)> cr;
    uint32_t tiles = 0, pieces = 0, codes = 0;       // issued so far
    bool good = true;
    pdl_wait_and_release();
    for (int64_t pos = first; pos < end && good;) {
      const TreeSeg sg = segment(pos);
      pos = sg.next;
      if (sg.t0 >= sg.t1) continue;
      const TreeSeq sq = seqs[sg.b];
      const int nq = NQ == 2 && sg.rows > kTreeRows ? 2 : 1;
      const int nblk = ctx_blocks(sq.ctx);
      const uint64_t pol = tree_units<NQ>(sq.n << shift) > 1 ? policy_evict_last() : policy_evict_first();
      const int32_t* row = p.block_tables + static_cast<int64_t>(sg.b) * p.max_blocks_per_seq;
      auto fetch_id = [&](int t) -> int {
        const int blk = t * kTTileBlocks + lane;
        return (t >= sg.t0 && lane < kTTileBlocks && blk < nblk) ? row[blk] : -1;
      };
      int id = fetch_id(sg.t1 - 1);
      // Q of the piece, once every Q K^T of the one before has read its tiles
      if (pieces > 0)
        good = __all_sync(0xffffffffu, mbar_wait(q_empty, (pieces - 1) & 1, p.err, p.wait_limit_ns) && !*abort_flag);
      if (!good) break;
      if (lane == 0) mbar_arrive_expect_tx(q_full, nq * (D / 64) * (p.q_box << shift) * 128);
      ++pieces;
      __syncwarp();
      if (lane < nq * (D / 64)) {
        const int c = lane / (D / 64), h = lane % (D / 64);
        tma_load_3d(sm + L::kQ + c * L::kTile + h * L::kHalfQ, &p.tmap_q, h * 64, sg.g << shift,
                    sq.start + ((sg.unit * kTreeRows * NQ + c * kTreeRows) >> shift), q_full, policy_evict_last());
      }
      __syncwarp();
      for (int t = sg.t1 - 1; t >= sg.t0 && good; --t) {
        // cache slab of this lane's block: -1 behind the context or for a bad id
        // (16-bit: read from outside the tensor, which fills with zeros)
        const int blk = t * kTTileBlocks + lane;
        bool have = lane < kTTileBlocks && blk < nblk;
        if (have && (id < 0 || id >= p.num_blocks)) {
          record_error(p.err, PKV_ERR_OOB);
          have = false;
        }
        const int64_t slab = have ? static_cast<int64_t>(id) * p.n_kv_heads + sg.g : -1;
        id = fetch_id(t - 1);
        if constexpr (!kFp8) {
          auto load = [&](bool is_v) -> bool {
            const uint32_t s = is_v ? vr.s : kr.s, ph = is_v ? vr.ph : kr.ph;
            const bool used = tiles >= static_cast<uint32_t>(is_v ? L::kVStages : L::kKStages);
            uint64_t* full = is_v ? &v_full[s] : &k_full[s];
            const bool freed =
                !used || mbar_wait(is_v ? &v_empty[s] : &k_empty[s], ph ^ 1u, p.err, p.wait_limit_ns);
            if (!__all_sync(0xffffffffu, freed && !*abort_flag)) return false;
            if (lane == 0) mbar_arrive_expect_tx(full, L::kTile);
            __syncwarp();
            if (lane < kTTileBlocks)
              tma_load_4d(sm + (is_v ? L::kV : L::kK) + s * L::kTile + lane * (kBlockSize * D * 2),
                          is_v ? &p.tmap_v : &p.tmap_k, static_cast<int>(slab) * 2, full, pol);
            __syncwarp();
            return true;
          };
          good = load(false);
          if (good) {
            kr.next();
            good = load(true);
          }
          if (good) {
            vr.next();
            ++tiles;
          } else if (!*abort_flag) {
            *abort_flag = 1;
          }
        } else {
          constexpr int kSlab = kBlockSize * D;
          for (int is_v = 0; is_v < 2 && good; ++is_v) {
            const bool freed = codes < static_cast<uint32_t>(L::kCodeStages) ||
                               mbar_wait(&c_empty[cr.s], cr.ph ^ 1u, p.err, p.wait_limit_ns);
            good = __all_sync(0xffffffffu, freed && !*abort_flag);
            if (!good) break;
            unsigned char* dst = sm + L::kCodes + cr.s * L::kStage + lane * kSlab;
            const uint32_t got = __ballot_sync(0xffffffffu, have);
            if (lane < kTTileBlocks && !have) {      // (codes of 0; rare but for the last tile)
              for (int x = 0; x < kSlab; x += 16)
                asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(smem_u32(dst + x)), "r"(0u) : "memory");
              fence_proxy_async_smem();
            }
            __syncwarp();
            if (lane == 0) mbar_arrive_expect_tx(&c_full[cr.s], __popc(got) * kSlab);
            __syncwarp();
            if (have)
              bulk_g2s(dst, (is_v ? p.v_codes : p.k_codes) + slab * kSlab, kSlab, &c_full[cr.s], pol);
            __syncwarp();
            ++codes;
            cr.next();
          }
        }
      }
    }
    if (!good) *abort_flag = 1;
    if (lane == 0) {
      // The last loads of every stage land before the block ends (bounded, with the
      // full limit): whoever should wait for them may have stopped.
      const unsigned long long deadline = global_ns() + kWaitLimitNs;
      if (pieces > 0) mbar_wait_until(q_full, (pieces - 1) & 1, deadline);
      if constexpr (!kFp8) {
        // (K of a tile whose V was not issued may be one further)
        for (uint32_t t = tiles > L::kVStages ? tiles - L::kVStages : 0; t < tiles; ++t)
          mbar_wait_until(&v_full[t % L::kVStages], (t / L::kVStages) & 1, deadline);
        const uint32_t kt = tiles + (kr.s != tiles % L::kKStages ? 1 : 0);
        for (uint32_t t = kt > L::kKStages ? kt - L::kKStages : 0; t < kt; ++t)
          mbar_wait_until(&k_full[t % L::kKStages], (t / L::kKStages) & 1, deadline);
      } else {
        constexpr uint32_t n = L::kCodeStages;
        for (uint32_t t = codes > n ? codes - n : 0; t < codes; ++t)
          mbar_wait_until(&c_full[t % n], (t / n) & 1, deadline);
      }
    }
    __syncwarp();
  } else if (warp < 11) {
    // ============================ MMA issuers (warps 9, 10) ============================
    // Warp 9 issues Q K^T, warp 10 P V, one elected lane each: a commit holds its
    // thread until the MMA queue has drained to a few entries; meanwhile the
    // other feeds the queue.
    constexpr int kPasses = kSplit ? 2 : 1;
    constexpr uint32_t kIdQK = umma_idesc<MT>(false, kTreeKeys), kIdPV = umma_idesc<MT>(true, D);
    const bool qk_warp = (warp == 9);
    bool ok = true;
    if (lane == 0) {
      Ring<NB> sr;
      Ring<L::kKStages> kr;
      Ring<L::kVStages> vr;
      uint32_t pieces = 0, ops = 0;
      for (int64_t pos = first; pos < end && ok;) {
        const TreeSeg sg = segment(pos);
        pos = sg.next;
        if (sg.t0 >= sg.t1) continue;
        const int nq = NQ == 2 && sg.rows > kTreeRows ? 2 : 1;
        if (qk_warp) {
          // (the producer loads nothing while the previous kernel runs)
          ok = mbar_wait_started_early(kFp8 && p.q_bf16 ? q_ready : q_full, pieces & 1, p.err, p.wait_limit_ns);
        }
        ++pieces;
        for (int t = sg.t1 - 1; t >= sg.t0 && ok; --t) {
          if (qk_warp)
            ok = mbar_wait(&k_full[kr.s], kr.ph, p.err, p.wait_limit_ns);
          else
            ok = mbar_wait_started_early(&v_ready[vr.s], vr.ph, p.err, p.wait_limit_ns);
#pragma unroll
          for (int c = 0; c < NQ; ++c) {
            if (c >= nq || !ok) break;
            const uint32_t d_s = tmem + sr.s * kTreeKeys;
            if (qk_warp) {
              // S once the P V that read P from its columns is done
              ok = (ops < NB || mbar_wait(&pv_done[sr.s], sr.ph ^ 1u, p.err, p.wait_limit_ns)) && !*abort_flag;
              if (!ok) break;
              tc_fence_after();
              const uint64_t a0 = umma_desc(smem_u32(sm + L::kQ + c * L::kTile), 16, 1024);
              const uint64_t b0 = umma_desc(smem_u32(sm + L::kK + kr.s * L::kTile), 16, L::kGroup);
#pragma unroll
              for (int ks = 0; ks < D / 16; ++ks)
                umma_f16(d_s, a0 + static_cast<uint64_t>(((ks >> 2) * L::kHalfQ + (ks & 3) * 32) >> 4),
                         b0 + static_cast<uint64_t>(((ks >> 2) * L::kHalf + (ks & 3) * 32) >> 4), kIdQK, ks > 0);
              umma_commit(&s_full[sr.s]);
            } else {
              ok = mbar_wait(&p_full[sr.s], sr.ph, p.err, p.wait_limit_ns) && !*abort_flag;
              if (!ok) break;
              tc_fence_after();
              const uint64_t b0 = umma_desc(smem_u32(sm + L::kV + vr.s * L::kTile), L::kHalf, L::kGroup);
              const uint32_t d_o = tmem + L::kOCol + c * D;
#pragma unroll
              for (int pass = 0; pass < kPasses; ++pass)
#pragma unroll
                for (int ks = 0; ks < kTreeKeys / 16; ++ks)
                  umma_f16_tmem_a(d_o, d_s + 32 * (ks >> 1) + 16 * pass + 8 * (ks & 1),
                                  b0 + static_cast<uint64_t>((ks * 2 * L::kGroup) >> 4), kIdPV,
                                  t < sg.t1 - 1 || ks > 0 || pass > 0);
              umma_commit(&pv_done[sr.s]);
            }
            ++ops;
            sr.next();
          }
          if (!ok) break;
          umma_commit(qk_warp ? &k_empty[kr.s] : &v_empty[vr.s]);
          if (qk_warp && t == sg.t0) umma_commit(q_empty);
          kr.next();
          vr.next();
        }
      }
      if (!ok) *abort_flag = 1;
      // every MMA of this lane has completed before TMEM is released
      umma_commit(&mma_idle[qk_warp ? 0 : 1]);
      mbar_wait(&mma_idle[qk_warp ? 0 : 1], 0, p.err);
    }
    __syncwarp();
  } else {
    // ============ warps 11-14: rows with drafted tokens, conversions ============
    const int x_tid = tid - 11 * 32, x_warp = x_tid >> 5;
    constexpr int kChunks = D / 8;                   // 16-byte chunks of a 16-bit row
    Ring<L::kKStages> kr;
    Ring<L::kVStages> vr;
    Ring<(kFp8 ? L::kCodeStages : 1)> cr;
    uint32_t pieces = 0, tiles = 0;
    bool ok = true;
    auto wait_all = [&](uint64_t* bar, uint32_t ph) {
      return __all_sync(0xffffffffu, mbar_wait(bar, ph, p.err, p.wait_limit_ns) && !*abort_flag);
    };
    pdl_wait();
    for (int64_t pos = first; pos < end && ok;) {
      const TreeSeg sg = segment(pos);
      pos = sg.next;
      if (sg.t0 >= sg.t1) continue;
      const TreeSeq sq = seqs[sg.b];
      const int base = sq.ctx - sq.n;
      uint32_t* my_bad = bad + (pieces % kTBadSlots) * (kTXform * 8) + x_warp * 8;
      if (lane < 8) my_bad[lane] = 0u;
      __syncwarp();
      auto store = [&](uint32_t addr, const uint4& v) {
        asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w)
                     : "memory");
      };
      // 16-byte chunk c of key row j of a K / V tile
      auto at = [&](int j, int c) -> uint32_t {
        return (j >> 3) * L::kGroup + (c >> 3) * L::kHalf + (j & 7) * 128 + (((c & 7) ^ (j & 7)) << 4);
      };
      // an element of V at position key: 0 behind the context; of a drafted token, 0
      // where it is not finite, and the token is remembered
      auto clean = [&](uint4 v, int key) -> uint4 {
        if (key >= sq.ctx) return make_uint4(0u, 0u, 0u, 0u);
        if (key >= base) {
          const uint4 f = make_uint4(nonfinite2<MT>(v.x), nonfinite2<MT>(v.y), nonfinite2<MT>(v.z), nonfinite2<MT>(v.w));
          if (f.x | f.y | f.z | f.w) {
            v.x ^= f.x, v.y ^= f.y, v.z ^= f.z, v.w ^= f.w;
            atomicOr(&my_bad[(key - base) >> 5], 1u << ((key - base) & 31));
          }
        }
        return v;
      };
      if constexpr (kFp8) {
        if (p.q_bf16) {
          // bf16 q to fp16, where it lies
          ok = wait_all(q_full, pieces & 1);
          if (!ok) break;
          const int nq = NQ == 2 && sg.rows > kTreeRows ? 2 : 1;
          for (int x = x_tid; x < nq * L::kTile / 16; x += kTXform * 32) {
            uint4* w = reinterpret_cast<uint4*>(sm + L::kQ) + x;
            const uint4 v = *w;
            auto half2 = [&](uint32_t u) {
              const float2 f = unpack2(u, BF16{});
              return pack2(f.x, f.y, F16{});
            };
            *w = make_uint4(half2(v.x), half2(v.y), half2(v.z), half2(v.w));
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(q_ready);
        }
      }
      ++pieces;
      for (int t = sg.t1 - 1; t >= sg.t0 && ok; --t, ++tiles) {
        const bool tail = (t + 1) * kTreeKeys > base;
        if constexpr (!kFp8) {
          ok = wait_all(&v_full[vr.s], vr.ph);
          if (!ok) break;
          if (tail) {
            const uint32_t tile = smem_u32(sm + L::kV + vr.s * L::kTile);
            const int j0 = max(0, base - t * kTreeKeys);
            for (int x = j0 * kChunks + x_tid; x < kTreeKeys * kChunks; x += kTXform * 32) {
              const int j = x / kChunks;
              const uint32_t addr = tile + at(j, x % kChunks);
              uint4 v;
              asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                           : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                           : "r"(addr));
              const uint4 w = clean(v, t * kTreeKeys + j);
              if ((v.x ^ w.x) | (v.y ^ w.y) | (v.z ^ w.z) | (v.w ^ w.w)) store(addr, w);
            }
            fence_proxy_async_smem();
            __syncwarp();
          }
          if (lane == 0) mbar_arrive(&v_ready[vr.s]);
          vr.next();
        } else {
          for (int is_v = 0; is_v < 2 && ok; ++is_v) {
            const uint32_t stages = is_v ? L::kVStages : L::kKStages;
            uint64_t* empty = is_v ? &v_empty[vr.s] : &k_empty[kr.s];
            ok = wait_all(&c_full[cr.s], cr.ph) &&
                 (tiles < stages || wait_all(empty, (is_v ? vr.ph : kr.ph) ^ 1u));
            if (!ok) break;
            const uint4* codes = reinterpret_cast<const uint4*>(sm + L::kCodes + cr.s * L::kStage);
            const uint32_t tile = smem_u32(sm + (is_v ? L::kV + vr.s * L::kTile : L::kK + kr.s * L::kTile));
            constexpr int kPer = kTreeKeys * D / 16 / (kTXform * 32);   // 16 codes each
            uint4 raw[kPer];
#pragma unroll
            for (int k = 0; k < kPer; ++k) raw[k] = codes[x_tid + k * kTXform * 32];
#pragma unroll
            for (int k = 0; k < kPer; ++k) {
              const int x = x_tid + k * kTXform * 32, j = x / (D / 16), c = x % (D / 16);
              uint4 h[2];
              const uint32_t w[4] = {raw[k].x, raw[k].y, raw[k].z, raw[k].w};
#pragma unroll
              for (int e = 0; e < 2; ++e)
                h[e] = make_uint4(byte2_to_f16x2(w[2 * e], KV{}), byte2_hi_to_f16x2(w[2 * e], KV{}),
                                  byte2_to_f16x2(w[2 * e + 1], KV{}), byte2_hi_to_f16x2(w[2 * e + 1], KV{}));
              if (is_v && tail) {
                h[0] = clean(h[0], t * kTreeKeys + j);
                h[1] = clean(h[1], t * kTreeKeys + j);
              }
              // (the upper half of a row's lanes stores its second chunk first: the two
              // halves of the row lie in the same banks)
              const bool up = D == 128 && (c & 4);
              store(tile + at(j, 2 * c + (up ? 1 : 0)), up ? h[1] : h[0]);
              store(tile + at(j, 2 * c + (up ? 0 : 1)), up ? h[0] : h[1]);
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
              mbar_arrive(&c_empty[cr.s]);
              mbar_arrive(is_v ? &v_ready[vr.s] : &k_full[kr.s]);
            }
            cr.next();
          }
          kr.next();
          vr.next();
        }
      }
    }
    if (!ok) *abort_flag = 1;
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 9)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512) : "memory");
}

// ---------------------------------------------------------------------------
// The merge: a thread block per 16 query rows of a (sequence, KV head), a warp per
// row in turn.  Lane x finds range r0 + x's piece of the row's unit (two divisions
// for all of a warp's rows of one unit); the states are joined as in the other
// merges, 8 pieces' loads at a time.  Units that one range held are done.
// ---------------------------------------------------------------------------
constexpr int kTMergeRows = 16;
constexpr int kTMergeWarps = 4;

template <int D, int NQ>
__global__ void __launch_bounds__(kTMergeWarps * 32)
    tree_merge_kernel(const __grid_constant__ TreeParams p, int ranges) {
  constexpr int N = D / 32, kBatch = 8, kUnit = kTreeRows * NQ;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int b = blockIdx.z, g = blockIdx.y, shift = p.group_shift;
  pdl_wait_and_release();
  const TreeSeq sq = p.seqs[b];
  const int64_t V = p.seqs[p.batch].cost, R = ranges;
  const int rows = sq.n << shift, row0 = blockIdx.x * kTMergeRows;
  if (row0 >= rows) return;
  const int units = tree_units<NQ>(rows), kt = tree_tiles(sq.ctx), unit = row0 / kUnit;   // (16 rows lie in one unit)
  const int64_t cost = tree_unit_cost(rows, kt), u0 = sq.cost + (static_cast<int64_t>(g) * units + unit) * cost;
  // ranges whose part of the axis meets the unit: r0 .. r1
  const int64_t r0 = div_nonneg((u0 + 1) * R + V - 1, V) - 1;
  const int64_t r1 = div_nonneg((u0 + cost) * R + V - 1, V) - 1;
  auto tiles_of = [&](int64_t r, int& t0, int& t1) {
    t0 = tree_tile_at(max(div_nonneg(r * V, R) - u0, static_cast<int64_t>(0)), rows, kt);
    t1 = tree_tile_at(max(min(div_nonneg((r + 1) * V, R) - u0, cost), static_cast<int64_t>(0)), rows, kt);
  };
  const int64_t base = tree_piece_row(sq.start, p.n_q_heads, g, rows, static_cast<int64_t>(unit) * kUnit, 0, kUnit);
  for (int row = row0 + warp; row < min(row0 + kTMergeRows, rows); row += kTMergeWarps) {
    float M = -INFINITY, Lsum = 0.f, O[N] = {};
    for (int64_t x0 = r0; x0 <= r1; x0 += 32) {
      const int64_t r = x0 + lane;
      int t0 = 0, t1 = 0;
      if (r <= r1) tiles_of(r, t0, t1);
      if (__any_sync(0xffffffffu, t0 == 0 && t1 == kt)) return;      // written where it was computed
      const bool have = t0 < t1;
      const int64_t at = base + r * kUnit + (row - unit * kUnit);
      const float2 st = have ? *reinterpret_cast<const float2*>(p.ml + at * 2) : make_float2(-INFINITY, 0.f);
      uint32_t left = __ballot_sync(0xffffffffu, have);
      float m = st.x;
#pragma unroll
      for (int k = 16; k >= 1; k >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, k));
      const float mn = fmaxf(M, m), ref = (mn == -INFINITY) ? 0.f : mn;
      const float keep = exp2f(M - ref), w = exp2f(st.x - ref);
      float l = w * st.y;
#pragma unroll
      for (int k = 16; k >= 1; k >>= 1) l += __shfl_xor_sync(0xffffffffu, l, k);
      Lsum = Lsum * keep + l;
      M = mn;
#pragma unroll
      for (int e = 0; e < N; ++e) O[e] *= keep;
      while (left) {
        float v[kBatch][N];
        int src[kBatch];
#pragma unroll
        for (int q = 0; q < kBatch; ++q) {
          src[q] = left ? __ffs(left) - 1 : -1;
          left &= left - 1;          // (0 stays 0)
          if (src[q] >= 0) {
            const float* from =
                p.o + (base + (x0 + src[q]) * kUnit + (row - unit * kUnit)) * D + N * lane;
            if constexpr (N == 4) {
              const float4 f = *reinterpret_cast<const float4*>(from);
              v[q][0] = f.x, v[q][1] = f.y, v[q][2] = f.z, v[q][3] = f.w;
            } else {
              const float2 f = *reinterpret_cast<const float2*>(from);
              v[q][0] = f.x, v[q][1] = f.y;
            }
          }
        }
#pragma unroll
        for (int q = 0; q < kBatch; ++q) {
          const float wq = __shfl_sync(0xffffffffu, w, src[q] < 0 ? 0 : src[q]);
          if (src[q] >= 0)
#pragma unroll
            for (int e = 0; e < N; ++e) O[e] = fmaf(wq, v[q][e], O[e]);
        }
      }
    }
    const float inv = Lsum > 0.f ? 1.f / Lsum : 0.f;
    const int node = row >> shift, head = (g << shift) + (row & ((1 << shift) - 1));
    uint16_t* out = static_cast<uint16_t*>(p.out) +
                    ((static_cast<int64_t>(sq.start) + node) * p.n_q_heads + head) * D + N * lane;
    uint32_t w[N / 2];
#pragma unroll
    for (int e = 0; e < N; e += 2)
      w[e / 2] = p.q_bf16 ? pack2(O[e] * inv, O[e + 1] * inv, BF16{}) : pack2(O[e] * inv, O[e + 1] * inv, F16{});
    if constexpr (N == 4)
      *reinterpret_cast<uint2*>(out) = make_uint2(w[0], w[1]);
    else
      *reinterpret_cast<uint32_t*>(out) = w[0];
  }
}

template <typename MT, typename KV, int D, int NQ>
pkv_status launch_tree(TreeParams& p, int ranges, cudaStream_t stream) {
  using L = TreeSmem<D, KV::kBytes == 1, NQ>;
  auto kern = tree_kernel<MT, KV, D, NQ>;
  constexpr int kDevices = 64;
  int dev = 0;
  if (cuda_failed(cudaGetDevice(&dev), "cudaGetDevice")) return PKV_ERR_CUDA;
  static std::mutex mu;
  static bool done[kDevices] = {};
  if (dev < 0 || dev >= kDevices) return PKV_ERR_UNSUPPORTED;
  {
    std::lock_guard<std::mutex> lock(mu);
    if (!done[dev]) {
      if (cuda_failed(cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                           static_cast<int>(L::bytes(kTreeMaxBatch))),
                      "cudaFuncSetAttribute"))
        return PKV_ERR_CUDA;
      done[dev] = true;
    }
  }
  if (cuda_failed(launch_pdl(kern, dim3(static_cast<unsigned>(ranges)), dim3(kTThreads), L::bytes(p.batch), stream, p),
                  "tree_kernel launch"))
    return PKV_ERR_CUDA;
  const unsigned chunks = ((p.max_nodes << p.group_shift) + kTMergeRows - 1) / kTMergeRows;
  const dim3 grid(chunks, static_cast<unsigned>(p.n_kv_heads), static_cast<unsigned>(p.batch));
  return cuda_failed(launch_pdl(tree_merge_kernel<D, NQ>, grid, dim3(kTMergeWarps * 32), 0, stream, p, ranges),
                     "tree_merge_kernel launch")
             ? PKV_ERR_CUDA
             : PKV_OK;
}

template <typename MT, typename KV>
TreeLauncher pick_tree(int head_dim, int q_tiles) {
  if (head_dim == 64) return q_tiles == 1 ? launch_tree<MT, KV, 64, 1> : launch_tree<MT, KV, 64, 2>;
  return q_tiles == 1 ? launch_tree<MT, KV, 128, 1> : launch_tree<MT, KV, 128, 2>;
}

}  // namespace pkv

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
//   S = Q K^T     into one of the S / P buffers in TMEM (three beside one row
//                 tile, one per group beside two)
//   softmax       two groups of 4 warps, one thread per row, take operations in
//                 turn, so that one group's waits and loads overlap the other's
//                 exponentials.  Of one row tile the groups take key tiles in turn
//                 and share its outputs: each passes the row's reference on through
//                 shared memory before its exponentials.  Of two row tiles, each
//                 has its own.  P overwrites S.  bf16 P is two bf16 parts (p
//                 truncated, the rounded remainder: exact to 2^-16, where one
//                 rounding, 2^-9, would be as large as the output's own); fp16 P
//                 (2^-12) is rounded once, and l sums the rounded values.  The row
//                 reference moves only when a tile's maximum exceeds it by more
//                 than 2^8; only then is O rescaled.  fp16 weights are held times
//                 2^7, so that the largest, 2^15, stays below fp16's and the
//                 smallest step is 2^-31 of a row's largest weight (unscaled, one
//                 key 17 nats above a long context took a fifth of the others).
//                 With one query head per KV head (ONE), where the dense decode
//                 keeps p in fp32, fp16 P is two fp16 parts.  (8 and 8 heads: the 32
//                 sequences below in fp16 124 us, 122 with one part; the 16 in E4M3
//                 109 us, 89: V is read twice from shared memory, which bounds it.)
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
// FP8 caches.  K's codes are an operand as they are (kind::f8f6f4, twice the rate
// of fp16), so q is too: per row q 2^k, k such that its largest element lies in
// [128, 256), is the sum of E4M3 parts -- the code of the element, of what is left,
// and (fp16 q) of what is left of that -- two for bf16's 8 bits, three for fp16's 11.
// They hold elements down to 2^-9 (2^-6) of the row's largest, and smaller ones to half
// a step of E4M3's denormals, 2^-17 of the largest.  Beside an outlier that is too little
// for the rest of a row: where an eighth of a row's elements or more are not held, its
// unit takes the parts behind the first in E5M2, which hold elements down to 2^-13 and
// smaller ones to 2^-21 (2^-24).  (Products with them take longer: E4M3 contexts 105 us
// where all units took them, else 97.)  2^-k joins the row's softmax scale, of which only
// K's sign goes with the parts: so the maximum of a row's scores is that of the scaled
// ones.  A scale may be 0 or not a number: scores are masked behind it.  A launch of its
// own writes the parts to the workspace (in the kernel, per piece, four warps took 6 to
// 13 us).  V's codes are converted to fp16 tiles, exactly, by eight warps (one
// instruction for two E4M3 codes, one byte permutation for two E5M2 ones; with four
// warps 106 us instead of 100).  With K converted as well, shared memory took 3900
// clocks a tile.
//
// Prompt chunks (CHUNK).  The same kernel attends the new tokens of a prompt to the
// first tokens and a window: a thread block per unit, whose key tiles are those
// that hold a key of one of its rows; what a row sees is a range of positions and
// the first num_sinks.
//
// Warps 0-7: softmax; 8 and 11: producers; 9: TMEM owner and Q K^T issuer; 10:
// P V issuer; from 12 on: rows of V with drafted tokens (four warps), or the
// conversions of V (eight).  The softmax warps take registers from the others.
// (Sixteen of them, two threads a row, were slower: 149 us instead of 136 for one
// document of 131072, 557 instead of 479 for the prompts below.)  Waits are bounded
// as in the other kernels.
//
// Measured (inputs taken in turn, everything with its launches; figures above and below
// that compare two forms are calls on one input): 32 sequences of 1024 to 16384 tokens
// with 20 to 32 drafted ones, 32 and 8 heads of 128, bf16: 136 us, of which 10 are the
// merge; the reads alone take 112 at 6.80 TB/s.  One of 131072 with 64, fp16: 132 us (79);
// each row tile's softmax, P V and next Q K^T wait for each other (4500 clocks, 2048 of
// them products).  16 of 4096 to 32768 with 10 to 31, E4M3 and E5M2: 100 us (57): shared
// memory feeds the products, the conversions and the loads in turn.  Four prompts of 2048
// tokens, window 4096: 474 us; the products with bf16's second part take 318.  A prompt
// chunk of 16 tokens alone: 41 us, eight thread blocks with 33 key tiles each, one after
// another (no split over the keys).
#pragma once

#include <cuda_runtime.h>

#include <algorithm>
#include <mutex>

#include "decode.cuh"
#include "pkv_common.cuh"
#include "tcgen05.cuh"
#include "tree.h"

namespace pkv {

constexpr int kTSoftmax = 256;
constexpr int kTTileBlocks = kTreeKeys / kBlockSize;
constexpr float kTRescaleLog2 = 8.f;
constexpr float kTHalfLog2 = 7.f;        // fp16 weights: of 2^15 at most
static_assert(kTRescaleLog2 + kTHalfLog2 < 16.f, "fp16 weights");
// Pieces whose remembered tokens live at once.  While a piece's outputs are read no P V
// of the next one runs, so the warps that look at V are at most kVStages tiles ahead,
// and clear the slot of the piece behind those.
constexpr int kTBadSlots = 5;

// Cost of a unit's set-up (Q, the first tile's latency, its outputs) and of a key
// tile against one row tile or two, in half tiles.  An FP8 tile is half the bytes, so
// the set-up is more of them.  Measured with 6, 12, 16: mixed contexts up to 16384
// over a 16-bit cache 132, 136, 138 us, up to 32768 over an FP8 one 99.6, 96.6, 96.3.
constexpr int tree_setup_cost(bool fp8) { return fp8 ? 14 : 6; }
__host__ __device__ constexpr int tree_tile_cost(int rows) { return rows > kTreeRows ? 3 : 2; }

template <int D, bool FP8, int NQ>
struct TreeSmem {
  // Warps that convert codes (or look at V rows) behind the first twelve, and the
  // registers that the softmax warps take from the others.  (144, 152 and 160 make little
  // difference over 16-bit caches: one document of 131072, fp16, 133.3, 132.8, 132.5 us,
  // four prompts 469.6, 473.5, 474.8.  E4M3 contexts with 120, 136, 144, 152: 97.6, 95.2,
  // 95.2, 98.1.)
  static constexpr int kXform = FP8 ? 8 : 4;
  static constexpr int kThreads = 384 + 32 * kXform;
  static constexpr int kRegs = 65536 / kThreads / 8 * 8;           // a thread, at launch
  static constexpr int kRegsSoftmax = FP8 ? 144 : 160, kRegsOther = FP8 ? 64 : 96;
  static_assert(kTSoftmax * kRegsSoftmax + (kThreads - kTSoftmax) * kRegsOther <= kThreads * kRegs, "registers");
  static constexpr int kTile = kTreeKeys * D * 2;                  // a Q, K or V tile
  static constexpr int kStage = kTile / 2;                         // FP8: a staged tile of codes
  static constexpr int kKStages = FP8 ? 4 - NQ : 2;
  static constexpr int kVStages = FP8 ? 3 - NQ : 4 - NQ;
  static constexpr int kCodeStages = FP8 ? 2 : 0;                  // of V
  static constexpr int kParts = FP8 ? 3 : 1;                       // of q
  static constexpr int kQTile = FP8 ? kParts * kStage : kTile;
  static constexpr int kKTile = FP8 ? kStage : kTile;
  static constexpr int kQ = 0;
  static constexpr int kK = NQ * kQTile;
  static constexpr int kV = kK + kKStages * kKTile;
  static constexpr int kCodes = kV + kVStages * kTile;
  static constexpr int kBar = kCodes + kCodeStages * kStage;       // 512 bytes
  static constexpr int kBad = kBar + 512;                          // uint32 [slots][warps][8]
  static constexpr int kRed = kBad + kTBadSlots * kXform * 32;     // float [128] references, [2][2][128] sums
  static constexpr int kSeqs = kRed + 5 * kTreeRows * 4;           // TreeSeq [batch + 1]
  static __host__ __device__ constexpr size_t bytes(int batch) {
    return 1024 + kSeqs + sizeof(TreeSeq) * (static_cast<size_t>(batch) + 1);
  }
  static_assert(kTBadSlots >= kVStages + 2, "slots");
  // S / P buffers, and the outputs behind them
  static constexpr int kSBufs = 4 - NQ;
  static constexpr int kOCol = kSBufs * kTreeKeys;
  // 8-key groups of a K / V tile and the 64-element halves of a row
  static constexpr int kGroup = 1024 * (D / 64);
  static constexpr int kHalf = 1024;
  static constexpr int kHalfQ = kTreeRows * 128;
  // FP8 operands: rows of D bytes, 8-row atoms of the D-byte swizzle
  static constexpr int kCodeGroup = 8 * D;
};
static_assert(TreeSmem<128, false, 1>::bytes(kTreeMaxBatch) <= 232448, "16-bit tiles");
static_assert(TreeSmem<128, false, 2>::bytes(kTreeMaxBatch) <= 232448, "16-bit tiles");
static_assert(TreeSmem<128, true, 1>::bytes(kTreeMaxBatch) <= 232448, "FP8 tiles");
static_assert(TreeSmem<128, true, 2>::bytes(kTreeMaxBatch) <= 232448, "FP8 tiles");

// a piece of a range: key tiles [t0, t1) of one unit
struct TreeSeg {
  int64_t next;                  // cost position behind it
  int64_t row;                   // first row of its states
  int b, g, unit, rows, t0, t1, kt;
  int gap_at, skip;              // CHUNK: skip tiles are left out in front of the gap_at-th one
  int pos0, pos1;                // CHUNK: positions of the unit's first and last token
  int low0, low1;                // and the first ones of their windows
};

// units of a sequence's rows, key tiles of its context, cost of one unit
template <int NQ>
__device__ __forceinline__ int tree_units(int rows) { return (rows + kTreeRows * NQ - 1) / (kTreeRows * NQ); }
__device__ __forceinline__ int tree_tiles(int ctx) { return ctx / kTreeKeys + (ctx % kTreeKeys != 0); }
__device__ __forceinline__ int64_t tree_unit_cost(int rows, int kt, int setup) {
  return setup + static_cast<int64_t>(kt) * tree_tile_cost(rows);
}
// sequence b with its own cost; one that is not to be attended has no tokens and cost 0
template <int NQ>
__device__ __forceinline__ TreeSeq tree_sequence(const TreeParams& p, int b, int32_t* err) {
  const int64_t t0 = p.cu_nodes[b], t1 = p.cu_nodes[b + 1], n = t1 - t0;
  const int ctx = p.context_lens[b];
  if (t0 < 0 || n < 0 || t1 > p.num_tokens || n > p.max_nodes || ctx < n ||
      ctx > static_cast<int64_t>(p.max_blocks_per_seq) * kBlockSize) {
    record_error(err, PKV_ERR_OOB);
    return TreeSeq{0, 0, 0, 0, 0};
  }
  if (n == 0) return TreeSeq{0, 0, 0, 0, 0};
  const int rows = static_cast<int>(n) << p.group_shift;
  return TreeSeq{p.n_kv_heads * tree_units<NQ>(rows) * tree_unit_cost(rows, tree_tiles(ctx), p.setup_cost),
                 static_cast<int>(t0), static_cast<int>(n), ctx, 0};
}
// first tile at or behind position x of its unit's cost
__device__ __forceinline__ int tree_tile_at(int64_t x, int rows, int kt, int setup) {
  if (x <= setup) return 0;
  const int w = tree_tile_cost(rows);
  return static_cast<int>(min(static_cast<int64_t>(kt), div_nonneg(x - setup + w - 1, w)));
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
                                                int64_t end, int64_t range, int setup) {
  int lo = 0, hi = batch - 1;    // the last sequence that starts at or before pos (a non-empty one)
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (seqs[mid].cost <= pos) lo = mid; else hi = mid - 1;
  }
  const TreeSeq sq = seqs[lo];
  const int rows = sq.n << shift, units = tree_units<NQ>(rows), kt = tree_tiles(sq.ctx);
  const int64_t cost = tree_unit_cost(rows, kt, setup), rem = pos - sq.cost;
  const int64_t u = div_nonneg(rem, cost), off = rem - u * cost;
  TreeSeg s;
  s.b = lo;
  s.g = static_cast<int>(u) / units;
  s.unit = static_cast<int>(u) - s.g * units;
  s.kt = kt;
  s.t0 = tree_tile_at(off, rows, kt, setup);
  s.t1 = tree_tile_at(off + (end - pos), rows, kt, setup);
  s.next = pos + min(cost - off, end - pos);
  s.rows = min(kTreeRows * NQ, rows - s.unit * kTreeRows * NQ);
  s.row = tree_piece_row(sq.start, n_q_heads, s.g, rows, static_cast<int64_t>(s.unit) * kTreeRows * NQ, range,
                         kTreeRows * NQ);
  return s;
}

// CHUNK: the only piece of a thread block, unit `unit` of sequence sq
__device__ __forceinline__ TreeSeg chunk_segment(const TreeSeq& sq, int b, int g, int unit, int unit_rows, int shift,
                                                 int window, int sinks) {
  TreeSeg s{};
  s.next = 1;
  s.b = b, s.g = g, s.unit = unit;
  s.rows = min(unit_rows, (sq.n << shift) - unit * unit_rows);
  if (s.rows <= 0) return s;     // (t0 == t1)
  const int tok = (unit * unit_rows) >> shift;
  s.pos0 = sq.ctx - sq.n + tok;
  s.pos1 = s.pos0 + (s.rows >> shift) - 1;
  s.low0 = max(0, s.pos0 - window + 1);
  s.low1 = max(0, s.pos1 - window + 1);
  s.gap_at = sinks / kTreeKeys + (sinks % kTreeKeys != 0);
  s.skip = max(0, s.low0 / kTreeKeys - s.gap_at);
  s.t1 = s.kt = s.pos1 / kTreeKeys + 1 - s.skip;
  return s;
}
// does every row of the unit see every key of tile t?
__device__ __forceinline__ bool chunk_plain(const TreeSeg& s, int t, int sinks) {
  const int k0 = t * kTreeKeys, k1 = k0 + kTreeKeys - 1;
  return k1 <= s.pos0 && (k0 >= s.low1 || k1 < sinks);
}
// bits of the 32 keys from key0 on that are below x
__device__ __forceinline__ uint32_t keys_below(int x, int key0) {
  const int d = x - key0;
  return d <= 0 ? 0u : d >= 32 ? 0xffffffffu : (1u << d) - 1u;
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

// four codes of a word -> halves
__device__ __forceinline__ uint2 codes4(uint32_t w, E5M2) {
  return make_uint2(__byte_perm(w, 0u, 0x1404), __byte_perm(w, 0u, 0x3424));
}
__device__ __forceinline__ uint2 codes4(uint32_t w, E4M3) {
  uint2 d;
  asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, lo;\n\tcvt.rn.f16x2.e4m3x2 %1, hi;\n\t}"
      : "=r"(d.x), "=r"(d.y)
      : "r"(w));
  return d;
}

// sums of an fp32 number and a 16-bit one, in one instruction each
__device__ __forceinline__ void add_halves(uint32_t w, float& a, float& b) {   // a, b += the halves of w
  asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %2;\n\tadd.f32.f16 %0, lo, %0;\n\tadd.f32.f16 %1, hi, %1;\n\t}"
      : "+f"(a), "+f"(b)
      : "r"(w));
}
__device__ __forceinline__ float2 less16(float a, float b, uint32_t w, F16) {  // a, b - the halves of w
  float2 d;
  asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %2;\n\t"
      "fma.rn.f32.f16 %0, lo, %5, %3;\n\tfma.rn.f32.f16 %1, hi, %5, %4;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "r"(w), "f"(a), "f"(b), "h"(static_cast<uint16_t>(0xbc00)));           // (times -1)
  return d;
}
__device__ __forceinline__ float2 less16(float a, float b, uint32_t w, BF16) { // a, b - the bf16 numbers of w
  float2 d;
  asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %2;\n\t"
      "fma.rn.f32.bf16 %0, lo, %5, %3;\n\tfma.rn.f32.bf16 %1, hi, %5, %4;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "r"(w), "f"(a), "f"(b), "h"(static_cast<uint16_t>(0xbf80)));           // (times -1)
  return d;
}

// descriptor of an FP8 operand: rows of D bytes, K-major, D-byte swizzle
template <int D>
__device__ __forceinline__ uint64_t umma_desc_codes(uint32_t saddr) {
  return static_cast<uint64_t>((saddr >> 4) & 0x3FFF) | (1ull << 16) |
         (static_cast<uint64_t>((8 * D) >> 4) << 32) | (1ull << 46) | ((D == 128 ? 2ull : 4ull) << 61);
}
// kind::f8f6f4: A in E4M3 or E5M2, B in KV, fp32 accumulate, both K-major, M = 128
template <typename KV>
__host__ __device__ constexpr uint32_t umma_idesc_codes(int n, bool a_e5m2) {
  return (1u << 4) | ((a_e5m2 ? 1u : 0u) << 7) | ((std::is_same<KV, E5M2>::value ? 1u : 0u) << 10) |
         (static_cast<uint32_t>(n >> 3) << 17) | (static_cast<uint32_t>(128 >> 4) << 24);
}
// D += A B over 32 STEPS elements of K: successive 32-byte steps of the descriptors.  (As
// statements of their own, E4M3 contexts took 104 us instead of 97 once the instruction
// descriptor was no constant: the issuer is in the chain of a tile's scores.)
template <int STEPS>
__device__ __forceinline__ void umma_f8(uint32_t d_tmem, uint64_t a, uint64_t b, uint32_t idesc, bool acc) {
  static_assert(STEPS == 2 || STEPS == 4, "rows of 64 or 128 bytes");
  if constexpr (STEPS == 4)
    asm volatile(
        "{\n\t.reg .pred p, t;\n\t.reg .b64 a1, a2, a3, b1, b2, b3;\n\t"
        "setp.ne.u32 p, %4, 0;\n\tsetp.eq.u32 t, 0, 0;\n\t"
        "add.u64 a1, %1, 2;\n\tadd.u64 a2, %1, 4;\n\tadd.u64 a3, %1, 6;\n\t"
        "add.u64 b1, %2, 2;\n\tadd.u64 b2, %2, 4;\n\tadd.u64 b3, %2, 6;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], a1, b1, %3, t;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], a2, b2, %3, t;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], a3, b3, %3, t;\n\t}" ::"r"(d_tmem),
        "l"(a), "l"(b), "r"(idesc), "r"(static_cast<uint32_t>(acc))
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p, t;\n\t.reg .b64 a1, b1;\n\tsetp.ne.u32 p, %4, 0;\n\tsetp.eq.u32 t, 0, 0;\n\t"
        "add.u64 a1, %1, 2;\n\tadd.u64 b1, %2, 2;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], a1, b1, %3, t;\n\t}" ::"r"(d_tmem),
        "l"(a), "l"(b), "r"(idesc), "r"(static_cast<uint32_t>(acc))
        : "memory");
}

// mbar_wait that gives up early once the block has stopped
__device__ __forceinline__ bool tree_wait(uint64_t* bar, uint32_t parity, const TreeParams& p,
                                          const volatile int* abort_flag) {
  if (mbar_try_wait(bar, parity)) return true;
  const unsigned long long t0 = global_ns();
  while (!mbar_try_wait(bar, parity)) {
    if (*abort_flag) return false;
    if (global_ns() - t0 > p.wait_limit_ns) {
      record_error(p.err, PKV_ERR_TIMEOUT);
      return false;
    }
  }
  return true;
}

template <int N>
__device__ __forceinline__ void set_max_regs_up() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void set_max_regs_down() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

// and for what another warp does only once the previous kernel is over: a limit that runs
// out while that kernel runs starts anew at its end
inline __device__ __noinline__ bool tree_wait_from_previous_end(uint64_t* bar, uint32_t parity, const TreeParams* p,
                                                                const volatile int* abort_flag) {
  pdl_wait();
  return tree_wait(bar, parity, *p, abort_flag);
}
__device__ __forceinline__ bool tree_wait_started_early(uint64_t* bar, uint32_t parity, const TreeParams& p,
                                                        const volatile int* abort_flag) {
  if (mbar_try_wait(bar, parity)) return true;
  const unsigned long long t0 = global_ns();
  while (!mbar_try_wait(bar, parity)) {
    if (*abort_flag) return false;
    if (global_ns() - t0 > p.wait_limit_ns) return tree_wait_from_previous_end(bar, parity, &p, abort_flag);
  }
  return true;
}

// MT: 16-bit type of the products; KV: the cache's (MT, or an FP8 format); ONE: one query
// head per KV head (fp16 products)
template <typename MT, typename KV, int D, int NQ, bool CHUNK, bool ONE>
__global__ void __launch_bounds__((TreeSmem<D, KV::kBytes == 1, NQ>::kThreads), 1) tree_kernel(const __grid_constant__ TreeParams p) {
  constexpr bool kFp8 = KV::kBytes == 1;
  using L = TreeSmem<D, kFp8, NQ>;
  constexpr bool kSplit = std::is_same<MT, BF16>::value || ONE;   // P in two parts
  constexpr int NB = L::kSBufs;
  static_assert(!CHUNK || !kFp8, "prompt chunks: 16-bit caches");
  static_assert(!ONE || (!CHUNK && std::is_same<MT, F16>::value), "one query head: fp16 products");
  constexpr int kBadWords = CHUNK ? 16 : 8;        // of remembered tokens
  static_assert(!CHUNK || L::kXform * 16 <= kTBadSlots * L::kXform * 8, "remembered tokens");
  extern __shared__ unsigned char tsm_raw[];
  unsigned char* sm = tsm_raw + ((1024 - (smem_u32(tsm_raw) & 1023)) & 1023);
  uint64_t* k_full = reinterpret_cast<uint64_t*>(sm + L::kBar);   // [kKStages] K tile landed
  uint64_t* k_empty = k_full + L::kKStages;        // its Q K^T done
  uint64_t* v_full = k_empty + L::kKStages;        // [kVStages] V tile landed (16-bit)
  uint64_t* v_ready = v_full + L::kVStages;        // its rows looked at, or converted
  uint64_t* v_empty = v_ready + L::kVStages;       // its P V done
  uint64_t* c_full = v_empty + L::kVStages;        // [kCodeStages] codes of V landed
  uint64_t* c_empty = c_full + L::kCodeStages;     // converted
  uint64_t* s_full = c_empty + L::kCodeStages;     // [NB] scores ready
  uint64_t* p_half = s_full + NB;                  // [NB] P of the upper keys written, O rescaled
  uint64_t* p_full = p_half + NB;                  // [NB] and of the lower ones
  uint64_t* pv_done = p_full + NB;                 // [NB] P V done
  uint64_t* q_full = pv_done + NB;                 // Q of a piece landed
  uint64_t* q_empty = q_full + 1;                  // its Q K^T done
  uint64_t* turn = q_empty + 1;                    // [2][4] a group's warp has passed its rows' references on
  uint64_t* joined = turn + 8;                     // [2][4] and its sums of a piece
  uint64_t* o_read = joined + 8;                   // 8 arrivals: a piece's outputs are out of TMEM
  uint64_t* mma_idle = o_read + 1;                 // [2] an issuer's MMAs done
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(mma_idle + 2);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  volatile int* far_parts = abort_flag + 1;        // FP8: the piece's parts behind the first are E5M2
  static_assert((2 * 3 + 3 * 3 + 2 * 2 + 4 * 3 + 5 + 17 + 2 + 2) * 8 <= 512, "barrier block overflows");
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
      mbar_init(&k_full[s], 1);
      mbar_init(&k_empty[s], 1);
    }
    for (int s = 0; s < L::kVStages; ++s) {
      mbar_init(&v_full[s], 1);
      mbar_init(&v_ready[s], L::kXform);
      mbar_init(&v_empty[s], 1);
    }
    for (int s = 0; s < L::kCodeStages; ++s) {
      mbar_init(&c_full[s], 1);
      mbar_init(&c_empty[s], L::kXform);
    }
    for (int s = 0; s < NB; ++s) {
      mbar_init(&s_full[s], 1);
      mbar_init(&p_half[s], kTSoftmax / 2);
      mbar_init(&p_full[s], kTSoftmax / 2);
      mbar_init(&pv_done[s], 1);
    }
    mbar_init(q_full, 1);
    mbar_init(q_empty, 1);
    for (int s = 0; s < 8; ++s) {
      mbar_init(&turn[s], 1);
      mbar_init(&joined[s], 1);
    }
    mbar_init(o_read, kTSoftmax / 32);
    mbar_init(&mma_idle[0], 1);
    mbar_init(&mma_idle[1], 1);
    fence_mbar_init();
  }
  // Until the waits below this kernel reads lengths, offsets and (in the producer)
  // tables only, which no kernel that releases early writes.

  // ---- the sequences: drafted (or new) tokens, context, cost ----
  if constexpr (CHUNK) {
    if (tid == 0) seqs[0] = tree_sequence<NQ>(p, blockIdx.z, p.err);
  } else {
    for (int b = tid; b < p.batch; b += L::kThreads) seqs[b] = tree_sequence<NQ>(p, b, p.err);
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
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (!CHUNK && blockIdx.x == 0) {
    pdl_wait();
    for (int b = tid; b <= p.batch; b += L::kThreads) p.seqs[b] = seqs[b];
  }
  const uint32_t tmem = *tmem_slot;
  const int64_t V = CHUNK ? 1 : seqs[p.batch].cost, R = CHUNK ? 1 : gridDim.x, range = CHUNK ? 0 : blockIdx.x;
  const int64_t first = div_nonneg(range * V, R), end = div_nonneg((range + 1) * V, R);
  auto segment = [&](int64_t pos) {
    if constexpr (CHUNK)   // (the longest units first)
      return chunk_segment(seqs[0], blockIdx.z, blockIdx.y, gridDim.x - 1 - blockIdx.x, kTreeRows * NQ, shift, p.window,
                           p.num_sinks);
    else
      return tree_segment<NQ>(seqs, p.batch, shift, p.n_q_heads, pos, end, range, p.setup_cost);
  };
  auto sequence_of = [&](const TreeSeg& sg) { return seqs[CHUNK ? 0 : sg.b]; };
  // key tile at place x of a piece's order
  auto tile_at = [&](const TreeSeg& sg, int x) { return CHUNK && x >= sg.gap_at ? x + sg.skip : x; };

  if (warp < 8) {
    // ============================ softmax / epilogue ============================
    set_max_regs_up<L::kRegsSoftmax>();
    const int grp = warp >> 2, quarter = warp & 3, r = tid & (kTreeRows - 1);
    const uint32_t lane_base = static_cast<uint32_t>(quarter * 32) << 16;
    uint64_t* my_turn = &turn[grp * 4 + quarter];
    uint64_t* their_turn = &turn[(1 - grp) * 4 + quarter];
    uint32_t ops = 0;                                // operations of the pieces before
    uint32_t turns = 0;                              // references taken over so far
    uint32_t joins = 0;                              // pieces whose sums were exchanged
    uint32_t slot = 0;                               // of remembered tokens
    bool ok = true;
    auto wait = [&](uint64_t* bar, uint32_t parity) {
      return __all_sync(0xffffffffu, tree_wait(bar, parity, p, abort_flag));
    };
    pdl_wait();
    for (int64_t pos = first; pos < end && ok;) {
      const TreeSeg sg = segment(pos);
      pos = sg.next;
      if (sg.t0 >= sg.t1) continue;
      const TreeSeq sq = sequence_of(sg);
      const int base = sq.ctx - sq.n, nt = sg.t1 - sg.t0;
      const bool two = NQ == 2 && sg.rows > kTreeRows;                // a row tile per group
      const int tile = two ? grp : 0, row0 = tile * kTreeRows + quarter * 32, row = row0 + lane;
      const bool live = row0 < sg.rows;                               // any row of this warp
      const int unit_row = sg.unit * kTreeRows * NQ + row;            // of the sequence's rows
      const int node = min(unit_row >> shift, sq.n - 1);
      const uint32_t* words = p.mask + (static_cast<int64_t>(sq.start) + node) * (2 * p.mask_words);
      // (FP8: q's parts, and so the scores, are scaled by row, and hold K's sign; the sign of
      // a row's scale tells which parts it needs)
      const float scale_log2 =
          p.qk_scale_log2 *
          (kFp8 ? fabsf(p.k_scale[sg.g] * p.part_scale[(static_cast<int64_t>(sq.start) + node) * p.n_q_heads +
                                                       (sg.g << shift) + (unit_row & ((1 << shift) - 1))])
                : 1.f);
      const uint32_t to = tmem + lane_base + L::kOCol + tile * D;
      float m_ref = -INFINITY, l_run = 0.f;
      // take over the row's reference of the operation before
      auto take_turn = [&]() -> bool {
        const bool got = wait(their_turn, turns & 1);
        ++turns;
        const float m = red[r];
        if (m != m_ref) l_run *= ex2_approx(m_ref - m);
        m_ref = m;
        return got;
      };
      // A warp waits for a phase of a barrier only where the phase behind it needs
      // that warp, and only once the phase before it is known to be over (a parity
      // tells no more than two apart).  So a warp without rows takes part in
      // everything but the arithmetic.
      for (int n = two ? 0 : grp; n < nt; n += two ? 1 : 2) {
        const uint32_t k = ops + (two ? 2 * n + grp : n), buf = k % NB, ph = (k / NB) & 1;
        if (!live) {
          ok = wait(&s_full[buf], ph) && (two || n == 0 || take_turn());
          if (!ok) break;
          if (!two && lane == 0) mbar_arrive(my_turn);
          mbar_arrive(&p_half[buf]);
          mbar_arrive(&p_full[buf]);
          continue;
        }
        const int t = tile_at(sg, sg.t1 - 1 - n);
        const bool tail = CHUNK ? !chunk_plain(sg, t, p.num_sinks) : t * kTreeKeys > base - kTreeKeys;
        uint32_t see[4] = {0xffffffffu, 0xffffffffu, 0xffffffffu, 0xffffffffu};
        if (tail) {
#pragma unroll
          for (int w = 0; w < 4; ++w) {
            const int key0 = t * kTreeKeys + 32 * w;
            if constexpr (CHUNK)
              see[w] = keys_below(base + node + 1, key0) &
                       (~keys_below(max(0, base + node + 1 - p.window), key0) | keys_below(p.num_sinks, key0));
            else
              see[w] = tree_bits(words, 2 * p.mask_words, sq.n, key0 - base);
          }
        }
        const uint32_t ts = tmem + lane_base + buf * kTreeKeys;
        // (the scores of two operations before, its own or before its last turn, are
        // known to be over, and so is the buffer's phase before, at least as old)
        ok = wait(&s_full[buf], ph);
        if (!ok) break;
        tc_fence_after();
        if (tail) {
          // masked where they lie: the loops below stay short (FP8: scaled first, for a
          // scale of 0 would make a NaN of -inf)
#pragma unroll 1
          for (int w = 0; w < 4; ++w) {
            const uint32_t bits = w < 2 ? (w == 0 ? see[0] : see[1]) : (w == 2 ? see[2] : see[3]);
            float x[32];
            tmem_ld32(ts + 32 * w, x);
#pragma unroll
            for (int i = 0; i < 32; ++i) x[i] = (bits >> i) & 1u ? (kFp8 ? x[i] * scale_log2 : x[i]) : -INFINITY;
            tmem_st32(ts + 32 * w, x);
          }
        }
        float mx = -INFINITY;
#pragma unroll 1
        for (int h = 0; h < 2; ++h) {
          float v[64];
          tmem_ld64(ts + 64 * h, v);
          mx = fmaxf(mx, max64(v));
        }
        // (the turn only now: between the groups only the references are in line)
        if (!two && n > 0) ok = take_turn();
        if (!ok) break;
        const float tile_scale = kFp8 && tail ? 1.f : scale_log2;
        const float m_tile = mx * tile_scale;
        float alpha = 1.f;
        if (m_tile > m_ref + kTRescaleLog2) {
          alpha = ex2_approx(m_ref - m_tile);
          m_ref = m_tile;
        }
        if (!two) {
          red[r] = m_ref;
          __syncwarp();
          if (lane == 0) mbar_arrive(my_turn);
        }
        if (n > 0 && __any_sync(0xffffffffu, alpha != 1.f)) {
          // O may be touched once the row tile's previous P V has completed
          const uint32_t before = k - (two ? 2 : 1);
          ok = wait(&pv_done[before % NB], (before / NB) & 1);
          if (!ok) break;
          tc_fence_after();
#pragma unroll 1
          for (int x = 0; x < D; x += 16) {
            float o[16];
            tmem_ld16(to + x, o);
#pragma unroll
            for (int i = 0; i < 16; ++i) o[i] *= alpha;
            tmem_st16(to + x, o);
          }
        }
        const float nref = (m_ref == -INFINITY) ? 0.f : (std::is_same<MT, F16>::value ? kTHalfLog2 : 0.f) - m_ref;
        const uint64_t scale2 = f32x2(tile_scale, tile_scale), nref2 = f32x2(nref, nref);
        uint64_t acc[4] = {0ull, 0ull, 0ull, 0ull};            // l's summands of this tile: two parts
        float sum[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};   // one
        // 32 keys at a time; the upper half first, whose product may run while the lower
        // keys' weights are computed.  P of a half: in two parts, for each 32 keys 16 columns
        // of pairs of the first and 16 of the second; in one, 32 columns of pairs.
        auto weights = [&](const uint32_t* x, uint32_t to_p) {
          uint32_t pk[kSplit ? 32 : 16];
#pragma unroll
          for (int j = 0; j < 32; j += 2) {
            const float2 y =
                f32x2_split(fma_f32x2(f32x2(__uint_as_float(x[j]), __uint_as_float(x[j + 1])), scale2, nref2));
            const float e0 = ex2_approx(y.x), e1 = ex2_approx(y.y);
            if constexpr (kSplit) {
              pk[j / 2] = std::is_same<MT, BF16>::value
                              ? __byte_perm(__float_as_uint(e0), __float_as_uint(e1), 0x7632)
                              : pack2(e0, e1, MT{});
              const float2 lo = less16(e0, e1, pk[j / 2], MT{});
              pk[16 + j / 2] = pack2(lo.x, lo.y, MT{});
              acc[(j / 2) & 3] = add_f32x2(acc[(j / 2) & 3], f32x2(e0, e1));
            } else {
              pk[j / 2] = pack2(e0, e1, MT{});
              add_halves(pk[j / 2], sum[j & 7], sum[(j & 7) + 1]);   // (l sums what is multiplied)
            }
          }
          if constexpr (kSplit)
            tmem_st32u(to_p, pk);
          else
            tmem_st16u(to_p, pk);
        };
        auto written = [&](int h) {
          tmem_wait_st();
          tc_fence_before();
          mbar_arrive(h ? &p_half[buf] : &p_full[buf]);
        };
        // 16-bit caches: the next 32 scores are on their way meanwhile (one long document
        // 130 -> 125 us).  Beside the conversions a shorter loop, and registers, are worth
        // more (long contexts in an E4M3 cache 104 -> 96 us).
        constexpr int kStepP = kSplit ? 32 : 16;     // columns of P of 32 keys
        uint32_t xa[32], xb[kFp8 ? 1 : 32];
        if constexpr (kFp8) {
#pragma unroll 1
          for (int i = 0; i < 4; ++i) {
            const int h = 1 - (i >> 1), c = i & 1;
            tmem_ld32_async(ts + 64 * h + 32 * c, xa);
            tmem_wait_ld32(xa);
            weights(xa, ts + 64 * h + kStepP * c);
            if (c) written(h);
          }
        } else {
          tmem_ld32_async(ts + 64, xa);
          tmem_wait_ld32(xa);
#pragma unroll 1
          for (int h = 1; h >= 0; --h) {
            tmem_ld32_async(ts + 64 * h + 32, xb);
            weights(xa, ts + 64 * h);
            tmem_wait_ld32(xb);
            tmem_ld32_async(ts, xa);                 // (behind the lower half: not used)
            weights(xb, ts + 64 * h + kStepP);
            tmem_wait_ld32(xa);
            written(h);
          }
        }
        const float2 s0 = f32x2_split(add_f32x2(add_f32x2(acc[0], acc[1]), add_f32x2(acc[2], acc[3])));
        const float s1 = ((sum[0] + sum[1]) + (sum[2] + sum[3])) + ((sum[4] + sum[5]) + (sum[6] + sum[7]));
        l_run = l_run * alpha + (kSplit ? s0.x + s0.y : s1);
      }
      if (!ok) break;
      const uint32_t last = ops + (two ? 2 * (nt - 1) + grp : nt - 1);
      ops += two ? 2 * nt : nt;
      const uint32_t piece_slot = slot++ % kTBadSlots;
      // the piece's outputs or states, once the last P V is done (with the last turn
      // taken, its scores are known to be over, and so is the buffer's P V before)
      if (!two && ((nt - 1) & 1) != grp) ok = take_turn();
      ok = ok && wait(&pv_done[last % NB], (last / NB) & 1);
      float l = l_run;
      if (!two && ok) {
        // (two slots: the other group may still read the piece's before)
        float* sums = red + kTreeRows + (joins & 1) * (2 * kTreeRows);
        sums[grp * kTreeRows + r] = l_run;
        __syncwarp();
        if (lane == 0) mbar_arrive(&joined[grp * 4 + quarter]);
        ok = ok && wait(&joined[(1 - grp) * 4 + quarter], joins & 1);
        ++joins;
        l = l_run + sums[(1 - grp) * kTreeRows + r];
      }
      if (!ok) break;
      tc_fence_after();
      if (!live) {
        if (lane == 0) mbar_arrive(o_read);
        continue;
      }
      // drafted tokens of this piece with elements of V that are not finite
      const uint32_t* noted = bad + piece_slot * (L::kXform * 8);     // [kXform][kBadWords]
      uint32_t any = 0;
      for (int w = lane; w < L::kXform * kBadWords; w += 32) any |= noted[w];
      const bool any_bad = __any_sync(0xffffffffu, any != 0u);
      const bool direct = sg.t0 == 0 && sg.t1 == sg.kt;
      const float v_scale = kFp8 ? p.v_scale[sg.g] : 1.f;
      const int n_rows = sg.rows - row0, head = (sg.g << shift) + (unit_row & ((1 << shift) - 1));
      const float weight = direct ? (l > 0.f ? v_scale / l : 0.f) : v_scale;
      // (of one row tile, each group writes half of the columns)
#pragma unroll 1
      for (int x = two ? 0 : grp * (D / 2); x < (two ? D : (grp + 1) * (D / 2)); x += 32) {
        float o[32];
        tmem_ld32(to + x, o);
#pragma unroll
        for (int i = 0; i < 32; ++i) o[i] *= weight;
        if (any_bad) {
          // (rare) every row adds what it sees of them
          for (int w = 0; w < (CHUNK ? kBadWords : 2 * p.mask_words); ++w) {
            uint32_t bits = 0;
#pragma unroll
            for (int k = 0; k < L::kXform; ++k) bits |= noted[k * kBadWords + w];
            if constexpr (!CHUNK) bits &= words[w];
            for (; bits != 0u; bits &= bits - 1u) {
              const int i0 = 32 * w + __ffs(bits) - 1;
              const int at = !CHUNK ? base + i0 : i0 < 256 ? sg.pos0 + 1 + i0 : sg.low0 + (i0 - 256);
              if (CHUNK && !(at <= base + node && (at > base + node - p.window || at < p.num_sinks))) continue;
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
                static_cast<uint16_t*>(p.out) + ((static_cast<int64_t>(sq.start) + node) * p.n_q_heads + head) * D + x);
            const bool bf16 = kFp8 ? p.q_bf16 != 0 : std::is_same<MT, BF16>::value;
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
      if (!direct && (two || grp == 0) && lane < n_rows)
        *reinterpret_cast<float2*>(p.ml + (sg.row + row) * 2) = make_float2(m_ref, l);
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(o_read);
    }
    if (!ok) *abort_flag = 1;
  } else {
    // (in front of the roles: setmaxnreg is one instruction for the four warps of a
    // warpgroup, and warps 8 to 11 have three roles)
    set_max_regs_down<L::kRegsOther>();
    if (warp == 8 || warp == 11) {
      // ============================ producers: Q and K, V ============================
      // (one warp each: V of a tile waits for an earlier P V than K of the tiles
      // behind it; one warp for both, K behind V, cost 15 % of the whole)
      const bool is_v = warp == 11;
      const bool codes_v = kFp8 && is_v;               // V's codes go to the conversion
      const uint32_t stages = codes_v ? L::kCodeStages : is_v ? L::kVStages : L::kKStages;
      uint64_t* full = codes_v ? c_full : is_v ? v_full : k_full;
      uint64_t* empty = codes_v ? c_empty : is_v ? v_empty : k_empty;
      unsigned char* ring = sm + (codes_v ? L::kCodes : is_v ? L::kV : L::kK);
      uint32_t s = 0, use = 0, tiles = 0, pieces = 0;  // stage and its use of the next tile; issued so far
      bool good = true;
      if (is_v)
        pdl_wait();
      else
        pdl_wait_and_release();
      for (int64_t pos = first; pos < end && good;) {
        const TreeSeg sg = segment(pos);
        pos = sg.next;
        if (sg.t0 >= sg.t1) continue;
        const TreeSeq sq = sequence_of(sg);
        const int nq = NQ == 2 && sg.rows > kTreeRows ? 2 : 1;
        const int nblk = ctx_blocks(sq.ctx);
        const uint64_t pol = tree_units<NQ>(sq.n << shift) > 1 ? policy_evict_last() : policy_evict_first();
        const int32_t* row = p.block_tables + static_cast<int64_t>(sg.b) * p.max_blocks_per_seq;
        // (CHUNK: blocks that no row sees a key of are not looked up)
        auto wanted = [&](int blk) -> bool {
          if (CHUNK && !(blk * kBlockSize <= sg.pos1 &&
                         (blk * kBlockSize > sg.low0 - kBlockSize || blk * kBlockSize < p.num_sinks)))
            return false;
          return lane < kTTileBlocks && blk < nblk;
        };
        auto fetch_id = [&](int x) -> int {
          const int blk = tile_at(sg, x) * kTTileBlocks + lane;
          return (x >= sg.t0 && wanted(blk)) ? row[blk] : -1;
        };
        int id = fetch_id(sg.t1 - 1);
        if (!is_v) {
          bool far = false;                            // does any row need the E5M2 parts?
          if constexpr (kFp8) {
            for (int x = lane; x < sg.rows; x += 32) {
              const int r = sg.unit * kTreeRows * NQ + x;
              far |= p.part_scale[(static_cast<int64_t>(sq.start) + (r >> shift)) * p.n_q_heads + (sg.g << shift) +
                                  (r & ((1 << shift) - 1))] < 0.f;
            }
            far = __any_sync(0xffffffffu, far);
          }
          // Q of the piece, once every Q K^T of the piece before has read it
          if (pieces > 0) good = __all_sync(0xffffffffu, tree_wait(q_empty, (pieces - 1) & 1, p, abort_flag));
          if (!good) break;
          const int parts = kFp8 ? (p.q_bf16 ? 2 : 3) : 1;
          if (kFp8 && lane == 0) *far_parts = far;
          if (lane == 0)
            mbar_arrive_expect_tx(q_full, nq * parts * (p.q_box << shift) * (kFp8 ? D : 2 * D));
          ++pieces;
          __syncwarp();
          if (kFp8 && lane < nq * parts) {
            const int c = lane / parts, part = lane % parts, kept = part + (far && part > 0 ? parts - 1 : 0);
            tma_load_3d(sm + L::kQ + c * L::kQTile + part * L::kStage, &p.tmap_q, 0, sg.g << shift,
                        static_cast<int>(kept * p.num_tokens) + sq.start +
                            ((sg.unit * kTreeRows * NQ + c * kTreeRows) >> shift),
                        q_full, policy_evict_last());
          }
          if (!kFp8 && lane < nq * (D / 64)) {
            const int c = lane / (D / 64), h = lane % (D / 64);
            tma_load_3d(sm + L::kQ + c * L::kTile + h * L::kHalfQ, &p.tmap_q, h * 64, sg.g << shift,
                        sq.start + ((sg.unit * kTreeRows * NQ + c * kTreeRows) >> shift), q_full,
                        policy_evict_last());
          }
          __syncwarp();
        }
        for (int t = sg.t1 - 1; t >= sg.t0; --t) {
          // cache slab of this lane's block: -1 behind the context or for a bad id
          bool have = wanted(tile_at(sg, t) * kTTileBlocks + lane);
          if (have && (id < 0 || id >= p.num_blocks)) {
            record_error(p.err, PKV_ERR_OOB);
            have = false;
          }
          const int64_t slab = have ? static_cast<int64_t>(id) * p.n_kv_heads + sg.g : -1;
          id = fetch_id(t - 1);
          good = __all_sync(0xffffffffu, use == 0 || tree_wait(&empty[s], (use - 1) & 1, p, abort_flag));
          if (!good) break;
          if constexpr (!kFp8) {
            if (lane == 0) mbar_arrive_expect_tx(&full[s], L::kTile);
            __syncwarp();
            // (slab -1 is outside the tensor, which fills with zeros)
            if (lane < kTTileBlocks)
              tma_load_4d(ring + s * L::kTile + lane * (kBlockSize * D * 2), is_v ? &p.tmap_v : &p.tmap_k,
                          static_cast<int>(slab) * 2, &full[s], pol);
          } else if (!is_v) {
            if (lane == 0) mbar_arrive_expect_tx(&full[s], L::kKTile);
            __syncwarp();
            if (lane < kTTileBlocks)
              tma_load_2d(ring + s * L::kKTile + lane * (kBlockSize * D), &p.tmap_k, 0,
                          static_cast<int>(slab) * kBlockSize, &full[s], pol);
          } else {
            constexpr int kSlab = kBlockSize * D;
            unsigned char* dst = ring + s * L::kStage + lane * kSlab;
            const uint32_t got = __ballot_sync(0xffffffffu, have);
            if (lane < kTTileBlocks && !have) {        // (codes of 0; rare but for the last tile)
              for (int x = 0; x < kSlab; x += 16)
                asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(smem_u32(dst + x)), "r"(0u) : "memory");
              fence_proxy_async_smem();
            }
            __syncwarp();
            if (lane == 0) mbar_arrive_expect_tx(&full[s], __popc(got) * kSlab);
            __syncwarp();
            if (have) bulk_g2s(dst, p.v_codes + slab * kSlab, kSlab, &full[s], pol);
          }
          __syncwarp();
          ++tiles;
          if (++s == stages) {
            s = 0;
            ++use;
          }
        }
      }
      if (!good) *abort_flag = 1;
      if (lane == 0) {
        // The last loads of every stage land before the block ends (bounded, with the
        // full limit): whoever should wait for them may have stopped.
        const unsigned long long deadline = global_ns() + kWaitLimitNs;
        if (pieces > 0) mbar_wait_until(q_full, (pieces - 1) & 1, deadline);
        for (uint32_t n = tiles > stages ? tiles - stages : 0; n < tiles; ++n)
          mbar_wait_until(&full[n % stages], (n / stages) & 1, deadline);
      }
      __syncwarp();
    } else if (warp < 11) {
      // ============================ MMA issuers (warps 9, 10) ============================
      // Warp 9 issues Q K^T, warp 10 P V, one elected lane each: a commit holds its
      // thread until the MMA queue has drained to a few entries; meanwhile the
      // other feeds the queue.
      constexpr int kPasses = kSplit ? 2 : 1;
      const int parts = p.q_bf16 ? 2 : 3;              // of an FP8 operand q
      constexpr uint32_t kIdQK = umma_idesc<MT>(false, kTreeKeys), kIdPV = umma_idesc<MT>(true, D);
      const bool qk_warp = (warp == 9);
      bool ok = true;
      if (lane == 0) {
        uint32_t id_rest = 0;                          // FP8: of the parts behind the first
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
            ok = tree_wait_started_early(q_full, pieces & 1, p, abort_flag);
            if constexpr (kFp8) id_rest = umma_idesc_codes<KV>(kTreeKeys, *far_parts != 0);
          }
          // (the piece's first P V overwrites the outputs of the piece before)
          if (!qk_warp && pieces > 0) ok = tree_wait(o_read, (pieces - 1) & 1, p, abort_flag);
          ++pieces;
          for (int t = sg.t1 - 1; t >= sg.t0 && ok; --t) {
            if (qk_warp)
              ok = tree_wait(&k_full[kr.s], kr.ph, p, abort_flag);
            else
              ok = tree_wait_started_early(&v_ready[vr.s], vr.ph, p, abort_flag);
#pragma unroll
            for (int c = 0; c < NQ; ++c) {
              if (c >= nq || !ok) break;
              const uint32_t d_s = tmem + sr.s * kTreeKeys;
              if (qk_warp) {
                // S once the P V that read P from its columns is done
                ok = ops < NB || tree_wait(&pv_done[sr.s], sr.ph ^ 1u, p, abort_flag);
                if (!ok) break;
                tc_fence_after();
                if constexpr (kFp8) {
                  const uint64_t a0 = umma_desc_codes<D>(smem_u32(sm + L::kQ + c * L::kQTile));
                  const uint64_t b0 = umma_desc_codes<D>(smem_u32(sm + L::kK + kr.s * L::kKTile));
                  constexpr uint32_t kIdFirst = umma_idesc_codes<KV>(kTreeKeys, false);
                  // (the smallest parts first)
#pragma unroll
                  for (int part = L::kParts - 1; part >= 0; --part)
                    if (part < parts)
                      umma_f8<D / 32>(d_s, a0 + static_cast<uint64_t>((part * L::kStage) >> 4), b0,
                                      part == 0 ? kIdFirst : id_rest, part < parts - 1);
                } else {
                  const uint64_t a0 = umma_desc(smem_u32(sm + L::kQ + c * L::kTile), 16, 1024);
                  const uint64_t b0 = umma_desc(smem_u32(sm + L::kK + kr.s * L::kTile), 16, L::kGroup);
#pragma unroll
                  for (int ks = 0; ks < D / 16; ++ks)
                    umma_f16(d_s, a0 + static_cast<uint64_t>(((ks >> 2) * L::kHalfQ + (ks & 3) * 32) >> 4),
                             b0 + static_cast<uint64_t>(((ks >> 2) * L::kHalf + (ks & 3) * 32) >> 4), kIdQK, ks > 0);
                }
                umma_commit(&s_full[sr.s]);
              } else {
                const uint64_t b0 = umma_desc(smem_u32(sm + L::kV + vr.s * L::kTile), L::kHalf, L::kGroup);
                const uint32_t d_o = tmem + L::kOCol + c * D;
                // the upper keys' P first
                auto half = [&](auto upper) {
                  constexpr int h = decltype(upper)::value;
                  tc_fence_after();
#pragma unroll
                  for (int pass = 0; pass < kPasses; ++pass)
#pragma unroll
                    for (int ks = 4 * h; ks < 4 * h + 4; ++ks)
                      umma_f16_tmem_a(d_o,
                                      d_s + (kSplit ? 32 * (ks >> 1) + 16 * pass + 8 * (ks & 1)
                                                    : 64 * (ks >> 2) + 8 * (ks & 3)),
                                      b0 + static_cast<uint64_t>((ks * 2 * L::kGroup) >> 4), kIdPV,
                                      t < sg.t1 - 1 || h == 0 || ks > 4 || pass > 0);
                };
                ok = tree_wait(&p_half[sr.s], sr.ph, p, abort_flag);
                if (ok) half(std::integral_constant<int, 1>{});
                ok = ok && tree_wait(&p_full[sr.s], sr.ph, p, abort_flag);
                if (!ok) break;
                half(std::integral_constant<int, 0>{});
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
      // ============ warps from 12 on: rows with drafted tokens, conversions ============
      const int x_tid = tid - 12 * 32, x_warp = x_tid >> 5;
      constexpr int kChunks = D / 8;                   // 16-byte chunks of a 16-bit row
      Ring<L::kVStages> vr;
      Ring<(kFp8 ? L::kCodeStages : 1)> cr;
      uint32_t pieces = 0, tiles = 0;
      bool ok = true;
      auto wait_all = [&](uint64_t* bar, uint32_t ph) {
        return __all_sync(0xffffffffu, tree_wait(bar, ph, p, abort_flag));
      };
      pdl_wait();
      for (int64_t pos = first; pos < end && ok;) {
        const TreeSeg sg = segment(pos);
        pos = sg.next;
        if (sg.t0 >= sg.t1) continue;
        const TreeSeq sq = sequence_of(sg);
        const int base = sq.ctx - sq.n;
        uint32_t* my_bad = bad + (pieces % kTBadSlots) * (L::kXform * 8) + x_warp * kBadWords;
        if (lane < kBadWords) my_bad[lane] = 0u;
        __syncwarp();
        auto store = [&](uint32_t addr, const uint4& v) {
          asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w)
                       : "memory");
        };
        auto load = [&](uint32_t addr) -> uint4 {
          uint4 v;
          asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                       : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                       : "r"(addr));
          return v;
        };
        // 16-byte chunk c of key row j of a K / V tile
        auto at = [&](int j, int c) -> uint32_t {
          return (j >> 3) * L::kGroup + (c >> 3) * L::kHalf + (j & 7) * 128 + (((c & 7) ^ (j & 7)) << 4);
        };
        // elements of V at position key: 0 where no row sees them; where only some do, 0
        // if they are not finite, and the token is remembered
        auto clean = [&](uint4 v, int key) -> uint4 {
          bool none, all;
          int note;
          if constexpr (CHUNK) {
            none = key > sg.pos1 || (key >= p.num_sinks && key < sg.low0);
            all = key <= sg.pos0 && (key < p.num_sinks || key >= sg.low1);
            note = key > sg.pos0 ? key - sg.pos0 - 1 : 256 + (key - sg.low0);
          } else {
            none = key >= sq.ctx;
            all = key < base;
            note = key - base;
          }
          if (none) return make_uint4(0u, 0u, 0u, 0u);
          if (!all) {
            const uint4 f =
                make_uint4(nonfinite2<MT>(v.x), nonfinite2<MT>(v.y), nonfinite2<MT>(v.z), nonfinite2<MT>(v.w));
            if (f.x | f.y | f.z | f.w) {
              v.x ^= f.x, v.y ^= f.y, v.z ^= f.z, v.w ^= f.w;
              atomicOr(&my_bad[note >> 5], 1u << (note & 31));
            }
          }
          return v;
        };
        ++pieces;
        for (int x0 = sg.t1 - 1; x0 >= sg.t0 && ok; --x0, ++tiles) {
          const int t = tile_at(sg, x0);
          if constexpr (!kFp8) {
            ok = wait_all(&v_full[vr.s], vr.ph);
            if (!ok) break;
            if (CHUNK ? !chunk_plain(sg, t, p.num_sinks) : t * kTreeKeys > base - kTreeKeys) {
              // (of drafted tokens: rows from the first one on)
              const uint32_t tile = smem_u32(sm + L::kV + vr.s * L::kTile);
              for (int x = (CHUNK ? 0 : max(0, base - t * kTreeKeys)) * kChunks + x_tid; x < kTreeKeys * kChunks;
                   x += L::kXform * 32) {
                const int j = x / kChunks;
                const uint32_t addr = tile + at(j, x % kChunks);
                const uint4 v = load(addr), w = clean(v, t * kTreeKeys + j);
                if ((v.x ^ w.x) | (v.y ^ w.y) | (v.z ^ w.z) | (v.w ^ w.w)) store(addr, w);
              }
              fence_proxy_async_smem();
              __syncwarp();
            }
            if (lane == 0) mbar_arrive(&v_ready[vr.s]);
            vr.next();
          } else {
            ok = wait_all(&c_full[cr.s], cr.ph) && (tiles < L::kVStages || wait_all(&v_empty[vr.s], vr.ph ^ 1u));
            if (!ok) break;
            const uint4* codes = reinterpret_cast<const uint4*>(sm + L::kCodes + cr.s * L::kStage);
            const uint32_t tile = smem_u32(sm + L::kV + vr.s * L::kTile);
            // Chunk k of 16 codes of this thread is kBytes of the tile behind chunk k - 1
            // (whole groups of 8 keys), so its two places are constants away.  The lanes of
            // a row's upper half convert and store its second 8 codes first: both halves of
            // a row lie in the same banks.
            constexpr int kAll = kTreeKeys * D / 16, kStep = L::kXform * 32;
            constexpr int kBytes = kStep / (D / 16) / 8 * L::kGroup;
            constexpr int kPer = kAll / kStep < 4 ? kAll / kStep : 4;   // chunks whose instructions interleave
            static_assert(kStep / (D / 16) % 8 == 0 && kAll % (kPer * kStep) == 0, "chunks");
            const int j0 = x_tid / (D / 16), c0 = x_tid % (D / 16);
            const bool up = D == 128 && (c0 & 4);
            const uint32_t first8 = tile + at(j0, 2 * c0 + (up ? 1 : 0)), last8 = tile + at(j0, 2 * c0 + (up ? 0 : 1));
#pragma unroll 1
            for (int k0 = 0; k0 < kAll / kStep; k0 += kPer) {
              uint4 raw[kPer];
#pragma unroll
              for (int k = 0; k < kPer; ++k) raw[k] = codes[x_tid + (k0 + k) * kStep];
#pragma unroll
              for (int k = 0; k < kPer; ++k) {
                const uint4 w = raw[k];
                const uint2 w0 = codes4(up ? w.z : w.x, KV{}), w1 = codes4(up ? w.w : w.y, KV{});
                const uint2 w2 = codes4(up ? w.x : w.z, KV{}), w3 = codes4(up ? w.y : w.w, KV{});
                store(first8 + (k0 + k) * kBytes, make_uint4(w0.x, w0.y, w1.x, w1.y));
                store(last8 + (k0 + k) * kBytes, make_uint4(w2.x, w2.y, w3.x, w3.y));
              }
            }
            if (t * kTreeKeys > base - kTreeKeys) {
              // V rows from the first drafted token on: each thread looks at what it wrote
#pragma unroll 1
              for (int x = x_tid; x < kAll; x += L::kXform * 32) {
                const int j = x / (D / 16), c = x % (D / 16);
#pragma unroll 1
                for (int e = 0; e < 2; ++e) {
                  const uint32_t addr = tile + at(j, 2 * c + e);
                  store(addr, clean(load(addr), t * kTreeKeys + j));
                }
              }
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
              mbar_arrive(&c_empty[cr.s]);
              mbar_arrive(&v_ready[vr.s]);
            }
            cr.next();
            vr.next();
          }
        }
      }
      if (!ok) *abort_flag = 1;
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 9)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512) : "memory");
}

// ---------------------------------------------------------------------------
// q as a sum of parts (FP8 caches): a warp per row of D elements, a lane per D / 32 of
// them, times the sign of its KV head's K scale.  parts [., rows, D] codes: the first in
// E4M3, the others (one of bf16, two of fp16) in E4M3, then the same in E5M2.  scale
// [rows], below 0 where the row needs the E5M2 ones.
// ---------------------------------------------------------------------------
constexpr int kTPartWarps = 8;

template <int D>
__global__ void __launch_bounds__(kTPartWarps * 32)
    tree_parts_kernel(const void* __restrict__ q, int q_bf16, int64_t rows, int n_q_heads, int group_shift,
                      const float* __restrict__ k_scale, uint8_t* __restrict__ parts, float* __restrict__ scale) {
  constexpr int N = D / 32;
  const int lane = threadIdx.x & 31;
  pdl_wait_and_release();   // (the next kernel waits for this one before it reads what this writes)
  const int64_t row = static_cast<int64_t>(blockIdx.x) * kTPartWarps + (threadIdx.x >> 5);
  if (row >= rows) return;
  // (rows fit 32 bits)
  const float ks = k_scale[(static_cast<uint32_t>(row) % static_cast<uint32_t>(n_q_heads)) >> group_shift];
  const uint32_t* src = reinterpret_cast<const uint32_t*>(static_cast<const uint16_t*>(q) + row * D) + lane * (N / 2);
  float f[N];
  float top = 0.f;
  bool nan = false;
#pragma unroll
  for (int e = 0; e < N / 2; ++e) {
    const float2 x = q_bf16 ? unpack2(src[e], BF16{}) : unpack2(src[e], F16{});
    f[2 * e] = x.x, f[2 * e + 1] = x.y;
    top = fmaxf(top, fmaxf(fabsf(x.x), fabsf(x.y)));
    nan |= !isfinite(x.x) | !isfinite(x.y);
  }
#pragma unroll
  for (int k = 16; k >= 1; k >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, k));
  nan = __any_sync(0xffffffffu, nan);
  // top in [2^e, 2^(e + 1)): times 2^(7 - e)
  const int e2 = max(static_cast<int>(__float_as_uint(top) >> 23) - 127, -113);
  const float mag = __uint_as_float(static_cast<uint32_t>(127 + 7 - e2) << 23);
  const float up = ks < 0.f ? -mag : mag;
#pragma unroll
  for (int e = 0; e < N; ++e) f[e] *= up;
  // the codes of r as part `at`; r: what is left
  auto put = [&](int at, float* r, auto fmt) {
    uint32_t w = 0;
#pragma unroll
    for (int e = 0; e < N; e += 2) {
      uint32_t code = fp8x2_from_f32(r[e], r[e + 1], fmt);
      float2 back;
      if constexpr (std::is_same<decltype(fmt), E4M3>::value)
        back = unpack2_e4m3(static_cast<uint16_t>(code));
      else
        back = unpack2_e5m2(code);
      r[e] -= back.x, r[e + 1] -= back.y;
      if (nan) code = 0x7f7fu;                       // (a NaN in both formats; so is the row's output)
      w |= code << (8 * e);
    }
    uint8_t* dst = parts + (at * rows + row) * D + lane * N;
    if constexpr (N == 4)
      *reinterpret_cast<uint32_t*>(dst) = w;
    else
      *reinterpret_cast<uint16_t*>(dst) = static_cast<uint16_t>(w);
  };
  put(0, f, E4M3{});
  float near[N];
#pragma unroll
  for (int e = 0; e < N; ++e) near[e] = f[e];
  put(1, near, E4M3{});
  if (q_bf16) {
    put(2, f, E5M2{});
  } else {
    put(2, near, E4M3{});
    put(3, f, E5M2{});
    put(4, f, E5M2{});
  }
  int left = 0;                                      // elements that the E4M3 parts do not hold
#pragma unroll
  for (int e = 0; e < N; ++e) left += __popc(__ballot_sync(0xffffffffu, near[e] != 0.f));
  const float back = nan ? 1.f : __uint_as_float(static_cast<uint32_t>(127 - 7 + e2) << 23);
  if (lane == 0) scale[row] = !nan && left >= D / 8 ? -back : back;
}

// ---------------------------------------------------------------------------
// The merge: a warp per NR query rows of a (sequence, KV head).  Lane x finds range
// r0 + x's piece of the rows' unit; the states are joined as in the other merges,
// with the first pieces' outputs loaded beside their weights.  Units that one range
// held are done.  It is all latency, so a warp takes one row and eight pieces at a
// time where the rows' warps fit the GPU at once (by the registers, five thread blocks
// an SM), and else four rows and two pieces.  (Calls with 19 tokens of 32 heads a
// sequence, contexts of 4096, one row a warp and four: 4 sequences, 2432 rows, 21.3 and
// 26.1 us; 8, where 3040 fit, 37.2 and 36.1; 16, 62.0 and 57.6; 64, 198 and 187.)
// With one row a warp, and all thread blocks on the GPU at once, the geometry is
// worked out from the inputs while the kernel before still runs (one document of
// 131072: 123 us instead of 125 then; four chats 9.0 instead of 9.9).
// Thread blocks of four warps, not eight: with four rows a warp the registers then
// hold 20 warps an SM instead of 16 (the 32 sequences 131.6 us instead of 132.8).
// ---------------------------------------------------------------------------
constexpr int kTMergeWarps = 4;

template <int D, int NQ, int NR>
__global__ void __launch_bounds__(kTMergeWarps * 32)
    tree_merge_kernel(const __grid_constant__ TreeParams p, int ranges, int ahead) {
  constexpr int N = D / 32, kBatch = 8 / NR, kUnit = kTreeRows * NQ;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int b = blockIdx.z, g = blockIdx.y, shift = p.group_shift;
  const bool early = NR == 1 && ahead;
  TreeSeq sq;
  int64_t V;
  if (early) {
    // (lengths and offsets only, as the kernel before)
    __shared__ int64_t sums[2][kTMergeWarps];
    int64_t before = 0, all = 0;
    for (int x = threadIdx.x; x < p.batch; x += kTMergeWarps * 32) {
      const int64_t c = tree_sequence<NQ>(p, x, nullptr).cost;
      all += c;
      before += x < b ? c : 0;
    }
#pragma unroll
    for (int k = 16; k >= 1; k >>= 1) {
      all += __shfl_xor_sync(0xffffffffu, all, k);
      before += __shfl_xor_sync(0xffffffffu, before, k);
    }
    if (lane == 0) sums[0][warp] = before, sums[1][warp] = all;
    __syncthreads();
    sq = tree_sequence<NQ>(p, b, nullptr);
    sq.cost = V = 0;
#pragma unroll
    for (int k = 0; k < kTMergeWarps; ++k) sq.cost += sums[0][k], V += sums[1][k];
  } else {
    pdl_wait_and_release();
    sq = p.seqs[b];
    V = p.seqs[p.batch].cost;
  }
  const int64_t R = ranges;
  const int rows = sq.n << shift, row0 = (blockIdx.x * kTMergeWarps + warp) * NR;
  if (row0 >= rows) {
    if (early) pdl_wait_and_release();
    return;
  }
  const int units = tree_units<NQ>(rows), kt = tree_tiles(sq.ctx), unit = row0 / kUnit;   // (NR divides kUnit)
  const int64_t cost = tree_unit_cost(rows, kt, p.setup_cost), u0 = sq.cost + (static_cast<int64_t>(g) * units + unit) * cost;
  // ranges whose part of the axis meets the unit: r0 .. r1
  const int64_t r0 = div_nonneg((u0 + 1) * R + V - 1, V) - 1;
  const int64_t r1 = div_nonneg((u0 + cost) * R + V - 1, V) - 1;
  // tiles of range r in the unit
  auto tiles_of = [&](int64_t r) -> int2 {
    if (r > r1) return make_int2(0, 0);
    return make_int2(
        tree_tile_at(max(div_nonneg(r * V, R) - u0, static_cast<int64_t>(0)), rows, kt, p.setup_cost),
        tree_tile_at(max(min(div_nonneg((r + 1) * V, R) - u0, cost), static_cast<int64_t>(0)), rows, kt, p.setup_cost));
  };
  int2 first = make_int2(0, 0);
  if (early) {
    first = tiles_of(r0 + lane);
    pdl_wait_and_release();
  }
  const int64_t base = tree_piece_row(sq.start, p.n_q_heads, g, rows, static_cast<int64_t>(unit) * kUnit, 0, kUnit) +
                       (row0 - unit * kUnit);
  float M[NR], Lsum[NR], O[NR][N];
#pragma unroll
  for (int i = 0; i < NR; ++i) {
    M[i] = -INFINITY, Lsum[i] = 0.f;
#pragma unroll
    for (int e = 0; e < N; ++e) O[i][e] = 0.f;
  }
  for (int64_t x0 = r0; x0 <= r1; x0 += 32) {
    const int64_t r = x0 + lane;
    const int2 of = early && x0 == r0 ? first : tiles_of(r);
    const int t0 = of.x, t1 = of.y;
    if (__any_sync(0xffffffffu, t0 == 0 && t1 == kt)) return;        // written where it was computed
    const bool have = t0 < t1;
    uint32_t left = __ballot_sync(0xffffffffu, have);
    float2 st[NR];
#pragma unroll
    for (int i = 0; i < NR; ++i)
      st[i] = have && row0 + i < rows ? *reinterpret_cast<const float2*>(p.ml + (base + i + r * kUnit) * 2)
                                      : make_float2(-INFINITY, 0.f);
    float v[kBatch][NR][N];
    int src[kBatch];
    auto load_batch = [&]() {
#pragma unroll
      for (int q = 0; q < kBatch; ++q) {
        src[q] = left ? __ffs(left) - 1 : -1;
        left &= left - 1;          // (0 stays 0)
#pragma unroll
        for (int i = 0; i < NR; ++i) {
          if (src[q] < 0 || row0 + i >= rows) continue;
          const float* from = p.o + (base + i + (x0 + src[q]) * kUnit) * D + N * lane;
          if constexpr (N == 4) {
            const float4 f = *reinterpret_cast<const float4*>(from);
            v[q][i][0] = f.x, v[q][i][1] = f.y, v[q][i][2] = f.z, v[q][i][3] = f.w;
          } else {
            const float2 f = *reinterpret_cast<const float2*>(from);
            v[q][i][0] = f.x, v[q][i][1] = f.y;
          }
        }
      }
    };
    load_batch();
    float w[NR];
#pragma unroll
    for (int i = 0; i < NR; ++i) {
      float m = st[i].x;
#pragma unroll
      for (int k = 16; k >= 1; k >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, k));
      const float mn = fmaxf(M[i], m), ref = (mn == -INFINITY) ? 0.f : mn;
      const float keep = exp2f(M[i] - ref);
      w[i] = exp2f(st[i].x - ref);
      float l = w[i] * st[i].y;
#pragma unroll
      for (int k = 16; k >= 1; k >>= 1) l += __shfl_xor_sync(0xffffffffu, l, k);
      Lsum[i] = Lsum[i] * keep + l;
      M[i] = mn;
#pragma unroll
      for (int e = 0; e < N; ++e) O[i][e] *= keep;
    }
    while (true) {
#pragma unroll
      for (int q = 0; q < kBatch; ++q)
#pragma unroll
        for (int i = 0; i < NR; ++i) {
          const float wq = __shfl_sync(0xffffffffu, w[i], src[q] < 0 ? 0 : src[q]);
          if (src[q] < 0 || row0 + i >= rows) continue;
#pragma unroll
          for (int e = 0; e < N; ++e) O[i][e] = fmaf(wq, v[q][i][e], O[i][e]);
        }
      if (left == 0) break;
      load_batch();
    }
  }
#pragma unroll
  for (int i = 0; i < NR; ++i) {
    const int row = row0 + i;
    if (row >= rows) break;
    const float inv = Lsum[i] > 0.f ? 1.f / Lsum[i] : 0.f;
    const int node = row >> shift, head = (g << shift) + (row & ((1 << shift) - 1));
    uint16_t* out = static_cast<uint16_t*>(p.out) +
                    ((static_cast<int64_t>(sq.start) + node) * p.n_q_heads + head) * D + N * lane;
    uint32_t x[N / 2];
#pragma unroll
    for (int e = 0; e < N; e += 2)
      x[e / 2] = p.q_bf16 ? pack2(O[i][e] * inv, O[i][e + 1] * inv, BF16{})
                          : pack2(O[i][e] * inv, O[i][e + 1] * inv, F16{});
    if constexpr (N == 4)
      *reinterpret_cast<uint2*>(out) = make_uint2(x[0], x[1]);
    else
      *reinterpret_cast<uint32_t*>(out) = x[0];
  }
}

template <typename MT, typename KV, int D, int NQ, bool ONE>
pkv_status launch_tree(TreeParams& p, int ranges, cudaStream_t stream) {
  using L = TreeSmem<D, KV::kBytes == 1, NQ>;
  auto kern = tree_kernel<MT, KV, D, NQ, false, ONE>;
  constexpr int kDevices = 64;
  int dev = 0;
  if (cuda_failed(cudaGetDevice(&dev), "cudaGetDevice")) return PKV_ERR_CUDA;
  static std::mutex mu;
  static int per_sm[kDevices] = {};   // thread blocks of the merge, one row a warp (0: not asked yet)
  if (dev < 0 || dev >= kDevices) return PKV_ERR_UNSUPPORTED;
  int merge_blocks;                   // of them on the GPU at once
  {
    std::lock_guard<std::mutex> lock(mu);
    if (per_sm[dev] == 0) {
      int n = 0;
      if (cuda_failed(cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                           static_cast<int>(L::bytes(kTreeMaxBatch))),
                      "cudaFuncSetAttribute") ||
          cuda_failed(cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, tree_merge_kernel<D, NQ, 1>,
                                                                    kTMergeWarps * 32, 0),
                      "cudaOccupancyMaxActiveBlocksPerMultiprocessor"))
        return PKV_ERR_CUDA;
      per_sm[dev] = std::max(n, 1);
    }
    merge_blocks = per_sm[dev] * sm_count();
  }
  p.setup_cost = tree_setup_cost(KV::kBytes == 1);
  if constexpr (KV::kBytes == 1) {
    const int64_t rows = p.num_tokens * p.n_q_heads;
    if (cuda_failed(launch_pdl(tree_parts_kernel<D>, dim3(static_cast<unsigned>((rows + kTPartWarps - 1) / kTPartWarps)),
                               dim3(kTPartWarps * 32), 0, stream, p.q, p.q_bf16, rows, p.n_q_heads, p.group_shift,
                               p.k_scale, p.parts, p.part_scale),
                    "tree_parts_kernel launch"))
      return PKV_ERR_CUDA;
  }
  if (cuda_failed(launch_pdl(kern, dim3(static_cast<unsigned>(ranges)), dim3(L::kThreads), L::bytes(p.batch), stream, p),
                  "tree_kernel launch"))
    return PKV_ERR_CUDA;
  const int nr = p.num_tokens * p.n_q_heads > static_cast<int64_t>(merge_blocks) * kTMergeWarps ? 4 : 1;
  const unsigned chunks = ((p.max_nodes << p.group_shift) + kTMergeWarps * nr - 1) / (kTMergeWarps * nr);
  const dim3 grid(chunks, static_cast<unsigned>(p.n_kv_heads), static_cast<unsigned>(p.batch));
  auto merge = nr == 4 ? tree_merge_kernel<D, NQ, 4> : tree_merge_kernel<D, NQ, 1>;
  const int ahead = static_cast<int64_t>(chunks) * p.n_kv_heads * p.batch <= merge_blocks;
  return cuda_failed(launch_pdl(merge, grid, dim3(kTMergeWarps * 32), 0, stream, p, ranges, ahead),
                     "tree_merge_kernel launch")
             ? PKV_ERR_CUDA
             : PKV_OK;
}

// grid: units of the longest sequence x KV heads x sequences
template <typename MT, int D, int NQ>
pkv_status launch_chunk(TreeParams& p, int units, cudaStream_t stream) {
  using L = TreeSmem<D, false, NQ>;
  auto kern = tree_kernel<MT, MT, D, NQ, true, false>;
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
                                           static_cast<int>(L::bytes(1))),
                      "cudaFuncSetAttribute"))
        return PKV_ERR_CUDA;
      done[dev] = true;
    }
  }
  const dim3 grid(static_cast<unsigned>(units), static_cast<unsigned>(p.n_kv_heads), static_cast<unsigned>(p.batch));
  return cuda_failed(launch_pdl(kern, grid, dim3(L::kThreads), L::bytes(1), stream, p), "tree_kernel launch (chunk)")
             ? PKV_ERR_CUDA
             : PKV_OK;
}

template <typename MT>
TreeLauncher pick_chunk(int head_dim, int q_tiles) {
  if (head_dim == 64) return q_tiles == 1 ? launch_chunk<MT, 64, 1> : launch_chunk<MT, 64, 2>;
  return q_tiles == 1 ? launch_chunk<MT, 128, 1> : launch_chunk<MT, 128, 2>;
}

template <typename MT, typename KV, bool ONE = false>
TreeLauncher pick_tree(int head_dim, int q_tiles) {
  if (head_dim == 64) return q_tiles == 1 ? launch_tree<MT, KV, 64, 1, ONE> : launch_tree<MT, KV, 64, 2, ONE>;
  return q_tiles == 1 ? launch_tree<MT, KV, 128, 1, ONE> : launch_tree<MT, KV, 128, 2, ONE>;
}

}  // namespace pkv

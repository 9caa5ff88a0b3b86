// Decode attention over prefixes that sequences share, and the merge with each
// sequence's own blocks (sm_103a).
//
// What is computed.  The sequences of a group hold the same blocks for their
// first P tokens.  For every query head of them
//   m = max_j s_j,  l = sum_j 2^(s_j - m),  o = sum_j 2^(s_j - m) V_j   (j < P)
// with s_j = scale log2(e) <q, K_j>: the state of an online softmax, which the
// merge joins with the state of the sequence's other blocks (the decode
// kernel's kRest variant) into
//   out = sum_i 2^(m_i - M) o_i / sum_i 2^(m_i - M) l_i.
//
// Why.  Read per sequence, the prefix costs n P rows of K and V; together, the
// group's n G query rows of a KV head (G query heads per KV head) are one
// matrix against it: P rows read once, and products that fill the tensor
// cores.  Up to about 256 rows the reads bound it, beyond that the products.
//
// Work.  A unit is up to 256 query rows of one (group, KV head); its cost is
// its number of 128-key tiles.  The units' costs lie on one axis, cut into
// equal ranges, one per thread block; a range meets one or more units, and
// each meeting leaves one fp32 state per row (a piece).
//
// Tiles.  Two chains of S = Q K^T -> softmax -> O += P V run at a time over
// 128-key tiles, each with its own S / P columns, O columns and four softmax
// warps, so that the tensor cores work for one while the other's softmax runs:
//   more than 128 rows   the chains are two row tiles against the same K / V
//                        tiles, each tile loaded once for both;
//   up to 128 rows       the chains are the even and the odd key tiles of one
//                        row tile; their states are joined in registers.
// Q tiles come by one TMA box per 64 columns (G heads x 128 / G sequences: the
// rows of a unit in order); K / V tiles are 8 cache blocks, gathered by boxes of
// [16 rows x 128 B] into 128-byte-swizzled K-major tiles (one stage of K; of V
// two beside one row tile, one beside two, where a tile serves both chains and
// its load has half of a period to arrive).  P overwrites its own S in TMEM (32 columns of scores become 16 of P
// pairs, and for bf16 16 more of the remainder); the product reads it from
// there.  bf16 P is multiplied as two bf16 parts (p truncated, and the rounded
// remainder: exact to 2^-16), because one bf16 rounding of p (2^-9) would be as
// large as the output's own.  fp16 P (2^-12) is rounded once, and l sums the
// rounded values, as in the dense decode; with one query head per KV head, where
// the dense decode keeps p in fp32, it is two fp16 parts.  (64 sequences behind
// 32768 tokens in fp16, 32 query and 8 KV heads: 58.4 us, 56.6 with l of the
// unrounded p; 8 and 8 heads 51.5 us, 49.8 with one part.)  The row
// reference m moves only when a tile's maximum exceeds it by more than 2^8.
// 64-key tiles with two score buffers per chain, which hide the softmax's
// latency entirely, were slower (67 us against 54 alone on 64 sequences behind
// 32768 tokens): a [128 x 64 x 16] MMA takes as long as a [128 x 128 x 16] one.
//
// Warps 0-3 and 4-7: softmax of chain 0 and 1, one thread per row; warp 8:
// TMA producer; warp 9: TMEM owner and Q K^T issuer, warp 10: P V issuer.
// Waits are bounded as in the other kernels.
//
// Beside it.  The kernel leaves room on its SM (registers: 128 a thread, three
// warps to a scheduler and two to one, so that a scheduler has room for one or
// two more; about 94 KiB of shared memory) for one thread block of five warps of
// the decode over the sequences' own blocks, which is bound by memory where this
// one is bound by the tensor cores; that kernel launches as soon as the wait for
// the previous one is over.  64 sequences of 16 to 2048 tokens behind 32768:
// 63.4 us.  (On another GPU 61.8, against 63.8 without the early start; 66.1 also
// with two stages of V, which leave the other block three consumer warps of two
// stages each instead of four; 103 where the two do not fit an SM together.)
#include <cuda_runtime.h>

#include <algorithm>
#include <mutex>

#include "host_util.h"
#include "pkv_common.cuh"
#include "prefix.h"
#include "tcgen05.cuh"

namespace pkv {

constexpr int kXThreads = 352;
constexpr int kXRows = 128;                       // query rows of a chain's tile
constexpr int kXKeys = 128;                       // keys of a K / V tile
constexpr int kXTileBlocks = kXKeys / kBlockSize;
// K tiles in shared memory: one; V tiles: two beside one row tile, one beside two
constexpr int kXVStages = 2;
constexpr float kXRescaleLog2 = 8.f;
// fp16 weights are held times 2^7 (below 2^16, and the smallest step is 2^-31 of a row's
// largest; unscaled, one key 18 nats above a prefix of 3000 tokens took a third of what
// the others give), and the states times 2^-7 as they leave
constexpr float kXHalfLog2 = 7.f, kXHalfDown = 1.f / 128.f;
static_assert(kXRescaleLog2 + kXHalfLog2 < 16.f, "fp16 weights");
constexpr int kXHalfQ = kXRows * 128;             // bytes of a 64-column half of a Q tile
constexpr int kXHalfKV = kXKeys * 128;            // and of a K / V tile

template <int D>
struct PrefixSmem {
  static constexpr int kQTile = kXRows * D * 2, kKVTile = kXKeys * D * 2;
  static_assert(kQTile == kKVTile, "the second row tile takes the second V stage's place");
  static constexpr int kK = 0;
  static constexpr int kV = kK + kKVTile;                      // V stage 0
  static constexpr int kV1 = kV + kKVTile;                     // V stage 1, or row tile 0
  static __host__ __device__ constexpr int q(int q_tiles) { return kV1 + (2 - q_tiles) * kQTile; }   // row tiles
  static constexpr int kBar = kV1 + 2 * kKVTile;               // 1024 bytes, of which barriers 256
  static constexpr int kRed = kBar + 1024;                     // float2 [2][128], a chain's (m, l)
  static constexpr int kGroups = kRed + 2 * kXRows * 8;        // PrefixGroup [num_groups + 1]
  static size_t bytes(int num_groups) {
    return 1024 + kGroups + sizeof(PrefixGroup) * (static_cast<size_t>(num_groups) + 1);
  }
};

// a piece of a range: key tiles [t0, t1) of one unit
struct PrefixSeg {
  int64_t next;                  // cost position behind it
  int64_t row;                   // first row of its states
  int group, g, unit, rows, t0, t1;
  bool share;                    // two row tiles (else two key streams)
};

__device__ __forceinline__ int prefix_units(int rows) { return (rows + kPrefixUnitRows - 1) / kPrefixUnitRows; }
__device__ __forceinline__ int prefix_tiles(int blocks) { return (blocks + kXTileBlocks - 1) / kXTileBlocks; }

__device__ __forceinline__ PrefixSeg prefix_segment(const PrefixGroup* groups, int num_groups, int n_q_heads,
                                                    int64_t pos, int64_t end, int64_t range) {
  int lo = 0, hi = num_groups - 1;   // the last group that starts at or before pos (a non-empty one)
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (groups[mid].cost <= pos) lo = mid; else hi = mid - 1;
  }
  const PrefixGroup gr = groups[lo];
  const int kt = prefix_tiles(gr.blocks), units = prefix_units(gr.rows);
  const int64_t rem = pos - gr.cost;
  const int64_t u = div_nonneg(rem, kt);
  PrefixSeg s;
  s.group = lo;
  s.g = static_cast<int>(div_nonneg(u, units));
  s.unit = static_cast<int>(u - static_cast<int64_t>(s.g) * units);
  s.t0 = static_cast<int>(rem - u * kt);
  s.t1 = static_cast<int>(min(static_cast<int64_t>(kt), s.t0 + (end - pos)));
  s.next = pos + (s.t1 - s.t0);
  s.rows = min(kPrefixUnitRows, gr.rows - s.unit * kPrefixUnitRows);
  s.share = s.rows > kXRows;
  s.row = piece_row(gr.start, n_q_heads, s.g, gr.rows, s.unit, range);
  return s;
}

// (512 threads a block as far as the registers go: 128 a thread)
template <typename QT, int D, int G>
__global__ void __launch_bounds__(512, 1) prefix_kernel(const __grid_constant__ PrefixParams p) {
  using L = PrefixSmem<D>;
  // (the dense decode keeps p in fp32 where a KV head has one query head)
  constexpr bool kSplit = std::is_same<QT, BF16>::value || G == 1;
  extern __shared__ unsigned char xsm_raw[];
  unsigned char* sm = xsm_raw + ((1024 - (smem_u32(xsm_raw) & 1023)) & 1023);
  uint64_t* bars = reinterpret_cast<uint64_t*>(sm + L::kBar);
  uint64_t* k_full = bars;                    // K tile landed
  uint64_t* k_empty = k_full + 1;             // its Q K^T done
  uint64_t* v_full = k_empty + 1;             // [kXVStages] V tile landed
  uint64_t* v_empty = v_full + kXVStages;     // [kXVStages] its P V done
  uint64_t* s_full = v_empty + kXVStages;     // [2] per chain: scores ready
  uint64_t* p_full = s_full + 2;              // [2] per chain, 128 arrivals: P written, O rescaled
  uint64_t* pv_done = p_full + 2;             // [2] per chain
  uint64_t* q_full = pv_done + 2;             // Q of a piece landed
  uint64_t* mma_idle = q_full + 1;            // [2] an issuer's MMAs done
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(mma_idle + 2);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  static_assert((2 + 2 * kXVStages + 2 + 2 + 2 + 1 + 2 + 1) * 8 <= 256, "barrier block overflows");
  float2* red = reinterpret_cast<float2*>(sm + L::kRed);
  PrefixGroup* groups = reinterpret_cast<PrefixGroup*>(sm + L::kGroups);
  // V stages, as a shift: tile t is in stage t & (stages - 1), its use t >> v_shift
  const uint32_t v_shift = 2 - p.q_tiles;
  auto v_stage = [&](uint32_t s) { return sm + (s == 0 ? L::kV : L::kV1); };
  unsigned char* q_sm = sm + L::q(p.q_tiles);

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (warp == 9) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_slot)),
                 "r"(512)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  if (tid == 8 * 32) {
    *abort_flag = 0;
    mbar_init(k_full, 1);
    mbar_init(k_empty, 1);
    for (int s = 0; s < kXVStages; ++s) {
      mbar_init(&v_full[s], 1);
      mbar_init(&v_empty[s], 1);
    }
    for (int c = 0; c < 2; ++c) {
      mbar_init(&s_full[c], 1);
      mbar_init(&p_full[c], kXRows);
      mbar_init(&pv_done[c], 1);
      mbar_init(&mma_idle[c], 1);
    }
    mbar_init(q_full, 1);
    fence_mbar_init();
  }
  // Early start, as in the decode kernel: until the waits below (the producer's
  // before Q, the softmax warps' before their first store) this kernel reads
  // lengths, group bounds and tables only, which no kernel that releases early
  // writes.  The producer then releases the next kernel, the decode over the
  // sequences' own blocks, which so starts after everything before this one.

  // ---- the groups: shared blocks, first covering sequence, cost ------------
  for (int j = warp; j < p.num_groups; j += kXThreads / 32) {
    const int raw0 = p.group_starts[j], raw1 = p.group_starts[j + 1], len = p.prefix_lens[j];
    const int s0 = min(max(raw0, 0), p.batch), s1 = min(max(raw1, s0), p.batch);
    if ((raw0 != s0 || raw1 != s1 || (j == 0 && raw0 != 0) || (j == p.num_groups - 1 && raw1 != p.batch)) && lane == 0)
      record_error(p.err, PKV_ERR_OOB);
    const int blocks = max(len, 0) / kBlockSize;
    int owner = -1;
    if (blocks > 0)
      for (int b0 = s0; b0 < s1 && owner < 0; b0 += 32) {
        const int b = b0 + lane;
        const bool covers = b < s1 && shares_prefix(blocks, p.context_lens[b], min(p.max_blocks_per_seq, p.max_nblk));
        const uint32_t m = __ballot_sync(0xffffffffu, covers);
        if (m) owner = b0 + __ffs(m) - 1;
      }
    if (lane == 0) {
      PrefixGroup gr;
      gr.start = s0;
      gr.rows = (s1 - s0) * G;
      gr.blocks = owner >= 0 ? blocks : 0;
      gr.owner = owner;
      gr.cost = static_cast<int64_t>(p.n_kv_heads) * prefix_units(gr.rows) * prefix_tiles(gr.blocks);
      groups[j] = gr;
    }
  }
  __syncthreads();
  if (warp == 0) {   // exclusive prefix of the costs
    int64_t carry = 0;
    for (int j0 = 0; j0 < p.num_groups; j0 += 32) {
      const int j = j0 + lane;
      const int64_t own = j < p.num_groups ? groups[j].cost : 0;
      int64_t x = own;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int64_t u = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += u;
      }
      if (j < p.num_groups) groups[j].cost = carry + x - own;
      carry += __shfl_sync(0xffffffffu, x, 31);
    }
    if (lane == 0) groups[p.num_groups] = PrefixGroup{carry, p.batch, 0, 0, -1};
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (blockIdx.x == 0) {
    pdl_wait();
    for (int j = tid; j <= p.num_groups; j += kXThreads) p.groups[j] = groups[j];
  }
  const uint32_t tmem = *tmem_slot;
  const int64_t V = groups[p.num_groups].cost, R = gridDim.x, range = blockIdx.x;
  const int64_t first = div_nonneg(range * V, R), end = div_nonneg((range + 1) * V, R);
  auto segment = [&](int64_t pos) { return prefix_segment(groups, p.num_groups, p.n_q_heads, pos, end, range); };
  // S / P of a chain at columns 128 chain, its O at 256 + chain D
  constexpr int kOCol = 2 * kXKeys;

  if (warp < 8) {
    // ============================ softmax / epilogue ============================
    const int chain = warp >> 2, r = tid & (kXRows - 1);
    const uint32_t lane_base = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t t_s = tmem + lane_base + chain * kXKeys, t_o = tmem + lane_base + kOCol;
    uint32_t ops = 0;                                            // this chain's operations so far
    // A failed wait ends a warp's work but not its walk over the pieces: the two
    // warpgroups meet at named barriers, which must find all of them.
    bool ok = true;
    pdl_wait();
    for (int64_t pos = first; pos < end;) {
      const PrefixSeg sg = segment(pos);
      pos = sg.next;
      const int n_tiles = sg.t1 - sg.t0;
      const int blocks = groups[sg.group].blocks;
      float m_ref = -INFINITY, l_run = 0.f;
      int mine = 0;                                              // operations of this chain in this piece
      const int step = sg.share ? 1 : 2;
      for (int n = sg.share ? 0 : chain; n < n_tiles && ok; n += step, ++mine, ++ops) {
        ok = __all_sync(0xffffffffu, mbar_wait(&s_full[chain], ops & 1, p.err, p.wait_limit_ns) && !*abort_flag);
        if (!ok) break;
        tc_fence_after();
        // keys of the tile that the prefix holds (whole blocks; the last tile may be short)
        const int valid = min(kXKeys, (blocks - (sg.t0 + n) * kXTileBlocks) * kBlockSize);
        float v[64];
        auto load_half = [&](int half) {
          tmem_ld64(t_s + 64 * half, v);
          if (valid < 64 * (half + 1)) {
#pragma unroll
            for (int i = 0; i < 64; ++i) v[i] = 64 * half + i < valid ? v[i] : -INFINITY;
          }
        };
        load_half(0);
        float mx = max64(v);
        load_half(1);
        mx = fmaxf(mx, max64(v));
        const float m_tile = mx * p.qk_scale_log2;
        float alpha = 1.f;
        if (m_tile > m_ref + kXRescaleLog2) {
          alpha = ex2_approx(m_ref - m_tile);
          m_ref = m_tile;
        }
        if (mine > 0 && __any_sync(0xffffffffu, alpha != 1.f)) {
          // (the chain's previous P V has completed: these scores were asked for behind it)
          ok = __all_sync(0xffffffffu, mbar_wait(&pv_done[chain], (ops - 1) & 1, p.err, p.wait_limit_ns));
          if (!ok) break;
          tc_fence_after();
#pragma unroll 1
          for (int c = 0; c < D; c += 16) {
            float o[16];
            tmem_ld16(t_o + chain * D + c, o);
#pragma unroll
            for (int i = 0; i < 16; ++i) o[i] *= alpha;
            tmem_st16(t_o + chain * D + c, o);
          }
        }
        const float nref = (m_ref == -INFINITY) ? 0.f : (std::is_same<QT, F16>::value ? kXHalfLog2 : 0.f) - m_ref;
        const uint64_t scale2 = f32x2(p.qk_scale_log2, p.qk_scale_log2), nref2 = f32x2(nref, nref);
        uint64_t acc[4] = {0ull, 0ull, 0ull, 0ull};
        // the columns in registers are the upper 64; the lower ones are read again
#pragma unroll 1
        for (int half = 1; half >= 0; --half) {
          if (half == 0) load_half(0);
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            uint32_t pk[32];
#pragma unroll
            for (int i = 0; i < 32; i += 2) {
              const float2 e2 = f32x2_split(fma_f32x2(f32x2(v[32 * c + i], v[32 * c + i + 1]), scale2, nref2));
              const float e0 = ex2_approx(e2.x), e1 = ex2_approx(e2.y);
              uint64_t e01 = f32x2(e0, e1);
              if constexpr (std::is_same<QT, BF16>::value) {
                const uint32_t b0 = __float_as_uint(e0), b1 = __float_as_uint(e1);
                pk[i / 2] = __byte_perm(b0, b1, 0x7632);
                const float2 lo = f32x2_split(
                    sub_f32x2(e01, f32x2(__uint_as_float(b0 & 0xffff0000u), __uint_as_float(b1 & 0xffff0000u))));
                pk[16 + i / 2] = pack2(lo.x, lo.y, QT{});
              } else {
                pk[i / 2] = pack2(e0, e1, QT{});
                const float2 hi = unpack2(pk[i / 2], QT{});
                if constexpr (kSplit) {
                  pk[16 + i / 2] = pack2(e0 - hi.x, e1 - hi.y, QT{});
                } else {
                  e01 = f32x2(hi.x, hi.y);   // (l sums what is multiplied)
                }
              }
              acc[(i / 2) & 3] = add_f32x2(acc[(i / 2) & 3], e01);
            }
            if constexpr (kSplit)
              tmem_st32u(t_s + 64 * half + 32 * c, pk);
            else
              tmem_st16u(t_s + 64 * half + 32 * c, pk);
          }
        }
        const float2 s0 = f32x2_split(add_f32x2(add_f32x2(acc[0], acc[1]), add_f32x2(acc[2], acc[3])));
        tmem_wait_st();
        l_run = l_run * alpha + (s0.x + s0.y);
        tc_fence_before();
        mbar_arrive(&p_full[chain]);
      }
      // the piece's states, once the last P V is done
      if (ok && mine > 0)
        ok = __all_sync(0xffffffffu, mbar_wait(&pv_done[chain], (ops - 1) & 1, p.err, p.wait_limit_ns));
      if (!ok) *abort_flag = 1;
      if (!sg.share) {
        red[chain * kXRows + r] = make_float2(m_ref, l_run);
        // (a failure on either side keeps both from writing)
        if (named_bar_red_or(1, 2 * kXRows, !ok)) ok = false;
      }
      tc_fence_after();
      const int row0 = (sg.share ? chain * kXRows : 0) + (warp & 3) * 32;   // the warp's first row of the unit
      const int n_rows = sg.rows - row0;                                    // those that exist (of 32)
      float* dst = p.o + (sg.row + row0) * D;
      constexpr float kDown = std::is_same<QT, F16>::value ? kXHalfDown : 1.f;
      if (sg.share) {
#pragma unroll 1
        for (int c = 0; c < D && ok; c += 32) {
          float o[32];
          tmem_ld32(t_o + chain * D + c, o);
#pragma unroll
          for (int i = 0; i < 32; ++i) o[i] *= kDown;
          store_rows32<D>(dst + c, o, n_rows, lane);
        }
        if (ok && lane < n_rows)
          *reinterpret_cast<float2*>(p.ml + (sg.row + row0 + lane) * 2) = make_float2(m_ref, l_run * kDown);
      } else {
        // join the two key streams: each warpgroup takes half of the columns
        const float2 a = red[r], b = red[kXRows + r];
        const float m = fmaxf(a.x, b.x), ref = (m == -INFINITY) ? 0.f : m;
        const float wa = ex2_approx(a.x - ref) * kDown, wb = ex2_approx(b.x - ref) * kDown;
        if (ok && n_rows > 0) {
#pragma unroll 1
          for (int c = chain * (D / 2); c < (chain + 1) * (D / 2); c += 32) {
            float o[32];
            tmem_ld32(t_o + c, o);
#pragma unroll
            for (int i = 0; i < 32; ++i) o[i] *= wa;
            if (n_tiles > 1) {
#pragma unroll
              for (int h = 0; h < 32; h += 16) {
                float o2[16];
                tmem_ld16(t_o + D + c + h, o2);
#pragma unroll
                for (int i = 0; i < 16; ++i) o[h + i] = fmaf(o2[i], wb, o[h + i]);
              }
            }
            store_rows32<D>(dst + c, o, n_rows, lane);
          }
          if (lane < n_rows && chain == 0)
            *reinterpret_cast<float2*>(p.ml + (sg.row + row0 + lane) * 2) = make_float2(m, a.y * wa + b.y * wb);
        }
        tc_fence_before();
        named_bar_sync(2, 2 * kXRows);   // both have read red and the other's O
        tc_fence_after();
      }
    }
  } else if (warp == 8) {
    // ============================ TMA producer ============================
    uint32_t tiles = 0;                  // tiles loaded so far (K and V alike)
    uint32_t issued_k = 0, issued_v = 0, issued_q = 0;
    bool good = true, waited = false;
    for (int64_t pos = first; pos < end && good;) {
      const PrefixSeg sg = segment(pos);
      pos = sg.next;
      const PrefixGroup gr = groups[sg.group];
      const uint64_t pol = prefix_units(gr.rows) > 1 ? policy_evict_last() : policy_evict_first();
      const int32_t* row = p.block_tables + static_cast<int64_t>(gr.owner) * p.max_blocks_per_seq;
      auto fetch_id = [&](int t) -> int {
        const int blk = t * kXTileBlocks + lane;
        return (t < sg.t1 && lane < kXTileBlocks && blk < gr.blocks) ? row[blk] : -1;
      };
      int id = fetch_id(sg.t0);
      if (!waited) pdl_wait_and_release();
      waited = true;
      // Q of the piece, once every Q K^T of the one before has read its tiles
      if (tiles > 0) {
        good = __all_sync(0xffffffffu, mbar_wait(k_empty, (tiles - 1) & 1, p.err, p.wait_limit_ns) && !*abort_flag);
        if (!good) break;
      }
      if (lane == 0) mbar_arrive_expect_tx(q_full, L::kQTile * (sg.share ? 2 : 1));
      ++issued_q;
      __syncwarp();
      if (lane < (sg.share ? 2 : 1) * (D / 64)) {
        const int c = lane / (D / 64), h = lane % (D / 64);
        tma_load_3d(q_sm + c * L::kQTile + h * kXHalfQ, &p.tmap_q, h * 64, sg.g * G,
                    gr.start + (sg.unit * kPrefixUnitRows + c * kXRows) / G, q_full, policy_evict_last());
      }
      __syncwarp();
      // cache row of this lane's block: a block behind the prefix, or a bad id,
      // is read from rows outside the tensor, which TMA fills with zeros
      auto to_row = [&](int t, int block_id) -> int {
        const int blk = t * kXTileBlocks + lane;
        if (lane < kXTileBlocks && blk < gr.blocks && (block_id < 0 || block_id >= p.num_blocks)) {
          record_error(p.err, PKV_ERR_OOB);
          block_id = -1;
        }
        return (block_id >= 0) ? (block_id * p.n_kv_heads + sg.g) * kBlockSize : -2 * kBlockSize;
      };
      // lane j + 8 h: half h of the tile's block j
      auto load = [&](bool is_v, int y) -> bool {
        const uint32_t shift = is_v ? v_shift : 0, s = tiles & ((1u << shift) - 1), use = tiles >> shift;
        uint64_t* full = is_v ? &v_full[s] : k_full;
        uint64_t* empty = is_v ? &v_empty[s] : k_empty;
        const bool freed = use == 0 || mbar_wait(empty, (use - 1) & 1, p.err, p.wait_limit_ns);
        if (!__all_sync(0xffffffffu, freed && !*abort_flag)) return false;
        if (lane == 0) mbar_arrive_expect_tx(full, L::kKVTile);
        __syncwarp();
        if (lane < kXTileBlocks * (D / 64)) {
          const int j = lane % kXTileBlocks, h = lane / kXTileBlocks;
          tma_load_2d((is_v ? v_stage(s) : sm + L::kK) + h * kXHalfKV + j * 2048,
                      is_v ? &p.tmap_v : &p.tmap_k, h * 64, y, full, pol);
        }
        __syncwarp();
        (is_v ? issued_v : issued_k) = tiles + 1;
        return true;
      };
      for (int t = sg.t0; t < sg.t1 && good; ++t) {
        const int y = __shfl_sync(0xffffffffu, to_row(t, id), lane % kXTileBlocks);
        id = fetch_id(t + 1);
        good = load(false, y) && load(true, y);
        ++tiles;
      }
    }
    if (!waited) pdl_wait_and_release();
    if (!good) *abort_flag = 1;
    if (lane == 0) {
      // The last loads of Q, K and every V stage land before the block ends
      // (bounded, with the full limit): whoever should wait for them may have
      // stopped, now or after this.
      const unsigned long long deadline = global_ns() + kWaitLimitNs;
      if (issued_q > 0) mbar_wait_until(q_full, (issued_q - 1) & 1, deadline);
      if (issued_k > 0) mbar_wait_until(k_full, (issued_k - 1) & 1, deadline);
      const uint32_t stages = 1u << v_shift;
      for (uint32_t t = issued_v > stages ? issued_v - stages : 0; t < issued_v; ++t)
        mbar_wait_until(&v_full[t & (stages - 1)], (t >> v_shift) & 1, deadline);
    }
  } else {
    // ============================ MMA issuers (warps 9, 10) ============================
    // Warp 9 issues Q K^T, warp 10 P V, one elected lane each: a commit holds its
    // thread until the MMA queue has drained to a few entries, and a wait costs
    // about 100 clocks even when it is over; meanwhile the other feeds the queue.
    constexpr int kPasses = kSplit ? 2 : 1;
    constexpr uint32_t kIdQK = umma_idesc<QT>(false, kXKeys), kIdPV = umma_idesc<QT>(true, D);
    const bool qk_warp = (warp == 9);
    bool ok = true;
    if (lane == 0) {
      uint32_t tile0 = 0, piece = 0;       // K / V tiles and pieces before the current piece
      uint32_t count[2] = {0, 0};          // this issuer's operations of each chain so far
      for (int64_t pos = first; pos < end && ok; ++piece) {
        const PrefixSeg sg = segment(pos);
        pos = sg.next;
        const int n_tiles = sg.t1 - sg.t0;
        const int n_ops = sg.share ? 2 * n_tiles : n_tiles;
        // (the producer loads nothing while the previous kernel runs)
        if (qk_warp) ok = mbar_wait_started_early(q_full, piece & 1, p.err, p.wait_limit_ns);
        for (int k = 0; k < n_ops && ok; ++k) {
          const uint32_t t = tile0 + (sg.share ? k >> 1 : k);
          const int c = k & 1;
          const bool last_use = !sg.share || c == 1;   // of the tile
          if (qk_warp) {
            // S of the chain once the P V that read P from its columns is done
            ok = mbar_wait(k_full, t & 1, p.err, p.wait_limit_ns) &&
                 (count[c] == 0 || mbar_wait(&pv_done[c], (count[c] - 1) & 1, p.err, p.wait_limit_ns)) && !*abort_flag;
            if (!ok) break;
            ++count[c];
            const uint64_t a0 = umma_desc(smem_u32(q_sm + (sg.share ? c * L::kQTile : 0)), 16, 1024);
            const uint64_t b0 = umma_desc(smem_u32(sm + L::kK), 16, 1024);
            tc_fence_after();
#pragma unroll
            for (int ks = 0; ks < D / 16; ++ks)
              umma_f16(tmem + c * kXKeys, a0 + static_cast<uint64_t>(((ks >> 2) * kXHalfQ + (ks & 3) * 32) >> 4),
                       b0 + static_cast<uint64_t>(((ks >> 2) * kXHalfKV + (ks & 3) * 32) >> 4), kIdQK, ks > 0);
            umma_commit(&s_full[c]);
            if (last_use) umma_commit(k_empty);
          } else {
            const uint32_t s = t & ((1u << v_shift) - 1);
            ok = mbar_wait_started_early(&v_full[s], (t >> v_shift) & 1, p.err, p.wait_limit_ns) &&
                 mbar_wait(&p_full[c], count[c] & 1, p.err, p.wait_limit_ns) && !*abort_flag;
            if (!ok) break;
            ++count[c];
            tc_fence_after();
            const uint64_t b0 = umma_desc(smem_u32(v_stage(s)), kXHalfKV, 1024);
            const uint32_t a0 = tmem + c * kXKeys, d = tmem + kOCol + c * D;
#pragma unroll
            for (int pass = 0; pass < kPasses; ++pass)
#pragma unroll
              for (int ks = 0; ks < kXKeys / 16; ++ks)
                umma_f16_tmem_a(d, a0 + 32 * (ks >> 1) + 16 * pass + 8 * (ks & 1),
                                b0 + static_cast<uint64_t>((ks * 2048) >> 4), kIdPV, k > 1 || ks > 0 || pass > 0);
            umma_commit(&pv_done[c]);
            if (last_use) umma_commit(&v_empty[s]);
          }
        }
        tile0 += n_tiles;
      }
      if (!ok) *abort_flag = 1;
      // every MMA of this lane has completed before TMEM is released
      umma_commit(&mma_idle[qk_warp ? 0 : 1]);
      mbar_wait(&mma_idle[qk_warp ? 0 : 1], 0, p.err);
    }
    __syncwarp();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 9)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512) : "memory");
}

// ---------------------------------------------------------------------------
// The merge: one warp per (sequence, query head).  Lane l owns D / 32
// consecutive outputs and joins the states of the prefix's pieces (one per
// range that the row's unit meets), then those of the sequence's own blocks:
// the pieces in the decode kernel's partial slots, or the one state it left
// for a pair that one range holds.
// It is all latency.  Small calls work out the geometry from the inputs while
// the other kernels run; others read what those left.  Then the lanes find the
// pieces (which take two divisions each) of 32 ranges at a time, prefix and own
// blocks in one list, and their states are loaded 8 at a time.  (Every lane
// dividing for every piece, one list after the other: 14 us of a 93 us call.)
// ---------------------------------------------------------------------------
constexpr int kMergeWarps = 4;

template <typename QT, int D, int G>
__global__ void __launch_bounds__(kMergeWarps * 32)
    prefix_merge_kernel(const __grid_constant__ PrefixParams p, int ranges, const __grid_constant__ DecodeParams rest,
                        int rest_grid) {
  constexpr int N = D / 32;
  constexpr int kBatch = 8;        // pieces whose loads are issued together
  const int lane = threadIdx.x & 31;
  const int64_t u = static_cast<int64_t>(blockIdx.x) * kMergeWarps + (threadIdx.x >> 5);
  // (every warp waits, at the latest here: this grid completes after the others)
  if (u >= static_cast<int64_t>(p.batch) * p.n_q_heads) {
    pdl_wait();
    return;
  }
  const int b = static_cast<int>(u / p.n_q_heads), head = static_cast<int>(u % p.n_q_heads);
  const int g = head / G, h = head % G;
  float M = -INFINITY, L = 0.f, O[N] = {};
  auto load = [&](const float* src, float* v) {
    if constexpr (N == 4) {
      const float4 x = *reinterpret_cast<const float4*>(src + 4 * lane);
      v[0] = x.x, v[1] = x.y, v[2] = x.z, v[3] = x.w;
    } else {
      const float2 x = *reinterpret_cast<const float2*>(src + 2 * lane);
      v[0] = x.x, v[1] = x.y;
    }
  };
  // ---- the geometry: this sequence's group, the cost of all groups, the
  // blocks of the sequences before it, its own and all ----
  const int cap = min(p.max_blocks_per_seq, p.max_nblk);
  const int ctx = p.context_lens[b];
  PrefixGroup gr{0, 0, 0, 0, -1};
  int64_t V, c0, tot, ne_b, tot_ne;
  int nb;
  const bool local = p.batch <= kCombineLocalPrefix && p.num_groups <= 32;
  if (local) {
    // small calls: from the inputs, as the two kernels take it, before the wait.
    // Lane j holds group j's bounds and whether a sequence covers its blocks.
    int start = INT32_MAX, stop = INT32_MAX, blocks = 0;
    if (lane < p.num_groups) {
      start = min(max(p.group_starts[lane], 0), p.batch);
      stop = min(max(p.group_starts[lane + 1], start), p.batch);
      blocks = max(p.prefix_lens[lane], 0) / kBlockSize;
    }
    uint32_t covered = 0;                                  // groups with a covering sequence
    int before = 0, mine = 0, all = 0, ne_before = 0, ne_all = 0;
    for (int i0 = 0; i0 < p.batch; i0 += 32) {
      const int i = i0 + lane;
      const int len = i < p.batch ? p.context_lens[i] : 0;
      int j = -1;                                          // its group: the last that starts at or before it
      for (int k = 0; k < p.num_groups; ++k)
        if (__shfl_sync(0xffffffffu, start, k) <= i) j = k;
      const int shared = __shfl_sync(0xffffffffu, blocks, max(j, 0));
      const int end = __shfl_sync(0xffffffffu, stop, max(j, 0));
      const bool shares = i < p.batch && j >= 0 && i < end && shares_prefix(shared, len, cap);
      int n = i < p.batch && len > 0 ? min(ctx_blocks(len), cap) : 0;
      if (shares) n -= shared;
      covered |= __reduce_or_sync(0xffffffffu, shares ? 1u << j : 0u);
      all += n;
      ne_all += n > 0;
      before += i < b ? n : 0;
      ne_before += i < b && n > 0;
      mine += i == b ? n : 0;
    }
    c0 = __reduce_add_sync(0xffffffffu, before);
    nb = __reduce_add_sync(0xffffffffu, mine);
    tot = __reduce_add_sync(0xffffffffu, all);
    ne_b = __reduce_add_sync(0xffffffffu, ne_before);
    tot_ne = __reduce_add_sync(0xffffffffu, ne_all);
    const int rows = lane < p.num_groups ? (stop - start) * G : 0;
    if (!((covered >> lane) & 1u)) blocks = 0;
    int64_t cost = static_cast<int64_t>(p.n_kv_heads) * prefix_units(rows) * prefix_tiles(blocks);
    const int64_t own = cost;
#pragma unroll
    for (int k = 1; k < 32; k <<= 1) {
      const int64_t x = __shfl_up_sync(0xffffffffu, cost, k);
      if (lane >= k) cost += x;
    }
    V = __shfl_sync(0xffffffffu, cost, 31);
    const uint32_t m = __ballot_sync(0xffffffffu, start <= b);
    const int from = m ? 31 - __clz(m) : 0;
    gr.cost = __shfl_sync(0xffffffffu, cost - own, from);
    gr.start = __shfl_sync(0xffffffffu, start, from);
    gr.rows = m ? __shfl_sync(0xffffffffu, rows, from) : 0;
    gr.blocks = __shfl_sync(0xffffffffu, blocks, from);
  } else {
    // else from what the two kernels leave in the workspace
    pdl_wait_and_release();
    c0 = rest.ws_cum[b];
    nb = rest.ws_cum[b + 1] - static_cast<int>(c0);
    tot = rest.ws_cum[rest.batch];
    ne_b = rest.ws_cum[rest.batch + 1 + b];
    tot_ne = rest.ws_cum[2 * rest.batch + 1];
    V = p.groups[p.num_groups].cost;
    for (int j0 = 0; j0 < p.num_groups; j0 += 32) {
      PrefixGroup own{0, INT32_MAX, 0, 0, -1};
      if (j0 + lane < p.num_groups) own = p.groups[j0 + lane];
      const uint32_t m = __ballot_sync(0xffffffffu, own.start <= b);
      if (m == 0) continue;
      const int from = 31 - __clz(m);
      gr.cost = __shfl_sync(0xffffffffu, own.cost, from);
      gr.start = __shfl_sync(0xffffffffu, own.start, from);
      gr.rows = __shfl_sync(0xffffffffu, own.rows, from);
      gr.blocks = __shfl_sync(0xffffffffu, own.blocks, from);
    }
  }
  const int row = (b - gr.start) * G + h;
  const int64_t R = ranges;
  int64_t lo = 0, hi = 0, r0 = 0, n_pre = 0, base = 0;     // the unit's cost span; its ranges r0 .. r0 + n_pre - 1
  // (row < 0: group starts that are not as documented, none at or before b)
  if (row >= 0 && row < gr.rows && shares_prefix(gr.blocks, ctx, cap)) {
    const int kt = prefix_tiles(gr.blocks), unit = row / kPrefixUnitRows;
    lo = gr.cost + (static_cast<int64_t>(g) * prefix_units(gr.rows) + unit) * kt;
    hi = lo + kt;
    r0 = div_nonneg((lo + 1) * R + V - 1, V) - 1;          // largest r with r V / R <= lo
    n_pre = div_nonneg(hi * R + V - 1, V) - r0;
    base = piece_row(gr.start, p.n_q_heads, g, gr.rows, unit, 0) + row % kPrefixUnitRows;
  }
  // ---- the sequence's own blocks ----
  CombineSpan sp{};
  int64_t n_own = 0;
  if (nb > 0) {
    sp = combine_span(rest, g, c0, nb, tot, ne_b, tot_ne, rest_grid);
    n_own = sp.r1 - sp.r0 + 1;
  }
  // state x of the list (null: its range holds none of the pair's)
  auto locate = [&](int64_t x, const float*& ml, const float*& o) {
    ml = o = nullptr;
    if (x < n_pre) {
      const int64_t r = r0 + x;
      if (max(lo, div_nonneg(r * V, R)) < min(hi, div_nonneg((r + 1) * V, R))) {
        const int64_t i = base + r * kPrefixUnitRows;
        ml = p.ml + i * 2;
        o = p.o + i * D;
      }
    } else if (x < n_pre + n_own) {
      const int64_t r = sp.r0 + (x - n_pre);
      if (n_own == 1) {
        ml = rest.rest_ml + u * 2;
        o = rest.rest_o + u * D;
      } else if (combine_has_piece(sp, rest, r, rest_grid)) {
        const int64_t i = combine_slot(sp, r) * G + h;
        ml = rest.ws_ml + i * 2;
        o = rest.ws_o + i * D;
      }
    }
  };
  const float *ml, *o;
  locate(lane, ml, o);
  if (local) pdl_wait_and_release();
  for (int64_t x0 = 0; x0 < n_pre + n_own; x0 += 32) {
    if (x0 > 0) locate(x0 + lane, ml, o);
    const float2 state = ml != nullptr ? *reinterpret_cast<const float2*>(ml) : make_float2(-INFINITY, 0.f);
    uint32_t left = __ballot_sync(0xffffffffu, ml != nullptr);
    // each piece's weight against the maximum over all of them (the lanes', then
    // the earlier rounds'), so that only the outputs are summed in turn
    float m = state.x;
#pragma unroll
    for (int k = 16; k >= 1; k >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, k));
    const float mn = fmaxf(M, m), ref = (mn == -INFINITY) ? 0.f : mn;
    const float keep = exp2f(M - ref), w = exp2f(state.x - ref);
    float l = w * state.y;
#pragma unroll
    for (int k = 16; k >= 1; k >>= 1) l += __shfl_xor_sync(0xffffffffu, l, k);
    L = L * keep + l;
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
        const float* from = reinterpret_cast<const float*>(
            __shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(o), src[q] < 0 ? 0 : src[q]));
        if (src[q] >= 0) load(from, v[q]);
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
  const float inv = L > 0.f ? 1.f / L : 0.f;
  auto* out = static_cast<typename QT::storage*>(rest.out) + u * D + N * lane;
  if constexpr (N == 4)
    *reinterpret_cast<uint2*>(out) =
        make_uint2(pack2(O[0] * inv, O[1] * inv, QT{}), pack2(O[2] * inv, O[3] * inv, QT{}));
  else
    *reinterpret_cast<uint32_t*>(out) = pack2(O[0] * inv, O[1] * inv, QT{});
}

namespace {

template <typename QT, int D, int G>
pkv_status prepare_prefix_variant() {
  auto kern = prefix_kernel<QT, D, G>;
  int dev = 0;
  if (cuda_failed(cudaGetDevice(&dev), "cudaGetDevice")) return PKV_ERR_CUDA;
  static std::mutex mu;
  static bool done[kMaxDevices] = {};
  if (dev < 0 || dev >= kMaxDevices) return PKV_ERR_UNSUPPORTED;
  std::lock_guard<std::mutex> lock(mu);
  if (!done[dev]) {
    if (cuda_failed(cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         static_cast<int>(PrefixSmem<D>::bytes(kMaxPrefixGroups))),
                    "cudaFuncSetAttribute") ||
        // (the SM's whole shared memory, so that what this kernel leaves is the next one's)
        cuda_failed(cudaFuncSetAttribute(kern, cudaFuncAttributePreferredSharedMemoryCarveout,
                                         cudaSharedmemCarveoutMaxShared),
                    "cudaFuncSetAttribute"))
      return PKV_ERR_CUDA;
    done[dev] = true;
  }
  return PKV_OK;
}

template <typename QT, int D, int G>
pkv_status launch_prefix_variant(PrefixParams& p, int ranges, cudaStream_t stream) {
  return cuda_failed(launch_pdl(prefix_kernel<QT, D, G>, dim3(static_cast<unsigned>(ranges)), dim3(kXThreads),
                                PrefixSmem<D>::bytes(p.num_groups), stream, p),
                     "prefix_kernel launch")
             ? PKV_ERR_CUDA
             : PKV_OK;
}

template <typename QT, int D, int G>
pkv_status launch_merge_variant(const PrefixParams& p, int ranges, const DecodeParams& rest, int rest_grid,
                                cudaStream_t stream) {
  const int64_t units = static_cast<int64_t>(p.batch) * p.n_q_heads;
  const int64_t grid = (units + kMergeWarps - 1) / kMergeWarps;
  if (grid > INT32_MAX) return PKV_ERR_UNSUPPORTED;
  return cuda_failed(launch_pdl(prefix_merge_kernel<QT, D, G>, dim3(static_cast<unsigned>(grid)),
                                dim3(kMergeWarps * 32), 0, stream, p, ranges, rest, rest_grid),
                     "prefix_merge_kernel launch")
             ? PKV_ERR_CUDA
             : PKV_OK;
}

// calls f with the type, head_dim and group as template arguments
template <typename F>
pkv_status dispatch(pkv_dtype dtype, int head_dim, int group, F&& f) {
  auto by_group = [&](auto qt, auto d) -> pkv_status {
    switch (group) {
      case 1: return f(qt, d, std::integral_constant<int, 1>{});
      case 2: return f(qt, d, std::integral_constant<int, 2>{});
      case 4: return f(qt, d, std::integral_constant<int, 4>{});
      case 8: return f(qt, d, std::integral_constant<int, 8>{});
      default: return PKV_ERR_UNSUPPORTED;
    }
  };
  auto by_dim = [&](auto qt) -> pkv_status {
    return head_dim == 64 ? by_group(qt, std::integral_constant<int, 64>{})
                          : by_group(qt, std::integral_constant<int, 128>{});
  };
  return dtype == PKV_F16 ? by_dim(F16{}) : by_dim(BF16{});
}

}  // namespace

size_t prefix_smem_bytes(int head_dim, int num_groups) {
  return head_dim == 64 ? PrefixSmem<64>::bytes(num_groups) : PrefixSmem<128>::bytes(num_groups);
}

pkv_status prepare_prefix(int group, int head_dim, pkv_dtype dtype) {
  return dispatch(dtype, head_dim, group, [](auto qt, auto d, auto g) {
    return prepare_prefix_variant<decltype(qt), decltype(d)::value, decltype(g)::value>();
  });
}

pkv_status launch_prefix(PrefixParams& p, int ranges, int group, int head_dim, pkv_dtype dtype, cudaStream_t stream) {
  return dispatch(dtype, head_dim, group, [&](auto qt, auto d, auto g) {
    return launch_prefix_variant<decltype(qt), decltype(d)::value, decltype(g)::value>(p, ranges, stream);
  });
}

pkv_status launch_prefix_merge(const PrefixParams& p, int ranges, const DecodeParams& rest, int rest_grid, int group,
                               int head_dim, pkv_dtype dtype, cudaStream_t stream) {
  return dispatch(dtype, head_dim, group, [&](auto qt, auto d, auto g) {
    return launch_merge_variant<decltype(qt), decltype(d)::value, decltype(g)::value>(p, ranges, rest, rest_grid,
                                                                                      stream);
  });
}

}  // namespace pkv

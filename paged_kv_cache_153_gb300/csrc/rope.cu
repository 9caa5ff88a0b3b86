// Rotary positions fused with the KV append (sm_103a), and the host function
// that lays out a rotation's frequencies.
//
// What is computed.  The first R = rot_dim elements of a head are R / 2 pairs;
// pair i of a token at position p turns by the angle p f_i:
//   x' = a (x cos - y sin),   y' = a (x sin + y cos)
// (a: the amplitude of a long-context scaling, 1 without one).  The pairs are
// (2 i, 2 i + 1) in the interleaved layout and (i, i + R / 2) in the half one;
// elements R.. of a head pass through.  q goes to q_out, the turned k and the
// unturned v to the token's cache slot.
//
// Angles.  f_i / (2 pi), a fraction of a turn per position, is given as a
// 64-bit fixed-point number: p times it, modulo 2^64, is the angle modulo one
// turn, exactly, in one integer product.  Only the remaining fraction of a turn
// in [-1/2, 1/2) is rounded to fp32 before sincospi, so positions of 2^20 and
// more keep fp32 accuracy, which p f_i in fp32 would not (its rounding at 10^6
// rad is 0.03 rad).  The rotation is fp32; each element is rounded once, to
// the output's or the cache's type.
//
// Bound and layout.  A token reads (Hq + 2 Hkv) D 16-bit elements and writes
// as many: memory-bound, and latency-bound below a few hundred tokens.  One
// thread block per token, so the R / 2 angles are computed once for all of its
// heads (in shared memory, while the block's first loads are in flight); a
// thread owns 16-byte chunks, in the half layout both chunks of its pairs, so
// q_out may be q.  On GB300, 8192 tokens of 32 query / 8 KV heads of 128 bf16
// (201 MB): 35.2 us, 5.72 TB/s of a 6.8 TB/s copy, with 128 threads and two items
// in flight each (256 threads 37.8, four items 36.0, one 37.2; loads that wait
// for the position and slot first 41.6).  Into an FP8 cache (185 MB) 39.2 us, for
// the exact quotient of each stored element (36.1 with a product in its place).
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>

#include "host_util.h"
#include "pkv_common.cuh"

namespace pkv {

struct RopeParams {
  const unsigned char* q;        // [T] rows of Hq D, q_stride bytes apart (null: no q)
  const unsigned char* k;        // [T] rows of Hkv D (null: no append)
  const unsigned char* v;
  unsigned char* q_out;
  unsigned char* k_cache;        // [NB, Hkv, 16, D]
  unsigned char* v_cache;
  const float* k_scale;          // [Hkv] (FP8 cache only)
  const float* v_scale;
  const int32_t* positions;      // [T]
  const int64_t* slots;          // [T]
  const uint64_t* turns;         // [R / 2]
  int32_t* err;
  int64_t q_stride, k_stride, v_stride, q_out_stride;   // bytes between tokens
  int64_t num_slots;
  int n_q_heads, n_kv_heads, head_dim, rot_dim;
  float amplitude;
};

constexpr int kRopeThreads = 128;
constexpr int kRopeUnroll = 2;   // items whose loads a thread issues before the angles

// eight floats -> eight elements of the output type at dst (16 or 8 bytes)
template <typename T>
__device__ __forceinline__ void store8(unsigned char* dst, const float* f, float scale, T) {
  if constexpr (T::kBytes == 2) {
    *reinterpret_cast<uint4*>(dst) = make_uint4(pack2(f[0], f[1], T{}), pack2(f[2], f[3], T{}),
                                                pack2(f[4], f[5], T{}), pack2(f[6], f[7], T{}));
  } else {
    uint32_t w[4];
#pragma unroll
    for (int e = 0; e < 4; ++e)
      w[e] = fp8x2_from_f32(__fdiv_rn(f[2 * e], scale), __fdiv_rn(f[2 * e + 1], scale), T{});
    *reinterpret_cast<uint2*>(dst) = make_uint2(w[0] | (w[1] << 16), w[2] | (w[3] << 16));
  }
}

// eight 16-bit elements, as they are, to the output type
template <typename IN, typename T>
__device__ __forceinline__ void copy8(unsigned char* dst, const uint4& raw, float scale) {
  if constexpr (T::kBytes == 2)
    *reinterpret_cast<uint4*>(dst) = raw;
  else
    *reinterpret_cast<uint2*>(dst) = quant8_fp8<T>(&raw, scale, IN{});
}

// IN: type of q, k_new, v_new and q_out; KV: the cache's (IN, or an FP8 format)
template <typename IN, typename KV, bool HALF>
__global__ void __launch_bounds__(kRopeThreads) rope_append_kernel(const __grid_constant__ RopeParams p) {
  __shared__ float2 cs[64];
  const int64_t t = blockIdx.x;
  const int tid = threadIdx.x;
  pdl_wait();   // (writes the cache and q_out: no early release of the next launch)
  // (the position and the slot travel together with the rows)
  const int32_t pos = p.positions[t];
  int64_t slot = p.k ? p.slots[t] : -1;
  const int D = p.head_dim, R = p.rot_dim;
  // a row's items: its pair chunks, then the chunks that pass through
  const int pairs = HALF ? R / 16 : R / 8;
  const int per_row = pairs + (D - R) / 8;
  const int q_rows = p.q ? p.n_q_heads : 0, kv_rows = p.k ? p.n_kv_heads : 0;
  const int qk_items = (q_rows + kv_rows) * per_row;
  const int items = qk_items + kv_rows * (D / 8);
  int64_t row0 = 0;

  struct Item {
    int chunk;                   // 16-byte chunk of the row (its first, for a pair)
    int row;                     // query or KV head
    int kind;                    // 0: q, 1: k, 2: v, -1: nothing to do
    bool turn;
  };
  auto item_at = [&](int i) -> Item {
    Item it{0, 0, -1, false};
    if (i >= items) return it;
    if (i < qk_items) {
      const int r = i / per_row, x = i - r * per_row;
      it.turn = x < pairs;
      it.chunk = it.turn ? x : R / 8 + (x - pairs);
      it.kind = r < q_rows ? 0 : 1;
      it.row = r < q_rows ? r : r - q_rows;
    } else {
      const int x = i - qk_items, per_v = D / 8;
      it.row = x / per_v;
      it.chunk = x - it.row * per_v;
      it.kind = 2;
    }
    return it;
  };
  auto load = [&](const Item& it, uint4& a, uint4& b) {
    if (it.kind < 0) return;
    const unsigned char* src = (it.kind == 0   ? p.q + t * p.q_stride
                                : it.kind == 1 ? p.k + t * p.k_stride
                                               : p.v + t * p.v_stride) +
                               (static_cast<int64_t>(it.row) * D + it.chunk * 8) * 2;
    a = *reinterpret_cast<const uint4*>(src);
    if (HALF && it.turn) b = *reinterpret_cast<const uint4*>(src + R);   // (R / 2 elements further)
  };
  auto finish = [&](const Item& it, const uint4& a, const uint4& b) {
    if (it.kind < 0 || (it.kind > 0 && slot < 0)) return;
    const float scale =
        (KV::kBytes == 1 && it.kind != 0) ? (it.kind == 1 ? p.k_scale[it.row] : p.v_scale[it.row]) : 1.f;
    const int esz = it.kind == 0 ? 2 : KV::kBytes;
    unsigned char* dst =
        it.kind == 0 ? p.q_out + t * p.q_out_stride + static_cast<int64_t>(it.row) * D * 2
                     : (it.kind == 1 ? p.k_cache : p.v_cache) +
                           (row0 + static_cast<int64_t>(it.row) * kBlockSize) * D * KV::kBytes;
    dst += it.chunk * 8 * esz;
    if (!it.turn) {
      if (it.kind == 0)
        copy8<IN, IN>(dst, a, 1.f);
      else
        copy8<IN, KV>(dst, a, scale);
      return;
    }
    float x[8], y[8];
    load8(&a, x, IN{});
    if constexpr (HALF) {
      load8(&b, y, IN{});
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float2 c = cs[8 * it.chunk + e];
        const float u = x[e], w = y[e];
        x[e] = u * c.x - w * c.y;
        y[e] = u * c.y + w * c.x;
      }
    } else {
#pragma unroll
      for (int e = 0; e < 8; e += 2) {
        const float2 c = cs[4 * it.chunk + e / 2];
        const float u = x[e], w = x[e + 1];
        x[e] = u * c.x - w * c.y;
        x[e + 1] = u * c.y + w * c.x;
      }
    }
    if (it.kind == 0) {
      store8(dst, x, 1.f, IN{});
      if constexpr (HALF) store8(dst + R, y, 1.f, IN{});   // (R / 2 elements further)
    } else {
      store8(dst, x, scale, KV{});
      if constexpr (HALF) store8(dst + R / 2 * KV::kBytes, y, scale, KV{});
    }
  };

  Item it[kRopeUnroll];
  uint4 a[kRopeUnroll], b[kRopeUnroll];
#pragma unroll
  for (int u = 0; u < kRopeUnroll; ++u) {
    it[u] = item_at(tid + u * kRopeThreads);
    load(it[u], a[u], b[u]);
  }
  if (pos < 0) return;   // a padding token (the whole block)
  if (slot >= p.num_slots) {
    if (tid == 0) record_error(p.err, PKV_ERR_OOB);
    slot = -1;
  }
  // first row of the slot in head 0's slab; heads are 16 rows apart
  row0 = (slot / kBlockSize) * p.n_kv_heads * kBlockSize + slot % kBlockSize;
  if (tid < R / 2) {
    const int64_t turn = static_cast<int64_t>(p.turns[tid] * static_cast<uint64_t>(pos));
    float s, c;
    sincospif(__ll2float_rn(turn) * 0x1p-63f, &s, &c);   // (half turns)
    cs[tid] = make_float2(c * p.amplitude, s * p.amplitude);
  }
  __syncthreads();
#pragma unroll
  for (int u = 0; u < kRopeUnroll; ++u) finish(it[u], a[u], b[u]);
  for (int i = tid + kRopeUnroll * kRopeThreads; i < items; i += kRopeThreads) {
    const Item x = item_at(i);
    uint4 xa, xb;
    load(x, xa, xb);
    finish(x, xa, xb);
  }
}

namespace {

template <typename IN, typename KV>
pkv_status launch_rope(const RopeParams& p, int64_t num_tokens, pkv_rope_layout layout, cudaStream_t stream) {
  auto kern = layout == PKV_ROPE_HALF ? rope_append_kernel<IN, KV, true> : rope_append_kernel<IN, KV, false>;
  const cudaError_t e =
      launch_pdl(kern, dim3(static_cast<unsigned>(num_tokens)), dim3(kRopeThreads), 0, stream, p);
  return cuda_failed(e, "rope_append_kernel launch") ? PKV_ERR_CUDA : PKV_OK;
}

// kv: 0 = the 16-bit type of q, 1 = E4M3, 2 = E5M2
pkv_status rope_common(int kv, const void* q, int64_t q_stride, const void* k_new, int64_t k_stride,
                       const void* v_new, int64_t v_stride, const int32_t* positions, const int64_t* slot_mapping,
                       int64_t num_tokens, const uint64_t* turns, int rot_dim, pkv_rope_layout layout,
                       float amplitude, void* q_out, int64_t q_out_stride, void* k_cache, void* v_cache,
                       int64_t num_blocks, const float* k_scale, const float* v_scale, int num_q_heads,
                       int num_kv_heads, int head_dim, int block_size, pkv_dtype dtype, int32_t* err_flag,
                       void* stream) {
  if (num_tokens < 0 || num_blocks < 0 || !std::isfinite(amplitude)) return PKV_ERR_INVALID_ARG;
  if (dtype != PKV_F16 && dtype != PKV_BF16) return PKV_ERR_INVALID_ARG;
  if (layout != PKV_ROPE_HALF && layout != PKV_ROPE_INTERLEAVED) return PKV_ERR_INVALID_ARG;
  if (block_size != kBlockSize || (head_dim != 64 && head_dim != 128)) return PKV_ERR_UNSUPPORTED;
  if (rot_dim <= 0 || rot_dim > head_dim) return PKV_ERR_INVALID_ARG;
  if (rot_dim % 16) return PKV_ERR_UNSUPPORTED;
  if ((q == nullptr) != (q_out == nullptr) || (k_new == nullptr) != (v_new == nullptr)) return PKV_ERR_INVALID_ARG;
  if (num_tokens == 0) return PKV_OK;
  if (num_tokens > INT32_MAX) return PKV_ERR_UNSUPPORTED;
  if (!positions || !turns || (q == nullptr && k_new == nullptr)) return PKV_ERR_INVALID_ARG;
  uintptr_t align = 0;
  if (q != nullptr) {
    if (num_q_heads <= 0) return PKV_ERR_INVALID_ARG;
    const int64_t row = static_cast<int64_t>(num_q_heads) * head_dim;
    if (q_stride < row || q_out_stride < row || q_stride % 8 || q_out_stride % 8) return PKV_ERR_INVALID_ARG;
    align |= reinterpret_cast<uintptr_t>(q) | reinterpret_cast<uintptr_t>(q_out);
  }
  if (k_new != nullptr) {
    if (num_kv_heads <= 0 || !slot_mapping || !k_cache || !v_cache) return PKV_ERR_INVALID_ARG;
    if (kv != 0 && (!k_scale || !v_scale)) return PKV_ERR_INVALID_ARG;
    const int64_t row = static_cast<int64_t>(num_kv_heads) * head_dim;
    if (k_stride < row || v_stride < row || k_stride % 8 || v_stride % 8) return PKV_ERR_INVALID_ARG;
    align |= reinterpret_cast<uintptr_t>(k_new) | reinterpret_cast<uintptr_t>(v_new) |
             reinterpret_cast<uintptr_t>(k_cache) | reinterpret_cast<uintptr_t>(v_cache);
  }
  if (align & 15u) return PKV_ERR_INVALID_ARG;
  RopeParams p{};
  p.q = static_cast<const unsigned char*>(q);
  p.k = static_cast<const unsigned char*>(k_new);
  p.v = static_cast<const unsigned char*>(v_new);
  p.q_out = static_cast<unsigned char*>(q_out);
  p.k_cache = static_cast<unsigned char*>(k_cache);
  p.v_cache = static_cast<unsigned char*>(v_cache);
  p.k_scale = k_scale;
  p.v_scale = v_scale;
  p.positions = positions;
  p.slots = slot_mapping;
  p.turns = turns;
  p.err = err_flag;
  p.q_stride = q_stride * 2;
  p.k_stride = k_stride * 2;
  p.v_stride = v_stride * 2;
  p.q_out_stride = q_out_stride * 2;
  p.num_slots = num_blocks * kBlockSize;
  p.n_q_heads = num_q_heads;
  p.n_kv_heads = num_kv_heads;
  p.head_dim = head_dim;
  p.rot_dim = rot_dim;
  p.amplitude = amplitude;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (dtype == PKV_F16)
    return kv == 0 ? launch_rope<F16, F16>(p, num_tokens, layout, s)
         : kv == 1 ? launch_rope<F16, E4M3>(p, num_tokens, layout, s)
                   : launch_rope<F16, E5M2>(p, num_tokens, layout, s);
  return kv == 0 ? launch_rope<BF16, BF16>(p, num_tokens, layout, s)
       : kv == 1 ? launch_rope<BF16, E4M3>(p, num_tokens, layout, s)
                 : launch_rope<BF16, E5M2>(p, num_tokens, layout, s);
}

}  // namespace
}  // namespace pkv

using namespace pkv;

extern "C" pkv_status pkv_rope_append(const void* q, int64_t q_stride, const void* k_new, int64_t k_stride,
                                      const void* v_new, int64_t v_stride, const int32_t* positions,
                                      const int64_t* slot_mapping, int64_t num_tokens, const uint64_t* turns,
                                      int rot_dim, pkv_rope_layout layout, float amplitude, void* q_out,
                                      int64_t q_out_stride, void* k_cache, void* v_cache, int64_t num_blocks,
                                      int num_q_heads, int num_kv_heads, int head_dim, int block_size,
                                      pkv_dtype dtype, int32_t* err_flag, void* stream) {
  return rope_common(0, q, q_stride, k_new, k_stride, v_new, v_stride, positions, slot_mapping, num_tokens, turns,
                     rot_dim, layout, amplitude, q_out, q_out_stride, k_cache, v_cache, num_blocks, nullptr, nullptr,
                     num_q_heads, num_kv_heads, head_dim, block_size, dtype, err_flag, stream);
}

extern "C" pkv_status pkv_rope_append_fp8(const void* q, int64_t q_stride, const void* k_new, int64_t k_stride,
                                          const void* v_new, int64_t v_stride, const int32_t* positions,
                                          const int64_t* slot_mapping, int64_t num_tokens, const uint64_t* turns,
                                          int rot_dim, pkv_rope_layout layout, float amplitude, void* q_out,
                                          int64_t q_out_stride, uint8_t* k_cache, uint8_t* v_cache,
                                          int64_t num_blocks, const float* k_scale, const float* v_scale,
                                          int num_q_heads, int num_kv_heads, int head_dim, int block_size,
                                          pkv_dtype dtype, int32_t* err_flag, void* stream) {
  return rope_common(1, q, q_stride, k_new, k_stride, v_new, v_stride, positions, slot_mapping, num_tokens, turns,
                     rot_dim, layout, amplitude, q_out, q_out_stride, k_cache, v_cache, num_blocks, k_scale, v_scale,
                     num_q_heads, num_kv_heads, head_dim, block_size, dtype, err_flag, stream);
}

extern "C" pkv_status pkv_rope_append_e5m2(const void* q, int64_t q_stride, const void* k_new, int64_t k_stride,
                                           const void* v_new, int64_t v_stride, const int32_t* positions,
                                           const int64_t* slot_mapping, int64_t num_tokens, const uint64_t* turns,
                                           int rot_dim, pkv_rope_layout layout, float amplitude, void* q_out,
                                           int64_t q_out_stride, uint8_t* k_cache, uint8_t* v_cache,
                                           int64_t num_blocks, const float* k_scale, const float* v_scale,
                                           int num_q_heads, int num_kv_heads, int head_dim, int block_size,
                                           pkv_dtype dtype, int32_t* err_flag, void* stream) {
  return rope_common(2, q, q_stride, k_new, k_stride, v_new, v_stride, positions, slot_mapping, num_tokens, turns,
                     rot_dim, layout, amplitude, q_out, q_out_stride, k_cache, v_cache, num_blocks, k_scale, v_scale,
                     num_q_heads, num_kv_heads, head_dim, block_size, dtype, err_flag, stream);
}

extern "C" pkv_status pkv_rope_plan(int rot_dim, double base, pkv_rope_scaling scaling, double factor,
                                    double original_context, double low_turns, double high_turns, uint64_t* turns,
                                    float* amplitude) {
  constexpr double kTwoPi = 6.283185307179586476925286766559;
  if (rot_dim <= 0 || rot_dim % 2 || turns == nullptr || amplitude == nullptr) return PKV_ERR_INVALID_ARG;
  if (!(base > 1.0) || !std::isfinite(base)) return PKV_ERR_INVALID_ARG;
  if (scaling < PKV_ROPE_NONE || scaling > PKV_ROPE_WAVELENGTH) return PKV_ERR_INVALID_ARG;
  if (scaling != PKV_ROPE_NONE && (!(factor >= 1.0) || !std::isfinite(factor))) return PKV_ERR_INVALID_ARG;
  if (scaling == PKV_ROPE_RAMP || scaling == PKV_ROPE_WAVELENGTH)
    if (!(original_context > 0.0) || !std::isfinite(original_context) || !(low_turns > 0.0) ||
        !(high_turns > low_turns) || !std::isfinite(high_turns))
      return PKV_ERR_INVALID_ARG;
  if (scaling == PKV_ROPE_BASE) {
    if (rot_dim == 2) return PKV_ERR_INVALID_ARG;   // (its only frequency is 1 for every base)
    base *= std::pow(factor, rot_dim / (rot_dim - 2.0));
    if (!std::isfinite(base)) return PKV_ERR_INVALID_ARG;
  }
  double ramp_lo = 0.0, ramp_hi = 0.0;
  if (scaling == PKV_ROPE_RAMP) {
    // pair index whose frequency makes `turns` full turns over the original context
    auto pair_of = [&](double n) { return rot_dim * std::log(original_context / (n * kTwoPi)) / (2.0 * std::log(base)); };
    ramp_lo = std::max(std::floor(pair_of(high_turns)), 0.0);
    ramp_hi = std::min(std::ceil(pair_of(low_turns)), rot_dim - 1.0);
  }
  for (int i = 0; i < rot_dim / 2; ++i) {
    double f = std::pow(base, -2.0 * i / rot_dim);
    if (scaling == PKV_ROPE_LINEAR) {
      f /= factor;
    } else if (scaling == PKV_ROPE_RAMP) {
      const double w = std::min(std::max((i - ramp_lo) / std::max(ramp_hi - ramp_lo, 0.001), 0.0), 1.0);
      f = f / factor * w + f * (1.0 - w);
    } else if (scaling == PKV_ROPE_WAVELENGTH) {
      const double n = original_context * f / kTwoPi;
      const double w = std::min(std::max((n - low_turns) / (high_turns - low_turns), 0.0), 1.0);
      f = f / factor * (1.0 - w) + f * w;
    }
    // f <= 1 radian, so the fraction of a turn is below 1 / 6
    turns[i] = static_cast<uint64_t>(std::rint(std::ldexp(f / kTwoPi, 64)));
  }
  *amplitude = scaling == PKV_ROPE_RAMP ? static_cast<float>(0.1 * std::log(factor) + 1.0) : 1.f;
  return PKV_OK;
}

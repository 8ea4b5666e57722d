// pa_norm_rope_write: what a layer does to its new queries, keys and values
// before the attention, in one pass: RMS norm of every query and key head,
// the position rotation, and the slot_mapping scatter of K and V.
//
// Per head row x of D elements (all arithmetic in fp32, rounded once on the
// way out):
//   y_i = x_i * rsqrt(mean(x^2) + eps) * w_i
//   (y_a, y_b) -> (y_a cos - y_b sin, y_b cos + y_a sin)
// over the pairs (i, i + R/2), or (2i, 2i + 1) interleaved, of the first R
// elements; the angle's cos and sin come from a table row per position.
// Queries go to q_out; keys and values to their slots, as bit copies of the
// rounded row or e4m3(y / scale) (one rounding, straight from fp32).
//
// Bound: HBM.  Every byte is read and written once: (2 Hq + 2 Hkv) D b_q +
// 2 Hkv D b_kv per token plus its table row.
//
// Layout: a head row is held by D / 8 lanes, eight elements each as two
// chunks of four.  A lane's two chunks hold both halves of its pairs (chunk
// c of the first half and of the second half; interleaved pairs sit inside a
// chunk), so the rotation needs no exchange between lanes and only the norm
// reduces over the row's lanes.  A row group takes a few head rows of one
// token, all loads first and kept as they came, and reads the token's cos and
// sin once.  e4m3 V, whose pool is d-major, goes by windows of 16 tokens: a
// lane takes two elements of 16 rows and stores 16 bytes per element where
// the window's slots fill an aligned part of a block (single bytes otherwise).
#include <cuda_runtime.h>

#include <algorithm>

#include "pa_device.cuh"
#include "pa_kernels.h"
#include "slot_window.cuh"

namespace pa {
namespace {

constexpr int kThreads = 256;

// Four elements as they lie in memory.
template <typename T> struct Four { using V = uint2; };
template <> struct Four<float> { using V = uint4; };

__device__ __forceinline__ void unpack(const uint2& v, float (&x)[4]) {
  x[0] = dev::bf16_bits_to_f32(v.x & 0xFFFFu);
  x[1] = dev::bf16_bits_to_f32(v.x >> 16);
  x[2] = dev::bf16_bits_to_f32(v.y & 0xFFFFu);
  x[3] = dev::bf16_bits_to_f32(v.y >> 16);
}
__device__ __forceinline__ void unpack(const uint4& v, float (&x)[4]) {
  x[0] = __uint_as_float(v.x);
  x[1] = __uint_as_float(v.y);
  x[2] = __uint_as_float(v.z);
  x[3] = __uint_as_float(v.w);
}
// The same as two packed pairs.
__device__ __forceinline__ void unpack2(const uint2& v, uint64_t (&x)[2]) {
  x[0] = dev::f2(__uint_as_float(v.x << 16), __uint_as_float(v.x & 0xFFFF0000u));
  x[1] = dev::f2(__uint_as_float(v.y << 16), __uint_as_float(v.y & 0xFFFF0000u));
}
__device__ __forceinline__ void unpack2(const uint4& v, uint64_t (&x)[2]) {
  x[0] = dev::f2(__uint_as_float(v.x), __uint_as_float(v.y));
  x[1] = dev::f2(__uint_as_float(v.z), __uint_as_float(v.w));
}
__device__ __forceinline__ void split2(const uint64_t (&x)[2], float (&y)[4]) {
  dev::f2_split(x[0], y[0], y[1]);
  dev::f2_split(x[1], y[2], y[3]);
}
template <typename T>
__device__ __forceinline__ typename Four<T>::V load4(const T* p) {
  return *reinterpret_cast<const typename Four<T>::V*>(p);
}
template <typename T>
__device__ __forceinline__ void store4(T* p, const float (&x)[4]) {
  if constexpr (sizeof(T) == 4) {
    *reinterpret_cast<float4*>(p) = make_float4(x[0], x[1], x[2], x[3]);
  } else {
    *reinterpret_cast<uint2*>(p) = make_uint2(dev::pack_bf16(x[0], x[1]), dev::pack_bf16(x[2], x[3]));
  }
}
__device__ __forceinline__ uint32_t quant2(float a, float b, float scale) {
  return dev::e4m3x2_from_f32(__fdiv_rn(a, scale), __fdiv_rn(b, scale));
}

// e4m3 V of one window of tokens and one kv head per D / 2 lanes.
template <typename T, int D>
__device__ __forceinline__ void write_v_window(const NormRopeParams& p, int64_t item) {
  constexpr int LANES = D / 2;  // whole warps
  const int hkv = p.num_kv_heads;
  const uint32_t win = dev::fdiv((uint32_t)item, p.heads);
  const int h = (int)((uint32_t)item - win * hkv);
  const int d0 = 2 * (threadIdx.x % LANES);
  const float scale = p.v_head ? __ldg(p.v_head + h) : p.v_scale;
  const int64_t end = dev::window_start(p.slots, p.num_tokens, (int64_t)win + 1);
  for (int64_t t = dev::window_start(p.slots, p.num_tokens, win); t < end; t += dev::kWindow) {
    const int n = (int)min((int64_t)dev::kWindow, end - t);
    int64_t s0;
    bool whole = dev::window_aligned(p.slots, t, n, p.num_slots, &s0);
    // a token whose position is outside the table is left out
    if (p.cos_sin) {
      const int pos = (threadIdx.x & 31) < n ? __ldg(p.positions + t + (threadIdx.x & 31)) : 0;
      whole = whole && __all_sync(0xffffffffu, pos >= 0 && pos < p.num_positions);
    }
    uint32_t code[2][4];  // [element][4 tokens]
    const T* src = reinterpret_cast<const T*>(p.v) + t * p.v_stride + h * D + d0;
    float2 x[dev::kWindow];
#pragma unroll
    for (int j = 0; j < dev::kWindow; ++j) {
      if constexpr (sizeof(T) == 4) {
        x[j] = *reinterpret_cast<const float2*>(src + min(j, n - 1) * p.v_stride);
      } else {  // kept as it came: the pair's upper element in y
        x[j].x = __uint_as_float(*reinterpret_cast<const uint32_t*>(src + min(j, n - 1) * p.v_stride));
      }
    }
#pragma unroll
    for (int j = 0; j < dev::kWindow; j += 2) {
      if constexpr (sizeof(T) != 4) {
#pragma unroll
        for (int k = j; k < j + 2; ++k) {
          const uint32_t w = __float_as_uint(x[k].x);
          x[k] = make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
        }
      }
      const uint32_t lo = quant2(x[j].x, x[j + 1].x, scale), hi = quant2(x[j].y, x[j + 1].y, scale);
      if (j & 2) {
        code[0][j >> 2] |= lo << 16;
        code[1][j >> 2] |= hi << 16;
      } else {
        code[0][j >> 2] = lo;
        code[1][j >> 2] = hi;
      }
    }
    if (whole) {
      uint8_t* dst = p.v_cache + (((s0 >> p.bs_shift) * hkv + h) * D + d0) * p.block_size + (s0 & (p.block_size - 1));
#pragma unroll
      for (int e = 0; e < 2; ++e)
        *reinterpret_cast<uint4*>(dst + e * p.block_size) = make_uint4(code[e][0], code[e][1], code[e][2], code[e][3]);
    } else {
#pragma unroll
      for (int j = 0; j < dev::kWindow; ++j) {
        if (j >= n) break;
        const int64_t slot = __ldg(p.slots + t + j);
        if (slot < 0 || slot >= p.num_slots) continue;
        if (p.cos_sin) {
          const int pos = __ldg(p.positions + t + j);
          if (pos < 0 || pos >= p.num_positions) continue;
        }
        uint8_t* dst =
            p.v_cache + (((slot >> p.bs_shift) * hkv + h) * D + d0) * p.block_size + (slot & (p.block_size - 1));
#pragma unroll
        for (int e = 0; e < 2; ++e) dst[e * p.block_size] = (uint8_t)(code[e][j >> 2] >> (8 * (j & 3)));
      }
    }
  }
}

// T: element type of the new rows; FP8: an e4m3 pool; HEADS: head rows of one
// token per row group; `block` counts CTA-sized pieces of the row groups.
// FULL: every head is normed and rotated over its whole width in halves (what
// a model with query and key norms asks for): issue slots bound the general
// form, so this one multiplies weights and angles together once per group,
// works on pairs of elements and moves V rows as they are (4344 tokens of 32 + 2
// x 8 heads, one call between events: 24.6 us; the general form 24.6 without
// norms, 26.6 with them, interleaved or over half the head).
template <typename T, int D, bool FP8, int HEADS, bool FULL>
__device__ __forceinline__ void prepare_rows(const NormRopeParams& p, uint32_t block) {
  constexpr int LANES = D / 8;  // lanes of a head row
  // A token's row groups: its query heads', its keys', its values' (in e4m3
  // the windows'), HEADS rows each: a group's rows are of one kind.
  const int hq = p.num_q_heads, hkv = p.num_kv_heads;
  const uint32_t item = block * (kThreads / LANES) + threadIdx.x / LANES;
  const uint32_t items = (uint32_t)p.num_tokens * p.per_token.d;
  const bool live = item < items;  // whole warps stay for the norm's shuffles
  const uint32_t t = live ? dev::fdiv(item, p.per_token) : 0;
  int g = live ? (int)(item - t * p.per_token.d) : 0;
  const int gq = (hq + HEADS - 1) / HEADS, gk = (hkv + HEADS - 1) / HEADS;
  const bool is_q = g < gq, is_v = g >= gq + gk;
  g -= is_q ? 0 : is_v ? gq + gk : gq;
  const int h0 = g * HEADS, nh = live ? (is_q ? hq : hkv) : 0;
  const int c = threadIdx.x % LANES;
  const int rot = p.rot_dim, half = rot >> 1;
  const bool turns = 8 * c < rot && !is_v;  // this lane's elements are rotated
  // the lane's two chunks of four elements
  int a0 = 8 * c, a1 = 8 * c + 4;
  if (FULL ? !is_v : turns && !p.interleaved) {
    a0 = 4 * c;
    a1 = half + 4 * c;
  }
  const int pos = p.cos_sin ? __ldg(p.positions + t) : 0;
  const int64_t slot = __ldg(p.slots + t);
  using V = typename Four<T>::V;
  V raw[HEADS][2];
  const T* rows = is_q   ? reinterpret_cast<const T*>(p.q) + t * p.q_stride
                  : is_v ? reinterpret_cast<const T*>(p.v) + t * p.v_stride
                         : reinterpret_cast<const T*>(p.k) + t * p.k_stride;
  rows += h0 * D;
#pragma unroll
  for (int j = 0; j < HEADS; ++j) {
    raw[j][0] = raw[j][1] = V{};
    if (h0 + j < nh) {
      raw[j][0] = load4(rows + j * D + a0);
      raw[j][1] = load4(rows + j * D + a1);
    }
  }
  const bool known = p.cos_sin == nullptr || (pos >= 0 && pos < p.num_positions);
  const bool in_pool = slot >= 0 && slot < p.num_slots;
  if constexpr (FULL) {
    if (!live || !known || (!is_q && !in_pool)) return;  // whole row groups: the sums below stay within one
    const uint32_t group = LANES == 32 ? 0xffffffffu : ((1u << LANES) - 1u) << (threadIdx.x & 31 & ~(LANES - 1));
    const int step = is_q ? D : p.block_size * D;
    const int64_t at = is_q ? ((int64_t)t * hq + h0) * D
                            : ((slot >> p.bs_shift) * hkv + h0) * step + (slot & (p.block_size - 1)) * D;
    if (is_v) {
      T* out = reinterpret_cast<T*>(p.v_cache) + at + a0;
#pragma unroll
      for (int j = 0; j < HEADS; ++j) {
        if (h0 + j >= nh) break;
        *reinterpret_cast<V*>(out + j * step) = raw[j][0];
        *reinterpret_cast<V*>(out + j * step + 4) = raw[j][1];
      }
      return;
    }
    const T* weight = reinterpret_cast<const T*>(is_q ? p.q_weight : p.k_weight);
    uint64_t w0[2], w1[2], c[2], s[2], ac[2], bs[2], bc[2], as[2];
    unpack2(load4(weight + a0), w0);
    unpack2(load4(weight + a1), w1);
    unpack2(__ldg(reinterpret_cast<const uint4*>(p.cos_sin + (int64_t)pos * D + a0)), c);
    unpack2(__ldg(reinterpret_cast<const uint4*>(p.cos_sin + (int64_t)pos * D + a1)), s);
    const uint64_t minus = dev::f2(-1.f, -1.f);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      ac[i] = dev::mul2(w0[i], c[i]);
      as[i] = dev::mul2(w0[i], s[i]);
      bc[i] = dev::mul2(w1[i], c[i]);
      bs[i] = dev::mul2(dev::mul2(w1[i], s[i]), minus);
    }
    T* out = reinterpret_cast<T*>(is_q ? p.q_out : p.k_cache) + at;
    uint8_t* out8 = p.k_cache + at;
#pragma unroll
    for (int j = 0; j < HEADS; ++j) {
      if (h0 + j >= nh) break;
      uint64_t a[2], b[2];
      unpack2(raw[j][0], a);
      unpack2(raw[j][1], b);
      uint64_t q2 = dev::mul2(a[0], a[0]);
      q2 = dev::fma2(a[1], a[1], q2);
      q2 = dev::fma2(b[0], b[0], q2);
      q2 = dev::fma2(b[1], b[1], q2);
      float ss, odd;
      dev::f2_split(q2, ss, odd);
      ss += odd;
#pragma unroll
      for (int o = LANES / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(group, ss, o);
      const float r = rsqrtf(ss * (1.f / D) + p.eps);
      const uint64_t r2 = dev::f2(r, r);
      uint64_t ya[2], yb[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        ya[i] = dev::mul2(dev::fma2(a[i], ac[i], dev::mul2(b[i], bs[i])), r2);
        yb[i] = dev::mul2(dev::fma2(b[i], bc[i], dev::mul2(a[i], as[i])), r2);
      }
      float x[2][4];
      split2(ya, x[0]);
      split2(yb, x[1]);
      if (!FP8 || is_q) {
        store4(out + j * step + a0, x[0]);
        store4(out + j * step + a1, x[1]);
      } else {
        const float scale = p.k_head ? __ldg(p.k_head + h0 + j) : p.k_scale;
        *reinterpret_cast<uint32_t*>(out8 + j * step + a0) =
            quant2(x[0][0], x[0][1], scale) | quant2(x[0][2], x[0][3], scale) << 16;
        *reinterpret_cast<uint32_t*>(out8 + j * step + a1) =
            quant2(x[1][0], x[1][1], scale) | quant2(x[1][2], x[1][3], scale) << 16;
      }
    }
    return;
  }
  // The norm's factor r is applied last (it commutes with weight and turn).
  float w[2][4], cs[4], sn[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) w[0][i] = w[1][i] = 1.f;
  const T* weight = reinterpret_cast<const T*>(is_q ? p.q_weight : p.k_weight);
  const bool norm = !is_v && weight != nullptr;
  if (norm) {
    unpack(load4(weight + a0), w[0]);
    unpack(load4(weight + a1), w[1]);
  }
  const bool turn = turns && known;  // (rot is 0 without a table)
  if (turn) {
    unpack(__ldg(reinterpret_cast<const uint4*>(p.cos_sin + (int64_t)pos * rot + 4 * c)), cs);
    unpack(__ldg(reinterpret_cast<const uint4*>(p.cos_sin + (int64_t)pos * rot + half + 4 * c)), sn);
  }
  T* dst;  // the group's first row in q_out or in a pool of T
  uint8_t* dst8 = nullptr;
  int step = D;
  if (is_q) {
    dst = reinterpret_cast<T*>(p.q_out) + ((int64_t)t * hq + h0) * D;
  } else {
    const int64_t blk = in_pool ? slot >> p.bs_shift : 0;
    const int off = in_pool ? (int)(slot & (p.block_size - 1)) : 0;
    step = p.block_size * D;
    const int64_t at = (blk * hkv + h0) * step + off * D;
    dst = reinterpret_cast<T*>(is_v ? p.v_cache : p.k_cache) + at;
    dst8 = p.k_cache + at;
  }
#pragma unroll
  for (int j = 0; j < HEADS; ++j) {
    float x[2][4];
    unpack(raw[j][0], x[0]);
    unpack(raw[j][1], x[1]);
    float r = 1.f;
    // the whole warp takes part in the sums: its row groups may be of
    // different kinds
    if (p.q_weight || p.k_weight) {
      float ss = 0.f;
#pragma unroll
      for (int i = 0; i < 4; ++i) ss += x[0][i] * x[0][i] + x[1][i] * x[1][i];
#pragma unroll
      for (int o = LANES / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
      if (norm) r = rsqrtf(ss * (1.f / D) + p.eps);
    }
    if (h0 + j >= nh || !known || (!is_q && !in_pool)) continue;
    if (!is_v) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        x[0][i] *= w[0][i];
        x[1][i] *= w[1][i];
      }
      if (turn && !p.interleaved) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float a = x[0][i], b = x[1][i];
          x[0][i] = a * cs[i] - b * sn[i];
          x[1][i] = b * cs[i] + a * sn[i];
        }
      } else if (turn) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          float(&ch)[4] = x[i >> 1];
          const float a = ch[2 * (i & 1)], b = ch[2 * (i & 1) + 1];
          ch[2 * (i & 1)] = a * cs[i] - b * sn[i];
          ch[2 * (i & 1) + 1] = b * cs[i] + a * sn[i];
        }
      }
      if (norm) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          x[0][i] *= r;
          x[1][i] *= r;
        }
      }
    }
    if (!FP8 || is_q) {
      store4(dst + j * step + a0, x[0]);
      store4(dst + j * step + a1, x[1]);
    } else {
      const float scale = p.k_head ? __ldg(p.k_head + h0 + j) : p.k_scale;
      uint8_t* out = dst8 + j * step;
      *reinterpret_cast<uint32_t*>(out + a0) = quant2(x[0][0], x[0][1], scale) | quant2(x[0][2], x[0][3], scale) << 16;
      *reinterpret_cast<uint32_t*>(out + a1) = quant2(x[1][0], x[1][1], scale) | quant2(x[1][2], x[1][3], scale) << 16;
    }
  }
}

// The first `v_blocks` of `blocks` pieces of work are windows of e4m3 V, the
// others row groups; a launch of more pieces than fit the GPU at once walks
// them with resident CTAs.
template <typename T, int D, bool FP8, int HEADS, bool FULL>
__global__ void __launch_bounds__(kThreads, sizeof(T) == 4 ? 3 : 4)
    norm_rope_write_kernel(const NormRopeParams p, uint32_t v_blocks, uint32_t blocks) {
  dev::grid_dep_wait();
  dev::grid_dep_launch();
  for (uint32_t w = blockIdx.x; w < blocks; w += gridDim.x) {
    if constexpr (FP8) {
      if (w < v_blocks) {
        const int64_t items = ((int64_t)p.num_tokens + dev::kWindow - 1) / dev::kWindow * p.num_kv_heads;
        const int64_t item = (int64_t)w * (kThreads / (D / 2)) + threadIdx.x / (D / 2);
        if (item < items) write_v_window<T, D>(p, item);
        continue;
      }
    }
    prepare_rows<T, D, FP8, HEADS, FULL>(p, w - (FP8 ? v_blocks : 0u));
  }
}

template <typename T, int D, bool FP8, int HEADS, bool FULL>
cudaError_t launch(const NormRopeParams& p, int num_sms, cudaStream_t stream) {
  NormRopeParams q = p;
  const int gk = (p.num_kv_heads + HEADS - 1) / HEADS;
  q.per_token = fast_div((uint32_t)((p.num_q_heads + HEADS - 1) / HEADS + (FP8 ? 1 : 2) * gk));
  const int64_t items = (int64_t)p.num_tokens * q.per_token.d;
  const int64_t rows = (items + kThreads / (D / 8) - 1) / (kThreads / (D / 8));
  int64_t vwin = 0;
  if (FP8) {
    const int64_t v = ((int64_t)p.num_tokens + dev::kWindow - 1) / dev::kWindow * p.num_kv_heads;
    vwin = (v + kThreads / (D / 2) - 1) / (kThreads / (D / 2));
    q.heads = fast_div((uint32_t)p.num_kv_heads);
  }
  if (items > INT32_MAX || rows + vwin > INT32_MAX) return cudaErrorNotSupported;
  norm_rope_write_kernel<T, D, FP8, HEADS, FULL>
      <<<(unsigned)std::min<int64_t>(rows + vwin, (int64_t)num_sms * (sizeof(T) == 4 ? 3 : 4)), kThreads, 0, stream>>>(q, (uint32_t)vwin, (uint32_t)(rows + vwin));
  return cudaGetLastError();
}

// Head rows per row group: one while the whole step then fits the GPU at once
// (latency: a decode step of 64 tokens), else four (bytes in flight).
template <typename T, int D, bool FP8>
cudaError_t launch_h(const NormRopeParams& p, int num_sms, cudaStream_t stream) {
  const int64_t rows = (int64_t)p.num_tokens * (p.num_q_heads + 2 * p.num_kv_heads);
  const bool full = p.cos_sin && p.rot_dim == D && !p.interleaved && p.q_weight && p.k_weight;
  if (rows * (D / 8) <= (int64_t)num_sms * 2048)
    return full ? launch<T, D, FP8, 1, true>(p, num_sms, stream) : launch<T, D, FP8, 1, false>(p, num_sms, stream);
  return full ? launch<T, D, FP8, 4, true>(p, num_sms, stream) : launch<T, D, FP8, 4, false>(p, num_sms, stream);
}

template <typename T, bool FP8>
cudaError_t launch_d(const NormRopeParams& p, int num_sms, cudaStream_t stream) {
  if (p.head_dim == 64) return launch_h<T, 64, FP8>(p, num_sms, stream);
  if (p.head_dim == 128) return launch_h<T, 128, FP8>(p, num_sms, stream);
  return cudaErrorNotSupported;
}

}  // namespace

cudaError_t launch_norm_rope_write(const NormRopeParams& p, int q_dtype, int kv_dtype, int num_sms,
                                   cudaStream_t stream) {
  if (q_dtype == kF32)
    return kv_dtype == kFP8 ? launch_d<float, true>(p, num_sms, stream) : launch_d<float, false>(p, num_sms, stream);
  return kv_dtype == kFP8 ? launch_d<__nv_bfloat16, true>(p, num_sms, stream)
                          : launch_d<__nv_bfloat16, false>(p, num_sms, stream);
}

}  // namespace pa

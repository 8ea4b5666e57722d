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
// reduces over the row's lanes.  A row group takes four head rows of one
// token, all loads first, and reads the token's cos and sin once.
#include <cuda_runtime.h>

#include "pa_device.cuh"
#include "pa_kernels.h"

namespace pa {
namespace {

constexpr int kThreads = 256;
constexpr int kHeads = 4;  // head rows of one token per row group

template <typename T>
__device__ __forceinline__ void load4(const T* p, float (&x)[4]) {
  if constexpr (sizeof(T) == 4) {
    const float4 v = *reinterpret_cast<const float4*>(p);
    x[0] = v.x;
    x[1] = v.y;
    x[2] = v.z;
    x[3] = v.w;
  } else {
    const uint2 v = *reinterpret_cast<const uint2*>(p);
    x[0] = dev::bf16_bits_to_f32(v.x & 0xFFFFu);
    x[1] = dev::bf16_bits_to_f32(v.x >> 16);
    x[2] = dev::bf16_bits_to_f32(v.y & 0xFFFFu);
    x[3] = dev::bf16_bits_to_f32(v.y >> 16);
  }
}
template <typename T>
__device__ __forceinline__ void store4(T* p, const float (&x)[4]) {
  if constexpr (sizeof(T) == 4) {
    *reinterpret_cast<float4*>(p) = make_float4(x[0], x[1], x[2], x[3]);
  } else {
    *reinterpret_cast<uint2*>(p) = make_uint2(dev::pack_bf16(x[0], x[1]), dev::pack_bf16(x[2], x[3]));
  }
}
__device__ __forceinline__ uint32_t quant4(const float (&x)[4], float scale) {
  const uint32_t lo = dev::e4m3x2_from_f32(__fdiv_rn(x[0], scale), __fdiv_rn(x[1], scale));
  const uint32_t hi = dev::e4m3x2_from_f32(__fdiv_rn(x[2], scale), __fdiv_rn(x[3], scale));
  return lo | (hi << 16);
}

// T: element type of the new rows; FP8: an e4m3 pool.
template <typename T, int D, bool FP8>
__global__ void __launch_bounds__(kThreads) norm_rope_write_kernel(const NormRopeParams p) {
  dev::grid_dep_wait();
  dev::grid_dep_launch();
  constexpr int LANES = D / 8;  // lanes of a head row
  const int hq = p.num_q_heads, hkv = p.num_kv_heads, nh = hq + 2 * hkv;
  const int per_token = (nh + kHeads - 1) / kHeads;
  const int64_t items = (int64_t)p.num_tokens * per_token;
  const int c = threadIdx.x % LANES;
  const int rot = p.rot_dim, half = rot >> 1;
  const bool turns = 8 * c < rot;  // this lane's elements are rotated
  // the lane's two chunks of four elements
  int a0 = 8 * c, a1 = 8 * c + 4;
  if (turns && !p.interleaved) {
    a0 = 4 * c;
    a1 = half + 4 * c;
  }
  float qw[2][4], kw[2][4];
#pragma unroll
  for (int i = 0; i < 4; ++i) qw[0][i] = qw[1][i] = kw[0][i] = kw[1][i] = 1.f;
  if (p.q_weight) {
    load4(reinterpret_cast<const T*>(p.q_weight) + a0, qw[0]);
    load4(reinterpret_cast<const T*>(p.q_weight) + a1, qw[1]);
  }
  if (p.k_weight) {
    load4(reinterpret_cast<const T*>(p.k_weight) + a0, kw[0]);
    load4(reinterpret_cast<const T*>(p.k_weight) + a1, kw[1]);
  }
  const int64_t step = (int64_t)gridDim.x * (kThreads / LANES);
  // whole warps iterate together (the norm's shuffles); a row group past the
  // end works on nothing
  const int64_t first = (int64_t)blockIdx.x * (kThreads / LANES) + threadIdx.x / LANES;
  const int64_t warp_first = first - (threadIdx.x & 31) / LANES;
  for (int64_t base = warp_first; base < items; base += step) {
    const int64_t item = base + (threadIdx.x & 31) / LANES;
    const bool live = item < items;
    const int64_t t = live ? item / per_token : 0;
    const int h0 = live ? (int)(item % per_token) * kHeads : nh;
    const int pos = p.cos_sin ? __ldg(p.positions + t) : 0;
    const int64_t slot = __ldg(p.slots + t);
    const bool known = p.cos_sin == nullptr || (pos >= 0 && pos < p.num_positions);
    const bool in_pool = slot >= 0 && slot < p.num_slots;
    const int64_t blk = in_pool ? slot / p.block_size : 0;
    const int off = in_pool ? (int)(slot % p.block_size) : 0;
    float x[kHeads][2][4];
#pragma unroll
    for (int j = 0; j < kHeads; ++j) {
      const int h = h0 + j;
#pragma unroll
      for (int i = 0; i < 4; ++i) x[j][0][i] = x[j][1][i] = 0.f;
      if (h < nh) {
        const T* row = h < hq ? reinterpret_cast<const T*>(p.q) + t * p.q_stride + (int64_t)h * D
                     : h < hq + hkv ? reinterpret_cast<const T*>(p.k) + t * p.k_stride + (int64_t)(h - hq) * D
                                    : reinterpret_cast<const T*>(p.v) + t * p.v_stride + (int64_t)(h - hq - hkv) * D;
        load4(row + a0, x[j][0]);
        load4(row + a1, x[j][1]);
      }
    }
    // cos and sin of the lane's four pairs
    float cs[4], sn[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      cs[i] = 1.f;
      sn[i] = 0.f;
    }
    if (turns && known && p.cos_sin) {
      const float4 cv = __ldg(reinterpret_cast<const float4*>(p.cos_sin + (int64_t)pos * rot + 4 * c));
      const float4 sv = __ldg(reinterpret_cast<const float4*>(p.cos_sin + (int64_t)pos * rot + half + 4 * c));
      cs[0] = cv.x, cs[1] = cv.y, cs[2] = cv.z, cs[3] = cv.w;
      sn[0] = sv.x, sn[1] = sv.y, sn[2] = sv.z, sn[3] = sv.w;
    }
#pragma unroll
    for (int j = 0; j < kHeads; ++j) {
      const int h = h0 + j;
      float ss = 0.f;
#pragma unroll
      for (int i = 0; i < 4; ++i) ss += x[j][0][i] * x[j][0][i] + x[j][1][i] * x[j][1][i];
#pragma unroll
      for (int o = LANES / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
      if (h >= nh || !known) continue;
      const bool is_q = h < hq, is_v = h >= hq + hkv;
      if (!is_q && !in_pool) continue;
      if (!is_v) {
        const bool norm = is_q ? p.q_weight != nullptr : p.k_weight != nullptr;
        const float inv = norm ? rsqrtf(ss * (1.f / D) + p.eps) : 1.f;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          x[j][0][i] *= inv * (is_q ? qw[0][i] : kw[0][i]);
          x[j][1][i] *= inv * (is_q ? qw[1][i] : kw[1][i]);
        }
        if (turns) {
          if (!p.interleaved) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const float a = x[j][0][i], b = x[j][1][i];
              x[j][0][i] = a * cs[i] - b * sn[i];
              x[j][1][i] = b * cs[i] + a * sn[i];
            }
          } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              float(&ch)[4] = x[j][i >> 1];
              const float a = ch[2 * (i & 1)], b = ch[2 * (i & 1) + 1];
              ch[2 * (i & 1)] = a * cs[i] - b * sn[i];
              ch[2 * (i & 1) + 1] = b * cs[i] + a * sn[i];
            }
          }
        }
      }
      if (is_q) {
        T* dst = reinterpret_cast<T*>(p.q_out) + (t * hq + h) * D;
        store4(dst + a0, x[j][0]);
        store4(dst + a1, x[j][1]);
        continue;
      }
      const int kvh = is_v ? h - hq - hkv : h - hq;
      uint8_t* pool = is_v ? p.v_cache : p.k_cache;
      if constexpr (!FP8) {
        T* dst = reinterpret_cast<T*>(pool) + ((blk * hkv + kvh) * p.block_size + off) * D;
        store4(dst + a0, x[j][0]);
        store4(dst + a1, x[j][1]);
      } else {
        const float* head = is_v ? p.v_head : p.k_head;
        const float scale = head ? __ldg(head + kvh) : (is_v ? p.v_scale : p.k_scale);
        const uint32_t w0 = quant4(x[j][0], scale), w1 = quant4(x[j][1], scale);
        if (!is_v) {
          uint8_t* dst = pool + ((blk * hkv + kvh) * p.block_size + off) * D;
          *reinterpret_cast<uint32_t*>(dst + a0) = w0;
          *reinterpret_cast<uint32_t*>(dst + a1) = w1;
        } else {  // d-major V: one byte per element
          uint8_t* dst = pool + (blk * hkv + kvh) * D * p.block_size + off;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            dst[(int64_t)(a0 + i) * p.block_size] = (uint8_t)(w0 >> (8 * i));
            dst[(int64_t)(a1 + i) * p.block_size] = (uint8_t)(w1 >> (8 * i));
          }
        }
      }
    }
  }
}

template <typename T, int D, bool FP8>
cudaError_t launch(const NormRopeParams& p, int num_sms, cudaStream_t stream) {
  const int per_token = (p.num_q_heads + 2 * p.num_kv_heads + kHeads - 1) / kHeads;
  const int groups = kThreads / (D / 8);
  const int64_t need = ((int64_t)p.num_tokens * per_token + groups - 1) / groups;
  const int64_t most = (int64_t)num_sms * 8;
  norm_rope_write_kernel<T, D, FP8><<<(unsigned)(need < most ? need : most), kThreads, 0, stream>>>(p);
  return cudaGetLastError();
}

template <typename T, bool FP8>
cudaError_t launch_d(const NormRopeParams& p, int num_sms, cudaStream_t stream) {
  if (p.head_dim == 64) return launch<T, 64, FP8>(p, num_sms, stream);
  if (p.head_dim == 128) return launch<T, 128, FP8>(p, num_sms, stream);
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

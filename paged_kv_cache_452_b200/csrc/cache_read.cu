// pa_cache_read: the pool's rows of given slots back as contiguous rows
// [tokens][kv heads][head_dim] in the query dtype, the inverse of
// pa_cache_write: bit copies of fp32 and bf16 rows, code * scale of e4m3 rows
// (exact in fp32 but for the product's rounding, rounded once more to bf16
// where that is the query dtype).
//
// Bound: HBM; every row is read and written once.  K, and V of fp32 and bf16
// pools, go by 16-byte vectors of the output, a few per thread in flight.
// e4m3 V, whose pool is d-major, goes by windows of 16 tokens: a lane loads 16
// tokens of four elements (four 16-byte vectors) and writes four elements of
// 16 rows, so that both sides move whole sectors.
#include <cuda_runtime.h>

#include "pa_device.cuh"
#include "pa_kernels.h"
#include "slot_window.cuh"

namespace pa {
namespace {

constexpr int kThreads = 256;

template <typename T>
__device__ __forceinline__ void store4(T* p, float a, float b, float c, float d) {
  if constexpr (sizeof(T) == 4) *reinterpret_cast<float4*>(p) = make_float4(a, b, c, d);
  else *reinterpret_cast<uint2*>(p) = make_uint2(dev::pack_bf16(a, b), dev::pack_bf16(c, d));
}

// Both halves of an f16 pair as fp32.
__device__ __forceinline__ float2 f16x2_to_f32(uint32_t w) {
  return __half22float2(*reinterpret_cast<const __half2*>(&w));
}

// e4m3 V of one window of tokens and one kv head per D / 4 lanes.
template <typename T, int D>
__device__ __forceinline__ void read_v_window(const CacheReadParams& p, int64_t item) {
  constexpr int LANES = D / 4;
  const int hkv = p.num_kv_heads;
  const int64_t heads = (hkv * LANES + 31) / 32 * (32 / LANES);  // heads per window, in whole warps
  const int64_t win = item / heads;
  const int h = (int)(item % heads);
  const int d0 = 4 * (threadIdx.x % LANES);
  const bool live = h < hkv;
  const float scale = !live ? 1.f : p.v_head ? __ldg(p.v_head + h) : p.v_scale;
  const int64_t end = dev::window_start(p.slots, p.num_tokens, win + 1);
  for (int64_t t = dev::window_start(p.slots, p.num_tokens, win); t < end; t += dev::kWindow) {
    const int n = (int)min((int64_t)dev::kWindow, end - t);
    int64_t s0;
    const bool whole = dev::window_aligned(p.slots, t, n, p.num_slots, &s0);
    if (!live) continue;
    T* dst = reinterpret_cast<T*>(p.v_out) + (t * hkv + h) * D + d0;
    if (whole) {
      const uint8_t* src = p.v_cache + (((s0 >> p.bs_shift) * hkv + h) * D + d0) * p.block_size + (s0 & (p.block_size - 1));
      uint4 raw[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) raw[e] = *reinterpret_cast<const uint4*>(src + (int64_t)e * p.block_size);
#pragma unroll
      for (int q = 0; q < 4; ++q) {  // four tokens
        float x[4][4];               // [element][token]
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const uint32_t w = q == 0 ? raw[e].x : q == 1 ? raw[e].y : q == 2 ? raw[e].z : raw[e].w;
          uint32_t lo, hi;
          dev::e4m3x4_to_f16x2(w, lo, hi);
          const float2 a = f16x2_to_f32(lo), b = f16x2_to_f32(hi);
          x[e][0] = a.x * scale;
          x[e][1] = a.y * scale;
          x[e][2] = b.x * scale;
          x[e][3] = b.y * scale;
        }
#pragma unroll
        for (int j = 0; j < 4; ++j)
          store4(dst + (int64_t)(4 * q + j) * hkv * D, x[0][j], x[1][j], x[2][j], x[3][j]);
      }
    } else {
      for (int j = 0; j < n; ++j) {
        const int64_t slot = __ldg(p.slots + t + j);
        if (slot < 0 || slot >= p.num_slots) continue;
        const uint8_t* src =
            p.v_cache + (((slot >> p.bs_shift) * hkv + h) * D + d0) * p.block_size + (slot & (p.block_size - 1));
        float x[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) x[e] = dev::e4m3_to_f32(src[(int64_t)e * p.block_size]) * scale;
        store4(dst + (int64_t)j * hkv * D, x[0], x[1], x[2], x[3]);
      }
    }
  }
}

// T: element type of the rows; FP8: an e4m3 pool; VECS: 16-byte vectors of the
// output per thread.  The first `v_blocks` blocks read e4m3 V.
template <typename T, int D, bool FP8, int VECS>
__global__ void __launch_bounds__(kThreads) cache_read_kernel(const CacheReadParams p, unsigned v_blocks) {
  dev::grid_dep_wait();
  dev::grid_dep_launch();
  const int hkv = p.num_kv_heads;
  if constexpr (FP8) {
    if (blockIdx.x < v_blocks) {
      const int64_t heads = (hkv * (D / 4) + 31) / 32 * (32 / (D / 4));
      const int64_t items = ((int64_t)p.num_tokens + dev::kWindow - 1) / dev::kWindow * heads;
      const int64_t item = (int64_t)blockIdx.x * (kThreads / (D / 4)) + threadIdx.x / (D / 4);
      if (item < items) read_v_window<T, D>(p, item);  // whole warps: items are a multiple of a warp's
      return;
    }
  }
  constexpr int VEC = 16 / sizeof(T), CH = D / VEC;  // elements of a vector, vectors of a row
  const int64_t per_side = (int64_t)p.num_tokens * hkv * CH, total = (FP8 ? 1 : 2) * per_side;
  const int64_t i0 = (int64_t)(blockIdx.x - (FP8 ? v_blocks : 0u)) * (kThreads * VECS) + threadIdx.x;
  int64_t row[VECS];  // element of the pool, -1: none
  int head[VECS];
#pragma unroll
  for (int j = 0; j < VECS; ++j) {
    const int64_t idx = i0 + j * kThreads;
    const int64_t r = idx >= per_side ? idx - per_side : idx;
    row[j] = -1;
    if (idx < total) {
      const uint32_t th = (uint32_t)(r / CH), t = dev::fdiv(th, p.heads);
      const int64_t slot = __ldg(p.slots + t);
      head[j] = (int)(th - t * hkv);
      if (slot >= 0 && slot < p.num_slots)
        row[j] = (((slot >> p.bs_shift) * hkv + head[j]) * p.block_size + (slot & (p.block_size - 1))) * D + r % CH * VEC;
    }
  }
  if constexpr (!FP8) {
    uint4 raw[VECS];
#pragma unroll
    for (int j = 0; j < VECS; ++j) {
      const uint8_t* pool = i0 + j * kThreads >= per_side ? p.v_cache : p.k_cache;
      if (row[j] >= 0) raw[j] = *reinterpret_cast<const uint4*>(reinterpret_cast<const T*>(pool) + row[j]);
    }
#pragma unroll
    for (int j = 0; j < VECS; ++j) {
      const int64_t idx = i0 + j * kThreads;
      const bool side = idx >= per_side;
      if (row[j] >= 0)
        reinterpret_cast<uint4*>(side ? p.v_out : p.k_out)[side ? idx - per_side : idx] = raw[j];
    }
  } else {
    uint2 raw[VECS];
#pragma unroll
    for (int j = 0; j < VECS; ++j) {
      if (row[j] >= 0) {
        if constexpr (VEC == 8) raw[j] = *reinterpret_cast<const uint2*>(p.k_cache + row[j]);
        else raw[j] = make_uint2(*reinterpret_cast<const uint32_t*>(p.k_cache + row[j]), 0u);
      }
    }
#pragma unroll
    for (int j = 0; j < VECS; ++j) {
      if (row[j] < 0) continue;
      const float scale = p.k_head ? __ldg(p.k_head + head[j]) : p.k_scale;
      T* dst = reinterpret_cast<T*>(p.k_out) + (i0 + j * kThreads) * VEC;
#pragma unroll
      for (int q = 0; q < VEC / 4; ++q) {
        uint32_t lo, hi;
        dev::e4m3x4_to_f16x2(q ? raw[j].y : raw[j].x, lo, hi);
        const float2 a = f16x2_to_f32(lo), b = f16x2_to_f32(hi);
        if constexpr (VEC == 4) {
          store4(dst, a.x * scale, a.y * scale, b.x * scale, b.y * scale);
        } else {
          store4(dst + 4 * q, a.x * scale, a.y * scale, b.x * scale, b.y * scale);
        }
      }
    }
  }
}

template <typename T, int D, bool FP8, int VECS>
cudaError_t launch(const CacheReadParams& p, cudaStream_t stream) {
  const int64_t total = (FP8 ? 1LL : 2LL) * p.num_tokens * p.num_kv_heads * (D * (int)sizeof(T) / 16);
  const int64_t rows = (total + kThreads * VECS - 1) / (kThreads * VECS);
  int64_t vwin = 0;
  if (FP8) {
    const int64_t heads = (p.num_kv_heads * (D / 4) + 31) / 32 * (32 / (D / 4));
    const int64_t v = ((int64_t)p.num_tokens + dev::kWindow - 1) / dev::kWindow * heads;
    vwin = (v + kThreads / (D / 4) - 1) / (kThreads / (D / 4));
  }
  if (rows + vwin > INT32_MAX) return cudaErrorNotSupported;
  CacheReadParams q = p;
  q.heads = fast_div((uint32_t)p.num_kv_heads);
  cache_read_kernel<T, D, FP8, VECS><<<(unsigned)(rows + vwin), kThreads, 0, stream>>>(q, (unsigned)vwin);
  return cudaGetLastError();
}

// Vectors per thread: one while the call then fits the GPU at once, else four
// in flight.
template <typename T, bool FP8>
cudaError_t launch_d(const CacheReadParams& p, int num_sms, cudaStream_t stream) {
  const bool few =
      2LL * p.num_tokens * p.num_kv_heads * (p.head_dim * (int)sizeof(T) / 16) <= (int64_t)num_sms * 2048;
  if (p.head_dim == 64) return few ? launch<T, 64, FP8, 1>(p, stream) : launch<T, 64, FP8, 4>(p, stream);
  if (p.head_dim == 128) return few ? launch<T, 128, FP8, 1>(p, stream) : launch<T, 128, FP8, 4>(p, stream);
  return cudaErrorNotSupported;
}

}  // namespace

cudaError_t launch_cache_read(const CacheReadParams& p, int q_dtype, int kv_dtype, int num_sms, cudaStream_t stream) {
  if (q_dtype == kF32)
    return kv_dtype == kFP8 ? launch_d<float, true>(p, num_sms, stream) : launch_d<float, false>(p, num_sms, stream);
  return kv_dtype == kFP8 ? launch_d<__nv_bfloat16, true>(p, num_sms, stream)
                          : launch_d<__nv_bfloat16, false>(p, num_sms, stream);
}

}  // namespace pa

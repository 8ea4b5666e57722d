// pa_cache_read: the pool's rows of given slots back as contiguous rows
// [tokens][kv heads][head_dim] in the query dtype, the inverse of
// pa_cache_write: bit copies of fp32 and bf16 rows, code * scale of e4m3 rows
// (exact in fp32, rounded once to bf16 where that is the query dtype).
//
// Bound: HBM; every row is read and written once.
#include <cuda_runtime.h>

#include "pa_device.cuh"
#include "pa_kernels.h"

namespace pa {
namespace {

constexpr int kThreads = 256;

// T: element type of the rows; FP8: an e4m3 pool.  A thread moves one
// 16-byte vector of an output row.
template <typename T, bool FP8>
__global__ void __launch_bounds__(kThreads) cache_read_kernel(const CacheReadParams p) {
  dev::grid_dep_wait();
  dev::grid_dep_launch();
  constexpr int VEC = 16 / sizeof(T);
  const int chunks = p.head_dim / VEC;
  const int64_t per_side = (int64_t)p.num_tokens * p.num_kv_heads * chunks;
  for (int64_t idx = (int64_t)blockIdx.x * kThreads + threadIdx.x; idx < 2 * per_side;
       idx += (int64_t)gridDim.x * kThreads) {
    const int side = idx >= per_side;  // 0: K, 1: V
    int64_t r = side ? idx - per_side : idx;
    const int64_t at = r * VEC;  // element of the output
    const int c = (int)(r % chunks);
    r /= chunks;
    const int h = (int)(r % p.num_kv_heads);
    const int64_t slot = __ldg(p.slots + r / p.num_kv_heads);
    if (slot < 0 || slot >= p.num_slots) continue;
    const int64_t blk = slot / p.block_size;
    const int off = (int)(slot % p.block_size);
    const uint8_t* pool = side ? p.v_cache : p.k_cache;
    T* dst = reinterpret_cast<T*>(side ? p.v_out : p.k_out) + at;
    const int64_t row = ((blk * p.num_kv_heads + h) * p.block_size + off) * p.head_dim + c * VEC;
    if constexpr (!FP8) {
      *reinterpret_cast<uint4*>(dst) = *reinterpret_cast<const uint4*>(reinterpret_cast<const T*>(pool) + row);
    } else {
      const float* head = side ? p.v_head : p.k_head;
      const float scale = head ? __ldg(head + h) : (side ? p.v_scale : p.k_scale);
      float x[VEC];
#pragma unroll
      for (int i = 0; i < VEC; ++i) {
        const int64_t e = side ? ((blk * p.num_kv_heads + h) * p.head_dim + c * VEC + i) * p.block_size + off : row + i;
        x[i] = dev::e4m3_to_f32(pool[e]) * scale;
      }
      if constexpr (sizeof(T) == 4) {
        *reinterpret_cast<float4*>(dst) = make_float4(x[0], x[1], x[2], x[3]);
      } else {
        *reinterpret_cast<uint4*>(dst) = make_uint4(dev::pack_bf16(x[0], x[1]), dev::pack_bf16(x[2], x[3]),
                                                    dev::pack_bf16(x[4], x[5]), dev::pack_bf16(x[6], x[7]));
      }
    }
  }
}

template <typename T, bool FP8>
cudaError_t launch(const CacheReadParams& p, int num_sms, cudaStream_t stream) {
  const int64_t total = 2LL * p.num_tokens * p.num_kv_heads * (p.head_dim * (int)sizeof(T) / 16);
  int64_t blocks = (total + kThreads - 1) / kThreads;
  if (blocks > (int64_t)num_sms * 64) blocks = (int64_t)num_sms * 64;
  cache_read_kernel<T, FP8><<<(unsigned)blocks, kThreads, 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_cache_read(const CacheReadParams& p, int q_dtype, int kv_dtype, int num_sms, cudaStream_t stream) {
  if (q_dtype == kF32)
    return kv_dtype == kFP8 ? launch<float, true>(p, num_sms, stream) : launch<float, false>(p, num_sms, stream);
  return kv_dtype == kFP8 ? launch<__nv_bfloat16, true>(p, num_sms, stream)
                          : launch<__nv_bfloat16, false>(p, num_sms, stream);
}

}  // namespace pa

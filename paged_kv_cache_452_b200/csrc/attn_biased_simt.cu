// Biased paged attention on CUDA cores: fp32 queries, whose 1e-4 rules out
// tensor-core inputs of fewer bits, over an fp32 or e4m3 pool; decode rows and
// chunks of new tokens alike.
//
// Row i of a sequence sees key j if j < prefix, or j <= i and (window) i - j <
// window; its score is cap * tanh(scale q k / cap) - slope |i - j|, all in
// fp32.  A CTA takes NP (position, head) pairs of one sequence and kv head, so
// that a key row read serves several queries; its warps take the visible
// 16-key tiles in turn, each with its own online softmax, and merge at the
// end.  With one pair per CTA (few rows: a chain of loads per tile is what
// bounds it) there are 16 warps and a tile's K and V are loaded together.
// Bound: latency for short contexts, FMA issue for long.
#include <cuda_runtime.h>

#include "pa_device.cuh"
#include "pa_kernels.h"

namespace pa {
namespace {

constexpr int kTile = 16;  // keys of a tile: block sizes are multiples of it
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kHalfLn2 = 0.34657359027997264f;  // cap_in holds 2 log2(e) times what tanh takes

template <typename T, int E>
__device__ __forceinline__ void load_elems(const uint8_t* base, int64_t idx, float (&x)[E]) {
  if constexpr (sizeof(T) == 4) {
    const float4* p = reinterpret_cast<const float4*>(reinterpret_cast<const float*>(base) + idx);
#pragma unroll
    for (int i = 0; i < E / 4; ++i) {
      const float4 v = __ldg(p + i);
      x[4 * i] = v.x, x[4 * i + 1] = v.y, x[4 * i + 2] = v.z, x[4 * i + 3] = v.w;
    }
  } else {
    const uint2* p = reinterpret_cast<const uint2*>(base + idx);
#pragma unroll
    for (int i = 0; i < E / 8; ++i) {
      const uint2 v = __ldg(p + i);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        x[8 * i + k] = dev::e4m3_to_f32((v.x >> (8 * k)) & 0xFFu);
        x[8 * i + 4 + k] = dev::e4m3_to_f32((v.y >> (8 * k)) & 0xFFu);
      }
    }
  }
}

template <int KV> struct KElem { using T = float; };
template <> struct KElem<kFP8> { using T = uint8_t; };

// (fp32 rows of 128 elements ahead need the registers of eight warps)
template <int KV, int D, int NP>
constexpr int warps_of() { return NP == 1 && (D == 64 || KV == kFP8) ? 16 : 8; }

template <int KV, int D, int NP>
__global__ void __launch_bounds__(warps_of<KV, D, NP>() * 32) attn_biased_simt_kernel(const BiasedSimtParams bp) {
  dev::grid_dep_wait();
  const SimtParams& p = bp.a;
  constexpr int kWarps = warps_of<KV, D, NP>();
  constexpr int E = D / 8;    // elements of a key row per lane (8 lanes a key, 4 keys a pass)
  constexpr int DV = D / 32;  // elements of the output per lane
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int hq = p.num_q_heads, hkv = p.num_kv_heads, G = hq / hkv, bs = p.block_size;
  const int kvh = blockIdx.y;
  // the CTA's pairs: block x of the batch, sequence s's blocks from
  // floor(first row * G / NP) + s on (at least as many as it needs)
  auto row0 = [&](int s) { return p.rows.qsl ? p.rows.qsl[s] : s; };
  auto base = [&](int s) { return (int64_t)row0(s) * G / NP + s; };
  int lo = 0, hi = p.rows.num_seqs - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (base(mid) <= (int64_t)blockIdx.x) lo = mid; else hi = mid - 1;
  }
  const int s = lo, first = row0(s), qlen = row0(s + 1) - first;
  const int64_t pair0 = ((int64_t)blockIdx.x - base(s)) * NP;
  const int64_t pairs = (int64_t)qlen * G;
  if (pair0 >= pairs) return;
  const int np = (int)min((int64_t)NP, pairs - pair0);
  int len = p.rows.seq_lens[s];
  if ((int64_t)len > (int64_t)p.max_blocks * bs) {  // longer than its table row: flag, clamp
    if (threadIdx.x == 0) atomicCAS(p.err, 0, 3);
    len = p.max_blocks * bs;
  }
  const int at0 = p.rows.seq_lens[s] - qlen;  // position of the sequence's first query row
  const int W = bp.mod.window;
  const int pfx = bp.mod.prefix ? max(0, min(len, bp.mod.prefix[s])) : 0;
  const float ks = p.k_head ? __ldg(p.k_head + kvh) : p.k_scale, vs = p.v_head ? __ldg(p.v_head + kvh) : p.v_scale;
  const float kmul = KV == kFP8 ? ks : 1.f;

  float q[NP][E], acc[NP][DV], m[NP], l[NP], slope[NP];
  int pos[NP];
  const int sub = lane & 7, kg = lane >> 3;
#pragma unroll
  for (int n = 0; n < NP; ++n) {
    const int64_t pr = pair0 + (n < np ? n : 0);
    const int row = (int)(pr / G), h = kvh * G + (int)(pr % G);
    pos[n] = at0 + row;
    slope[n] = bp.mod.slopes ? __ldg(bp.mod.slopes + h) * kLog2e : 0.f;
    load_elems<float, E>(p.q, ((int64_t)(first + row) * hq + h) * D + sub * E, q[n]);
    m[n] = -1e30f;
    l[n] = 0.f;
#pragma unroll
    for (int e = 0; e < DV; ++e) acc[n][e] = 0.f;
  }
  // tiles with a key that some pair sees: [0, tp) of the prefix and [tl, te)
  const int plo = at0 + (int)(pair0 / G), phi = at0 + (int)((pair0 + np - 1) / G);
  const int end = min(len, max(phi + 1, pfx));
  const int wlo = W > 0 ? max(0, plo - W + 1) : 0;
  const int tp = (pfx + kTile - 1) / kTile, tl = max(tp, wlo / kTile), te = (end + kTile - 1) / kTile;
  const int ntiles = tp + max(0, te - tl);
  const int32_t* table = p.block_tables + (int64_t)s * p.max_blocks;
  for (int i = warp; i < ntiles; i += kWarps) {
    const int tile = i < tp ? i : i - tp + tl;
    const int key0 = tile * kTile;
    int64_t blk = __ldg(table + key0 / bs);
    if (blk < 0 || blk >= p.num_blocks) {  // bad table entry: flag it, read block 0
      if (lane == 0) atomicCAS(p.err, 0, 2);
      blk = 0;
    }
    const int off = key0 % bs;
    const int64_t kb = ((blk * hkv + kvh) * bs + off) * D;
    // key 4 j + kg of the tile, and this lane's V elements (with several pairs
    // loaded where they are used: registers)
    constexpr bool kAhead = NP == 1;
    float kall[kAhead ? 4 : 1][E];
    float2 vall[kAhead && KV != kFP8 ? kTile : 1][DV / 2];
    uint4 raw[KV == kFP8 ? DV : 1];
    if constexpr (kAhead) {
#pragma unroll
      for (int j = 0; j < 4; ++j)
        load_elems<typename KElem<KV>::T, E>(p.k_cache, kb + (4 * j + kg) * D + sub * E, kall[j]);
      if constexpr (KV != kFP8) {
#pragma unroll
        for (int k = 0; k < kTile; ++k)
#pragma unroll
          for (int e = 0; e < DV / 2; ++e)
            vall[k][e] = __ldg(reinterpret_cast<const float2*>(p.v_cache) + (kb + k * D + lane * DV) / 2 + e);
      }
    }
    if constexpr (KV == kFP8) {
#pragma unroll
      for (int e = 0; e < DV; ++e)
        raw[e] = __ldg(reinterpret_cast<const uint4*>(p.v_cache + ((blk * hkv + kvh) * D + lane * DV + e) * bs + off));
    }
    float sc[NP][4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      float kx[E];
      if constexpr (kAhead) {
#pragma unroll
        for (int e = 0; e < E; ++e) kx[e] = kall[j][e];
      } else {
        load_elems<typename KElem<KV>::T, E>(p.k_cache, kb + (4 * j + kg) * D + sub * E, kx);
      }
      const int key = key0 + 4 * j + kg;
#pragma unroll
      for (int n = 0; n < NP; ++n) {
        float dot = 0.f;
#pragma unroll
        for (int e = 0; e < E; ++e) dot = fmaf(q[n][e], kx[e], dot);
#pragma unroll
        for (int o = 4; o > 0; o >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, o);
        const bool seen = key < len && (key < pfx || (key <= pos[n] && (W <= 0 || pos[n] - key < W)));
        // (tanhf: fp32 rows are held to fp32's rounding, and latency bounds)
        const float x = bp.mod.cap_out > 0.f ? bp.mod.cap_out * tanhf(dot * (bp.mod.cap_in * kmul * kHalfLn2))
                                             : dot * (p.scale * kLog2e * kmul);
        sc[n][j] = seen ? fmaf(-slope[n], fabsf((float)(pos[n] - key)), x) : -INFINITY;
      }
    }
    float pr[NP][4];
#pragma unroll
    for (int n = 0; n < NP; ++n) {
      float mx = fmaxf(fmaxf(sc[n][0], sc[n][1]), fmaxf(sc[n][2], sc[n][3]));
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
      const float mn = fmaxf(m[n], mx), al = dev::ex2(m[n] - mn);
      m[n] = mn;
      l[n] *= al;
#pragma unroll
      for (int e = 0; e < DV; ++e) acc[n][e] *= al;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        pr[n][j] = dev::ex2(sc[n][j] - mn);
        l[n] += pr[n][j];  // per key group: the groups are added at the end
      }
    }
    // O += P V, key by key; a key that no pair sees is skipped (its V may be
    // anything: 0 * NaN)
    if constexpr (KV != kFP8) {
#pragma unroll
      for (int k = 0; k < kTile; ++k) {
        const int key = key0 + k;
        const bool any = key < len && (key < pfx || (key <= phi && key >= wlo));
        if (!any) continue;
        float vx[DV];
        const int64_t vb = kb + (int64_t)k * D + lane * DV;
#pragma unroll
        for (int e = 0; e < DV; e += 2) {
          float2 v;
          if constexpr (kAhead) v = vall[k][e / 2];
          else v = __ldg(reinterpret_cast<const float2*>(reinterpret_cast<const float*>(p.v_cache) + vb + e));
          vx[e] = v.x;
          vx[e + 1] = v.y;
        }
#pragma unroll
        for (int n = 0; n < NP; ++n) {
          const float w = __shfl_sync(0xffffffffu, pr[n][k >> 2], (k & 3) * 8);
#pragma unroll
          for (int e = 0; e < DV; ++e) acc[n][e] = fmaf(w, vx[e], acc[n][e]);
        }
      }
    } else {  // d-major: 16 keys of an element are contiguous
#pragma unroll
      for (int k = 0; k < kTile; ++k) {
        const int key = key0 + k;
        const bool any = key < len && (key < pfx || (key <= phi && key >= wlo));
        if (!any) continue;
        float w[NP];
#pragma unroll
        for (int n = 0; n < NP; ++n) w[n] = __shfl_sync(0xffffffffu, pr[n][k >> 2], (k & 3) * 8);
#pragma unroll
        for (int e = 0; e < DV; ++e) {
          const uint32_t r[4] = {raw[e].x, raw[e].y, raw[e].z, raw[e].w};
          const float v = dev::e4m3_to_f32((r[k >> 2] >> (8 * (k & 3))) & 0xFFu);
#pragma unroll
          for (int n = 0; n < NP; ++n) acc[n][e] = fmaf(w[n], v, acc[n][e]);
        }
      }
    }
  }
  // ---- merge the warps ----
  __shared__ float sm[kWarps][NP], sl[kWarps][NP], sa[kWarps][NP][D];
#pragma unroll
  for (int n = 0; n < NP; ++n) {
    float t = l[n];  // lanes of a key group hold the same sum
    t += __shfl_xor_sync(0xffffffffu, t, 8);
    t += __shfl_xor_sync(0xffffffffu, t, 16);
    if (lane == 0) {
      sm[warp][n] = m[n];
      sl[warp][n] = t;
    }
#pragma unroll
    for (int e = 0; e < DV; ++e) sa[warp][n][lane * DV + e] = acc[n][e];
  }
  __syncthreads();
  for (int i = threadIdx.x; i < np * D; i += kWarps * 32) {
    const int n = i / D, d = i % D;
    float M = sm[0][n];
#pragma unroll
    for (int w = 1; w < kWarps; ++w) M = fmaxf(M, sm[w][n]);
    float L = 0.f, o = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const float a = dev::ex2(sm[w][n] - M);
      L = fmaf(sl[w][n], a, L);
      o = fmaf(sa[w][n][d], a, o);
    }
    const int64_t pr = pair0 + n;
    const int64_t at = ((int64_t)(first + pr / G) * hq + kvh * G + pr % G) * D + d;
    const float x = L > 0.f ? o / L * (KV == kFP8 ? vs : 1.f) : 0.f;  // an empty context: a zero row
    reinterpret_cast<float*>(p.out)[at] = x;
  }
}

template <int KV, int D, int NP>
cudaError_t launch(const BiasedSimtParams& p, cudaStream_t stream) {
  const int G = p.a.num_q_heads / p.a.num_kv_heads;
  const int64_t blocks = (int64_t)p.a.rows.num_rows * G / NP + p.a.rows.num_seqs;
  if (blocks > INT32_MAX || p.a.num_kv_heads > 65535) return cudaErrorNotSupported;
  attn_biased_simt_kernel<KV, D, NP><<<dim3((unsigned)blocks, (unsigned)p.a.num_kv_heads),
                                             warps_of<KV, D, NP>() * 32, 0, stream>>>(p);
  return cudaGetLastError();
}

// Pairs per CTA: one where there are few (a decode batch: short chains per
// warp count), else four.
template <int KV>
cudaError_t launch_d(const BiasedSimtParams& p, cudaStream_t stream) {
  const int64_t pairs = (int64_t)p.a.rows.num_rows * p.a.num_q_heads;
  const bool few = pairs <= 1024 || (p.a.num_q_heads == p.a.num_kv_heads && !p.a.rows.qsl);
  if (p.a.head_dim == 64) return few ? launch<KV, 64, 1>(p, stream) : launch<KV, 64, 4>(p, stream);
  if (p.a.head_dim == 128) return few ? launch<KV, 128, 1>(p, stream) : launch<KV, 128, 4>(p, stream);
  return cudaErrorNotSupported;
}

}  // namespace

cudaError_t launch_attn_biased_simt(const BiasedSimtParams& p, int kv_dtype, cudaStream_t stream) {
  if (kv_dtype == kF32) return launch_d<kF32>(p, stream);
  if (kv_dtype == kFP8) return launch_d<kFP8>(p, stream);
  return cudaErrorNotSupported;
}

}  // namespace pa

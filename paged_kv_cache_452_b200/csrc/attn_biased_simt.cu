// Biased paged attention on CUDA cores: fp32 queries, whose 1e-4 rules out
// tensor-core inputs of fewer bits, over an fp32 or e4m3 pool.
//
// Row i of a sequence sees key j if j < prefix, or j <= i and (window) i - j <
// window; its score is cap * tanh(scale q k / cap) - slope |i - j|, all in
// fp32.
//
// Row kernel: a CTA takes one (row, head); its warps take the visible 16-key
// tiles in turn, each with its own online softmax, and merge at the end.  A
// chain of loads per tile bounds it for short contexts, so there are up to 16
// warps and a tile's K and V are loaded together (4 sequences of up to 301
// keys: 9.4 us a call; 16.4 with eight warps and V loaded behind the softmax).
// Tile kernel, further down: chunks with rows enough to fill it.
#include <cuda_runtime.h>

#include "pa_device.cuh"
#include "pa_kernels.h"

namespace pa {
namespace {

constexpr int kTile = 16;  // keys of a tile: block sizes are multiples of it
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kHalfLn2 = 0.34657359027997264f;  // cap_in holds 2 log2(e) times what tanh takes

// E elements of a key row as fp32: fp32, or e4m3 codes (exact).
template <int KV, int E>
__device__ __forceinline__ void load_elems(const uint8_t* base, int64_t idx, float (&x)[E]) {
  if constexpr (KV == kF32) {
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

// (fp32 rows of 128 elements ahead need the registers of eight warps)
template <int KV, int D>
constexpr int row_warps() { return D == 64 || KV == kFP8 ? 16 : 8; }

template <int KV, int D>
__global__ void __launch_bounds__(row_warps<KV, D>() * 32)
    attn_biased_row_kernel(const BiasedSimtParams bp, bool chunks) {
  dev::grid_dep_wait();
  const SimtParams& p = bp.a;
  constexpr int kWarps = row_warps<KV, D>();
  constexpr int E = D / 8;    // elements of a key row per lane (8 lanes a key, 4 keys a pass)
  constexpr int DV = D / 32;  // elements of the output per lane
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int hq = p.num_q_heads, hkv = p.num_kv_heads, bs = p.block_size;
  const int row = blockIdx.x, h = blockIdx.y, kvh = h / (hq / hkv);
  int s = row, first = row, qlen = 1;
  if (p.rows.qsl) {  // the last s with qsl[s] <= row
    int lo = 0, hi = p.rows.num_seqs - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (p.rows.qsl[mid] <= row) lo = mid; else hi = mid - 1;
    }
    s = lo;
    first = p.rows.qsl[s];
    qlen = p.rows.qsl[s + 1] - first;
    if (row < first || row >= first + qlen || (qlen > 1 && !chunks)) return;
  }
  int len = p.rows.seq_lens[s];
  const int pos = len - qlen + row - first;
  if ((int64_t)len > (int64_t)p.max_blocks * bs) {  // longer than its table row: flag, clamp
    if (threadIdx.x == 0) atomicCAS(p.err, 0, 3);
    len = p.max_blocks * bs;
  }
  const int W = bp.mod.window;
  const int pfx = bp.mod.prefix ? max(0, min(len, bp.mod.prefix[s])) : 0;
  const float vs = KV != kFP8 ? 1.f : p.v_head ? __ldg(p.v_head + kvh) : p.v_scale;
  const float kmul = KV != kFP8 ? 1.f : p.k_head ? __ldg(p.k_head + kvh) : p.k_scale;
  const float slope = bp.mod.slopes ? __ldg(bp.mod.slopes + h) * kLog2e : 0.f;
  const int sub = lane & 7, kg = lane >> 3;
  float q[E], acc[DV], m = -1e30f, l = 0.f;
  load_elems<kF32, E>(p.q, ((int64_t)row * hq + h) * D + sub * E, q);
#pragma unroll
  for (int e = 0; e < DV; ++e) acc[e] = 0.f;
  // tiles with a visible key: [0, tp) of the prefix and [tl, te)
  const int end = min(len, max(pos + 1, pfx)), wlo = W > 0 ? max(0, pos - W + 1) : 0;
  const int tp = (pfx + kTile - 1) / kTile, tl = max(tp, wlo / kTile), te = (end + kTile - 1) / kTile;
  const int ntiles = tp + max(0, te - tl);
  auto seen = [&](int key) { return key < len && (key < pfx || (key <= pos && key >= wlo)); };
  const int32_t* table = p.block_tables + (int64_t)s * p.max_blocks;
  for (int i = warp; i < ntiles; i += kWarps) {
    const int key0 = (i < tp ? i : i - tp + tl) * kTile;
    int64_t blk = __ldg(table + key0 / bs);
    if (blk < 0 || blk >= p.num_blocks) {  // bad table entry: flag it, read block 0
      if (lane == 0) atomicCAS(p.err, 0, 2);
      blk = 0;
    }
    const int off = key0 % bs;
    const int64_t kb = ((blk * hkv + kvh) * bs + off) * D;
    float kx[4][E];  // keys 4 j + kg
    float2 vx[KV == kF32 ? kTile : 1][DV / 2];
    uint4 raw[KV == kFP8 ? DV : 1];  // d-major: 16 keys of an element are contiguous
#pragma unroll
    for (int j = 0; j < 4; ++j) load_elems<KV, E>(p.k_cache, kb + (4 * j + kg) * D + sub * E, kx[j]);
    if constexpr (KV == kF32) {
#pragma unroll
      for (int k = 0; k < kTile; ++k)
#pragma unroll
        for (int e = 0; e < DV / 2; ++e)
          vx[k][e] = __ldg(reinterpret_cast<const float2*>(p.v_cache) + (kb + k * D + lane * DV) / 2 + e);
    } else {
#pragma unroll
      for (int e = 0; e < DV; ++e)
        raw[e] = __ldg(reinterpret_cast<const uint4*>(p.v_cache + ((blk * hkv + kvh) * D + lane * DV + e) * bs + off));
    }
    float sc[4], w[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      float dot = 0.f;
#pragma unroll
      for (int e = 0; e < E; ++e) dot = fmaf(q[e], kx[j][e], dot);
#pragma unroll
      for (int o = 4; o > 0; o >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, o);
      const int key = key0 + 4 * j + kg;
      // (tanhf: fp32 rows are held to fp32's rounding, and latency bounds)
      const float x = bp.mod.cap_out > 0.f ? bp.mod.cap_out * tanhf(dot * (bp.mod.cap_in * kmul * kHalfLn2))
                                           : dot * (p.scale * kLog2e * kmul);
      sc[j] = seen(key) ? fmaf(-slope, fabsf((float)(pos - key)), x) : -INFINITY;
    }
    float mx = fmaxf(fmaxf(sc[0], sc[1]), fmaxf(sc[2], sc[3]));
    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
    const float mn = fmaxf(m, mx), al = dev::ex2(m - mn);
    m = mn;
    l *= al;
#pragma unroll
    for (int e = 0; e < DV; ++e) acc[e] *= al;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      w[j] = dev::ex2(sc[j] - mn);
      l += w[j];  // per key group: the groups are added at the end
    }
    // O += P V, key by key; a hidden key is skipped (its V may be anything: 0 * NaN)
#pragma unroll
    for (int k = 0; k < kTile; ++k) {
      if (!seen(key0 + k)) continue;
      const float wk = __shfl_sync(0xffffffffu, w[k >> 2], (k & 3) * 8);
#pragma unroll
      for (int e = 0; e < DV; ++e) {
        float v;
        if constexpr (KV == kF32) {
          v = e & 1 ? vx[k][e / 2].y : vx[k][e / 2].x;
        } else {
          const uint32_t r[4] = {raw[e].x, raw[e].y, raw[e].z, raw[e].w};
          v = dev::e4m3_to_f32((r[k >> 2] >> (8 * (k & 3))) & 0xFFu);
        }
        acc[e] = fmaf(wk, v, acc[e]);
      }
    }
  }
  // ---- merge the warps ----
  __shared__ float sm[kWarps], sl[kWarps], sa[kWarps][D];
  l += __shfl_xor_sync(0xffffffffu, l, 8);  // (the lanes of a key group hold the same sum)
  l += __shfl_xor_sync(0xffffffffu, l, 16);
  if (lane == 0) {
    sm[warp] = m;
    sl[warp] = l;
  }
#pragma unroll
  for (int e = 0; e < DV; ++e) sa[warp][lane * DV + e] = acc[e];
  __syncthreads();
  if (threadIdx.x < D) {
    float M = sm[0];
#pragma unroll
    for (int i = 1; i < kWarps; ++i) M = fmaxf(M, sm[i]);
    float L = 0.f, o = 0.f;
#pragma unroll
    for (int i = 0; i < kWarps; ++i) {
      const float a = dev::ex2(sm[i] - M);
      L = fmaf(sl[i], a, L);
      o = fmaf(sa[i][threadIdx.x], a, o);
    }
    // nothing visible: a zero row; NaN stays
    reinterpret_cast<float*>(p.out)[((int64_t)row * hq + h) * D + threadIdx.x] =
        L > 0.f ? o / L * vs : (L == 0.f ? 0.f : L);
  }
}

// ---- chunks ----------------------------------------------------------------
// The rows of sequences with more than one: 64 (position, head) pairs of one
// sequence and kv head against tiles of 64 keys, both products in registers:
// a thread has 4 x 4 scores and 4 x D / 16 outputs, so that eight (then ten)
// shared-memory vectors feed 64 (128) FMAs.  Bound: FMA issue and the shared
// memory's loads (256 rows of 32 heads over 4000 keys, twice: 1.85 ms, 18
// TFLOP/s; the row kernel with four pairs per CTA took 6.7 ms).
constexpr int kR = kBiasedTileRows;  // pairs of a CTA
constexpr int kKT = 64;  // keys of a tile
constexpr int kTileThreads = 256;
template <int D>
constexpr int tile_smem() { return (kR * (D + 4) + 2 * kKT * (D + 4) + kR * (kKT + 4)) * 4; }

template <int KV, int D>
__global__ void __launch_bounds__(kTileThreads, 2) attn_biased_tile_kernel(const BiasedSimtParams bp) {
  dev::grid_dep_wait();
  extern __shared__ float4 smem4[];
  constexpr int LD = D + 4, LP = kKT + 4, DC = D / 64;  // padded rows; 64-column groups of the outputs
  float* qs = reinterpret_cast<float*>(smem4);
  float* ks = qs + kR * LD;
  float* vs = ks + kKT * LD;
  float* ps = vs + kKT * LD;
  const SimtParams& p = bp.a;
  const int hq = p.num_q_heads, hkv = p.num_kv_heads, G = hq / hkv, bs = p.block_size, kvh = blockIdx.y;
  auto base = [&](int s) { return (int64_t)p.rows.qsl[s] * G / kR + s; };
  int lo = 0, hi = p.rows.num_seqs - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (base(mid) <= (int64_t)blockIdx.x) lo = mid; else hi = mid - 1;
  }
  const int s = lo, first = p.rows.qsl[s], qlen = p.rows.qsl[s + 1] - first;
  if (qlen <= 1 || first < 0) return;  // single rows are the other kernel's
  // (never past the rows that q and out have, whatever query_start_loc says)
  const int64_t pair0 = ((int64_t)blockIdx.x - base(s)) * kR, pairs = (int64_t)min(qlen, p.rows.num_rows - first) * G;
  if (pair0 >= pairs) return;
  const int np = (int)min((int64_t)kR, pairs - pair0);
  int len = p.rows.seq_lens[s];
  const int at0 = len - qlen;  // position of the sequence's first query row
  if ((int64_t)len > (int64_t)p.max_blocks * bs) {  // longer than its table row: flag, clamp
    if (threadIdx.x == 0) atomicCAS(p.err, 0, 3);
    len = p.max_blocks * bs;
  }
  const int W = bp.mod.window;
  const int pfx = bp.mod.prefix ? max(0, min(len, bp.mod.prefix[s])) : 0;
  const float kmul = KV != kFP8 ? 1.f : p.k_head ? __ldg(p.k_head + kvh) : p.k_scale;
  const float vmul = KV != kFP8 ? 1.f : p.v_head ? __ldg(p.v_head + kvh) : p.v_scale;
  const int tid = threadIdx.x, ty = tid >> 4, tx = tid & 15;

  for (int i = tid; i < kR * (D / 4); i += kTileThreads) {
    const int r = i / (D / 4), c = i % (D / 4);
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
    if (r < np) {
      const int64_t pr = pair0 + r;
      x = __ldg(reinterpret_cast<const float4*>(p.q) + (((int64_t)(first + pr / G)) * hq + kvh * G + pr % G) * (D / 4) + c);
    }
    *reinterpret_cast<float4*>(qs + r * LD + 4 * c) = x;
  }
  float acc[4][4 * DC], m[4], l[4], slope[4];
  int pos[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int64_t pr = pair0 + min(4 * ty + i, np - 1);
    pos[i] = at0 + (int)(pr / G);
    slope[i] = bp.mod.slopes ? __ldg(bp.mod.slopes + kvh * G + pr % G) * kLog2e : 0.f;
    m[i] = -1e30f;
    l[i] = 0.f;
#pragma unroll
    for (int e = 0; e < 4 * DC; ++e) acc[i][e] = 0.f;
  }
  // tiles with a key that some pair sees: [0, tp) of the prefix and [tl, te)
  const int plo = at0 + (int)(pair0 / G), phi = at0 + (int)((pair0 + np - 1) / G);
  const int end = min(len, max(phi + 1, pfx)), wlo = W > 0 ? max(0, plo - W + 1) : 0;
  const int tp = (pfx + kKT - 1) / kKT, tl = max(tp, wlo / kKT), te = (end + kKT - 1) / kKT;
  const int ntiles = tp + max(0, te - tl);
  const int32_t* table = p.block_tables + (int64_t)s * p.max_blocks;
  auto seen_by_some = [&](int key) { return key < end && (key < pfx || (key >= wlo && key <= phi)); };
  auto block_of = [&](int key) {
    int64_t blk = __ldg(table + key / bs);
    if (blk < 0 || blk >= p.num_blocks) {  // bad table entry: flag it, read block 0
      atomicCAS(p.err, 0, 2);
      blk = 0;
    }
    return blk;
  };
  const float scale2 = p.scale * kLog2e * kmul;
  for (int t = 0; t < ntiles; ++t) {
    const int key0 = (t < tp ? t : t - tp + tl) * kKT;
    __syncthreads();  // the previous tile has been read
    // K and V rows; those that no pair sees are 0 (their V may be anything: 0 * NaN)
    for (int i = tid; i < kKT * (D / 4); i += kTileThreads) {
      const int k = i / (D / 4), c = i % (D / 4), key = key0 + k;
      float4 kx = make_float4(0.f, 0.f, 0.f, 0.f), vx = kx;
      if (seen_by_some(key)) {
        const int64_t at = ((block_of(key) * hkv + kvh) * bs + key % bs) * D + 4 * c;
        if constexpr (KV == kF32) {
          kx = __ldg(reinterpret_cast<const float4*>(reinterpret_cast<const float*>(p.k_cache) + at));
          vx = __ldg(reinterpret_cast<const float4*>(reinterpret_cast<const float*>(p.v_cache) + at));
        } else {
          const uint32_t w = __ldg(reinterpret_cast<const uint32_t*>(p.k_cache + at));
          kx = make_float4(dev::e4m3_to_f32(w & 0xFFu), dev::e4m3_to_f32((w >> 8) & 0xFFu),
                           dev::e4m3_to_f32((w >> 16) & 0xFFu), dev::e4m3_to_f32(w >> 24));
        }
      }
      *reinterpret_cast<float4*>(ks + k * LD + 4 * c) = kx;
      if constexpr (KV == kF32) *reinterpret_cast<float4*>(vs + k * LD + 4 * c) = vx;
    }
    if constexpr (KV == kFP8) {  // d-major: 16 keys of an element are contiguous
      for (int i = tid; i < D * (kKT / 16); i += kTileThreads) {
        const int d = i % D, k0 = i / D * 16, key = key0 + k0;
        bool any = false;
#pragma unroll
        for (int k = 0; k < 16; ++k) any = any || seen_by_some(key + k);
        uint4 raw = make_uint4(0, 0, 0, 0);
        if (any)
          raw = __ldg(reinterpret_cast<const uint4*>(p.v_cache + ((block_of(key) * hkv + kvh) * D + d) * bs + key % bs));
        const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
        for (int k = 0; k < 16; ++k)
          vs[(k0 + k) * LD + d] = seen_by_some(key + k) ? dev::e4m3_to_f32((w[k >> 2] >> (8 * (k & 3))) & 0xFFu) : 0.f;
      }
    }
    __syncthreads();
    // ---- scores of rows 4 ty + i and keys tx + 16 j ----
    float sc[4][4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) sc[i][j] = 0.f;
#pragma unroll 4
    for (int c = 0; c < D; c += 4) {
      float4 a[4], b[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        a[i] = *reinterpret_cast<const float4*>(qs + (4 * ty + i) * LD + c);
        b[i] = *reinterpret_cast<const float4*>(ks + (tx + 16 * i) * LD + c);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          sc[i][j] = fmaf(a[i].x, b[j].x, sc[i][j]);
          sc[i][j] = fmaf(a[i].y, b[j].y, sc[i][j]);
          sc[i][j] = fmaf(a[i].z, b[j].z, sc[i][j]);
          sc[i][j] = fmaf(a[i].w, b[j].w, sc[i][j]);
        }
    }
    // ---- cap, bias, masks, online softmax per row (16 lanes) ----
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float mx = -INFINITY;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int key = key0 + tx + 16 * j;
        const bool seen = key < len && (key < pfx || (key <= pos[i] && (W <= 0 || pos[i] - key < W)));
        const float x = bp.mod.cap_out > 0.f ? bp.mod.cap_out * tanhf(sc[i][j] * (bp.mod.cap_in * kmul * kHalfLn2))
                                             : sc[i][j] * scale2;
        sc[i][j] = seen ? fmaf(-slope[i], fabsf((float)(pos[i] - key)), x) : -INFINITY;
        mx = fmaxf(mx, sc[i][j]);
      }
#pragma unroll
      for (int o = 8; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
      const float mn = fmaxf(m[i], mx), al = dev::ex2(m[i] - mn);
      m[i] = mn;
      l[i] *= al;
#pragma unroll
      for (int e = 0; e < 4 * DC; ++e) acc[i][e] *= al;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float w = dev::ex2(sc[i][j] - mn);
        l[i] += w;  // this lane's keys: the lanes are added at the end
        ps[(4 * ty + i) * LP + tx + 16 * j] = w;
      }
    }
    __syncwarp();  // a row's weights are written and read by the same half warp
    // ---- O += P V: rows 4 ty + i, columns 64 c + 4 tx .. + 3 ----
#pragma unroll 2
    for (int k = 0; k < kKT; k += 4) {
      float4 w[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) w[i] = *reinterpret_cast<const float4*>(ps + (4 * ty + i) * LP + k);
#pragma unroll
      for (int kk = 0; kk < 4; ++kk)
#pragma unroll
        for (int c = 0; c < DC; ++c) {
          const float4 v = *reinterpret_cast<const float4*>(vs + (k + kk) * LD + 64 * c + 4 * tx);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float x = kk == 0 ? w[i].x : kk == 1 ? w[i].y : kk == 2 ? w[i].z : w[i].w;
            acc[i][4 * c] = fmaf(x, v.x, acc[i][4 * c]);
            acc[i][4 * c + 1] = fmaf(x, v.y, acc[i][4 * c + 1]);
            acc[i][4 * c + 2] = fmaf(x, v.z, acc[i][4 * c + 2]);
            acc[i][4 * c + 3] = fmaf(x, v.w, acc[i][4 * c + 3]);
          }
        }
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float sum = l[i];
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if (4 * ty + i >= np) continue;
    const float inv = sum > 0.f ? vmul / sum : (sum == 0.f ? 0.f : sum);  // nothing visible: 0; NaN stays
    const int64_t pr = pair0 + 4 * ty + i;
    float4* out = reinterpret_cast<float4*>(p.out) + ((int64_t)(first + pr / G) * hq + kvh * G + pr % G) * (D / 4);
#pragma unroll
    for (int c = 0; c < DC; ++c)
      out[16 * c + tx] = make_float4(acc[i][4 * c] * inv, acc[i][4 * c + 1] * inv, acc[i][4 * c + 2] * inv,
                                     acc[i][4 * c + 3] * inv);
  }
}

template <int KV, int D>
cudaError_t launch_tiles(const BiasedSimtParams& p, cudaStream_t stream) {
  const int G = p.a.num_q_heads / p.a.num_kv_heads;
  const int64_t blocks = (int64_t)p.a.rows.num_rows * G / kR + p.a.rows.num_seqs;
  auto kern = attn_biased_tile_kernel<KV, D>;
  static int set_for[64] = {0};  // the shared memory limit is raised once per device
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= 64 || !set_for[dev]) {
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, tile_smem<D>());
    if (e != cudaSuccess) return e;
    if (dev < 64) set_for[dev] = 1;
  }
  kern<<<dim3((unsigned)blocks, (unsigned)p.a.num_kv_heads), kTileThreads, tile_smem<D>(), stream>>>(p);
  return cudaGetLastError();
}

// The tile kernel where the chunks' pairs make 32 CTAs of it or more (below
// that the row kernel's many short CTAs are faster: 33 rows of 8 heads over 500
// keys 33 us against 120, 512 over 1000 580 against 309; beside 62 single rows
// of 32 heads over 500 keys a 2-row chunk 181 us a step against 276).
template <int KV, int D>
cudaError_t launch_rows(const BiasedSimtParams& p, cudaStream_t stream) {
  const bool tiles = (int64_t)p.chunk_rows * p.a.num_q_heads >= 32 * kR;
  if (!biased_simt_fits(p.a.rows.num_rows, p.a.rows.num_seqs, p.a.num_q_heads, p.a.num_kv_heads))
    return cudaErrorNotSupported;  // (before either launch)
  attn_biased_row_kernel<KV, D><<<dim3((unsigned)p.a.rows.num_rows, (unsigned)p.a.num_q_heads),
                                  row_warps<KV, D>() * 32, 0, stream>>>(p, !tiles);
  const cudaError_t e = cudaGetLastError();
  return e == cudaSuccess && tiles ? launch_tiles<KV, D>(p, stream) : e;
}

template <int KV>
cudaError_t launch_d(const BiasedSimtParams& p, cudaStream_t stream) {
  if (p.a.head_dim == 64) return launch_rows<KV, 64>(p, stream);
  if (p.a.head_dim == 128) return launch_rows<KV, 128>(p, stream);
  return cudaErrorNotSupported;
}

}  // namespace

cudaError_t launch_attn_biased_simt(const BiasedSimtParams& p, int kv_dtype, cudaStream_t stream) {
  if (kv_dtype == kF32) return launch_d<kF32>(p, stream);
  if (kv_dtype == kFP8) return launch_d<kFP8>(p, stream);
  return cudaErrorNotSupported;
}

}  // namespace pa

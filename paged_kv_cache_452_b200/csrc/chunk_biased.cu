// Chunks of new tokens under a biased score, over a paged bf16 or e4m3 pool,
// on the 5th-generation tensor cores (pa_decode_chunked_prefill_biased's rows
// of more than one per sequence).
//
// What it computes: row i of a sequence sees key j if j < prefix, or j <= i
// and (window) i - j < window; s = cap tanh(scale q k / cap) - slope |i - j|
// (or scale q k - slope |i - j|), out = softmax(s) V over the visible keys.
//
// Unit = (sequence, kv head, 2 x (128 / G) query positions): two query tiles A
// and B of 128 rows (positions x the group's heads), one warpgroup of softmax
// warps each, a thread per row.  While A's softmax runs, the tensor core does
// B's products and the other way round, and both tiles use every K/V tile that
// is brought in.  One persistent CTA per SM claims units from a counter.
//  * Steps of 64 keys: half a 128-key K/V tile.  TMEM (512 columns): two S
//    buffers of 64 columns and O (head_dim columns) per query tile; a step's
//    weights P (16 bit) go over the first half of its own S buffer.  One warp
//    per query tile issues its MMAs, PV(j) then S(j + 2): MMAs of one thread run
//    in order, so S(j + 2) finds P(j) consumed, and the softmax of step j + 1
//    runs under both.  (Steps of 128 keys with one S buffer: 205 us instead of
//    182 on six 640-row chunks with a distance bias; one warp issuing for both
//    tiles in turn 196; a lock around each tile's products 210.)
//  * Steps run from the last key to the first: with a distance bias the
//    nearest keys carry the largest weights, so the reference that a row's
//    exponents get from its first step serves the others.  A later step skips
//    the row max: its weights 2^(s - ref) only have to stay finite, and a sum
//    above BIG sends the warp to the long way that moves the reference and
//    rescales O.  Tiles between the prefix and the window are skipped.
//  * The cap's tanh is an odd polynomial of degree 9 on |y| <= 0.8 (minimax,
//    3.5e-7 absolute), which leaves one special-function operation per score,
//    the exponential; a step with a larger |y| takes the exact form, which
//    needs three.
//  * Few units (a chunk or two): their keys are cut into up to eight parts,
//    each a unit of the queue that leaves (reference, sum, O) per row; for each
//    warp's rows the part that arrives last joins them in the order of the
//    parts.  Nobody waits for another, and results do not depend on the order
//    of arrival.  (One 512-row chunk over 8300 keys, 32 heads: 155 -> 90 us.)
//  * e4m3 pools: blocks land raw (bulk copies), four converter warps write them
//    as f16 (exact) into the swizzled K and V tiles, V as rows of d with
//    their keys contiguous (what its d-major blocks give), and the queries
//    become f16, each row times a power of two that keeps it in range; P is f16.
//
// What bounds it (measured on B200, clocks per step of both query tiles): the
// products 1280 (S at N = 64 reads its 6 KB of operands per MMA at the shared
// memory's 128 bytes a clock, 48 instead of 32; PV 64), 2 x 4 x 64 x 32
// exponentials 1024 at 16 lanes a clock (with what surrounds them 1174 under a
// distance bias, 1466 under a cap), and 1750 to 2000 in all, the rest being the
// hand-offs between the two (a step's weights to its next scores).  Six
// 640-row chunks over up to 2048 cached keys, 32 heads, distance bias: 161 us,
// 724 TFLOP/s; two 1024-row chunks over 4096 to 8192 keys in e4m3, cap: 343 us,
// 765 TFLOP/s.
// A mixed step of many sequences over a bf16 pool launches this kernel twice
// around its decode kernel, which is bound by HBM: some CTAs before it, which run beside it on
// SMs of their own, and CTAs behind it that take SMs as its CTAs leave.  All
// claim units of one queue.
// Every wait is bounded (2 s, then the error word); TMEM is freed on every path.
#include <cuda_runtime.h>

#include "pa_device.cuh"
#include "pa_kernels.h"

namespace pa {
namespace {

constexpr int kRows = 128;   // rows of a query tile: the MMA's M
constexpr int kKeys = 128;   // keys of a K/V tile
constexpr int kHalf = 64;    // keys of a step: half a tile
constexpr int kTileRow = 128 * 128;  // bytes of a 64-element-wide chunk of a 128-row tile
constexpr int kUQ = 4;       // unit queue entries
constexpr int kMaxParts = 8;
constexpr float kPartCost = 6.f;  // tiles (3 and 10 choose the same almost everywhere)
static_assert(kMaxParts == 8, "a candidate per lane of eight");
constexpr int kGroup = 64;   // sequences of a group in the unit search
constexpr int kMaxGroups = 256;  // groups: 16384 sequences
constexpr int kMaxOrder = 64;    // up to so many chunks are taken longest context first
constexpr int kKWarp = 8, kVWarp = 9, kMmaWarp = 10, kConvWarp = 12;  // warps 0..7: softmax of A, of B
constexpr uint32_t kTmemCols = 512;
constexpr int kSmemOptIn = 232448;  // 227 KB per block
constexpr int kMask = 0, kSlope = 1, kCap = 2, kCapSlope = 3;

// tanh(y) = y P(y^2) on |y| <= kCapFast: minimax in the absolute error (3.5e-7;
// 4.2e-7 as evaluated in fp32), fitted by an exchange iteration in fp64.  (A fit
// of the relative error reaches 1.0e-6, 7e-7 absolute: better only for scores
// far below a cap, worse at the caps that models use.)
constexpr float kCapFast = 0.8f;
constexpr float kTanh[5] = {0.999995135f, -0.333174266f, 0.131862197f, -0.0482613155f, 0.0114646552f};

template <int KV, int D, int BS>
struct C {
  static constexpr bool FP8 = KV == kFP8;
  static constexpr int NCH = D / 64;                // 64-element chunks of a row
  static constexpr int TILE = NCH * kTileRow;       // bytes of a 16-bit Q, K or V tile
  static constexpr int RAW = kKeys * D;             // bytes of a raw e4m3 tile
  static constexpr int BPT = kKeys / BS;            // blocks per tile
  static constexpr int NK = FP8 ? 2 : D == 64 ? 4 : 3, NV = FP8 || D == 128 ? 2 : 4;  // K and V tiles in shared memory
  static constexpr int NR = FP8 ? 2 : 0;            // raw tiles
  static constexpr int THREADS = FP8 ? 512 : 384;
  // warps that read a queue entry: the V loader, the two MMA warps, the eight
  // softmax warps, in e4m3 the four converters
  static constexpr int READERS = 1 + 2 + 8 + (FP8 ? 4 : 0);
  // weights stay at most this in a tile's sum before the reference moves:
  // bf16 has fp32's range, f16 ends at 65504
  static constexpr float BIG = FP8 ? 16384.f : 18446744073709551616.f;
  // shared memory
  static constexpr int Q = 0, K = 2 * TILE, V = K + NK * TILE, R = V + NV * TILE, BARS = R + NR * RAW;
  static constexpr int NBARS = 2 * NK + 2 * NV + 2 * NR + 14 + 4 + 2 * kUQ;
  static constexpr int UQ = (BARS + NBARS * 8 + 15) / 16 * 16, TSLOT = UQ + kUQ * 48, GROUPS = TSLOT + 16;
  static constexpr int ORDER = GROUPS + (kMaxGroups + 1) * 4;  // bases, then sequences
  static constexpr int TOTAL = ORDER + (kMaxOrder + 1) * 4 + kMaxOrder * 2 + 1024;
  static_assert(TOTAL <= kSmemOptIn, "shared memory");
  static_assert(256 + 2 * D <= (int)kTmemCols, "TMEM columns");
};

// One unit, published in shared memory by the claiming warp.
struct __align__(16) Unit {
  int s, h;        // sequence (-1: no more units), kernel kv head
  int row0, qn;    // first query row, positions (at most two tiles' worth)
  int p0;          // position of the first query
  int len, pfx;    // context, visible prefix
  int unit;        // the unit's number, where its keys are cut into parts
  int part, parts; // this part of them
  int pad[2];
};
static_assert(sizeof(Unit) == 48, "queue entry");

// A unit's key tiles: [0, npt) and [npt + gap, npt + gap + ...), visited from
// the last; nt of them are this part's.
template <int BS>
struct Tiles {
  int kend, lo, nb, nt, npt, gap, window, pfx;
  int all, from;  // tiles of the unit, and where this part of it starts
  __device__ __forceinline__ Tiles(const Unit& u, const PrefillParams& p) {
    window = p.mod.window;
    pfx = u.pfx;
    kend = max(min(u.len, u.p0 + u.qn), u.pfx);
    lo = window > 0 ? max(0, u.p0 - window + 1) : 0;
    nb = min((max(kend, 0) + BS - 1) / BS, p.max_blocks);
    const int tiles = (nb * BS + kKeys - 1) / kKeys;
    npt = min((pfx + kKeys - 1) / kKeys, tiles);
    gap = max(0, min(lo / kKeys, tiles) - npt);
    all = tiles - gap;
    from = 0;
    nt = all;
    if (u.parts > 1) {
      from = all * u.part / u.parts;
      nt = all * (u.part + 1) / u.parts - from;
    }
  }
  __device__ __forceinline__ int tile(int k) const {
    const int t = all - 1 - from - k;
    return t < npt ? t : t + gap;
  }
  // Half tiles, 64 keys each, in the order of the visits: step j is half 1 - j
  // % 2 of tile(j / 2).  first() is step 0's half (64-key index), next() the one after.
  __device__ __forceinline__ int first_half() const { return nt > 0 ? 2 * tile(0) + 1 : 0; }
  __device__ __forceinline__ int next_half(int h) const {
    return gap > 0 && h == 2 * (npt + gap) ? 2 * npt - 1 : h - 1;
  }
};
// Whether rows at positions [a, a + n) see a key of half h.
struct Seen {
  int hp, f, e;
  template <int BS>
  __device__ __forceinline__ Seen(const Tiles<BS>& t, int a, int n) {
    hp = n > 0 ? (t.pfx + kHalf - 1) / kHalf : 0;
    f = (t.window > 0 ? max(0, a - t.window + 1) : 0) / kHalf;
    e = n > 0 ? (max(a + n, 0) + kHalf - 1) / kHalf : 0;
  }
  __device__ __forceinline__ bool operator()(int h) const { return h < hp || (h >= f && h < e); }
};

// Registers move from the loaders', the MMA's and the converters' warpgroups
// to the two softmax warpgroups: 2 x 128 x 208 + 128 x 88 of the 384 x 168 at
// launch, and with the converters 2 x 128 x 176 + 2 x 128 x 80 of 512 x 128.
template <bool FP8>
__device__ __forceinline__ void reg_inc() {
  if constexpr (FP8) asm volatile("setmaxnreg.inc.sync.aligned.u32 176;");
  else asm volatile("setmaxnreg.inc.sync.aligned.u32 208;");
}
template <bool FP8>
__device__ __forceinline__ void reg_dec() {
  if constexpr (FP8) asm volatile("setmaxnreg.dec.sync.aligned.u32 80;");
  else asm volatile("setmaxnreg.dec.sync.aligned.u32 88;");
}

template <int KV, int D, int BS, int MOD>
__global__ void __launch_bounds__(C<KV, D, BS>::THREADS, 1)
    chunk_biased_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                        const __grid_constant__ CUtensorMap tm_q, const PrefillParams p) {
  using T = C<KV, D, BS>;
  constexpr bool CAPS = MOD >= kCap, SLOPES = MOD == kSlope || MOD == kCapSlope;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* kfull = reinterpret_cast<uint64_t*>(smem + T::BARS);
  uint64_t* kempty = kfull + T::NK;
  uint64_t* vfull = kempty + T::NK;
  uint64_t* vempty = vfull + T::NV;
  uint64_t* rfull = vempty + T::NV;
  uint64_t* rempty = rfull + T::NR;
  // per query tile x and S buffer b, at 2 x + b
  uint64_t* s_full = rempty + T::NR;  // [4] S is complete
  uint64_t* p_full = s_full + 4;      // [4] P is written
  uint64_t* pv_done = p_full + 4;     // [4] its PV is complete
  uint64_t* o_free = pv_done + 4;     // [2] a unit's O has been read out
  uint64_t* q_full = o_free + 2;      // the Q tiles are in place
  uint64_t* q_raw = q_full + 1;       // e4m3: ... as bf16, before their conversion
  uint64_t* q_free = q_raw + 1;       // the unit's last S MMA is complete
  uint64_t* done = q_free + 1;        // every MMA issued is complete
  uint64_t* uq_full = done + 1;
  uint64_t* uq_empty = uq_full + kUQ;
  Unit* uq = reinterpret_cast<Unit*>(smem + T::UQ);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + T::TSLOT);
  int32_t* gsum = reinterpret_cast<int32_t*>(smem + T::GROUPS);  // unit blocks before each group of sequences
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int G = p.group, hq = p.num_q_heads, hkv = p.num_kv_heads, S = p.rows.num_seqs;
  const int QB = kRows / G, QB2 = 2 * QB;

  if (!p.after_decode) dev::grid_dep_wait();
  // ---- unit blocks of each group of sequences, exclusive prefix --------------
  auto blocks_of = [&](int s) {
    const int q = s < S ? p.rows.qsl[s + 1] - p.rows.qsl[s] : 0;
    return q > 1 || (q == 1 && p.singles) ? (q + QB2 - 1) / QB2 : 0;
  };
  const int groups = (S + kGroup - 1) / kGroup;
  // The chunks by falling context where there are few (long units first leave
  // a shorter tail; more of them even out by their number): obase, the unit
  // blocks before each, and oseq, the sequence
  int32_t* obase = reinterpret_cast<int32_t*>(smem + T::ORDER);
  int16_t* oseq = reinterpret_cast<int16_t*>(obase + kMaxOrder + 1);
  int32_t* found = reinterpret_cast<int32_t*>(tmem_slot + 1);
  int32_t* longest = found + 1;  // context of the first
  if (tid == 0) *found = 0;
  __syncthreads();
  for (int g = warp; g < groups; g += T::THREADS / 32) {
    int n = 0;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int s = kGroup * g + 2 * lane + e, nb = blocks_of(s);
      n += nb;
      if (nb > 0) {
        const int at = atomicAdd(found, 1);
        if (at < kMaxOrder) {
          oseq[at] = (int16_t)s;
          obase[at] = p.rows.seq_lens[s];
        }
      }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) n += __shfl_xor_sync(0xffffffffu, n, o);
    if (lane == 0) gsum[g] = n;
  }
  if (tid == 0) {
    for (int i = 0; i < T::NK; ++i) {
      dev::mbar_init(&kfull[i], T::FP8 ? 4 : 1);
      dev::mbar_init(&kempty[i], 2);  // both query tiles' MMAs
    }
    for (int i = 0; i < T::NV; ++i) {
      dev::mbar_init(&vfull[i], T::FP8 ? 4 : 1);
      dev::mbar_init(&vempty[i], 2);
    }
    for (int i = 0; i < T::NR; ++i) {
      dev::mbar_init(&rfull[i], 1);
      dev::mbar_init(&rempty[i], 4);
    }
    for (int i = 0; i < 4; ++i) {
      dev::mbar_init(&s_full[i], 1);
      dev::mbar_init(&p_full[i], 4);
      dev::mbar_init(&pv_done[i], 1);
    }
    for (int x = 0; x < 2; ++x) dev::mbar_init(&o_free[x], 4);
    dev::mbar_init(q_full, T::FP8 ? 8 : 1);
    dev::mbar_init(q_raw, 1);
    dev::mbar_init(q_free, 2);
    dev::mbar_init(done, 2);
    for (int i = 0; i < kUQ; ++i) {
      dev::mbar_init(&uq_full[i], 1);
      dev::mbar_init(&uq_empty[i], T::READERS);
    }
    dev::fence_barrier_init();
  }
  __syncthreads();
  if (warp == 0) {
    int run = 0;
    for (int g0 = 0; g0 < groups; g0 += 32) {
      const int n = g0 + lane < groups ? gsum[g0 + lane] : 0;
      int x = n;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
      }
      if (g0 + lane < groups) gsum[g0 + lane] = run + x - n;
      run += __shfl_sync(0xffffffffu, x, 31);
    }
    if (lane == 0) gsum[groups] = run;
  }
  const int chunks = *found;
  const bool ordered = chunks <= kMaxOrder;
  {
    // rank by (context, sequence): the same whatever order they were found in
    int mine = -1, rank = 0, nb = 0, len = 0;
    if (ordered && tid < chunks) {
      mine = oseq[tid];
      nb = blocks_of(mine);
      len = obase[tid];
      for (int j = 0; j < chunks; ++j) rank += obase[j] > len || (obase[j] == len && oseq[j] < mine);
    }
    __syncthreads();
    if (mine >= 0) {
      oseq[rank] = (int16_t)mine;
      obase[rank] = nb;
      if (rank == 0) *longest = len;
    }
    __syncthreads();
    if (ordered && warp == 1) {
      int v[2], run = 0;
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int i = 32 * e + lane;
        const int n = i < chunks ? obase[i] : 0;
        int x = n;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int y = __shfl_up_sync(0xffffffffu, x, o);
          if (lane >= o) x += y;
        }
        v[e] = run + x - n;
        run += __shfl_sync(0xffffffffu, x, 31);
      }
      __syncwarp();
      obase[lane] = v[0];
      obase[32 + lane] = v[1];
      if (lane == 0) obase[kMaxOrder] = run;
    }
  }
  __syncthreads();
  dev::grid_dep_launch();
  // With few units their keys are cut into parts, so that every SM gets some
  // and the last ones are short; a unit's parts leave (reference, sum, O) per
  // row, and for each warp's rows the part that arrives last joins them.
  const int whole = gsum[groups] * hkv;
  // A part costs its tiles and about kPartCost more (start, first step, join);
  // parts are as many as make the rounds over the SMs shortest (as many as
  // there are slots for: 6 chunks of 27 rows over 3200 keys 45 us, so 30; one of
  // 512 over 8500, 32 heads, 106 and 90).
  int parts = 1;
  if (!ordered && whole > 0) {  // (contexts not at hand: one round)
    parts = max(1, min(kMaxParts, p.part_slots / (kPartSlots * whole)));
  } else if (whole > 0 && p.part_slots >= 2 * whole) {
    int tiles = (min(*longest, p.max_blocks * BS) + kKeys - 1) / kKeys;
    if (p.mod.window > 0) tiles = min(tiles, (p.mod.window - 1) / kKeys + QB2 / kKeys + 2);
    const int sms = p.part_slots / kPartSlots;
    parts = (lane & 7) + 1;  // a candidate per lane, then the best of them
    float cost = parts * whole > p.part_slots ? 1e30f
                                              : (float)((whole * parts + sms - 1) / sms) * ((float)tiles / (float)parts + kPartCost);
#pragma unroll
    for (int x = 1; x < 8; x <<= 1) {
      const float c = __shfl_xor_sync(0xffffffffu, cost, x);
      const int n = __shfl_xor_sync(0xffffffffu, parts, x);
      if (c < cost || (c == cost && n < parts)) {
        cost = c;
        parts = n;
      }
    }
  }
  const int nunits = whole * parts;
  auto finish_queue = [&]() {  // the step's last CTA puts the claim counter back to zero
    if (tid == 0) {
      __threadfence();
      if (atomicAdd(p.unit_exit, 1) == p.exits - 1) {
        atomicExch(p.unit_ctr, 0);
        atomicExch(p.unit_exit, 0);
      }
    }
    // this grid does not wait for the step's decode grid before it works, and
    // a later grid of the stream may wait for this one alone
    if (p.after_decode) dev::grid_dep_wait();
  };
  if ((int)blockIdx.x >= nunits) {
    finish_queue();
    return;
  }
  if (warp == kMmaWarp) {
    dev::tmem_alloc(tmem_slot, kTmemCols);
    dev::tmem_relinquish();
  }
  dev::tc_fence_before();
  __syncthreads();
  dev::tc_fence_after();
  const uint32_t tbase = *tmem_slot;

  // queue entry n, as one warp's (or thread's) copy; ok false: none
  auto read_unit = [&](int n, Unit& u, bool& ok) {
    const int slot = n % kUQ;
    if (ok) ok = dev::mbar_wait_clk(&uq_full[slot], (uint32_t)((n / kUQ) & 1), p.err);
    if (ok) u = uq[slot];
    else u.s = -1;
  };

  if (warp == kKWarp || warp == kVWarp) {
    // ================= claims, and the loads of K / V and Q ======================
    reg_dec<T::FP8>();
    const bool is_v = warp == kVWarp;
    const uint64_t pol = dev::policy_evict_last();  // the sequence's other units read the same tiles
    const uint64_t qpol = dev::policy_evict_first();
    const int ph_div = p.mod.sub;
    bool ok = true;
    int st = 0, g = 0, qlast = -1;
    uint32_t ph = 0;
    for (int n = 0;; ++n) {
      Unit u;
      u.s = -1;
      if (!is_v) {
        // claim the next unit (part) and publish it; parts that a short unit
        // does not have are passed over
        while (ok && u.s < 0) {
          int idx = 0;
          if (lane == 0) idx = atomicAdd(p.unit_ctr, 1);
          idx = __shfl_sync(0xffffffffu, idx, 0);
          if (idx >= nunits) break;
          const int id = idx / parts, x = id / hkv;
          bool hit;
          int before, mine;
          if (ordered) {
            const int r = __popc(__ballot_sync(0xffffffffu, lane < chunks && obase[lane] <= x)) +
                          __popc(__ballot_sync(0xffffffffu, 32 + lane < chunks && obase[32 + lane] <= x)) - 1;
            hit = true;
            u.s = oseq[r];
            before = obase[r];
            mine = (r + 1 < chunks ? obase[r + 1] : obase[kMaxOrder]) - before;
            before -= x;  // (below: the block's place among the sequence's)
          } else {
            int lo = 0, hi = groups - 1;  // the last group with gsum <= x
            while (lo < hi) {
              const int mid = (lo + hi + 1) >> 1;
              if (gsum[mid] <= x) lo = mid; else hi = mid - 1;
            }
            const int s0 = kGroup * lo + 2 * lane;  // this lane's two sequences
            const int nb0 = blocks_of(s0), nb = nb0 + blocks_of(s0 + 1);
            int inc = nb;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
              const int y = __shfl_up_sync(0xffffffffu, inc, o);
              if (lane >= o) inc += y;
            }
            const int local = x - gsum[lo];
            const uint32_t who = __ballot_sync(0xffffffffu, local >= inc - nb && local < inc);
            hit = who != 0;
            const int src = hit ? __ffs(who) - 1 : 0;
            const int pair0 = __shfl_sync(0xffffffffu, inc - nb, src);
            const int n0 = __shfl_sync(0xffffffffu, nb0, src), n1 = __shfl_sync(0xffffffffu, nb, src) - n0;
            const int second = local - pair0 >= n0;
            u.s = hit ? kGroup * lo + 2 * src + second : -1;
            mine = second ? n1 : n0;
            before = pair0 + (second ? n0 : 0) - local;
          }
          if (hit) {
            u.h = id % hkv;
            u.unit = id;
            u.part = idx - id * parts;
            u.parts = 1;
            const int first = p.rows.qsl[u.s], qlen = p.rows.qsl[u.s + 1] - first;
            const int qb = mine - 1 + before;  // a sequence's last (longest) rows first
            int len = p.rows.seq_lens[u.s];  // (u.s is a sequence here; below it may be given up)
            u.p0 = len - qlen + qb * QB2;
            u.row0 = first + qb * QB2;
            // (never past the rows that q and out have, whatever query_start_loc says)
            u.qn = min(min(QB2, qlen - qb * QB2), p.rows.num_rows - u.row0);
            if (u.row0 < 0 || u.qn <= 0) u.s = -1;
            if (len > p.max_blocks * BS) {  // longer than its table row: flag, clamp
              if (lane == 0) atomicCAS(p.err, 0, 3);
              len = p.max_blocks * BS;
            }
            u.len = len;
            u.pfx = p.mod.prefix && u.s >= 0 ? max(0, min(len, __ldg(p.mod.prefix + u.s))) : 0;
            if (parts > 1 && u.s >= 0) {  // at least two tiles a part
              u.parts = min(parts, max(1, Tiles<BS>(u, p).all / 2));
              if (u.part >= u.parts) u.s = -1;
            }
          }
        }
        const int slot = n % kUQ;
        if (n >= kUQ && ok)
          ok = __all_sync(0xffffffffu, dev::mbar_wait_clk(&uq_empty[slot], (uint32_t)(((n / kUQ) - 1) & 1), p.err));
        if (!ok) u.s = -1;
        if (lane == 0) {
          uq[slot] = u;
          dev::mbar_arrive(&uq_full[slot]);
        }
        __syncwarp();
      } else {
        read_unit(n, u, ok);
        ok = __all_sync(0xffffffffu, ok);
        __syncwarp();
        if (lane == 0) dev::mbar_arrive(&uq_empty[n % kUQ]);
      }
      if (u.s < 0) break;
      const Tiles<BS> tl(u, p);
      if (is_v) {
        // the unit's queries, once the previous unit's S MMAs are done with
        // them: two boxes of 128 / G positions (rows past the unit are other
        // rows or zeros: computed, not kept)
        if (n > 0 && ok) ok = __all_sync(0xffffffffu, dev::mbar_wait_clk(q_free, (uint32_t)((n - 1) & 1), p.err));
        if (!ok) continue;
        if (lane == 0) {
          uint64_t* bar = T::FP8 ? q_raw : q_full;
          dev::mbar_arrive_expect_tx(bar, (uint32_t)(2 * T::NCH * QB * G * 128));
#pragma unroll
          for (int i = 0; i < 2 * T::NCH; ++i)
            dev::tma_load_3d(smem + T::Q + (i / T::NCH) * T::TILE + (i % T::NCH) * kTileRow, &tm_q, (i % T::NCH) * 64,
                             u.h * G, u.row0 + (i / T::NCH) * QB, bar, qpol);
        }
        qlast = n;
        __syncwarp();
        if constexpr (T::FP8) continue;  // K and V both come raw, by the K warp
      }
      const int32_t* table = p.block_tables + (int64_t)u.s * p.max_blocks;
      const int head = u.h / ph_div, pool_heads = hkv / ph_div;
      // a block is read if a row of the unit may see one of its keys
      auto entry = [&](int k, int j) -> int32_t {
        const int b = tl.tile(k) * T::BPT + j;
        return k < tl.nt && b < tl.nb && (b * BS < u.pfx || b >= tl.lo / BS) ? __ldg(table + b) : -2;
      };
      auto checked = [&](int32_t blk) {
        if (blk < 0 || blk >= p.num_blocks) {  // bad table entry: flag, read block 0
          atomicCAS(p.err, 0, 2);
          blk = 0;
        }
        return blk;
      };
      if constexpr (!T::FP8) {
        uint64_t* fullb = is_v ? vfull : kfull;
        uint64_t* emptyb = is_v ? vempty : kempty;
        uint8_t* ring = smem + (is_v ? T::V : T::K);
        const int nst = is_v ? T::NV : T::NK;
        const CUtensorMap* tm = is_v ? &tm_v : &tm_k;
        const int c = lane / T::BPT, j = lane % T::BPT;
        const bool mine = lane < T::NCH * T::BPT;
        int32_t next = mine ? entry(0, j) : -2;
        for (int k = 0; k < tl.nt && ok; ++k, ++g) {
          if (g >= nst) ok = __all_sync(0xffffffffu, dev::mbar_wait_clk(&emptyb[st], ph ^ 1u, p.err));
          if (!ok) break;
          const int32_t blk = next;
          if (mine) next = entry(k + 1, j);
          int32_t y = p.num_blocks * pool_heads * BS;  // past the pool: zeros
          if (blk != -2) y = (checked(blk) * pool_heads + head) * BS;
          if (lane == 0) dev::mbar_arrive_expect_tx(&fullb[st], (uint32_t)T::TILE);
          __syncwarp();
          if (mine) dev::tma_load_2d(ring + st * T::TILE + c * kTileRow + j * BS * 128, tm, c * 64, y, &fullb[st], pol);
          if (++st == nst) {
            st = 0;
            ph ^= 1u;
          }
        }
      } else {
        // raw K, then raw V of each tile, a bulk copy per block
        const int j = lane % T::BPT;
        int32_t next = lane < T::BPT ? entry(0, j) : -2;
        for (int k = 0; k < tl.nt && ok; ++k) {
          int32_t blk = next;
          if (lane < T::BPT) next = entry(k + 1, j);
          const bool mine = blk != -2;
          if (mine) blk = checked(blk);
          const uint32_t bytes = (uint32_t)(__popc(__ballot_sync(0xffffffffu, mine)) * BS * D);
          for (int side = 0; side < 2 && ok; ++side, ++g) {
            if (g >= T::NR) ok = __all_sync(0xffffffffu, dev::mbar_wait_clk(&rempty[st], ph ^ 1u, p.err));
            if (!ok) break;
            if (lane == 0) dev::mbar_arrive_expect_tx(&rfull[st], bytes);
            __syncwarp();
            if (mine)
              dev::bulk_load(smem + T::R + st * T::RAW + j * BS * D,
                             (side ? p.v_raw : p.k_raw) + ((int64_t)blk * pool_heads + head) * BS * D,
                             (uint32_t)(BS * D), &rfull[st], pol);
            if (++st == T::NR) {
              st = 0;
              ph ^= 1u;
            }
          }
        }
      }
    }
    // drain: what is still in flight must land before the CTA may exit
    if (lane == 0) {
      uint64_t* fullb = T::FP8 ? rfull : is_v ? vfull : kfull;
      const int nst = T::FP8 ? T::NR : is_v ? T::NV : T::NK;
      for (int d = max(0, g - nst); d < g; ++d)
        dev::mbar_wait_clk(&fullb[d % nst], (uint32_t)((d / nst) & 1), nullptr, 1ll << 28);
      if (qlast >= 0) dev::mbar_wait_clk(T::FP8 ? q_raw : q_full, (uint32_t)(qlast & 1), nullptr, 1ll << 28);
    }
    __syncwarp();
  } else if (warp == kMmaWarp || warp == kMmaWarp + 1) {
    // ==================== MMA issue: one thread per query tile ====================
    reg_dec<T::FP8>();
    {
      // the whole warp runs this loop, converged; lane 0 issues
      auto uni = [](auto v) { return __shfl_sync(0xffffffffu, v, 0); };
      const uint32_t on = lane == 0;
      const int x = uni(warp) - kMmaWarp;
      auto wait = [&](uint64_t* bar, uint32_t parity) {
        return (bool)__all_sync(0xffffffffu, dev::mbar_wait_clk(bar, parity, p.err));
      };
      const uint32_t idesc_s = T::FP8 ? dev::umma_idesc_f16(kHalf, false) : dev::umma_idesc_bf16(kHalf, false);
      const uint32_t idesc_o = T::FP8 ? dev::umma_idesc_f16(D, false) : dev::umma_idesc_bf16(D, true);
      const uint64_t dq = dev::umma_desc_sw128(dev::smem_u32(smem + T::Q + x * T::TILE), 16, 1024);
      const uint64_t dk = dev::umma_desc_sw128(dev::smem_u32(smem + T::K), 16, 1024);
      // V: bf16 MN-major (d contiguous, 64-wide chunks kTileRow apart); e4m3's
      // converted tile K-major (keys contiguous, 64-key chunks of D rows)
      const uint64_t dv = dev::umma_desc_sw128(dev::smem_u32(smem + T::V), T::FP8 ? 16 : kTileRow, 1024);
      const uint32_t tb = uni(tbase), ts = tb + x * 2 * kHalf, to = tb + 4 * kHalf + x * D;
      // ring positions and barrier phases by counters: every instruction here
      // delays the tensor core's next tile
      int kst = 0, vst = 0;
      uint32_t kph = 0, vph = 0, oph = 1;
      uint32_t cs = 0, cp = 0;  // S's and PV's issued
      bool ok = true, used = false;
      for (int n = 0;; ++n) {
        Unit u;
        read_unit(n, u, ok);
        u.s = uni(u.s);
        ok = ok && u.s >= 0;
        u.p0 = uni(u.p0);
        u.qn = uni(u.qn);
        u.len = uni(u.len);
        u.pfx = uni(u.pfx);
        u.part = uni(u.part);
        u.parts = uni(u.parts);
        __syncwarp();
        if (on) dev::mbar_arrive(&uq_empty[n % kUQ]);
        if (u.s < 0) break;
        const Tiles<BS> tl(u, p);
        const int na = min(u.qn, QB);  // positions of tile A; B has the rest
        const Seen seen(tl, u.p0 + x * QB, x ? u.qn - na : na);
        ok = ok && wait(q_full, (uint32_t)(n & 1));
        const int steps = 2 * tl.nt;
        bool begun = false;
        if (steps == 0) dev::umma_commit_if(on, q_free);
        int hs = tl.first_half(), hv = hs;  // the halves of the next S and the next PV
        // step j: the PV of half j and the S of half j + 2, into the buffer
        // that this PV (or an earlier one) has read.  A stage is given back by
        // both threads, also by one whose query tile does not take it, and
        // only once it has landed (so neither can give it back twice in a row)
        for (int j = -2; j < steps && ok; ++j) {
          if (j >= 0) {
            const int hf = 1 - (j & 1);
            if (hf) ok = wait(&vfull[vst], vph);
            if (ok && seen(hv)) {
              const uint32_t b = cp & 1;
              ok = wait(&p_full[2 * x + b], (cp >> 1) & 1);
              if (!begun && used) ok = ok && wait(&o_free[x], oph);
              if (!ok) break;
              dev::tc_fence_after();
              const uint64_t vb = dv + (uint64_t)(vst * (T::TILE >> 4)) +
                                  (uint64_t)((T::FP8 ? hf * (D * 128) : hf * 4 * 16 * 128) >> 4);
#pragma unroll
              for (int ks = 0; ks < kHalf / 16; ++ks)
                dev::umma_ts_if(on, to, ts + b * kHalf + 8 * ks, vb + (uint64_t)((T::FP8 ? ks * 32 : ks * 16 * 128) >> 4),
                             idesc_o, (begun || ks > 0) ? 1u : 0u);
              dev::umma_commit_if(on, &pv_done[2 * x + b]);
              begun = true;
              ++cp;
            }
            if (!ok) break;
            hv = tl.next_half(hv);
            if (!hf) {
              dev::umma_commit_if(on, &vempty[vst]);
              if (++vst == T::NV) {
                vst = 0;
                vph ^= 1u;
              }
            }
          }
          if (j + 2 < steps) {
            const int hf = 1 - (j & 1);
            if (hf) ok = wait(&kfull[kst], kph);
            if (!ok) break;
            if (seen(hs)) {
              const uint32_t b = cs & 1;
              dev::tc_fence_after();
              const uint64_t kb = dk + (uint64_t)(kst * (T::TILE >> 4)) + (uint64_t)((hf * kHalf * 128) >> 4);
#pragma unroll
              for (int ks = 0; ks < D / 16; ++ks) {
                const uint64_t off = (uint64_t)(((ks >> 2) * kTileRow + (ks & 3) * 32) >> 4);
                dev::umma_ss_if(on, ts + b * kHalf, dq + off, kb + off, idesc_s, ks > 0 ? 1u : 0u);
              }
              dev::umma_commit_if(on, &s_full[2 * x + b]);
              ++cs;
            }
            hs = tl.next_half(hs);
            if (!hf) {
              dev::umma_commit_if(on, &kempty[kst]);
              if (++kst == T::NK) {
                kst = 0;
                kph ^= 1u;
              }
            }
            if (j + 3 == steps) dev::umma_commit_if(on, q_free);
          }
        }
        if (begun) {
          used = true;
          oph ^= 1u;
        }
      }
      // every MMA issued has completed before TMEM may be freed
      dev::umma_commit_if(on, done);
      dev::mbar_wait_clk(done, 0, nullptr, 1ll << 28);
    }
    __syncwarp();
  } else if (warp < 8) {
    // ============================ softmax rows =================================
    reg_inc<T::FP8>();
    const int x = warp >> 2, quarter = warp & 3;
    const int r = 32 * quarter + lane;  // this thread's row of tile x: its TMEM lane
    const uint32_t lane_addr = (uint32_t)(32 * quarter) << 16;
    const uint32_t ts0 = tbase + x * 2 * kHalf + lane_addr, to = tbase + 4 * kHalf + x * D + lane_addr;
    uint8_t* qs = smem + T::Q + x * T::TILE;
    uint32_t sc = 0;  // half tiles done
    uint64_t poly2[5];
#pragma unroll
    for (int i = 0; i < 5; ++i) poly2[i] = dev::f2(p.mod.poly[i], p.mod.poly[i]);
    int gv = 0;  // key tiles before this unit (the V ring's position)
    bool ok = true;
    auto wait_ok = [&](uint64_t* bar, uint32_t parity) {
      if (ok) ok = __all_sync(0xffffffffu, dev::mbar_wait_clk(bar, parity, p.err));
    };
    for (int n = 0;; ++n) {
      Unit u;
      read_unit(n, u, ok);
      ok = __all_sync(0xffffffffu, ok);
      __syncwarp();
      if (lane == 0) dev::mbar_arrive(&uq_empty[n % kUQ]);
      if (!ok || u.s < 0) break;
      const Tiles<BS> tl(u, p);
      const int na = min(u.qn, QB);
      const int px = u.p0 + x * QB, nx = x ? u.qn - na : na;  // this tile's positions
      const Seen seen(tl, px, nx);
      const bool valid = r < nx * G;
      const int pos = px + r / G;
      const int qh = u.h * G + r % G;
      float scale = p.scale_log2, cap_in = p.mod.cap_in, osc = p.out_scale, slope = 0.f;
      if constexpr (T::FP8) {
        const int head = u.h / p.mod.sub;
        if (p.k_head) {
          const float ks = __ldg(p.k_head + head);
          scale *= ks;
          cap_in *= ks;
        }
        if (p.v_head) osc *= __ldg(p.v_head + head);
        // the queries as f16, in place, each row by a power of two that keeps
        // it in f16's range (its scores' factors take it back)
        wait_ok(q_raw, (uint32_t)(n & 1));
        uint32_t most = 0;
#pragma unroll 4  // (whole, its registers spill others': two 1024-row chunks 350 us, so 344)
        for (int v = 0; v < T::NCH * 8; ++v) {
          const uint4 b = *reinterpret_cast<const uint4*>(qs + (v >> 3) * kTileRow + r * 128 + (v & 7) * 16);
          most = dev::max_bf16_bits(dev::max_bf16_bits(most, b.x), b.y);
          most = dev::max_bf16_bits(dev::max_bf16_bits(most, b.z), b.w);
        }
        float up, down;
        dev::f16_row_scale(most, up, down);
        scale *= down;
        cap_in *= down;
#pragma unroll
        for (int v = 0; v < T::NCH * 8; ++v) {
          uint4* w = reinterpret_cast<uint4*>(qs + (v >> 3) * kTileRow + r * 128 + (v & 7) * 16);
          uint4 b = *w;
          uint32_t* e = &b.x;
#pragma unroll
          for (int i = 0; i < 4; ++i)
            e[i] = dev::pack_f16(dev::bf16_bits_to_f32(e[i] & 0xFFFFu) * up, dev::bf16_bits_to_f32(e[i] >> 16) * up);
          *w = b;
        }
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncwarp();
        if (lane == 0) dev::mbar_arrive(q_full);
      }
      if constexpr (SLOPES) {
        if (valid) slope = __ldg(p.mod.slopes + qh) * 1.4426950408889634f;
      }
      // y = x * y_in is what the cap's tanh takes (a row past the unit holds
      // anything and must not ask for the exact form)
      const float y_in = valid ? cap_in * (0.5f / 1.4426950408889634f) : 0.f;
      // Halves that are plain to every row of this warp: each of their keys is
      // seen and none lies past a row's position: h < ppre, or pbeg <= h < pend
      const int rlo = min(32 * quarter, max(0, nx * G - 1)), rhi = min(32 * quarter + 31, max(0, nx * G - 1));
      const int pmin = px + rlo / G, pmax = px + rhi / G;
      const int pend = (min(pmin + 1, u.len)) / kHalf;
      const int pbeg = tl.window > 0 ? (max(0, pmax - tl.window + 1) + kHalf - 1) / kHalf : 0;
      const int ppre = (SLOPES ? min(u.pfx, pmin + 1) : u.pfx) / kHalf;
      float ref = -1e30f, lsum = 0.f;
      bool first = true;
      int h = tl.first_half();
      for (int j = 0; j < 2 * tl.nt;) {
        if (!seen(h)) {
          ++j;
          h = tl.next_half(h);
          continue;
        }
        // the plain halves from here on, one under the other
        int run = 0;
        if (!first) {
          if (h >= pbeg && h < pend) run = h + 1 - max(pbeg, tl.gap > 0 && h >= 2 * (tl.npt + tl.gap) ? 2 * (tl.npt + tl.gap) : 0);
          else if (h < ppre) run = h + 1;
          run = min(run, 2 * tl.nt - j);
        }
        bool landed = false;  // the scores of half h have been waited for
        const bool ran = run > 0;
        for (float dist = (float)(pos - h * kHalf); run > 0; --run, dist += (float)kHalf) {
          const uint32_t b = sc & 1, ts = ts0 + b * kHalf;
          wait_ok(&s_full[2 * x + b], (sc >> 1) & 1);
          dev::tc_fence_after();
          // Weights over the reference in hand, kept in registers until they
          // are known to be in range (the scores are needed again if not).
          // Arithmetic on pairs: with two warps per SM sub-partition issue
          // slots count as much as the exponentials.
          uint32_t pk[kHalf / 2];
          uint64_t sum2 = 0;
          float z2[2] = {0.f, 0.f};
          const uint64_t in = CAPS ? dev::f2(y_in, y_in) : dev::f2(scale, scale);
          const uint64_t step = dev::f2(2.f * slope, 2.f * slope);
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            uint32_t w[32];
            dev::tmem_ld32(ts + 32 * c, w);
            const float base = SLOPES ? fmaf(-slope, dist - (float)(32 * c), -ref) : -ref;
            uint64_t off = dev::f2(base, SLOPES ? base + slope : base);
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              const uint64_t v = dev::f2(__uint_as_float(w[2 * i]), __uint_as_float(w[2 * i + 1]));
              uint64_t a;
              if constexpr (CAPS) {
                const uint64_t y = dev::mul2(v, in), z = dev::mul2(y, y);
                float z0, z1;
                dev::f2_split(z, z0, z1);
                z2[i & 1] = dev::max3(z2[i & 1], z0, z1);
                uint64_t q = dev::fma2(z, poly2[4], poly2[3]);
                q = dev::fma2(z, q, poly2[2]);
                q = dev::fma2(z, q, poly2[1]);
                q = dev::fma2(z, q, poly2[0]);
                a = dev::fma2(y, q, off);
              } else {
                a = dev::fma2(v, in, off);
              }
              if (SLOPES) off = dev::add2(off, step);
              float e0, e1;
              dev::f2_split(a, e0, e1);
              e0 = dev::ex2(e0);
              e1 = dev::ex2(e1);
              sum2 = dev::add2(sum2, dev::f2(e0, e1));
              pk[16 * c + i] = T::FP8 ? dev::pack_f16(e0, e1) : dev::pack_bf16(e0, e1);
            }
          }
          float sum, odd;
          dev::f2_split(sum2, sum, odd);
          sum += odd;
          landed = __any_sync(0xffffffffu, valid && (!(sum <= T::BIG) ||
                                                      (CAPS && !(fmaxf(z2[0], z2[1]) <= kCapFast * kCapFast))));
          if (landed) break;  // out of range: the long way below
          lsum += sum;
          dev::tmem_st32(ts, pk);
          dev::tc_fence_before();
          __syncwarp();
          if (lane == 0) dev::mbar_arrive(&p_full[2 * x + b]);
          ++sc;
          ++j;
          --h;
        }
        if (ran && !landed) {
          if (tl.gap > 0 && h == 2 * (tl.npt + tl.gap) - 1) h = 2 * tl.npt - 1;
          continue;
        }
        const uint32_t b = sc & 1, ts = ts0 + b * kHalf;
        if (!landed) {
          wait_ok(&s_full[2 * x + b], (sc >> 1) & 1);
          dev::tc_fence_after();
        }
        const int key0 = h * kHalf;
        const float dist = (float)(pos - key0);
        // The first step of a unit, a step with hidden keys, or weights (a
        // score) that left the fast form's range: the row max, then the
        // weights, 16 keys at a time over scores already read.  Rolled loops:
        // this path is taken a few times per unit, and what it costs is
        // above all fetching its instructions.
        // The row sees keys [wlo, hi) and [0, pl) of the half tile, a bit each.
        const int hi = valid ? min(pos + 1, u.len) - key0 : 0;
        const int wlo = tl.window > 0 ? pos - tl.window + 1 - key0 : 0;
        const int pl = valid ? u.pfx - key0 : 0;
        auto below = [](int n) { return n <= 0 ? 0ull : n >= 64 ? ~0ull : (1ull << n) - 1ull; };
        const uint64_t vis = below(pl) | (below(hi) & ~below(wlo));
        // 16 scores -> exponents s - rf in log2 units: masks, keys past the
        // row's position (their distance has the other sign), and with
        // `exact` the cap's exact form
        // the capped pair (y P(y^2)) of two raw scores
        auto cap2 = [&](float x0, float x1, uint64_t& z) {
          const uint64_t y = dev::mul2(dev::f2(x0, x1), dev::f2(y_in, y_in));
          z = dev::mul2(y, y);
          uint64_t q = dev::fma2(z, poly2[4], poly2[3]);
          q = dev::fma2(z, q, poly2[2]);
          q = dev::fma2(z, q, poly2[1]);
          q = dev::fma2(z, q, poly2[0]);
          return dev::mul2(y, q);
        };
        auto args = [&](int c, float (&a)[16], float rf, bool exact, float& zmax) {
          uint32_t w[16];
          dev::tmem_ld16(ts + 16 * c, w);
          const uint32_t v = (uint32_t)(vis >> (16 * c));
          const float d = dist - (float)(16 * c);
#pragma unroll
          for (int i = 0; i < 16; ++i)  // (what a hidden key holds must not choose the cap's form)
            a[i] = !CAPS || (v & (1u << i)) ? __uint_as_float(w[i]) : 0.f;
          if constexpr (CAPS) {
            if (exact) {
#pragma unroll
              for (int i = 0; i < 16; ++i) a[i] = dev::capped(a[i], cap_in, p.mod.cap_out);
            } else {
#pragma unroll
              for (int i = 0; i < 16; i += 2) {
                uint64_t z;
                const uint64_t y = cap2(a[i], a[i + 1], z);
                if (SLOPES) {  // (without slopes the raw maximum has decided)
                  float z0, z1;
                  dev::f2_split(z, z0, z1);
                  zmax = dev::max3(zmax, z0, z1);
                }
                dev::f2_split(y, a[i], a[i + 1]);
              }
            }
          }
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const float off = SLOPES ? fmaf(-slope, fabsf(d - (float)i), -rf) : -rf;
            a[i] = (v & (1u << i)) ? (CAPS ? a[i] + off : fmaf(a[i], scale, off)) : -INFINITY;
          }
        };
        bool exact = false;
        float m, zmax = 0.f;
        if constexpr (!SLOPES) {
          // scale and cap are monotone: the raw maximum decides (and with the
          // raw minimum whether the cap's polynomial serves)
          float hi_raw = -INFINITY, lo_raw = INFINITY;
#pragma unroll 1
          for (int c = 0; c < kHalf / 16; ++c) {
            uint32_t w[16];
            dev::tmem_ld16(ts + 16 * c, w);
            const uint32_t v = (uint32_t)(vis >> (16 * c));
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              const float x = __uint_as_float(w[i]);
              hi_raw = fmaxf(hi_raw, (v & (1u << i)) ? x : -INFINITY);
              if (CAPS) lo_raw = fminf(lo_raw, (v & (1u << i)) ? x : INFINITY);
            }
          }
          if constexpr (CAPS) {
            const float most = vis ? fmaxf(fabsf(hi_raw), fabsf(lo_raw)) * y_in : 0.f;
            exact = __any_sync(0xffffffffu, !(most <= kCapFast));
            uint64_t z;
            float capped, other;
            dev::f2_split(cap2(hi_raw, 0.f, z), capped, other);
            m = !vis ? -INFINITY : exact ? dev::capped(hi_raw, cap_in, p.mod.cap_out) : capped;
          } else {
            m = hi_raw * scale;
          }
        } else {
          for (;;) {
            m = -INFINITY;
            zmax = 0.f;
#pragma unroll 1
            for (int c = 0; c < kHalf / 16; ++c) {
              float a[16];
              args(c, a, 0.f, exact, zmax);
#pragma unroll
              for (int i = 0; i < 16; i += 2) m = dev::max3(m, a[i], a[i + 1]);
            }
            if (!CAPS || exact || !__any_sync(0xffffffffu, !(zmax <= kCapFast * kCapFast))) break;
            exact = true;
          }
        }
        // the reference moves where the weights would grow past 2^8; O is
        // rescaled once the previous PV is complete
        const bool move = m > ref + 8.f;
        const float alpha = move ? dev::ex2(ref - m) : 1.f;
        if (move) ref = m;
        lsum *= alpha;
        if (!first && __any_sync(0xffffffffu, move)) {
          wait_ok(&pv_done[2 * x + (b ^ 1)], ((sc - 1) >> 1) & 1);
          dev::tc_fence_after();
#pragma unroll 1
          for (int c = 0; c < D / 16; ++c) {
            uint32_t w[16];
            dev::tmem_ld16(to + 16 * c, w);
#pragma unroll
            for (int i = 0; i < 16; ++i) w[i] = __float_as_uint(__uint_as_float(w[i]) * alpha);
            dev::tmem_st16(to + 16 * c, w);
          }
        }
#pragma unroll 1
        for (int c = 0; c < kHalf / 16; ++c) {
          float a[16], s2[2] = {0.f, 0.f};
          args(c, a, ref, exact, zmax);
          uint32_t pk[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const float e0 = dev::ex2(a[2 * i]), e1 = dev::ex2(a[2 * i + 1]);
            s2[i & 1] += e0 + e1;
            pk[i] = T::FP8 ? dev::pack_f16(e0, e1) : dev::pack_bf16(e0, e1);
          }
          lsum += s2[0] + s2[1];
          dev::tmem_st8(ts + 8 * c, pk);
        }
        if constexpr (!T::FP8) {
          // V rows that no row of the unit sees may hold anything (0 * NaN):
          // each query tile zeroes them before its own PV (neither waits for
          // the other's)
          auto zero_v = [&](int z0, int z1) {
            if (z0 >= z1) return;
            const int gg = gv + (j >> 1);
            wait_ok(&vfull[gg % T::NV], (uint32_t)((gg / T::NV) & 1));
            uint8_t* vt = smem + T::V + (gg % T::NV) * T::TILE + (1 - (j & 1)) * kHalf * 128;
            for (int i = tid & 127; i < (z1 - z0) * T::NCH * 8; i += 128) {
              const int key = z0 + i / (T::NCH * 8), rest = i % (T::NCH * 8);
              *reinterpret_cast<uint4*>(vt + (rest >> 3) * kTileRow + key * 128 + (rest & 7) * 16) =
                  make_uint4(0, 0, 0, 0);
            }
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
          };
          zero_v(max(0, max(u.len, u.pfx) - key0), min(kHalf, tl.nb * BS - key0));
          zero_v(max(u.pfx, key0) - key0, min(tl.lo, key0 + kHalf) - key0);
        }
        first = false;
        dev::tc_fence_before();
        __syncwarp();
        if (lane == 0) dev::mbar_arrive(&p_full[2 * x + b]);
        ++sc;
        ++j;
        h = tl.next_half(h);
      }
      gv += tl.nt;
      // ---- O / sum -> the output row; then O is free ----
      const int64_t at = ((int64_t)(u.row0 + x * QB + r / G) * hq + qh) * D;
      uint4* dst = reinterpret_cast<uint4*>(p.out + at * 2);
      if (u.parts > 1) {
        // this part's rows, lane by lane side by side, then the join
        const int64_t slot = ((int64_t)u.unit * parts + u.part) * 8 + warp;
        float2* ml = reinterpret_cast<float2*>(p.part_ml) + slot * 32 + lane;
        float4* po = reinterpret_cast<float4*>(p.part_o) + slot * (D / 4) * 32 + lane;
        if (!first) {
          wait_ok(&pv_done[2 * x + ((sc - 1) & 1)], ((sc - 1) >> 1) & 1);
          dev::tc_fence_after();
#pragma unroll 1
          for (int c = 0; c < D / 16; ++c) {
            uint32_t w[16];
            dev::tmem_ld16(to + 16 * c, w);
#pragma unroll
            for (int i = 0; i < 4; ++i)
              __stcg(po + (4 * c + i) * 32, make_float4(__uint_as_float(w[4 * i]), __uint_as_float(w[4 * i + 1]),
                                                        __uint_as_float(w[4 * i + 2]), __uint_as_float(w[4 * i + 3])));
          }
          dev::tc_fence_before();
          __syncwarp();
          if (lane == 0) dev::mbar_arrive(&o_free[x]);
        }
        __stcg(ml, make_float2(ref, lsum));  // (no tile: the starting reference, 0)
        __threadfence();
        __syncwarp();
        unsigned int* cnt = p.part_cnt + (int64_t)u.unit * 8 + warp;
        int last = 0;
        if (lane == 0) last = ok && atomicAdd(cnt, 1u) == (unsigned)u.parts - 1u;
        last = __shfl_sync(0xffffffffu, last, 0);
        if (last) {
          __threadfence();
          const float2* pml = reinterpret_cast<const float2*>(p.part_ml) + ((int64_t)u.unit * parts * 8 + warp) * 32 + lane;
          const float4* pp = reinterpret_cast<const float4*>(p.part_o) +
                             ((int64_t)u.unit * parts * 8 + warp) * (D / 4) * 32 + lane;
          float M = -1e30f, L = 0.f, wt[kMaxParts];
#pragma unroll
          for (int q = 0; q < kMaxParts; ++q)
            if (q < u.parts) M = fmaxf(M, __ldcg(pml + q * 8 * 32).x);
#pragma unroll
          for (int q = 0; q < kMaxParts; ++q) {
            wt[q] = 0.f;
            if (q < u.parts) {
              const float2 v = __ldcg(pml + q * 8 * 32);
              if (v.x > -1e29f) wt[q] = dev::ex2(v.x - M);  // (a row without a tile there left no O)
              L = fmaf(v.y, wt[q], L);
            }
          }
          const float inv = L > 0.f ? osc / L : (L == 0.f ? 0.f : L);
#pragma unroll 1
          for (int c = 0; c < D / 16; ++c) {  // (all parts' loads of a chunk are in flight together)
            float4 o[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) o[i] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int q = 0; q < kMaxParts; ++q) {
              if (q >= u.parts || wt[q] == 0.f) continue;
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const float4 v = __ldcg(pp + ((int64_t)q * 8 * (D / 4) + 4 * c + i) * 32);
                o[i].x = fmaf(v.x, wt[q], o[i].x);
                o[i].y = fmaf(v.y, wt[q], o[i].y);
                o[i].z = fmaf(v.z, wt[q], o[i].z);
                o[i].w = fmaf(v.w, wt[q], o[i].w);
              }
            }
            uint32_t out[8];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              out[2 * i] = dev::pack_bf16(o[i].x * inv, o[i].y * inv);
              out[2 * i + 1] = dev::pack_bf16(o[i].z * inv, o[i].w * inv);
            }
            if (valid && ok) dev::store32(dst + 2 * c, out);
          }
          if (lane == 0) *cnt = 0u;  // ready for the next call
        }
      } else if (!first) {
        wait_ok(&pv_done[2 * x + ((sc - 1) & 1)], ((sc - 1) >> 1) & 1);
        dev::tc_fence_after();
        const float inv = lsum > 0.f ? osc / lsum : (lsum == 0.f ? 0.f : lsum);  // nothing visible: 0; NaN stays
#pragma unroll
        for (int c = 0; c < D / 32; ++c) {
          uint32_t w[32];
          dev::tmem_ld32(to + 32 * c, w);
          if (valid && ok) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              uint32_t o[8];
#pragma unroll
              for (int e = 0; e < 8; ++e)
                o[e] = dev::pack_bf16(__uint_as_float(w[16 * i + 2 * e]) * inv, __uint_as_float(w[16 * i + 2 * e + 1]) * inv);
              dev::store32(dst + 4 * c + 2 * i, o);
            }
          }
        }
        dev::tc_fence_before();
        __syncwarp();
        if (lane == 0) dev::mbar_arrive(&o_free[x]);
      } else if (valid && ok) {  // no tile at all
#pragma unroll
        for (int i = 0; i < D / 8; ++i) dst[i] = make_uint4(0, 0, 0, 0);
      }
    }
  } else if (T::FP8 && warp >= kConvWarp) {
    // ==================== e4m3 -> f16 tiles ====================================
    if constexpr (T::FP8) {
      reg_dec<true>();
      const int ct = tid - 32 * kConvWarp;  // 0..127
      bool ok = true;
      int g = 0;   // tiles of K (and of V) converted
      int rst = 0;
      uint32_t rph = 0;
      auto wait_ok = [&](uint64_t* bar, uint32_t parity) {
        if (ok) ok = __all_sync(0xffffffffu, dev::mbar_wait_clk(bar, parity, p.err));
      };
      auto to_f16 = [&](const uint4& b, uint4& lo, uint4& hi) {
        dev::e4m3x4_to_f16x2(b.x, lo.x, lo.y);
        dev::e4m3x4_to_f16x2(b.y, lo.z, lo.w);
        dev::e4m3x4_to_f16x2(b.z, hi.x, hi.y);
        dev::e4m3x4_to_f16x2(b.w, hi.z, hi.w);
      };
      for (int n = 0;; ++n) {
        Unit u;
        read_unit(n, u, ok);
        ok = __all_sync(0xffffffffu, ok);
        __syncwarp();
        if (lane == 0) dev::mbar_arrive(&uq_empty[n % kUQ]);
        if (!ok || u.s < 0) break;
        const Tiles<BS> tl(u, p);
        for (int k = 0; k < tl.nt; ++k, ++g) {
          const int key0 = tl.tile(k) * kKeys;
          const int ring = g % 2;
          const uint32_t par = (uint32_t)((g / 2) & 1);
          static_assert(T::NK == 2 && T::NV == 2, "rings of two");
          // ---- K: rows of D bytes -> rows of D f16, 64-element chunks
          wait_ok(&rfull[rst], rph);
          if (g >= 2) wait_ok(&kempty[ring], par ^ 1u);
          {
            const uint8_t* raw = smem + T::R + rst * T::RAW;
            uint8_t* out = smem + T::K + ring * T::TILE;
#pragma unroll
            for (int i = 0; i < T::RAW / 16 / 128; ++i) {
              const int idx = i * 128 + ct, key = idx / (D / 16), pc = idx % (D / 16);
              uint4 a, b;
              to_f16(*reinterpret_cast<const uint4*>(raw + idx * 16), a, b);
              uint8_t* row = out + (pc >> 2) * kTileRow + key * 128;
              *reinterpret_cast<uint4*>(row + (((2 * (pc & 3)) ^ (key & 7)) << 4)) = a;
              *reinterpret_cast<uint4*>(row + (((2 * (pc & 3) + 1) ^ (key & 7)) << 4)) = b;
            }
          }
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
          __syncwarp();
          if (lane == 0) {
            dev::mbar_arrive(&kfull[ring]);
            dev::mbar_arrive(&rempty[rst]);
          }
          if (++rst == T::NR) {
            rst = 0;
            rph ^= 1u;
          }
          // ---- V: blocks [D][BS] -> rows of d, keys contiguous, 64-key chunks;
          // keys that no row of the unit sees become 0 (0 * NaN)
          wait_ok(&rfull[rst], rph);
          if (g >= 2) wait_ok(&vempty[ring], par ^ 1u);
          {
            const uint8_t* raw = smem + T::R + rst * T::RAW;
            uint8_t* out = smem + T::V + ring * T::TILE;
            const int d = ct % D;
            // keys [0, za) and [zb, ze) of the tile are seen
            const int za = u.pfx - key0, zb = tl.lo - key0, ze = min(tl.kend, tl.nb * BS) - key0;
#pragma unroll
            for (int i = 0; i < 8 * D / 128; ++i) {
              const int kg = i * (128 / D) + ct / D;  // 16 keys
              const int jb = kg * 16 / BS, off = kg * 16 % BS;
              uint4 a, b;
              to_f16(*reinterpret_cast<const uint4*>(raw + jb * BS * D + d * BS + off), a, b);
              const int f = kg * 16;
              if (!((f + 16 <= za) || (f >= zb && f + 16 <= ze))) {
                uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                  const int k0 = f + 2 * e, k1 = k0 + 1;
                  if (!(k0 < za || (k0 >= zb && k0 < ze))) w[e] &= 0xFFFF0000u;
                  if (!(k1 < za || (k1 >= zb && k1 < ze))) w[e] &= 0x0000FFFFu;
                }
                a = make_uint4(w[0], w[1], w[2], w[3]);
                b = make_uint4(w[4], w[5], w[6], w[7]);
              }
              uint8_t* row = out + (kg >> 2) * (D * 128) + d * 128;
              *reinterpret_cast<uint4*>(row + (((2 * (kg & 3)) ^ (d & 7)) << 4)) = a;
              *reinterpret_cast<uint4*>(row + (((2 * (kg & 3) + 1) ^ (d & 7)) << 4)) = b;
            }
          }
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
          __syncwarp();
          if (lane == 0) {
            dev::mbar_arrive(&vfull[ring]);
            dev::mbar_arrive(&rempty[rst]);
          }
          if (++rst == T::NR) {
            rst = 0;
            rph ^= 1u;
          }
        }
      }
    }
  }

  // ---- free TMEM once every warp is past its last tcgen05 access ----
  dev::tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    dev::tc_fence_after();
    dev::tmem_dealloc(tbase, kTmemCols);
  }
  finish_queue();
}

template <int KV, int D, int BS, int MOD>
cudaError_t launch(const PrefillParams& p, const CUtensorMap& tm_k, const CUtensorMap& tm_v, const CUtensorMap& tm_q,
                   int grid, cudaStream_t stream) {
  using T = C<KV, D, BS>;
  auto kern = chunk_biased_kernel<KV, D, BS, MOD>;
  static int set_for[64] = {0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= 64 || !set_for[dev]) {
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, T::TOTAL);
    if (e != cudaSuccess) return e;
    if (dev < 64) set_for[dev] = 1;
  }
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3(T::THREADS);
  cfg.dynamicSmemBytes = T::TOTAL;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, tm_k, tm_v, tm_q, p);
}

template <int KV, int D, int BS>
cudaError_t launch_mod(const PrefillParams& p, const CUtensorMap& tm_k, const CUtensorMap& tm_v,
                       const CUtensorMap& tm_q, int grid, cudaStream_t stream) {
  if (p.mod.cap_out > 0.f)
    return p.mod.slopes ? launch<KV, D, BS, kCapSlope>(p, tm_k, tm_v, tm_q, grid, stream)
                        : launch<KV, D, BS, kCap>(p, tm_k, tm_v, tm_q, grid, stream);
  if (p.mod.slopes) return launch<KV, D, BS, kSlope>(p, tm_k, tm_v, tm_q, grid, stream);
  return launch<KV, D, BS, kMask>(p, tm_k, tm_v, tm_q, grid, stream);
}

template <int KV>
cudaError_t launch_kv(const PrefillParams& p, const CUtensorMap& tm_k, const CUtensorMap& tm_v, const CUtensorMap& tm_q,
                      int head_dim, int block_size, int grid, cudaStream_t stream) {
  if (head_dim == 128)
    return block_size == 16 ? launch_mod<KV, 128, 16>(p, tm_k, tm_v, tm_q, grid, stream)
                            : launch_mod<KV, 128, 32>(p, tm_k, tm_v, tm_q, grid, stream);
  return block_size == 16 ? launch_mod<KV, 64, 16>(p, tm_k, tm_v, tm_q, grid, stream)
                          : launch_mod<KV, 64, 32>(p, tm_k, tm_v, tm_q, grid, stream);
}

}  // namespace

cudaError_t launch_chunk_biased(const PrefillParams& p_in, const CUtensorMap& tm_k, const CUtensorMap& tm_v,
                                const CUtensorMap& tm_q, int kv, int head_dim, int block_size, int num_tokens,
                                int num_sms, int ahead, bool front, cudaStream_t stream) {
  PrefillParams p = p_in;
  if (p.group < 1 || p.group > kRows || p.rows.num_seqs > kGroup * kMaxGroups) return cudaErrorNotSupported;
  for (int i = 0; i < 5; ++i) p.mod.poly[i] = kTanh[i] * p.mod.cap_out;
  static_assert(kRows == 128, "chunk_biased_units counts query tiles of 128 rows");
  const int64_t bound = chunk_biased_units(num_tokens, p.rows.num_seqs, p.group, p.num_kv_heads);
  if (bound <= 0) return cudaSuccess;
  if (bound >= INT32_MAX) return cudaErrorNotSupported;
  // units are cut into at most kMaxParts parts each
  const int64_t most = p.part_slots > 0 ? bound * kMaxParts : bound;
  const int rest = (int)(most < num_sms ? most : num_sms), first = (int)(most < ahead ? most : ahead);
  const int grid = front ? first : rest;
  p.exits = first + rest;
  if (front) p.after_decode = 0;
  return kv == kBF16 ? launch_kv<kBF16>(p, tm_k, tm_v, tm_q, head_dim, block_size, grid, stream)
                     : launch_kv<kFP8>(p, tm_k, tm_v, tm_q, head_dim, block_size, grid, stream);
}

}  // namespace pa

// Internal: kernel parameter blocks and launchers (host <-> device contract).
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace pa {

// dtype codes match pa_dtype in pa.h
enum : int { kF32 = 0, kBF16 = 1, kFP8 = 2 };

struct CacheWriteParams {
  const uint8_t* k_new;
  const uint8_t* v_new;
  const int64_t* slots;
  uint8_t* k_cache;
  uint8_t* v_cache;
  int32_t num_tokens, num_kv_heads, head_dim, block_size;
  int64_t num_slots;  // num_blocks * block_size
  float k_scale, v_scale;
  const float* k_head;  // per-kv-head scales (device) or nullptr: k_scale / v_scale
  const float* v_head;
};
cudaError_t launch_cache_write(const CacheWriteParams& p, int in_dtype, int kv_dtype, cudaStream_t stream);

// Division of n < 2^31 by a fixed d >= 1 as a multiplication (Granlund and
// Montgomery, "Division by Invariant Integers using Multiplication", PLDI
// 1994): the quotient is (umulhi(n, mul) + n) >> shift (mul = floor(2^32 (2^shift -
// d) / d) + 1 with shift = ceil(log2 d)).
struct FastDiv {
  uint32_t mul, shift, d;
};
inline FastDiv fast_div(uint32_t d) {
  FastDiv f = {0, 0, d};
  while (f.shift < 31 && (1u << f.shift) < d) ++f.shift;
  f.mul = (uint32_t)((((uint64_t)1 << 32) * (((uint64_t)1 << f.shift) - d)) / d + 1);
  return f;
}

// pa_norm_rope_write: norms, rotation and cache write of a step's new rows.
struct NormRopeParams {
  const uint8_t* q;
  const uint8_t* k;
  const uint8_t* v;
  int64_t q_stride, k_stride, v_stride;  // elements between tokens
  const uint8_t* q_weight;               // [head_dim] or nullptr: no norm of the queries
  const uint8_t* k_weight;               // [head_dim] or nullptr: no norm of the keys
  float eps;
  const float* cos_sin;  // [num_positions][rot_dim] or nullptr: no rotation
  int32_t num_positions, rot_dim, interleaved;
  const int32_t* positions;
  const int64_t* slots;
  uint8_t* q_out;
  uint8_t* k_cache;
  uint8_t* v_cache;
  int32_t num_tokens, num_q_heads, num_kv_heads, head_dim, block_size;
  int64_t num_slots;
  float k_scale, v_scale;
  const float* k_head;  // per-kv-head scales (device) or nullptr: k_scale / v_scale
  const float* v_head;
  int32_t bs_shift;      // log2 of block_size
  FastDiv per_token;     // the launch's: row groups of a token
  FastDiv heads;         // the launch's: num_kv_heads
};
cudaError_t launch_norm_rope_write(const NormRopeParams& p, int q_dtype, int kv_dtype, int num_sms,
                                   cudaStream_t stream);

// pa_cache_read: rows of given slots out of the pools.
struct CacheReadParams {
  const int64_t* slots;
  const uint8_t* k_cache;
  const uint8_t* v_cache;
  uint8_t* k_out;
  uint8_t* v_out;
  int32_t num_tokens, num_kv_heads, head_dim, block_size;
  int64_t num_slots;
  float k_scale, v_scale;
  const float* k_head;  // per-kv-head scales (device) or nullptr: k_scale / v_scale
  const float* v_head;
  int32_t bs_shift;      // log2 of block_size
  FastDiv heads;         // num_kv_heads
};
cudaError_t launch_cache_read(const CacheReadParams& p, int q_dtype, int kv_dtype, int num_sms, cudaStream_t stream);

// Whole-block copies inside both pools (copy-on-write): K and V block dst[i]
// become copies of block src[i]; pairs with an id outside [0, num_blocks)
// or src == dst are skipped.
struct CopyBlocksParams {
  const int32_t* src;
  const int32_t* dst;
  int32_t n;
  int32_t num_blocks;
  int64_t block_bytes;  // bytes of one block of one pool
  uint8_t* k_cache;
  uint8_t* v_cache;
};
cudaError_t launch_copy_blocks(const CopyBlocksParams& p, int num_sms, cudaStream_t stream);

// Rows of a decode or mixed step.  Sequence s owns query rows
// qsl[s] .. qsl[s+1]-1 (qsl == nullptr: exactly row s), the last of which
// sits at position seq_lens[s] - 1.
struct AttnRows {
  const int32_t* seq_lens;
  const int32_t* qsl;
  int32_t num_seqs;
  int32_t num_rows;
};

// What the biased attention (pa_decode_biased and the mixed step's form) does
// to the scores of a row at position i: s = cap * tanh(scale q k / cap), minus
// slope * |i - j|; key j is visible if j < prefix, or j <= i and, with a
// window, i - j < window.
struct ScoreMod {
  float cap_in, cap_out;  // 2 log2(e) scale / cap and log2(e) cap: see capped(); cap_out 0: no cap
  int32_t window;         // 0: none
  const float* slopes;    // [num_q_heads] (device) or nullptr
  const int32_t* prefix;  // [num_seqs] (device) or nullptr
  float poly[5];          // the chunk kernel's: cap_out times its tanh polynomial
  int32_t sub;            // kernel kv heads per pool kv head (a group too large for the kernel is cut)
};

// Workspace carve-up of the split-K decode kernel.
struct DecodeWorkspace {
  int32_t* err;             // error word (first 4 bytes of the caller's buffer)
  unsigned int* cnt;        // [num_seqs * num_kv_heads] arrival counters: zero between calls
  float* ml;                // [workers][G][2] partial (max, sum), one cut piece per warp
  float* o;                 // [workers][G][D] partial unnormalised outputs
};

struct DecodeParams {
  const uint8_t* q;  // bf16 [rows][Hq][D]
  uint8_t* out;      // bf16 [rows][Hq][D]
  const uint8_t* v_cache;
  const int32_t* block_tables;
  int32_t max_blocks;
  AttnRows rows;
  int32_t num_q_heads, num_kv_heads, group;
  int32_t num_blocks;  // table entries outside [0, num_blocks) are flagged and read as block 0
  int32_t nstages;
  int32_t grid;
  float scale_log2;  // softmax scale * log2(e), times the per-tensor K dequant factor for fp8
  float out_scale;   // 1, or the per-tensor V dequant factor for fp8
  const float* k_head;  // fp8 per-kv-head scales (device; they multiply scale_log2 / out_scale) or nullptr
  const float* v_head;
  // fused cache write (pa_decode_fused): the new token's rows [rows][Hkv][D]
  // (bf16) and the pools to store them in; k_new == nullptr: no write
  const uint8_t* k_new;
  const uint8_t* v_new;
  uint8_t* k_pool;
  uint8_t* v_pool;
  float k_scale_w, v_scale_w;  // per-tensor quantisation scales of the write (fp8)
  // shared prefixes (pa_decode_prefix; pfx_of == nullptr: none): sequence s
  // with pfx_of[s] = p >= 0 skips the first pfx_blocks[p] blocks of its row
  // and folds the chunk partials of member slot pfx_slot[s] into its result
  const int32_t* pfx_of;
  const int32_t* pfx_slot;
  const int32_t* pfx_blocks;
  const float* pfx_ml;  // [chunks][num_members][Hq][2]
  const float* pfx_o;   // [chunks][num_members][Hq][D]
  int32_t pfx_members;
  int32_t pfx_chunk_blocks;  // blocks per prefix chunk (prefix_chunk_keys / block_size)
  ScoreMod mod;              // the biased kernel's
  int32_t beside_chunks;     // the biased kernel's: launched behind chunk CTAs that run beside it
  DecodeWorkspace ws;
};

// kv: kBF16 or kFP8; returns cudaErrorNotSupported for unsupported shapes.
cudaError_t launch_decode_tc(const DecodeParams& p, const CUtensorMap& tm_k, const CUtensorMap& tm_v,
                             int kv, int head_dim, int block_size, int num_sms, cudaStream_t stream);
// The same with p.mod applied; groups 1..8, head_dim 64 and 128 for both
// pools.  p.num_kv_heads counts kernel kv heads (mod.sub per pool kv head).
cudaError_t launch_decode_biased(const DecodeParams& p, const CUtensorMap& tm_k, const CUtensorMap& tm_v,
                                 int kv, int head_dim, int block_size, int num_sms, cudaStream_t stream);
size_t decode_tc_smem_bytes(int kv, int head_dim, int block_size, int group, int num_seqs, int nstages);
int decode_tc_workers(int num_sms);  // the most worker warps a launch can have (workspace sizing)
size_t decode_tc_workspace_bytes(int num_seqs, int num_kv_heads, int group, int head_dim, int num_sms);

// Prompt rows (q_len > 1) of a mixed step on the tensor-core path.
struct PrefillParams {
  const uint8_t* q;  // bf16 [rows][Hq][D]
  uint8_t* out;      // bf16 [rows][Hq][D]
  const int32_t* block_tables;
  int32_t max_blocks;
  AttnRows rows;  // qsl required
  int32_t num_q_heads, num_kv_heads, group, num_blocks;
  int32_t nstages;    // ring stages (the tcgen05 kernel: K stages)
  int32_t nstages_v;  // the tcgen05 kernel's V stages
  float scale_log2;
  int32_t* err;  // workspace error word
  // the tcgen05 kernel's unit queue: a claim counter and a count of CTAs
  // done, both zero between launches (workspace header words 2 and 3)
  int32_t* unit_ctr;
  int32_t* unit_exit;
  int32_t after_decode;  // 1: launched right behind this step's decode kernel
  // Shared-prefix mode of the tcgen05 kernel (pa_decode_prefix): units are
  // (prefix, kv head, tile of members, chunk of prefix keys) and each writes
  // partial (max reference, sum, unnormalised O) rows instead of outputs.
  // rows.num_seqs then counts prefixes; the other rows fields are unused.
  const int32_t* pfx_start;    // [P + 1] CSR into pfx_members
  const int32_t* pfx_members;  // [M] sequence of each member slot (= its decode row)
  const int32_t* pfx_blocks;   // [P] blocks in each prefix
  int32_t num_members;         // M
  int32_t chunk_keys;          // prefix keys per unit, a multiple of 128
  float* pfx_ml;               // [chunks][M][Hq][2] (max reference, sum), log2 domain
  float* pfx_o;                // [chunks][M][Hq][D]
  ScoreMod mod;                // the biased kernel's
  int32_t singles;             // the biased kernel's: 1: single rows are units too (no decode kernel has them)
  int32_t exits;               // the biased kernel's: CTAs of this step that unit_exit counts
  // the biased kernel's cut units (part_slots 0: none are cut): counters, zero
  // between calls, [slots][8]; (reference, sum) [slots][256][2]; O [slots][256][D]
  int32_t part_slots;
  unsigned int* part_cnt;
  float* part_ml;
  float* part_o;
  const uint8_t* k_raw;        // an e4m3 pool
  const uint8_t* v_raw;
  float out_scale;             // the biased kernel's: 1, or an e4m3 pool's V scale
  const float* k_head;         // e4m3 per-kv-head scales (device) or nullptr
  const float* v_head;
};

// The split of a prefix into chunks of keys that pa_decode_prefix uses: a
// unit of the prefix kernel is (prefix, kv head, 128 / G members, chunk).
// Chunks are whole 128-key tiles, at least two, and as few as give about
// kPrefixUnits units in all: every chunk adds a partial per member row that
// the prefix kernel writes and the decode folds in one after the other, and
// measured on B200 that fold outweighs spreading the prefix over more SMs
// (a 32768-token prefix shared by 64 sequences: 91 us at about 128 units,
// 131 us at 512; a 1024-token prefix: 194 us with 256-key chunks, 237 us
// with 128).  A function of the batch's sizes alone, so the workspace size
// does not depend on the device.
constexpr int kPrefixUnits = 128;
inline int prefix_chunk_keys(int max_prefix_blocks, int block_size, int num_members, int group, int num_kv_heads) {
  const long long keys = (long long)max_prefix_blocks * block_size;
  const int per_tile = 128 / group;  // members per unit
  const long long member_tiles = num_members > per_tile ? (num_members + per_tile - 1) / per_tile : 1;
  const long long per_chunk = member_tiles * (num_kv_heads > 0 ? num_kv_heads : 1);
  const long long chunks = per_chunk >= kPrefixUnits ? 1 : (kPrefixUnits + per_chunk - 1) / per_chunk;
  const long long ck = ((keys + chunks - 1) / chunks + 127) / 128 * 128;
  return (int)(ck < 256 ? 256 : ck);
}
cudaError_t launch_prefix_umma(const PrefillParams& p, const CUtensorMap& tm_k, const CUtensorMap& tm_v,
                               int head_dim, int block_size, int num_sms, cudaStream_t stream);
bool prefill_tc_supported(int kv, int q, int head_dim, int block_size, int group);
// The same rows on tcgen05 (TMEM accumulators); cudaErrorNotSupported when
// the shape or the batch's unit table does not fit (the caller falls back).
bool prefill_umma_supported(int kv, int q, int head_dim, int block_size, int group);
// tm_q: the queries as [tokens][Hq][D] bf16, boxes of [128 / G tokens][G
// heads][64 elements] with 128-byte swizzle (one box per 64-column chunk of
// a unit's Q tile).
cudaError_t launch_prefill_umma(const PrefillParams& p, const CUtensorMap& tm_k, const CUtensorMap& tm_v,
                                const CUtensorMap& tm_q, int head_dim, int block_size, int num_tokens, int num_sms,
                                cudaStream_t stream);
// Rows of more than one per sequence with p.mod applied, any group up to 128;
// an e4m3 pool comes through k_raw and v_raw, a bf16 one through the maps.
// ahead > 0: the step launches its chunks twice, `ahead` CTAs (front) before
// its decode kernel and the rest behind it.
cudaError_t launch_chunk_biased(const PrefillParams& p, const CUtensorMap& tm_k, const CUtensorMap& tm_v,
                                const CUtensorMap& tm_q, int kv, int head_dim, int block_size, int num_tokens,
                                int num_sms, int ahead, bool front, cudaStream_t stream);
// Its units, at most: two query tiles of 128 / group positions each, per
// kernel kv head.
inline int64_t chunk_biased_units(int num_tokens, int num_seqs, int group, int heads) {
  return ((int64_t)num_tokens / (2 * (128 / group)) + num_seqs) * heads;
}
// Slots per SM for cut units (a slot: one part of one unit, 256 rows).  Two
// keep the workspace at 39 MB (head_dim 128) and leave steps of more units than
// SMs whole.
constexpr int kPartSlots = 2;
cudaError_t launch_prefill_tc(const PrefillParams& p, const CUtensorMap& tm_k, const CUtensorMap& tm_v,
                              int head_dim, int block_size, int num_tokens, cudaStream_t stream);

struct SimtParams {
  const uint8_t* q;  // [rows][Hq][D] in q dtype
  uint8_t* out;
  const uint8_t* k_cache;
  const uint8_t* v_cache;
  const int32_t* block_tables;
  int32_t max_blocks;
  AttnRows rows;
  int32_t num_q_heads, num_kv_heads, head_dim, block_size;
  float scale;
  float k_scale, v_scale;
  const float* k_head;  // fp8 per-kv-head scales (device) or nullptr: k_scale / v_scale
  const float* v_head;
  int32_t only_multi_row;  // 1: skip sequences with exactly one query row
  int32_t num_blocks;      // table entries outside [0, num_blocks) are flagged and read as block 0
  int32_t* err;            // error word of the caller's workspace
};
// Biased attention on CUDA cores (fp32 queries), of every row (qsl nullptr: one
// per sequence).
constexpr int kBiasedTileRows = 64;  // (row, head) pairs of a tile kernel's CTA
struct BiasedSimtParams {
  SimtParams a;
  ScoreMod mod;
  int32_t chunk_rows;  // rows of sequences with more than one, about: chooses the kernel that takes those
};
// Whether both kernels' grids hold the step.
inline bool biased_simt_fits(int num_rows, int num_seqs, int num_q_heads, int num_kv_heads) {
  return num_q_heads <= 65535 &&
         (int64_t)num_rows * (num_q_heads / num_kv_heads) / kBiasedTileRows + num_seqs <= INT32_MAX;
}
cudaError_t launch_attn_biased_simt(const BiasedSimtParams& p, int kv_dtype, cudaStream_t stream);
cudaError_t launch_attn_simt(const SimtParams& p, int q_dtype, int kv_dtype, cudaStream_t stream);

}  // namespace pa

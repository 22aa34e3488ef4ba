// fa_kernels.h — launch interface between the C ABI (fa_api.cu) and the
// kernel translation units.  Internal to libfa.so.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace fa {

// Watchdog codes written to the device error word: (kernel << 8) | wait site.
enum : unsigned int {
  kKernFwd = 1,
  kKernDecode = 2,
  kKernBwd = 3,
  kKernTree = 4,
  kKernCache = 5,
  kKernSelftest = 15,  // fa_watchdog_selftest
};

struct FwdParams {
  CUtensorMap tm_q;  // 4-D maps {d, N, H, B}, box {64, 128, 1, 1}, 128-byte swizzle
  CUtensorMap tm_k;
  CUtensorMap tm_v;
  void* o;
  float* lse;  // may be null
  int B, H, Nq, Nkv;
  int64_t o_sb, o_sh, o_sn;  // element strides of O
  float scale_log2;          // σ·log2(e) (FP8: also × the Q and K descale factors)
  int causal;                // query i sees keys j <= i + (Nkv − Nq); needs Nq <= Nkv
  unsigned int* err;
  float o_scale = 1.f;       // multiplies O before the 1/ℓ (FP8: the V descale factor)
  CUtensorMap tm_o;          // O as {d, N_q, H, B} (its strides), box {64, 128, 1, 1}, 128-byte swizzle
};

struct FwdF32Params {
  const float* q;
  const float* k;
  const float* v;
  float* o;
  float* lse;
  int B, H, Nq, Nkv;
  int64_t q_sb, q_sh, q_sn, k_sb, k_sh, k_sn, v_sb, v_sh, v_sn, o_sb, o_sh, o_sn;
  float scale;
  int causal;
};

struct DecodeParams {
  const void* q;  // [B,H,d] bf16 (H query heads)
  const void* k;  // [B,Hkv,N,d] bf16
  const void* v;
  void* o;        // [B,H,d] bf16
  float* lse;     // [B,H] or null
  float* part_o;  // [B,H,S,d] fp32
  float* part_ml; // [B,H,S,2] fp32: (m in log2 units, ℓ)
  int B, H, Nkv, n_splits, chunk;
  float scale_log2;
  unsigned int* err;
  int Hkv = 0;    // key/value heads (informational; this kernel needs Hkv = H)
  int G = 1;      // query heads per key/value head; the CUDA-core kernel handles G = 1
  // Paged cache (k, v are [num_blocks, H, block_size, d]); null block_table = contiguous.
  const int* block_table = nullptr;  // [B, max_blocks]
  const int* seq_lens = nullptr;     // [B]
  int max_blocks = 0, block_size = 0, num_blocks = 0;
  int d = 128;  // head dim: 64 or 128
};

// Device-side argument checks report with these sites in the word after the
// watchdog's, which no pipeline wait looks at: a bad page of one sequence leaves
// the others' results, and other kernels, alone.
enum : unsigned int { kSiteBadBlock = 0xE1, kSiteBadLength = 0xE2 };

// Grouped-query split-KV decode on tensor cores (fa_decode_tc.cu).
struct DecodeTcParams {
  CUtensorMap tm_q;  // q viewed as [B·Hq rows, d]: 4-D map {d, B·Hq, 1, 1}, box {64, 128, 1, 1}
  CUtensorMap tm_k;  // {d, N, Hkv, B}, box {64, 128, 1, 1}; paged: {d, bs, Hkv, num_blocks}, box {64, bs, 1, 1}
  CUtensorMap tm_v;
  const int* block_table;  // paged cache only: [B, max_blocks]
  const int* seq_lens;     // paged cache only: [B]
  int max_blocks, block_size, num_blocks;
  float* part_o;     // [B,Hq,S,d] fp32
  float* part_ml;    // [B,Hq,S,2] fp32
  int B, Hq, Hkv, G, Nkv, n_splits, chunk;
  int d;             // head dim: 64 or 128
  float scale_log2;
  unsigned int* err;
};

struct BwdParams {
  CUtensorMap tm_q;   // {d, N, H, B}, box {64, 128, 1, 1}
  CUtensorMap tm_k;
  CUtensorMap tm_v;
  CUtensorMap tm_do;
  const void* q;
  const void* o;
  const void* dout;
  const float* lse;
  void* dq;
  void* dk;
  void* dv;
  float* dq_acc;      // [B,H,N,d] fp32, zeroed before the main kernel
  float* delta;       // [B,H,N]   D_i
  float* lse_log2;    // [B,H,N]   LSE·log2(e)
  int B, H, N;
  float scale;        // σ
  float scale_log2;   // σ·log2(e)
  int causal;         // key j visible to query i when j <= i
  unsigned int* err;
  CUtensorMap tm_dk;  // dK, dV as {d, N, H, B}, box {64, 128, 1, 1}, 128-byte swizzle (TMA stores)
  CUtensorMap tm_dv;
};

// Rotary positions of q and k (fa_rope.cu).
struct RopeParams {
  const void* q;
  const void* k;        // null with Hk = 0
  void* q_out;
  void* k_out;
  const int32_t* positions;  // positions[b·pos_stride_b + n], or null for n
  int64_t pos_stride_b;
  int64_t sq[3], sk[3], sqo[3], sko[3];  // element strides (b, h, n)
  int B, Hq, Hk, N, d, rot;
  int rot_cols, copy_cols, heads_per_thread, q_groups;  // set by the launcher
  int64_t position0;
  float magnitude, sign;
  uint64_t turns[128];  // w_i / 2π as 64-bit fractions of a turn
};

// Paged cache writes and reads (fa_cache.cu).
struct CacheParams {
  void* k_rows;  // [B, Hkv, N, d] bf16, read by the append and written by the gather
  void* v_rows;
  int64_t sk[3], sv[3];  // their element strides (b, h, n)
  void* k_cache;  // [num_blocks, Hkv, block_size, d] bf16 or E4M3
  void* v_cache;
  uint8_t* k_scale;  // E4M3: [num_blocks, Hkv, block_size] E8M0 bytes
  uint8_t* v_scale;
  const int* block_table;  // [B, max_blocks]
  const int* start;        // append: logical position of the first new token
  const int* lens;         // append: new tokens (null: N each); gather: sequence lengths
  int B, Hkv, N, num_blocks, block_size, max_blocks;
  unsigned int* err;
};

// Attention of drafted tokens over a paged cache (fa_tree.cu).
struct TreeParams {
  CUtensorMap tm_k;  // pages of one head, as for DecodeTcParams; E4M3: {d bytes, bs, Hkv, num_blocks}, box {d, bs, 1, 1}
  CUtensorMap tm_v;
  const void* q;  // bf16, element strides sq (b, h, t)
  void* o;        // bf16, so
  float* lse;     // [B, Hq, T] or null
  int64_t sq[3], so[3];
  const void* k_cache;  // [num_blocks, Hkv, block_size, d] bf16 or E4M3
  const void* v_cache;
  const uint8_t* k_scale;  // E4M3: [num_blocks, Hkv, block_size] E8M0 bytes
  const uint8_t* v_scale;
  const int* block_table;  // [B, max_blocks]
  const int* seq_lens;     // [B] keys, the drafted ones included
  const int* draft_lens;   // [B] or null (T each)
  const uint8_t* mask;     // mask[b·mask_sb + t·T + u], or null: u <= t
  int64_t mask_sb;
  int2* pieces;    // [B·Hkv]: first part of a pair and the number of parts it lies in
  float* part_o;   // [slot, tree_piece_rows(T·G), d] fp32: o/ℓ of a cut pair's pieces
  float* part_ml;  // [slot, T·G, 2] fp32: (m in log2 units, ℓ)
  int B, Hq, Hkv, G, T, num_blocks, block_size, max_blocks;
  unsigned g_magic;   // ceil(2^32 / G), for rows / G (G > 1)
  int row_tiles;      // CTA tiles of the T·G rows of a pair
  int parts;          // equal parts that the line of key tiles is cut into
  int slots_by_pair;  // a piece's slot: pair + part, else two per part
  float scale_log2;
  unsigned int* err;
};

cudaError_t launch_rope(const RopeParams& p, bool fp32, bool inter, bool in_place, cudaStream_t s);
cudaError_t launch_cache_append(const CacheParams& p, int d, bool fp8, cudaStream_t s);
cudaError_t launch_cache_gather(const CacheParams& p, int d, bool fp8, cudaStream_t s);
int tree_cta_rows(int64_t rows);  // rows one CTA takes, for T·G rows in all
constexpr int kTreeNarrowRows = 32;  // up to here a kernel of its own
// Rows of a cut pair's piece in part_o: beyond the narrow kernel whole groups of 32.
__host__ __device__ constexpr int64_t tree_piece_rows(int64_t rows) {
  return rows > kTreeNarrowRows ? (rows + 31) / 32 * 32 : rows;
}
cudaError_t launch_tree_wide(const TreeParams& p, int d, bool fp8, cudaStream_t s);  // more rows than that
cudaError_t launch_decode_tree(const TreeParams& p, int d, bool fp8, cudaStream_t s);

cudaError_t launch_fwd_bf16(int d, const FwdParams& p, cudaStream_t s);
// Unmasked bf16 forward at d = 64 with 3 or 4 query tiles of 128 rows per CTA
// (fa_fwd_d64.cu); K/V maps with 64-row boxes.
cudaError_t launch_fwd_d64_tiles(int query_tiles, const FwdParams& p, cudaStream_t s);
cudaError_t launch_fwd_fp8(int d, const FwdParams& p, cudaStream_t s);  // E4M3 Q/K/V, bf16 O
cudaError_t launch_fwd_f32(int d, const FwdF32Params& p, cudaStream_t s);
cudaError_t launch_decode_bf16(int d, const DecodeParams& p, cudaStream_t s);
cudaError_t launch_decode_merge(const DecodeParams& p, cudaStream_t s);
cudaError_t launch_decode_gqa_tc(const DecodeTcParams& p, cudaStream_t s);
cudaError_t launch_decode_paged_bf16(const DecodeParams& p, cudaStream_t s);
cudaError_t launch_decode_gqa_tc_paged(const DecodeTcParams& p, cudaStream_t s);
cudaError_t launch_bwd_bf16(int d, const BwdParams& p, cudaStream_t s, int* launches);

// Size of the library-owned decode scratch (fa_decode_splitkv_noalloc).
constexpr size_t kDecodeStaticScratchBytes = static_cast<size_t>(36) << 20;
// Device address of that scratch on the current device (looked up once per
// device and context).
cudaError_t decode_static_scratch(void** out);
// The calling thread's current CUDA context (null if the runtime has not bound
// one to the thread yet); keys the per-device caches of symbol addresses.
cudaError_t current_context(void** ctx);

}  // namespace fa

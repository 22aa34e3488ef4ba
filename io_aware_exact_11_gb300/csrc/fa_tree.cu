// fa_tree.cu — attention of T drafted tokens per sequence over a paged cache
// (T = 1: plain decode), bf16 or E4M3.
//
// Sequence b holds len keys, the last m of them those of its m ≤ T drafted
// tokens.  Token t sees every key of the context [0, len − m) and drafted key u
// where mask[t][u] is set (u ≤ t without a mask).  Rows that see nothing, the
// padding rows t ≥ m among them, give O = 0 and LSE = −∞.
//
// One warp walks one row (b, h, t) over one chunk of the keys with the online
// softmax; a second kernel joins the chunks' (m, ℓ, o) with the block-merge
// rule.
#include <cuda_fp8.h>

#include "fa_kernels.h"
#include "sm103.cuh"

namespace fa {
namespace {

constexpr int kWarps = 4;

// Lengths of sequence b, checked: keys in all and drafted keys among them.
// Lengths that cannot be are reported and taken as an empty sequence.
__device__ __forceinline__ void seq_lengths(const TreeParams& p, int b, int& len, int& drafts) {
  len = p.seq_lens[b];
  drafts = p.draft_lens != nullptr ? p.draft_lens[b] : p.T;
  if (p.draft_lens == nullptr && len == 0) drafts = 0;  // an unused batch slot
  if (drafts < 0 || drafts > p.T || len < drafts || len > static_cast<int64_t>(p.max_blocks) * p.block_size) {
    atomicCAS(p.err, 0u, (kKernTree << 8) | kSiteBadLength);
    len = drafts = 0;
  }
}

template <int D, bool FP8>
__global__ void __launch_bounds__(kWarps * 32) tree_rows_kernel(const __grid_constant__ TreeParams p) {
  constexpr int E = D / 32;
  const int lane = threadIdx.x & 31;
  const int64_t r = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5);  // (b, h, t)
  const int c = blockIdx.y;
  if (r >= static_cast<int64_t>(p.B) * p.Hq * p.T) return;
  const int t = static_cast<int>(r % p.T);
  const int64_t bh = r / p.T;
  const int h = static_cast<int>(bh % p.Hq);
  const int b = static_cast<int>(bh / p.Hq);
  const int hkv = h / p.G;
  int len, drafts;
  seq_lengths(p, b, len, drafts);
  const int context = len - drafts;
  const int chunk = (((len + p.n_splits - 1) / p.n_splits) + 127) & ~127;
  const int key0 = c * chunk, key1 = t < drafts ? min(len, key0 + chunk) : 0;

  float q[E], o[E];
  const __nv_bfloat16* qr = static_cast<const __nv_bfloat16*>(p.q) + b * p.sq[0] + h * p.sq[1] + t * p.sq[2] + lane * E;
#pragma unroll
  for (int e = 0; e < E; ++e) {
    q[e] = __bfloat162float(qr[e]) * p.scale_log2;
    o[e] = 0.f;
  }
  float m = -INFINITY, l = 0.f;
  for (int j = key0; j < key1; ++j) {
    if (j >= context) {
      const int u = j - context;
      const bool seen = p.mask != nullptr ? p.mask[b * p.mask_sb + static_cast<int64_t>(t) * p.T + u] != 0 : u <= t;
      if (!seen) continue;
    }
    int blk = p.block_table[static_cast<int64_t>(b) * p.max_blocks + j / p.block_size];
    if (blk < 0 || blk >= p.num_blocks) {
      atomicCAS(p.err, 0u, (kKernTree << 8) | kSiteBadBlock);
      blk = 0;
    }
    const int64_t row = (static_cast<int64_t>(blk) * p.Hkv + hkv) * p.block_size + j % p.block_size;
    float k[E], v[E];
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const int64_t at = row * D + lane * E + e;
      if (FP8) {
        __half_raw a = __nv_cvt_fp8_to_halfraw(static_cast<const uint8_t*>(p.k_cache)[at], __NV_E4M3);
        __half_raw w = __nv_cvt_fp8_to_halfraw(static_cast<const uint8_t*>(p.v_cache)[at], __NV_E4M3);
        k[e] = __half2float(a) * exp2f(static_cast<float>(p.k_scale[row]) - 127.f);
        v[e] = __half2float(w) * exp2f(static_cast<float>(p.v_scale[row]) - 127.f);
      } else {
        k[e] = __bfloat162float(static_cast<const __nv_bfloat16*>(p.k_cache)[at]);
        v[e] = __bfloat162float(static_cast<const __nv_bfloat16*>(p.v_cache)[at]);
      }
    }
    float s = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) s = fmaf(q[e], k[e], s);
#pragma unroll
    for (int x = 16; x > 0; x >>= 1) s += __shfl_xor_sync(0xffffffffu, s, x);
    const float m_new = fmaxf(m, s);
    const float corr = exp2f(m - m_new), w = exp2f(s - m_new);
    l = l * corr + w;
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] = o[e] * corr + w * v[e];
    m = m_new;
  }
  const int64_t slot = r * p.n_splits + c;
#pragma unroll
  for (int e = 0; e < E; ++e) p.part_o[slot * D + lane * E + e] = o[e];
  if (lane == 0) {
    p.part_ml[slot * 2] = m;
    p.part_ml[slot * 2 + 1] = l;
  }
}

// Joins a row's chunks: weights 2^(m_c − m), then O = Σ w o / Σ w ℓ.  One warp per row.
template <int D>
__global__ void __launch_bounds__(kWarps * 32) tree_merge_kernel(const __grid_constant__ TreeParams p) {
  constexpr int E = D / 32;
  const int lane = threadIdx.x & 31;
  const int64_t r = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
  if (r >= static_cast<int64_t>(p.B) * p.Hq * p.T) return;
  const int t = static_cast<int>(r % p.T);
  const int64_t bh = r / p.T;
  const int h = static_cast<int>(bh % p.Hq);
  const int b = static_cast<int>(bh / p.Hq);
  const float2* ml = reinterpret_cast<const float2*>(p.part_ml) + r * p.n_splits;
  float m = -INFINITY;
  for (int c = 0; c < p.n_splits; ++c) m = fmaxf(m, ml[c].x);
  float l = 0.f, o[E];
#pragma unroll
  for (int e = 0; e < E; ++e) o[e] = 0.f;
  for (int c = 0; c < p.n_splits; ++c) {
    const float2 x = ml[c];
    if (x.y == 0.f) continue;
    const float w = exp2f(x.x - m);
    l += w * x.y;
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] += w * p.part_o[(r * p.n_splits + c) * D + lane * E + e];
  }
  __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(p.o) + b * p.so[0] + h * p.so[1] + t * p.so[2] + lane * E;
  const float inv = l != 0.f ? 1.f / l : 0.f;
#pragma unroll
  for (int e = 0; e < E; ++e) dst[e] = __float2bfloat16_rn(o[e] * inv);
  if (p.lse != nullptr && lane == 0) p.lse[r] = l != 0.f ? (m + log2f(l)) * 0.6931471805599453f : -INFINITY;
}

template <int D>
cudaError_t launch_d(const TreeParams& p, bool fp8, cudaStream_t s) {
  const int64_t rows = static_cast<int64_t>(p.B) * p.Hq * p.T;
  const int64_t blocks = (rows + kWarps - 1) / kWarps;
  if (blocks > 0x7fffffff) return cudaErrorInvalidValue;
  const dim3 grid(static_cast<unsigned>(blocks), p.n_splits);
  if (fp8)
    tree_rows_kernel<D, true><<<grid, kWarps * 32, 0, s>>>(p);
  else
    tree_rows_kernel<D, false><<<grid, kWarps * 32, 0, s>>>(p);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  tree_merge_kernel<D><<<static_cast<unsigned>(blocks), kWarps * 32, 0, s>>>(p);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_decode_tree(const TreeParams& p, int d, bool fp8, cudaStream_t s) {
  if (d == 128) return launch_d<128>(p, fp8, s);
  if (d == 64) return launch_d<64>(p, fp8, s);
  return cudaErrorInvalidValue;
}

}  // namespace fa

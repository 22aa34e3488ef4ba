// fa_tree.cu — attention of T drafted tokens per sequence over a paged cache
// (T = 1: plain decode), bf16 or E4M3, on tcgen05 tensor cores.
//
// Sequence b holds len keys, the last m of them those of its m ≤ T drafted
// tokens.  Token t sees every key of the context [0, len − m) and drafted key u
// where mask[t][u] is set (u ≤ t without a mask).  Rows that see nothing, the
// padding rows t ≥ m among them, give O = 0 and LSE = −∞.
//
// The T·G query rows of one (b, key/value head) are cut into tiles of NR = 16,
// 32 or 64 rows, the keys into n_splits chunks; a CTA takes one row tile over
// one chunk.  Bound: the cache is read once per row tile; up to 64 rows that is
// device memory, with more tiles the tensor cores and exponentials.
//
// Both products run transposed, with the keys (or the head dim) on the 128
// matrix rows and the query rows on the N side:
//   Sᵀ[key, row] = K Qᵀ,  Oᵀ[dim, row] += Vᵀ P̃ᵀ.
// N is as small as the rows are few, where putting 1 … 64 query rows on the
// 128-row side would pay for 128 rows of products and exponentials.  K and V go
// from the pages into shared memory as they lie (a page of one head is one TMA
// box) and are used as the A operand both times: K with its head dim
// contiguous, V with its head dim along M.  A softmax thread owns one key of
// the tile (TMEM lane) and walks over the rows (TMEM columns); P̃ᵀ goes to
// shared memory as 128 bytes per key with the rows contiguous.
//
// Row maxima lie across threads in this layout, so they are not recomputed per
// tile: a row keeps its reference m while every score is below m + 2^lazy, which
// one barrier with an OR tells; only then the tile's maxima are exchanged and O
// and ℓ rescaled.  ℓ stays in per-thread partial sums until the end.
//
// bf16 cache: P̃ enters as two bf16 terms, p ≈ hi + lo, two MMAs into one
// accumulator; p is then good to 2⁻¹⁷ at the price of N more columns, where one
// term alone would add an error as large as O's own rounding to bf16.
// E4M3 cache: K is multiplied as it is; q enters as two E4M3 terms
// q·2⁻ᵃ = hi + lo/16 in separate columns (exact for elements down to 2⁻¹⁴ of the
// row's largest, below that off by 2⁻²² of it), and the key's power of two
// multiplies the score in fp32.  V is widened to fp16 (exact) by four converter
// warps while the scores are worked on, so P̃ is fp16 (2⁻¹¹); the value row's
// power of two is folded into P̃ relative to a running maximum.  fp16 P̃ is kept
// near 2⁷ … 2¹⁵ by the reference m, so its subnormals begin 2⁻²¹ below a row's
// largest weight.
//
// Values in masked places.  Cache slots past the sequence end are zeroed in
// shared memory before V is used.  A drafted key's value row is seen by some
// rows and not by others, and 0·NaN would reach the others through the product:
// non-finite elements of drafted rows are zeroed there too, and added to the
// rows that do see them at the end.
#include <cuda_fp16.h>

#include "fa_kernels.h"
#include "sm103.cuh"

namespace fa {
namespace {

constexpr int kBN = 128;                 // keys per tile
constexpr int kPBlock = kBN * 128;       // P̃ᵀ: one 128-byte row per key
constexpr int kMaxStagedPages = 1024;
constexpr int kMaxRing = 8;
constexpr uint64_t kDrainNs = 200000000ull;

template <int D, bool FP8, int NR>
struct Cfg {
  static constexpr int kThreads = FP8 ? 320 : 192;  // softmax 0–3, producer 4, MMA 5, converters 6–9
  static constexpr int kSlot = kBN * D * (FP8 ? 1 : 2);
  static constexpr int kRK = (FP8 ? 3 : 2) * (128 / D);  // K and V ring slots: 160 KB (bf16), 112 KB (E4M3)
  static constexpr int kRV = (FP8 ? 4 : 3) * (128 / D);
  static constexpr int kV16 = FP8 ? kBN * D * 2 : 0;     // one widened V tile, double buffered
  static constexpr int kQ = FP8 ? 2 * NR * D : NR * D * 2;
  static constexpr int kOffK = 0;
  static constexpr int kOffV = kOffK + kRK * kSlot;
  static constexpr int kOffV16 = kOffV + kRV * kSlot;
  static constexpr int kOffP = kOffV16 + 2 * kV16;
  static constexpr int kOffQ = kOffP + kPBlock * (FP8 ? 1 : 2);
  static constexpr int kOffPages = kOffQ + kQ;
  static constexpr int kOffMisc = kOffPages + kMaxStagedPages * 4;
  static constexpr int kSW = FP8 ? 2 * NR : NR;          // TMEM columns of one S buffer
  static constexpr int kColO = 2 * kSW;
  static constexpr uint32_t kTmemCols = kColO + NR <= 64 ? 64 : kColO + NR <= 128 ? 128 : kColO + NR <= 256 ? 256 : 512;
  static_assert(kRK <= kMaxRing && kRV <= kMaxRing, "ring barriers");
  static_assert(kQ % 1024 == 0 && kSlot % 1024 == 0, "swizzle atoms");
};

template <int NR>
struct Misc {
  uint64_t k_full[kMaxRing], k_empty[kMaxRing], v_full[kMaxRing], v_empty[kMaxRing];
  uint64_t s_full[2], s_free[2], p_full, p_free, v16_full[2], v16_empty[2], drain;
  alignas(16) float m[NR];  // reference maxima (log2 units), −∞ while a row has seen nothing
  alignas(16) float f[NR];  // what a raw score is multiplied by (per row for E4M3)
  float corr[NR];    // factor of the last rescale
  float red[4][NR];  // per-warp maxima or sums
  int64_t row[NR];   // (b·Hq + h)·T + t, or −1 for a row that is not there
  int64_t o_off[NR]; // element offset of the row in O
  int token[NR];
  int kv_red[4];
  uint32_t bad[8];   // drafted keys with non-finite values (one bit each)
  uint32_t tmem_base;
  int abort_flag;
};

__device__ __forceinline__ unsigned int site(unsigned int s) { return (kKernTree << 8) | s; }

// Lengths of sequence b, checked: keys in all and drafted keys among them.
// Lengths that cannot be are reported and taken as an empty sequence.
__device__ __forceinline__ void seq_lengths(const TreeParams& p, int b, int& len, int& drafts) {
  len = p.seq_lens[b];
  drafts = p.draft_lens != nullptr ? p.draft_lens[b] : p.T;
  if (p.draft_lens == nullptr && len == 0) drafts = 0;  // an unused batch slot
  if (drafts < 0 || drafts > p.T || len < drafts || len > static_cast<int64_t>(p.max_blocks) * p.block_size) {
    atomicCAS(p.err + 1, 0u, (kKernTree << 8) | kSiteBadLength);
    len = drafts = 0;
  }
}

__device__ __forceinline__ int checked_page(const TreeParams& p, int b, int index) {
  const int blk = p.block_table[static_cast<int64_t>(b) * p.max_blocks + index];
  if (blk >= 0 && blk < p.num_blocks) return blk;
  atomicCAS(p.err + 1, 0u, (kKernTree << 8) | kSiteBadBlock);
  return 0;
}

struct OpMax {
  __device__ __forceinline__ float operator()(float a, float b) const { return fmaxf(a, b); }
};
struct OpAdd {
  __device__ __forceinline__ float operator()(float a, float b) const { return a + b; }
};

// Reduces each of NR columns over the warp's 32 lanes by halving: at every step
// a lane hands over the half of its columns that its partner keeps.  Ends with
// max(1, NR/32) totals in v[0 …], of the columns from the returned one on.
template <int NR, class Op>
__device__ __forceinline__ int reduce_cols(float (&v)[NR], int lane, Op op) {
  int base = 0;
#pragma unroll
  for (int step = 0; step < 5; ++step) {
    const int mask = 16 >> step;
    const int half = NR >> (step + 1);
    if (half >= 1) {
      const bool up = (lane & mask) != 0;
#pragma unroll
      for (int i = 0; i < (half >= 1 ? half : 1); ++i) {
        const float send = up ? v[i] : v[i + half];
        const float keep = up ? v[i + half] : v[i];
        v[i] = op(keep, __shfl_xor_sync(0xffffffffu, send, mask));
      }
      base += up ? half : 0;
    } else {
      v[0] = op(v[0], __shfl_xor_sync(0xffffffffu, v[0], mask));
    }
  }
  return base;
}

// One tile's raw scores of this thread's key, all rows.
template <bool FP8, int NR>
__device__ __forceinline__ void load_scores(uint32_t addr, float (&s)[NR]) {
  constexpr int C = NR < 32 ? NR : 32;
#pragma unroll
  for (int c = 0; c < NR; c += C) {
    uint32_t a[C];
    if constexpr (C == 32) tmem_ld32(addr + c, a); else tmem_ld16(addr + c, a);
    if constexpr (FP8) {
      uint32_t b[C];
      if constexpr (C == 32) tmem_ld32(addr + NR + c, b); else tmem_ld16(addr + NR + c, b);
      tmem_wait_ld();
      reg_fence(a);
      reg_fence(b);
#pragma unroll
      for (int i = 0; i < C; i += 2)
        ffma2(s[c + i], s[c + i + 1], __uint_as_float(b[i]), __uint_as_float(b[i + 1]), 0.0625f, 0.0625f,
              __uint_as_float(a[i]), __uint_as_float(a[i + 1]));
    } else {
      tmem_wait_ld();
      reg_fence(a);
#pragma unroll
      for (int i = 0; i < C; ++i) s[c + i] = __uint_as_float(a[i]);
    }
  }
}

template <int D, bool FP8, int NR>
__global__ void __launch_bounds__(Cfg<D, FP8, NR>::kThreads, 1) tree_kernel(const __grid_constant__ TreeParams p) {
  using C = Cfg<D, FP8, NR>;
  constexpr bool kPg5 = !FP8 && D == 128;  // K/V pages as [row group][half][8 rows][128 bytes]
  constexpr int kSlot = C::kSlot;
  // Rescale once a score exceeds the reference by this; the reference is taken kBase below the maximum.
  constexpr float kLazy = FP8 ? 11.f : 8.f;
  constexpr float kBase = FP8 ? 7.f : 0.f;
  constexpr int kKvLazy = 4;  // fp16 P̃ stays below 2^(11 + 4)
  extern __shared__ uint8_t smem_raw[];
  const uint32_t pad = (1024u - (smem_u32(smem_raw) & 1023u)) & 1023u;
  uint8_t* smem = smem_raw + pad;
  Misc<NR>* ms = reinterpret_cast<Misc<NR>*>(smem + C::kOffMisc);
  int* staged = reinterpret_cast<int*>(smem + C::kOffPages);
  volatile int* abort_flag = &ms->abort_flag;

  const int tid = threadIdx.x;
  const int warp = tid >> 5;
  const int lane = tid & 31;
  // Row tiles of one chunk are neighbours in the grid, so that they share its keys in L2.
  int idx = blockIdx.x;
  const int rt = idx % p.row_tiles;
  idx /= p.row_tiles;
  const int c = idx % p.n_splits;
  idx /= p.n_splits;
  const int hkv = idx % p.Hkv;
  const int b = idx / p.Hkv;

  int len, drafts;
  seq_lengths(p, b, len, drafts);
  const int context = len - drafts;
  const int chunk = (((len + p.n_splits - 1) / p.n_splits) + kBN - 1) & ~(kBN - 1);
  const int key0 = min(c * chunk, len);
  const int kend = min(len, key0 + chunk);
  const int row0 = rt * NR;
  const int live_rows = drafts * p.G - row0;  // rows of this tile that belong to a drafted token
  const int nt = live_rows > 0 ? (kend - key0 + kBN - 1) / kBN : 0;

  if (tid < NR) {
    const int rr = row0 + tid;
    const int t = rr / p.G;
    const int h = hkv * p.G + (rr - t * p.G);
    const bool there = t < p.T;
    ms->row[tid] = there ? (static_cast<int64_t>(b) * p.Hq + h) * p.T + t : -1;
    ms->o_off[tid] = b * p.so[0] + h * p.so[1] + static_cast<int64_t>(t) * p.so[2];
    ms->token[tid] = t;
    ms->m[tid] = -INFINITY;
    ms->f[tid] = p.scale_log2;
    if (nt == 0 && there) {  // nothing to see in this chunk
      if (p.n_splits > 1) {
        p.part_ml[(ms->row[tid] * p.n_splits + c) * 2 + 0] = -INFINITY;
        p.part_ml[(ms->row[tid] * p.n_splits + c) * 2 + 1] = 0.f;
      } else if (p.lse != nullptr) {
        p.lse[ms->row[tid]] = -INFINITY;
      }
    }
  }
  if (nt == 0) {
    if (p.n_splits == 1) {
      __syncthreads();
      for (int i = tid; i < NR * (D / 8); i += C::kThreads) {
        const int n = i / (D / 8);
        if (ms->row[n] >= 0)
          *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.o) + ms->o_off[n] + (i % (D / 8)) * 8) =
              make_uint4(0, 0, 0, 0);
      }
    }
    return;
  }

  if (tid == 0) {
    for (int s = 0; s < C::kRK; ++s) {
      mbar_init(&ms->k_full[s], 1);
      mbar_init(&ms->k_empty[s], 1);
    }
    for (int s = 0; s < C::kRV; ++s) {
      mbar_init(&ms->v_full[s], 1);
      mbar_init(&ms->v_empty[s], FP8 ? 4 : 1);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(&ms->s_full[s], 1);
      mbar_init(&ms->s_free[s], 128);
      mbar_init(&ms->v16_full[s], 128);
      mbar_init(&ms->v16_empty[s], 1);
    }
    mbar_init(&ms->p_full, 128);
    mbar_init(&ms->p_free, 1);
    mbar_init(&ms->drain, 1);
    ms->abort_flag = 0;
    for (int i = 0; i < 8; ++i) ms->bad[i] = 0;
    fence_barrier_init();
  }
  if (warp == 5) {
    tmem_alloc(&ms->tmem_base, C::kTmemCols);
    tmem_relinquish();
  }
  // The chunk's page ids, checked.
  const int page0 = key0 / p.block_size;
  const int npages = (kend - 1) / p.block_size - page0 + 1;
  for (int i = tid; i < min(npages, kMaxStagedPages); i += C::kThreads) staged[i] = checked_page(p, b, page0 + i);
  auto page_id = [&](int key) -> int {
    const int rel = key / p.block_size - page0;
    return rel < kMaxStagedPages ? staged[rel] : checked_page(p, b, page0 + rel);
  };
  // The tile's query rows as a K-major operand (rows that are not there as zeros).
  for (int i0 = 0; i0 < NR * (D / 8); i0 += C::kThreads) {
    const int i = i0 + tid;
    const bool in = i < NR * (D / 8);
    const int n = in ? i / (D / 8) : 0, ch = i % (D / 8);
    uint4 v = make_uint4(0, 0, 0, 0);
    if (in && n < live_rows) {
      const int rr = row0 + n;
      const int t = rr / p.G;
      v = *reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p.q) + b * p.sq[0] +
                                          (hkv * p.G + rr - t * p.G) * p.sq[1] + t * p.sq[2] + ch * 8);
    }
    if constexpr (!FP8) {
      if (in)
        *reinterpret_cast<uint4*>(smem + C::kOffQ + (ch >> 3) * NR * 128 + n * 128 + (((ch & 7) ^ (n & 7)) << 4)) = v;
    } else {
      // 2⁻ᵃ brings the row's largest magnitude to at most 448.
      const uint32_t w[4] = {v.x, v.y, v.z, v.w};
      float x[8];
      uint32_t top = 0;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        x[e] = __uint_as_float(e & 1 ? w[e >> 1] & 0xffff0000u : w[e >> 1] << 16);
        const uint32_t a = __float_as_uint(x[e]) & 0x7fffffffu;
        if (a < 0x7f800000u) top = max(top, a);
        else x[e] = __uint_as_float(0x7fffffffu);
      }
#pragma unroll
      for (int mk = D / 16; mk > 0; mk >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, mk));
      const int a = max(-126, static_cast<int>(top >> 23) - 135 + ((top & 0x7fffffu) > 0x600000u ? 1 : 0));
      const float inv = __uint_as_float(static_cast<uint32_t>(127 - a) << 23);
      uint32_t hi[2] = {0, 0}, lo[2] = {0, 0};
#pragma unroll
      for (int e = 0; e < 8; e += 2) {
        const float y0 = x[e] * inv, y1 = x[e + 1] * inv;
        const uint32_t h = pack_e4m3x2(y0, y1);
        const uint32_t back = e4m3x2_to_f16x2(h);
        const float2 z = __half22float2(*reinterpret_cast<const __half2*>(&back));
        hi[e >> 2] |= h << ((e & 2) * 8);
        lo[e >> 2] |= pack_e4m3x2((y0 - z.x) * 16.f, (y1 - z.y) * 16.f) << ((e & 2) * 8);
      }
      if (in) {
        // Rows of D bytes; chunk of 16 bytes XORed with the row (128-byte rows) or half of it (64-byte rows).
        const int sw = D == 128 ? n & 7 : (n >> 1) & 3;  // NR is a multiple of 16: the same for rows n and NR + n
        uint8_t* dst = smem + C::kOffQ + n * D + (((ch >> 1) ^ sw) << 4) + (ch & 1) * 8;
        *reinterpret_cast<uint2*>(dst) = make_uint2(hi[0], hi[1]);
        *reinterpret_cast<uint2*>(dst + NR * D) = make_uint2(lo[0], lo[1]);
        if (ch == 0) ms->f[n] = p.scale_log2 * __uint_as_float(static_cast<uint32_t>(a + 127) << 23);
      }
    }
  }
  fence_proxy_async_smem();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = ms->tmem_base;

  if (warp == 4) {
    // ------------------------------------------------------------ producer
    if (lane == 0) {
      tma_prefetch_desc(&p.tm_k);
      tma_prefetch_desc(&p.tm_v);
    }
    int ki = 0, vi = 0;
    bool ok = true;
    const int bs = p.block_size;
    auto load = [&](bool is_v) {
      const int j = is_v ? vi : ki;
      const int ring = is_v ? C::kRV : C::kRK;
      const int slot = j % ring;
      uint64_t* full = is_v ? &ms->v_full[slot] : &ms->k_full[slot];
      uint64_t* empty = is_v ? &ms->v_empty[slot] : &ms->k_empty[slot];
      bool got = true;
      if (lane == 0) {
        got = mbar_wait(empty, ((j / ring) & 1) ^ 1, abort_flag, p.err, site(is_v ? 2 : 1));
        if (got) mbar_arrive_expect_tx(full, kSlot);
      }
      ok = __shfl_sync(0xffffffffu, got, 0);
      if (!ok) return;
      const CUtensorMap* tm = is_v ? &p.tm_v : &p.tm_k;
      uint8_t* dst = smem + (is_v ? C::kOffV : C::kOffK) + slot * kSlot;
      if (lane < kBN / bs) {
        const int t0 = key0 + j * kBN + lane * bs;
        int blk = 0, row = bs;  // a row past the page: TMA fills the box with zeros
        if (t0 < kend) {
          blk = page_id(t0);
          row = 0;
        }
        if constexpr (kPg5)
          tma_load_5d(dst + lane * bs * 256, tm, full, 0, 0, 0, row >> 3, blk * p.Hkv + hkv);
        else
          tma_load_4d(dst + lane * bs * (kSlot / kBN), tm, full, 0, row, hkv, blk);
      }
      (is_v ? vi : ki) += 1;
    };
    load(false);
    for (int j = 0; ok && j < nt; ++j) {
      if (j + 1 < nt) load(false);
      if (ok) load(true);
    }
    if (lane == 0 && *abort_flag) {  // let the copies in flight land before the CTA ends
      for (int j = max(0, ki - C::kRK); j < ki; ++j)
        mbar_wait_drain(&ms->k_full[j % C::kRK], (j / C::kRK) & 1, kDrainNs);
      for (int j = max(0, vi - C::kRV); j < vi; ++j)
        mbar_wait_drain(&ms->v_full[j % C::kRV], (j / C::kRV) & 1, kDrainNs);
    }
  } else if (warp == 5) {
    // ------------------------------------------------------------ MMA issuer
    if (lane == 0) {
      constexpr uint32_t kIdescS = FP8 ? idesc_e4m3_f32(128, 2 * NR, false, false) : idesc_bf16_f32(128, NR, false, false);
      constexpr uint32_t kIdescO = FP8 ? idesc_f16_f32(128, NR, true, true) : idesc_bf16_f32(128, NR, true, true);
      const uint32_t sQ = smem_u32(smem + C::kOffQ), sK = smem_u32(smem + C::kOffK), sP = smem_u32(smem + C::kOffP);
      auto issue_pv = [&](int j) -> bool {
        const int slot = j % C::kRV;
        if (!mbar_wait(&ms->p_full, j & 1, abort_flag, p.err, site(3))) return false;
        if constexpr (FP8) {
          if (!mbar_wait(&ms->v16_full[j & 1], (j >> 1) & 1, abort_flag, p.err, site(4))) return false;
        } else {
          if (!mbar_wait(&ms->v_full[slot], (j / C::kRV) & 1, abort_flag, p.err, site(4))) return false;
        }
        tc_fence_after();
        const uint32_t sV = smem_u32(smem + (FP8 ? C::kOffV16 + (j & 1) * C::kV16 : C::kOffV + slot * kSlot));
#pragma unroll
        for (int term = 0; term < (FP8 ? 1 : 2); ++term)
#pragma unroll
          for (int kk = 0; kk < kBN / 16; ++kk) {
            // A: 16 keys, the head dim along M in 64-element blocks (D = 64: the one block twice, the upper
            // 64 rows of the result are not read).  B: 16 keys of P̃ᵀ.
            const uint64_t ad = kPg5 ? sdesc_sw128(sV + kk * 4096, 1024, 2048)
                                     : sdesc_sw128(sV + kk * 2048, D == 128 ? kBN * 128 : 0, 1024);
            const uint64_t bd = sdesc_sw128(sP + term * kPBlock + kk * 2048, kPBlock, 1024);
            mma_bf16_ss(tmem + C::kColO, ad, bd, kIdescO, (j > 0 || term > 0 || kk > 0) ? 1u : 0u);
          }
        mma_commit(&ms->p_free);
        mma_commit(FP8 ? &ms->v16_empty[j & 1] : &ms->v_empty[slot]);
        return true;
      };
      bool ok = true;
      for (int j = 0; ok && j < nt; ++j) {
        const int slot = j % C::kRK;
        ok = mbar_wait(&ms->k_full[slot], (j / C::kRK) & 1, abort_flag, p.err, site(5)) &&
             mbar_wait(&ms->s_free[j & 1], ((j >> 1) & 1) ^ 1, abort_flag, p.err, site(6));
        if (!ok) break;
        tc_fence_after();
        const uint32_t kb = sK + slot * kSlot;
        const uint32_t ds = tmem + (j & 1) * C::kSW;
        if constexpr (FP8) {
#pragma unroll
          for (int kk = 0; kk < D / 32; ++kk) {
            if constexpr (D == 128)
              mma_e4m3_ss(ds, sdesc_sw128(kb + kk * 32, 16, 1024), sdesc_sw128(sQ + kk * 32, 16, 1024), kIdescS,
                          kk > 0 ? 1u : 0u);
            else
              mma_e4m3_ss(ds, sdesc_sw64(kb + kk * 32, 16, 512), sdesc_sw64(sQ + kk * 32, 16, 512), kIdescS,
                          kk > 0 ? 1u : 0u);
          }
        } else {
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk) {
            const uint64_t ad = kPg5 ? sdesc_sw128(kb + (kk >> 2) * 1024 + (kk & 3) * 32, 16, 2048)
                                     : sdesc_sw128(kb + kk * 32, 16, 1024);
            const uint64_t bd = sdesc_sw128(sQ + (kk >> 2) * NR * 128 + (kk & 3) * 32, 16, 1024);
            mma_bf16_ss(ds, ad, bd, kIdescS, kk > 0 ? 1u : 0u);
          }
        }
        mma_commit(&ms->s_full[j & 1]);
        mma_commit(&ms->k_empty[slot]);
        if (j >= 1) ok = issue_pv(j - 1);
      }
      if (ok) issue_pv(nt - 1);
      if (*abort_flag) {
        mma_commit(&ms->drain);
        mbar_wait_drain(&ms->drain, 0, kDrainNs);
      }
    }
  } else if (warp < 4) {
    // --------------------------------------- softmax: one key per thread, all rows
    const uint32_t lane_base = static_cast<uint32_t>(warp * 32) << 16;
    float l[NR];
#pragma unroll
    for (int n = 0; n < NR; ++n) l[n] = 0.f;
    int kv_ref = -1024;
    bool ok = true;
    // E4M3: the scale bytes of this thread's key, two tiles ahead.
    int sk[3] = {0, 0, 0}, sv[3] = {0, 0, 0};
    auto fetch_scales = [&](int j, int& a, int& v) {
      const int key = key0 + j * kBN + tid;
      if (key < kend) {
        const int64_t at = (static_cast<int64_t>(page_id(key)) * p.Hkv + hkv) * p.block_size + key % p.block_size;
        a = p.k_scale[at];
        v = p.v_scale[at];
      }
    };
    if constexpr (FP8) {
      fetch_scales(0, sk[0], sv[0]);
      fetch_scales(1, sk[1], sv[1]);
    }
    for (int j = 0; j < nt; ++j) {
      if constexpr (FP8) fetch_scales(j + 2, sk[2], sv[2]);
      const int key = key0 + j * kBN + tid;
      const bool tail = key0 + (j + 1) * kBN > context;  // the tile holds drafted keys or the end
      // Which rows see this key (bit per row); context keys are seen by all.
      uint64_t seen = ~0ull;
      if (tail && key >= context) {
        seen = 0;
        const int u = key - context;
        if (key < kend) {
          bool sees = false;
          int last = -1;
          for (int n = 0; n < NR; ++n) {
            const int t = ms->token[n];
            if (t >= drafts) break;
            if (t != last) {
              sees = p.mask != nullptr ? p.mask[b * p.mask_sb + static_cast<int64_t>(t) * p.T + u] != 0 : u <= t;
              last = t;
            }
            seen |= static_cast<uint64_t>(sees) << n;
          }
        }
      }
      ok = mbar_wait(&ms->s_full[j & 1], (j >> 1) & 1, abort_flag, p.err, site(7));
      tc_fence_after();
      const uint32_t sa = tmem + lane_base + (j & 1) * C::kSW;
      // 2^(k of the key) for E4M3; s = 0 stands for 2^−127, which only its double times ½ can build.
      float ks = 1.f;
      int kv = -1024;
      if constexpr (FP8) {
        ks = sk[0] == 0 ? 5.877471754111438e-39f : __uint_as_float(static_cast<uint32_t>(sk[0]) << 23);
        if (key < kend) kv = sv[0] - 127;
      }
      // x = score − reference, masked to −∞ where the row does not see the key.
      float x[NR];
      auto scores = [&](bool relative) {
        load_scores<FP8, NR>(sa, x);
#pragma unroll
        for (int n = 0; n < NR; n += 4) {
          const float4 m4 = relative ? *reinterpret_cast<const float4*>(&ms->m[n]) : make_float4(0.f, 0.f, 0.f, 0.f);
          float4 f4;
          if constexpr (FP8) {
            f4 = *reinterpret_cast<const float4*>(&ms->f[n]);
            fmul2(f4.x, f4.y, f4.x, f4.y, ks, ks);
            fmul2(f4.z, f4.w, f4.z, f4.w, ks, ks);
          } else {
            f4 = make_float4(p.scale_log2, p.scale_log2, p.scale_log2, p.scale_log2);
          }
          ffma2(x[n], x[n + 1], x[n], x[n + 1], f4.x, f4.y, -m4.x, -m4.y);
          ffma2(x[n + 2], x[n + 3], x[n + 2], x[n + 3], f4.z, f4.w, -m4.z, -m4.w);
        }
        if (tail) {
#pragma unroll
          for (int n = 0; n < NR; ++n)
            if (!((seen >> n) & 1)) x[n] = -INFINITY;
        }
      };
      scores(true);
      float mx[4] = {x[0], x[1], x[2], x[3]};
#pragma unroll
      for (int n = 4; n < NR; n += 4)
#pragma unroll
        for (int i = 0; i < 4; ++i) mx[i] = fmaxf(mx[i], x[n + i]);
      const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
      const bool over = top > kLazy || (FP8 && kv > kv_ref + kKvLazy);
      if (named_any(1, 128, over || !ok)) {
        // A reference moves (the first tile always does): exchange the tile's maxima, rescale ℓ and O.
        if (named_any(1, 128, !ok)) {
          ok = false;
          break;
        }
        scores(false);
        const int col = reduce_cols<NR>(x, lane, OpMax());
        if (NR >= 32 || !(lane & 1)) {
#pragma unroll
          for (int i = 0; i < (NR >= 32 ? NR / 32 : 1); ++i) ms->red[warp][col + i] = x[i];
        }
        if constexpr (FP8) {
          const int top_kv = __reduce_max_sync(0xffffffffu, kv);
          if (lane == 0) ms->kv_red[warp] = top_kv;
        }
        named_sync(1, 128);
        int kv_new = kv_ref;
        if constexpr (FP8)
          kv_new = max(kv_ref, max(max(ms->kv_red[0], ms->kv_red[1]), max(ms->kv_red[2], ms->kv_red[3])));
        if (tid < NR) {
          const float old = ms->m[tid];
          const float now = fmaxf(fmaxf(ms->red[0][tid], ms->red[1][tid]), fmaxf(ms->red[2][tid], ms->red[3][tid]));
          const bool up = now > -INFINITY && now - kBase > old;
          ms->corr[tid] = up ? exp2f(old - (now - kBase)) : 1.f;  // 0 from −∞: nothing was summed yet
          if (up) ms->m[tid] = now - kBase;
        }
        named_sync(1, 128);
#pragma unroll
        for (int n = 0; n < NR; ++n) l[n] *= ms->corr[n];
        if (j > 0) {
          ok = mbar_wait(&ms->p_free, (j - 1) & 1, abort_flag, p.err, site(8));
          tc_fence_after();
          const float kf = FP8 ? exp2f(static_cast<float>(max(kv_ref - kv_new, -200))) : 1.f;
          constexpr int W = NR < 32 ? NR : 32;
#pragma unroll
          for (int cc = 0; cc < NR; cc += W) {
            uint32_t r[W];
            const uint32_t oa = tmem + lane_base + C::kColO + cc;
            if constexpr (W == 32) tmem_ld32(oa, r); else tmem_ld16(oa, r);
            tmem_wait_ld();
            reg_fence(r);
#pragma unroll
            for (int i = 0; i < W; ++i) r[i] = __float_as_uint(__uint_as_float(r[i]) * (ms->corr[cc + i] * kf));
            if constexpr (W == 32) tmem_st32(oa, r); else tmem_st16(oa, r);
          }
          tmem_wait_st();
        }
        kv_ref = kv_new;
        scores(true);
        // A row that has seen nothing has the reference −∞, and only masked scores: −∞ − (−∞) is −∞ here.
#pragma unroll
        for (int n = 0; n < NR; ++n)
          if (ms->m[n] == -INFINITY) x[n] = -INFINITY;
      }
      tc_fence_before();
      mbar_arrive(&ms->s_free[j & 1]);

#pragma unroll
      for (int n = 0; n < NR; n += 2) {
        x[n] = ex2_approx(x[n]);
        x[n + 1] = ex2_approx(x[n + 1]);
        fadd2(l[n], l[n + 1], l[n], l[n + 1], x[n], x[n + 1]);
      }
      // P̃ᵀ in the matrix type, 8 rows per 16-byte chunk.
      uint32_t hi[NR / 2], lo[FP8 ? 1 : NR / 2];
      if constexpr (FP8) {
        // The value row's scale relative to the running maximum: a power of two, at most 2^kKvLazy.
        const float w = kv - kv_ref < -126 ? 0.f : __uint_as_float(static_cast<uint32_t>(kv - kv_ref + 127) << 23);
#pragma unroll
        for (int n = 0; n < NR; n += 2) {
          float a, d;
          fmul2(a, d, x[n], x[n + 1], w, w);
          hi[n / 2] = pack_f16x2(a, d);
        }
      } else {
#pragma unroll
        for (int n = 0; n < NR; n += 2) {
          hi[n / 2] = pack_bf16x2(x[n], x[n + 1]);
          lo[n / 2] = pack_bf16x2(x[n] - __uint_as_float(hi[n / 2] << 16),
                                  x[n + 1] - __uint_as_float(hi[n / 2] & 0xffff0000u));
        }
      }
      // P̃'s buffer is free once the product of the tile before has run.
      if (j > 0) ok = mbar_wait(&ms->p_free, (j - 1) & 1, abort_flag, p.err, site(8)) && ok;
      uint8_t* prow = smem + C::kOffP + tid * 128;
#pragma unroll
      for (int ch = 0; ch < NR / 8; ++ch) {
        *reinterpret_cast<uint4*>(prow + ((ch ^ (tid & 7)) << 4)) =
            make_uint4(hi[4 * ch], hi[4 * ch + 1], hi[4 * ch + 2], hi[4 * ch + 3]);
        if constexpr (!FP8)
          *reinterpret_cast<uint4*>(prow + kPBlock + ((ch ^ (tid & 7)) << 4)) =
              make_uint4(lo[4 * ch], lo[4 * ch + 1], lo[4 * ch + 2], lo[4 * ch + 3]);
      }
      if (!FP8 && tail && key >= context) {
        // This key's value row: zeros past the end, and in place of what a drafted row holds that is not finite.
        const int slot = j % C::kRV;
        ok = mbar_wait(&ms->v_full[slot], (j / C::kRV) & 1, abort_flag, p.err, site(9)) && ok;
        uint8_t* vt = smem + C::kOffV + slot * kSlot;
        bool bad = false;
#pragma unroll
        for (int kb = 0; kb < D / 64; ++kb) {
          uint8_t* vr = vt + (kPg5 ? (tid >> 3) * 2048 + kb * 1024 + (tid & 7) * 128 : tid * 128);
#pragma unroll
          for (int q = 0; q < 8; ++q) {
            uint4* at = reinterpret_cast<uint4*>(vr + q * 16);
            uint32_t w[4] = {0, 0, 0, 0};
            if (key < kend) {
              const uint4 v = *at;
              w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                if ((w[i] & 0x7f80u) == 0x7f80u) w[i] &= 0xffff0000u, bad = true;
                if ((w[i] & 0x7f800000u) == 0x7f800000u) w[i] &= 0xffffu, bad = true;
              }
            }
            *at = make_uint4(w[0], w[1], w[2], w[3]);
          }
        }
        if (bad) atomicOr(&ms->bad[(key - context) >> 5], 1u << ((key - context) & 31));
      }
      fence_proxy_async_smem();
      tc_fence_before();
      mbar_arrive(&ms->p_full);
      sk[0] = sk[1], sk[1] = sk[2];
      sv[0] = sv[1], sv[1] = sv[2];
    }
    // ------------------------------------------------------------ epilogue
    // (Barrier 1 is joined by all 128 threads whatever the waits said.)
    ok = ok && mbar_wait(&ms->p_free, (nt - 1) & 1, abort_flag, p.err, site(10));
    tc_fence_after();
    {
      const int col = reduce_cols<NR>(l, lane, OpAdd());
      if (NR >= 32 || !(lane & 1)) {
#pragma unroll
        for (int i = 0; i < (NR >= 32 ? NR / 32 : 1); ++i) ms->red[warp][col + i] = l[i];
      }
    }
    named_sync(1, 128);
    if (tid < NR) {  // fixed order: the same sums every time
      const float sum = (ms->red[0][tid] + ms->red[1][tid]) + (ms->red[2][tid] + ms->red[3][tid]);
      const int64_t r = ms->row[tid];
      const bool live = tid < live_rows;
      if (ok && r >= 0) {
        const float m = live ? ms->m[tid] : -INFINITY;
        const float s = live ? sum : 0.f;
        if (p.n_splits > 1) {
          p.part_ml[(r * p.n_splits + c) * 2 + 0] = m;
          p.part_ml[(r * p.n_splits + c) * 2 + 1] = s;
        } else if (p.lse != nullptr) {
          p.lse[r] = s != 0.f ? (m + log2f(s)) * 0.6931471805599453f : -INFINITY;
        }
      }
      ms->corr[tid] = live && sum != 0.f ? 1.f / sum : 0.f;
    }
    named_sync(1, 128);
    const bool mine = __all_sync(0xffffffffu, ok) && tid < D;
    if (__any_sync(0xffffffffu, mine)) {
      const float kf = FP8 ? exp2f(static_cast<float>(max(kv_ref, -300))) : 1.f;
      bool any_bad = false;
      for (int i = 0; i < 8; ++i) any_bad = any_bad || ms->bad[i] != 0;
      constexpr int W = NR < 32 ? NR : 32;
#pragma unroll
      for (int cc = 0; cc < NR; cc += W) {
        uint32_t r[W];
        if constexpr (W == 32) tmem_ld32(tmem + lane_base + C::kColO + cc, r);
        else tmem_ld16(tmem + lane_base + C::kColO + cc, r);
        tmem_wait_ld();
        reg_fence(r);
        if (any_bad) {
          for (int u = 0; u < drafts; ++u) {
            if (!((ms->bad[u >> 5] >> (u & 31)) & 1)) continue;
            const int key = context + u;
            const int64_t at =
                ((static_cast<int64_t>(page_id(key)) * p.Hkv + hkv) * p.block_size + key % p.block_size) * D + tid;
            float v;
            if (FP8)
              v = (static_cast<const uint8_t*>(p.v_cache)[at] & 0x7f) == 0x7f ? NAN : 0.f;
            else
              v = __bfloat162float(static_cast<const __nv_bfloat16*>(p.v_cache)[at]);
            if (fabsf(v) <= 3.4028234663852886e38f) continue;
#pragma unroll
            for (int i = 0; i < W; ++i) {
              const int t = ms->token[cc + i];
              if (t < drafts &&
                  (p.mask != nullptr ? p.mask[b * p.mask_sb + static_cast<int64_t>(t) * p.T + u] != 0 : u <= t))
                r[i] = __float_as_uint(__uint_as_float(r[i]) + v);
            }
          }
        }
#pragma unroll
        for (int i = 0; i < W; ++i) {
          const int n = cc + i;
          const int64_t row = ms->row[n];
          if (row >= 0) {
            const float f = ms->corr[n];
            const float o = f != 0.f ? __uint_as_float(r[i]) * f * kf : 0.f;
            if (p.n_splits > 1)
              p.part_o[(row * p.n_splits + c) * D + tid] = o;
            else
              static_cast<__nv_bfloat16*>(p.o)[ms->o_off[n] + tid] = __float2bfloat16_rn(o);
          }
        }
      }
    }
  } else if constexpr (FP8) {
    // ------------------------------------------ converters: one value row per thread
    const int r = tid - 192;
    for (int j = 0; j < nt; ++j) {
      const int slot = j % C::kRV;
      bool ok = mbar_wait(&ms->v_full[slot], (j / C::kRV) & 1, abort_flag, p.err, site(11)) &&
                mbar_wait(&ms->v16_empty[j & 1], ((j >> 1) & 1) ^ 1, abort_flag, p.err, site(12));
      if (!__all_sync(0xffffffffu, ok)) break;
      const int key = key0 + j * kBN + r;
      const uint8_t* src = smem + C::kOffV + slot * kSlot + r * D;
      uint8_t* dst = smem + C::kOffV16 + (j & 1) * C::kV16 + r * 128;
      bool bad = false;
#pragma unroll
      for (int ch = 0; ch < D / 16; ++ch) {
        const int sw = D == 128 ? r & 7 : (r >> 1) & 3;
        const uint4 v = *reinterpret_cast<const uint4*>(src + ((ch ^ sw) << 4));
        uint32_t w[4] = {v.x, v.y, v.z, v.w};
        if (key >= context) {  // drafted keys: NaN codes out; past the end: everything out
#pragma unroll
          for (int i = 0; i < 4; ++i) {
#pragma unroll
            for (int q = 0; q < 4; ++q)
              if (((w[i] >> (8 * q)) & 0x7f) == 0x7f) w[i] &= ~(0xffu << (8 * q)), bad = key < kend;
            if (key >= kend) w[i] = 0;
          }
        }
        uint32_t o[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) o[i] = e4m3x2_to_f16x2(w[i >> 1] >> (16 * (i & 1)));
        uint8_t* half = dst + (ch >> 2) * kBN * 128;  // 64 elements per 128-byte row
        *reinterpret_cast<uint4*>(half + ((((ch & 3) * 2) ^ (r & 7)) << 4)) = make_uint4(o[0], o[1], o[2], o[3]);
        *reinterpret_cast<uint4*>(half + ((((ch & 3) * 2 + 1) ^ (r & 7)) << 4)) = make_uint4(o[4], o[5], o[6], o[7]);
      }
      if (bad) atomicOr(&ms->bad[(key - context) >> 5], 1u << ((key - context) & 31));
      fence_proxy_async_smem();
      mbar_arrive(&ms->v16_full[j & 1]);
      __syncwarp();
      if (lane == 0) mbar_arrive(&ms->v_empty[slot]);
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 5) {
    tc_fence_after();
    tmem_dealloc(tmem, C::kTmemCols);
  }
}

// Joins a row's chunks, which hold o_c/ℓ_c: weights w_c = 2^(m_c − m)·ℓ_c, O = Σ w_c (o_c/ℓ_c) / Σ w_c.
// One warp per row.
constexpr int kMergeWarps = 4;
template <int D>
__global__ void __launch_bounds__(kMergeWarps * 32) tree_merge_kernel(const __grid_constant__ TreeParams p) {
  constexpr int E = D / 32;
  const int lane = threadIdx.x & 31;
  const int64_t r = static_cast<int64_t>(blockIdx.x) * kMergeWarps + (threadIdx.x >> 5);
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
    const float w = exp2f(x.x - m) * x.y;
    l += w;
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] += w * p.part_o[(r * p.n_splits + c) * D + lane * E + e];
  }
  __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(p.o) + b * p.so[0] + h * p.so[1] + t * p.so[2] + lane * E;
  const float inv = l != 0.f ? 1.f / l : 0.f;
#pragma unroll
  for (int e = 0; e < E; ++e) dst[e] = __float2bfloat16_rn(l != 0.f ? o[e] * inv : 0.f);
  if (p.lse != nullptr && lane == 0) p.lse[r] = l != 0.f ? (m + log2f(l)) * 0.6931471805599453f : -INFINITY;
}

template <int D, bool FP8, int NR>
cudaError_t launch_rows(const TreeParams& p, int64_t blocks, cudaStream_t s) {
  constexpr int kSmem = Cfg<D, FP8, NR>::kOffMisc + static_cast<int>(sizeof(Misc<NR>)) + 1024;
  static_assert(kSmem <= 227 * 1024, "shared memory");
  cudaError_t e =
      cudaFuncSetAttribute(tree_kernel<D, FP8, NR>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
  if (e != cudaSuccess) return e;
  tree_kernel<D, FP8, NR><<<static_cast<unsigned>(blocks), Cfg<D, FP8, NR>::kThreads, kSmem, s>>>(p);
  return cudaGetLastError();
}

template <int D, bool FP8>
cudaError_t launch_d(const TreeParams& p, cudaStream_t s) {
  const int64_t blocks = static_cast<int64_t>(p.B) * p.Hkv * p.n_splits * p.row_tiles;
  if (blocks > 0x7fffffff) return cudaErrorInvalidValue;
  cudaError_t e = p.tile_rows == 16   ? launch_rows<D, FP8, 16>(p, blocks, s)
                  : p.tile_rows == 32 ? launch_rows<D, FP8, 32>(p, blocks, s)
                                      : launch_rows<D, FP8, 64>(p, blocks, s);
  if (e != cudaSuccess || p.n_splits == 1) return e;
  const int64_t rows = static_cast<int64_t>(p.B) * p.Hq * p.T;
  tree_merge_kernel<D><<<static_cast<unsigned>((rows + kMergeWarps - 1) / kMergeWarps), kMergeWarps * 32, 0, s>>>(p);
  return cudaGetLastError();
}

}  // namespace

int tree_tile_rows(int64_t rows) { return rows <= 16 ? 16 : rows <= 32 ? 32 : 64; }

cudaError_t launch_decode_tree(const TreeParams& p, int d, bool fp8, cudaStream_t s) {
  if (d == 128) return fp8 ? launch_d<128, true>(p, s) : launch_d<128, false>(p, s);
  if (d == 64) return fp8 ? launch_d<64, true>(p, s) : launch_d<64, false>(p, s);
  return cudaErrorInvalidValue;
}

}  // namespace fa

// fa_tree.cu — attention of T drafted tokens per sequence over a paged cache
// (T = 1: plain decode), bf16, E4M3 or E2M1, on tcgen05 tensor cores: the kernel for
// up to 32 query rows (T·G, G query heads per key/value head) and the joining kernel.
//
// Sequence b holds len keys, the last m of them those of its m ≤ T drafted
// tokens.  Token t sees every key of the context [0, len − m) and drafted key u
// where mask[t][u] is set (u ≤ t without a mask).  Rows that see nothing, the
// padding rows t ≥ m among them, give O = 0 and LSE = −∞.
//
// Products.  Both run transposed, with the keys (or the head dim) on the 128
// matrix rows and the T·G query rows of a key/value head on the N side:
//   Sᵀ[key, row] = K Qᵀ,  Oᵀ[dim, row] += Vᵀ P̃ᵀ.
// N is as small as the rows are few (16 or 32), where putting them on the 128-row
// side would pay for 128 rows of products and exponentials.  K and V go
// from the pages into shared memory as they lie (a page of one head is one TMA
// box) and are the A operand both times: K with its head dim contiguous, V with
// its head dim along M.  A softmax thread owns one key of the tile (TMEM lane)
// and walks over the rows (TMEM columns); P̃ᵀ goes to shared memory as 128 bytes
// per key with the rows contiguous.
//
// Two streams.  A tile's softmax is a chain of waits (scores out of TMEM, the
// group's vote, exponentials, P̃ into shared memory, the second product), so two
// warpgroups run two of them at once on alternate key tiles, each with its own S,
// P̃, O and statistics, and are joined at the end of a piece.
//
// Row maxima lie across threads in this layout, so they are not recomputed per
// tile: a row keeps its reference m while every score is less than 2^8 above it,
// which one barrier with an OR tells; only then the tile's maxima are exchanged
// and O and ℓ rescaled.  ℓ stays in per-thread partial sums until the end.
//
// Work.  The 128-key tiles of all (b, key/value head) pairs form one line that is
// cut into equal parts, one per CTA, so ragged batches load every SM alike and
// short ones spread over the machine.  A CTA walks over its part without draining its pipeline between
// pairs.  A pair that is cut leaves o/ℓ, m, ℓ of each piece in the workspace,
// and a second kernel joins them.
//
// bf16 cache: P̃ enters as two bf16 terms p ≈ hi + lo in separate columns (good to
// 2⁻¹⁵; one term alone adds an error as large as O's own rounding to bf16), which
// costs nothing here, where device memory bounds it.  Both terms are positive, so
// that an infinite value stays one.
// E4M3 cache: K is multiplied as it is; q enters as two E4M3 terms
// q·2⁻ᵃ = hi + lo/16 in separate columns (exact for elements down to 2⁻¹⁴ of the
// row's largest, below that off by 2⁻²² of it), and the key's power of two
// multiplies the score in fp32.  V is widened to fp16 by the softmax warps, times the
// row's power of two relative to a running reference; from 2⁻¹⁵ to 2^7 that is exact
// (E4M3's smallest step, 2⁻⁹, becomes fp16's, 2⁻²⁴).  So P̃ is fp16 (2⁻¹¹): its reference is
// taken 2^3 below the maximum and P̃ stays below 2^11, fp16's subnormals begin
// 2⁻¹⁷ below a row's largest weight and weights are off by at most 2⁻²⁸ of it.
// (Folded into P̃ instead, the powers of two of small value rows cost their weights as
// many bits: rows made of such weights came out wrong by several times that.)
// A tile with value rows further below the reference than 2^15 is widened to bf16 with its
// powers of two, P̃ goes as two bf16 terms, and the product runs as bf16.
// E2M1 cache: a key's groups have a power of two each, which kind::mxf8f6f4 products apply
// to 32 elements at a time: K's codes stay E2M1 (spread to 16 bytes for sixteen, which is how
// the products read them), their scales go to tensor memory, and q enters as E4M3's two terms
// with scales of one.  V, whose groups lie across the second product's sum, is widened to fp16
// and P̃ is fp16, as with E4M3; from 2⁻²³ to 2^13 of the reference that is exact.  Both take
// warps of their own, as the codes need work before every product: one warpgroup for the keys
// of both streams and one for each stream's values.
//
// Values in masked places.  Cache slots past the sequence end are zeroed in
// shared memory before V is used.  A drafted key's value row is seen by some
// rows and not by others, and 0·NaN would reach the others through the product:
// non-finite elements of drafted rows are zeroed there too, and added to the
// rows that do see them at the end.
//
// Measured on GB300, 8 sequences of 16384 keys, 8 key/value heads of 128 elements (replaying a graph over two caches):
//   4 / 16 / 32 rows, bf16   91 / 92 / 95 us   5.9 / 5.8 / 5.7 TB/s, 0.88 of a device copy: bound by device memory
//   4 / 16 / 32 rows, E4M3   58 / 59 / 68 us   4.7 / 4.6 / 4.0 TB/s: inside a piece 4 and 16 rows run at the memory's
//                            rate; start, piece ends and the joining kernel take 15 us, and with 32 rows the softmax
//                            warps, which also widen V, are the bound
//   4 / 16 / 32 rows, E2M1   54 / 62 / 80 us   2.6 / 2.3 / 1.8 TB/s (8 rows 55, E4M3 58): a stream's tile is a chain of 3300 cycles (its values'
//                            codes 550, their reference 600, the place of the widened tile 400, widening 1450) and both
//                            streams' instructions take two thirds of it; with 32 rows the softmax adds to that
// E2M1, not kept: both halves written out as bf16 tiles by four warps, 195 us at 16 rows; codes of both halves fetched by one
// warp, 72 at 4 rows; and where the version at hand took 60 at 4 rows: both value warpgroups on one tile after the other and its
// reference found by the keys' warpgroup, 80; a ring of three widened tiles for both streams, 61, and with the references
// found by the fetching warp, 90.  Every role's instructions are fetched anew each tile, so that more of them on a chain
// cost more than the waits they save.
// E4M3, not kept: four or eight converter warps beside the softmax warps (7 and 12 % more at 4 rows, 15 % at 32);
// V widened by integer operations instead of the conversion instruction (slower, and it loses NaN); P̃ as two E4M3
// terms over V as it is (the terms span too few binades).
#include <stddef.h>

#include <atomic>

#include "fa_tree.cuh"

namespace fa {
namespace {

constexpr int kBN = kTreeBN;
constexpr int kPBlock = kBN * 128;       // P̃ᵀ: one 128-byte row per key
constexpr int kMaxRing = 8;
// Warps: streams 0–3 and 4–7, K loads 8, MMA 9, V loads 10, Q loads 11; E2M1: value converters 12–19, key converters 20–23.
// Registers per thread at launch and after the warpgroups' split.  A softmax thread holds its scores and partial
// sums, 2·NR values, and a spilled one would go to L2, shared memory leaving next to no L1.
constexpr int kScaleRing = 16;           // E4M3: tiles whose scale bytes are staged (V slots and four more)
constexpr int kFRing = 4;                // pieces whose row factors may be live at once
constexpr int kBadRing = 8;              // pieces whose flags of bad values may be

// NR rows of a pair, shared by both streams.
template <int D, int F, int NR>
struct Cfg {
  static constexpr bool FP8 = F == kCacheE4m3, FP4 = F == kCacheE2m1;
  static constexpr bool kWiden = FP8 || FP4;  // V is widened to fp16
  // E2M1: a warpgroup more for each stream, which widens the values, and one which lays out the keys.
  static constexpr int kThreads = FP4 ? 768 : 384;
  static constexpr int kRegsLaunch = FP4 ? 80 : 168;
  static constexpr int kRegsSoftmax = FP4 ? 120 : 208;
  static constexpr int kRegsConvert = FP4 ? 64 : 0;
  static constexpr int kRegsOther = FP4 ? 56 : 88;
  static_assert(2 * kRegsSoftmax + 2 * kRegsConvert + (FP4 ? 2 : 1) * kRegsOther <= kThreads / 128 * kRegsLaunch,
                "register split");
  static constexpr int kSlot = kBN * D * (kWiden ? 1 : 2);    // of a K tile as the products read it
  static constexpr int kTerms = kWiden ? 1 : 2;               // of P̃
  static constexpr int kPCols = kTerms * NR;                  // columns of P̃ᵀ and of Oᵀ
  // A key's P̃ᵀ row is 2·kPCols bytes (twice that for two terms of a tile in bf16); the streams' rows lie side by side in
  // 128 bytes where both fit.
  static constexpr int kPRow = FP8 ? 128 : FP4 ? 4 * NR : 2 * kPCols;
  static constexpr int kPNext = kPRow <= 64 ? kPRow : kPBlock;  // from a stream's rows to the other's
  static constexpr int kP = kPRow <= 64 ? kPBlock : 2 * kPBlock;
  static constexpr int kQTile = kWiden ? 2 * NR * D : NR * D * 2;
  static constexpr int kV16 = kWiden ? kBN * D * 2 : 0;       // a stream's widened V tile
  static constexpr int kFixed = 2 * kV16 + kP + kQTile;
  // K and V ring slots in what is left of 227 KB after this, the bookkeeping and the alignment pad.
  static constexpr int kMisc = (FP8 ? 9 : 6) * 1024;
  static constexpr int kRoom = 226 * 1024 - kMisc - kFixed;
  static constexpr int kRing = kRoom / kSlot < 14 ? kRoom / kSlot : 14;
  static constexpr int kRK = FP4 ? 4 : kRing / 2;  // (E2M1: two for each stream)
  // E2M1: codes of as many tiles as fit, in two rings.  The keys' are taken up sooner: three places of eight for them
  // (8 x 16384 keys, 8 heads, 32 rows 81 us; with one half 88, with a quarter 98).
  static constexpr int kCodeRoom = (kRoom - kRK * kSlot) / FourBit<D>::kHalf;
  static constexpr int kForKeys = kCodeRoom * 3 / 8;
  static constexpr int kRC = !FP4 ? 1 : kForKeys < kMaxRing ? kForKeys : kMaxRing;
  static constexpr int kRV = !FP4 ? kRing - kRK : kCodeRoom - kRC < kMaxRing ? kCodeRoom - kRC : kMaxRing;
  static constexpr int kOffK = 0;
  static constexpr int kOffV16 = kOffK + kRK * kSlot + (FP4 ? 0 : kRV * kSlot);
  static constexpr int kOffP = kOffV16 + 2 * kV16;
  static constexpr int kOffQ = kOffP + kP;
  static constexpr int kOffCodes = kOffQ + kQTile;            // E2M1: of keys, then of values
  static constexpr int kOffV = FP4 ? kOffCodes + kRC * FourBit<D>::kHalf : kOffK + kRK * kSlot;
  static constexpr int kOffMisc = FP4 ? kOffV + kRV * FourBit<D>::kHalf : kOffCodes;
  static constexpr int kSCols = kWiden ? 2 * NR : NR;         // TMEM columns of one stream's S
  static constexpr int kColO = 2 * kSCols;
  static constexpr int kColScales = kColO + 2 * kPCols;       // E2M1: of each K tile's scales, and of ones
  static constexpr int kCols = kColScales + (FP4 ? 20 : 0);
  static constexpr uint32_t kTmemCols = kCols <= 64 ? 64 : kCols <= 128 ? 128 : kCols <= 256 ? 256 : 512;
  static_assert(kRK >= 2 && kRV >= 2 && (!FP4 || kRC >= 2) && kRV <= kMaxRing && (!FP8 || kRV + 4 <= kScaleRing), "rings");
  static_assert(kQTile % 1024 == 0 && kSlot % 1024 == 0 && kCols <= 512, "swizzle atoms, TMEM");
};

template <int NR, int F>
struct Misc {
  static constexpr bool FP8 = F == kCacheE4m3;
  uint64_t k_full[kMaxRing], k_empty[kMaxRing], v_full[kMaxRing], v_empty[kMaxRing];
  uint64_t code_full[F == kCacheE2m1 ? kMaxRing : 1], code_empty[F == kCacheE2m1 ? kMaxRing : 1];
  uint64_t ref_full[2][2], v16_full[2];  // E2M1: per stream (and tile)
  int ref[2][2];                       // E2M1: 2·(exponent that a stream's widened tile is relative to) + (it is bf16)
  int range[2][4];                     // E2M1: per stream and warp
  uint64_t s_full[2], s_free[2], p_full[2], p_free[2], sc_full[kScaleRing], q_full, q_empty, drain;
  alignas(16) float nm[2][NR];         // minus the reference maxima (log2 units), 0 while a row has seen nothing
  alignas(16) float f[kFRing][NR];     // E4M3, E2M1: what a row's raw scores are multiplied by
  float corr[2][NR];                   // factor of the last rescale
  float red[2][4][NR];                 // per-warp maxima or sums
  float scale[2][NR];                  // what a stream's O is multiplied by in the end
  float kv_scale[2];                   // E4M3, E2M1: and by this
  int64_t row[2][NR];                  // (b·Hq + h)·T + t of a live row, or −1
  int64_t o_off[2][NR];                // its element offset in O
  int fresh[2][NR];                    // a live row that has seen nothing yet
  int far[2];                          // E4M3, E2M1: the stream's tile has gone over to bf16
  int kv_red[2][4];                    // per stream and warp
  alignas(16) uint8_t k_scale[FP8 ? kScaleRing : 1][kBN];  // written by bulk copies
  alignas(16) uint8_t v_scale[FP8 ? kScaleRing : 1][kBN];
  uint32_t bad[kBadRing][8];           // drafted keys with non-finite values (one bit each)
  long long warp_sum[24];
  int start[3];
  uint32_t tmem_base;
  int abort_flag;
};

struct OpMax {
  __device__ __forceinline__ float operator()(float a, float b) const { return fmaxf(a, b); }
};
struct OpAdd {
  __device__ __forceinline__ float operator()(float a, float b) const { return a + b; }
};

// Reduces each of N columns over the warp's 32 lanes by halving: at every step a
// lane hands over the half of its columns that its partner keeps.  The totals go
// to out[0 … N − 1].
template <int N, class Op>
__device__ __forceinline__ void reduce_cols(float (&v)[N], int lane, Op op, float* out) {
  int base = 0;
#pragma unroll
  for (int step = 0; step < 5; ++step) {
    const int mask = 16 >> step;
    const int half = N >> (step + 1);
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
  static_assert(N <= 32, "one total per lane");
  if ((lane & (32 / N - 1)) == 0) out[base] = v[0];
}

// Widens one value row of D E4M3 codes to fp16, times the pair of scales (all of context keys).  src: the row in its slot,
// swizzled as TMA wrote it; dst: the row in the first 64-column block of the fp16 tile.
template <int D>
__device__ __forceinline__ void widen_row(const uint8_t* src, uint8_t* dst, int r, uint32_t scale2) {
  const int sw = D == 128 ? r & 7 : (r >> 1) & 3;
#pragma unroll
  for (int ch = 0; ch < D / 16; ++ch) {
    const uint4 v = *reinterpret_cast<const uint4*>(src + ((ch ^ sw) << 4));
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    uint32_t o[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const uint32_t h = e4m3x2_to_f16x2(w[e >> 1] >> (16 * (e & 1)));
      const __half2 x = __hmul2(*reinterpret_cast<const __half2*>(&h), *reinterpret_cast<const __half2*>(&scale2));
      o[e] = *reinterpret_cast<const uint32_t*>(&x);
    }
    uint8_t* block = dst + (ch >> 2) * kBN * 128;  // 64 elements per 128-byte row
    *reinterpret_cast<uint4*>(block + ((((ch & 3) * 2) ^ (r & 7)) << 4)) = make_uint4(o[0], o[1], o[2], o[3]);
    *reinterpret_cast<uint4*>(block + ((((ch & 3) * 2 + 1) ^ (r & 7)) << 4)) = make_uint4(o[4], o[5], o[6], o[7]);
  }
}

// Multiplies N columns of this thread's lane by w[i]·k.
template <int N>
__device__ __forceinline__ void rescale_cols(uint32_t addr, const float* w, float k) {
  constexpr int C = N < 32 ? N : 32;
#pragma unroll
  for (int c = 0; c < N; c += C) {
    uint32_t r[C];
    tmem_ld(addr + c, r);
    tmem_wait_ld();
    reg_fence(r);
#pragma unroll
    for (int i = 0; i < C; ++i) r[i] = __float_as_uint(__uint_as_float(r[i]) * (w[c + i] * k));
    tmem_st(addr + c, r);
  }
  tmem_wait_st();
}

// The query rows of a piece as a K-major operand (rows that are not there as
// zeros), by NT threads.  E4M3, E2M1: two terms per element and the factor of the row.
template <int D, int F, int NR, int NT, int kBatchMax>
__device__ __forceinline__ void load_q(const TreeParams& p, const TreeWalk& w, uint8_t* q_smem, float* f, int id) {
  constexpr int kChunks = D / 8;  // 16-byte chunks of a row
  constexpr int kPer = (NR * kChunks + NT - 1) / NT;
  constexpr int kBatch = kPer < kBatchMax ? kPer : kBatchMax;  // loads in flight per thread
  const int live = w.drafts * p.G;
#pragma unroll 1
  for (int i0 = 0; i0 < kPer; i0 += kBatch) {
    uint4 q4[kBatch];
#pragma unroll
    for (int e = 0; e < kBatch; ++e) {
      const int i = (i0 + e) * NT + id;
      const int n = i / kChunks, ch = i % kChunks;
      q4[e] = make_uint4(0, 0, 0, 0);
      if (n < live) {
        const int t = token_of(p, n);
        q4[e] = *reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p.q) + w.b * p.sq[0] +
                                                (w.h * p.G + n - t * p.G) * p.sq[1] + t * p.sq[2] + ch * 8);
      }
    }
#pragma unroll
    for (int e8 = 0; e8 < kBatch; ++e8) {
      const int i = (i0 + e8) * NT + id;
      const int r = i / kChunks, ch = i % kChunks;
      if (r >= NR) continue;  // whole warps: a row is held by neighbouring lanes
      const uint4 v = q4[e8];
      if constexpr (F == kCacheBf16) {
        *reinterpret_cast<uint4*>(q_smem + (ch >> 3) * NR * 128 + r * 128 + (((ch & 7) ^ (r & 7)) << 4)) = v;
      } else {
        uint2 hi, lo;
        const int a = split_q8<kChunks, 4>(v, hi, lo);
        // Rows of D bytes; chunk of 16 bytes XORed with the row (128-byte rows) or half of it (64-byte rows).
        const int sw = D == 128 ? r & 7 : (r >> 1) & 3;  // NR is a multiple of 16: the same for rows r and NR + r
        uint8_t* dst = q_smem + r * D + (((ch >> 1) ^ sw) << 4) + (ch & 1) * 8;
        *reinterpret_cast<uint2*>(dst) = hi;
        *reinterpret_cast<uint2*>(dst + NR * D) = lo;
        if (ch == 0) f[r] = p.scale_log2 * __uint_as_float(static_cast<uint32_t>(a + 127) << 23);
      }
    }
  }
  fence_proxy_async_smem();
}

// E2M1: one warpgroup lays out the keys of both streams.  It spreads their codes as kind::mxf8f6f4 takes E2M1 elements
// (sixteen to 16 bytes, in the lower eight: rows of as many bytes as E4M3 rows) and puts their scales into tensor memory.
// Rows past the end become zeros.
template <int D, int NR>
__device__ __forceinline__ void convert_keys(const TreeParams& p, const TreePart& my, uint8_t* smem,
                                             Misc<NR, kCacheE2m1>* ms, uint32_t tmem) {
  using C = Cfg<D, kCacheE2m1, NR>;
  constexpr int kGroups = D / kE2m1Group;          // of a row
  constexpr int kItems = kTreeBN * kGroups / 128;  // 16-byte pieces of codes per thread
  constexpr int kItemRows = 128 / kGroups;
  volatile int* abort_flag = &ms->abort_flag;
  const int lane = threadIdx.x & 31, warp = (threadIdx.x >> 5) & 3, r = threadIdx.x & 127;
  const uint32_t scales = tmem + (static_cast<uint32_t>(warp * 32) << 16) + C::kColScales;
  const int r0 = r / kGroups, piece = r % kGroups;
  const int sw = D == 128 ? r0 & 7 : (r0 >> 1) & 3;  // the same for all of a thread's rows
  constexpr uint32_t kOnes = 0x7f7f7f7fu;            // the queries' scales, before the first keys are announced
  tmem_st4(scales + 16, kOnes, kOnes, kOnes, kOnes);
  Ring<C::kRC> rc;
  uint32_t used[2] = {0, 0};  // tiles of each stream so far
  bool ok = true;
  TreeWalk w;
  w.begin(p, my);
  do {
#pragma unroll 1
    for (int i = w.t0; i < w.t1; ++i) {
      // One of the stream's two K tiles and its scales.
      const int g = (i - w.t0) & 1;
      const uint32_t u = g == 0 ? used[0] : used[1];
      const uint32_t place = 2 * g + (u & 1);
      ok = mbar_wait_inl(&ms->code_full[rc.slot], rc.parity, abort_flag, p.err, tree_site(0x10)) &&
           mbar_wait_inl(&ms->k_empty[place], ((u >> 1) & 1) ^ 1, abort_flag, p.err, tree_site(0x11));
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      tc_fence_after();
      const uint8_t* src = smem + C::kOffCodes + rc.slot * FourBit<D>::kHalf;
      uint32_t s[4];
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const uint8_t* at = src + FourBit<D>::kCodes + (q * 32 + lane) * kGroups;
        s[q] = D == 128 ? *reinterpret_cast<const uint32_t*>(at) : *reinterpret_cast<const uint16_t*>(at);
      }
      tmem_st4(scales + place * 4, s[0], s[1], s[2], s[3]);
      const uint4* codes = reinterpret_cast<const uint4*>(src) + r;
      const int live = w.len - i * kTreeBN - r0;
      uint8_t* dst = smem + C::kOffK + place * C::kSlot + r0 * D;
      uint4 c[kItems];
#pragma unroll
      for (int it = 0; it < kItems; ++it) c[it] = codes[it * 128];
#pragma unroll
      for (int it = 0; it < kItems; ++it) {
        if (live < kTreeBN && it * kItemRows >= live) c[it] = make_uint4(0, 0, 0, 0);
        uint8_t* to = dst + it * kItemRows * D;
        *reinterpret_cast<uint4*>(to + (((2 * piece) ^ sw) << 4)) = make_uint4(c[it].x, c[it].y, 0, 0);
        *reinterpret_cast<uint4*>(to + (((2 * piece + 1) ^ sw) << 4)) = make_uint4(c[it].z, c[it].w, 0, 0);
      }
      fence_proxy_async_smem();
      __syncwarp();
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(&ms->k_full[place]);
        mbar_arrive(&ms->code_empty[rc.slot]);
      }
      __syncwarp();
      rc.advance();
      used[0] += g == 0;
      used[1] += g;
    }
  } while (ok && w.next(p));
}

// E2M1: a warpgroup of each stream widens the values to fp16, each group times its power of two relative to a running
// reference, which it tells the softmax.  Rows past the end become zeros.
//
// A tile with value groups too far below the reference is widened to bf16 instead, as with E4M3.
template <int D, int NR>
__device__ __forceinline__ void convert_values(const TreeParams& p, const TreePart& my, uint8_t* smem,
                                              Misc<NR, kCacheE2m1>* ms, int g) {
  using C = Cfg<D, kCacheE2m1, NR>;
  constexpr int kGroups = D / kE2m1Group;          // of a row
  volatile int* abort_flag = &ms->abort_flag;
  const int lane = threadIdx.x & 31, r = threadIdx.x & 127;
  uint8_t* const v_tile = smem + C::kOffV16 + g * C::kV16 + r * 128;
  // A wait that fails raises the abort flag, and all leave together, after a vote on it: until then a thread whose wait
  // has failed goes on, since the others wait for it at the vote without a limit.
  bool ok = true;
  int used = 0, ref = 0;  // tiles of this stream so far, and what the last one's values were relative to
  int tile0 = 0;  // tiles of the pieces before
  TreeWalk w;
  w.begin(p, my);
  do {
    const int n_tiles = w.t1 - w.t0, context = w.len - w.drafts;
#pragma unroll 1
    for (int i = g; i < n_tiles; i += 2) {
      // The values' powers of two: the largest and the smallest that count set the reference.  (Groups of NaN, rows that no
      // row sees, and 2^−126, next to nothing or zeros, do not.)
      const int slot = (tile0 + i) % C::kRV, key = (w.t0 + i) * kTreeBN + r;
      mbar_wait_inl(&ms->v_full[slot], ((tile0 + i) / C::kRV) & 1, abort_flag, p.err, tree_site(0x12));
      __syncwarp();
      const uint8_t* src = smem + C::kOffV + slot * FourBit<D>::kHalf;
      const uint8_t* at = src + FourBit<D>::kCodes + r * kGroups;
      const uint32_t bytes = D == 128 ? *reinterpret_cast<const uint32_t*>(at) : *reinterpret_cast<const uint16_t*>(at);
      bool counts = key < w.len;
      if (counts && key >= context && p.mask != nullptr)
        counts = any_token_sees(p.mask + w.b * p.mask_sb + (key - context), w.drafts, p.T);
      bool far = false;
      __syncwarp();
      if (named_any(4 + g, 128, i == g || (counts && outside_reference<kGroups>(bytes, ref)) || *abort_flag != 0)) {
        ok = !named_any(4 + g, 128, *abort_flag != 0);
        if (!ok) break;
        const int2 range = exponent_range<kGroups>(bytes, counts, 4 + g, ms->range[g]);
        if (i == g || range.x - 127 > ref + kFourLazy) ref = range.x - 127;
        far = range.y - 127 < ref - kFourFar;
      }
      // (The softmax has read the one two tiles ago: its product was waited for below.  It may not have read the last one,
      // so there are two barriers.)
      if (r == 0) {
        ms->ref[g][used & 1] = ref * 2 + (far ? 1 : 0);
        mbar_arrive(&ms->ref_full[g][used & 1]);
      }
      // The stream's widened tile is free once the second product before has run.
      if (used > 0) mbar_wait_inl(&ms->p_free[g], (used - 1) & 1, abort_flag, p.err, tree_site(0x13));
      __syncwarp();
      if (!far && (w.t0 + i + 1) * kTreeBN <= context) {
        // (Groups at a time 1, 2, 4: 54, 54, 53 us at 4 rows, 93, 84, 88 for 64 ragged sequences of up to 8192 keys in pages
        // of 16; 1, 2, 4 with 32 rows: 88, 88, 94.)
        widen_codes<D, NR == 16 ? 2 : 1>(src + r * (D / 2), bytes, v_tile, r, ref);
      } else if (widen_codes_edge<D>(src + r * (D / 2), bytes, v_tile, r, ref, key >= context, !counts, far)) {
        atomicOr(&ms->bad[w.index % kBadRing][(key - context) >> 5], 1u << ((key - context) & 31));
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(&ms->v16_full[g]);
        mbar_arrive(&ms->v_empty[slot]);
      }
      ++used;
    }
    tile0 += n_tiles;
    // Both streams' converters begin a piece together: one whose stream has no tiles in some pieces would run ahead of the
    // loads by more than a barrier's two phases can tell.  (And the piece's last waits have had no vote.)
    __syncwarp();
    ok = !named_any(6, 256, !ok || *abort_flag != 0);
  } while (ok && w.next(p));
}

// E2M1: the products of one stream, by a warp each.  The whole warp runs the loop, which keeps descriptors warp-uniform,
// and one elected lane issues, in loops that are not unrolled (64 ragged sequences of up to 8192 keys: 84 us instead of 86;
// all roles compete for instruction fetches).
template <int D, int NR>
__device__ __forceinline__ void issue_products(const TreeParams& p, const TreePart& my, uint8_t* smem,
                                               Misc<NR, kCacheE2m1>* ms, uint32_t tmem, int g) {
  using C = Cfg<D, kCacheE2m1, NR>;
  constexpr uint32_t kIdescO = idesc_f16_f32(128, NR, true, true), kIdescFar = idesc_bf16_f32(128, NR, true, true);
  volatile int* abort_flag = &ms->abort_flag;
  const uint32_t sQ = smem_u32(smem + C::kOffQ), sK = smem_u32(smem + C::kOffK) + 2 * g * C::kSlot;
  const uint64_t q_desc = D == 64 ? sdesc_sw64(sQ, 16, 512) : sdesc_sw128(sQ, 16, 1024);
  const uint64_t k_desc = D == 64 ? sdesc_sw64(sK, 16, 512) : sdesc_sw128(sK, 16, 1024);
  const uint64_t v_desc = sdesc_sw128(smem_u32(smem + C::kOffV16) + g * C::kV16, D == 128 ? kBN * 128 : 0, 1024);
  const uint64_t p_desc = sdesc_sw128(smem_u32(smem + C::kOffP) + g * C::kPNext, kPBlock, 1024);
  const uint32_t ds = tmem + g * C::kSCols, dst = tmem + C::kColO + g * C::kPCols;
  const uint32_t scales = tmem + C::kColScales + 8 * g, ones = tmem + C::kColScales + 16;
  const bool leader = elect_one_lane();
  uint32_t u = 0;  // tiles of this stream whose scores have been issued
  bool ok = true;
  TreeWalk w;
  w.begin(p, my);
  do {
    const int tiles = __shfl_sync(0xffffffffu, (w.t1 - w.t0 + 1 - g) >> 1, 0);  // of the piece, this stream's
    ok = mbar_wait_inl(&ms->q_full, w.index & 1, abort_flag, p.err, tree_site(14));
    // S runs a tile ahead, so that the next scores are ready when the softmax has stored P̃.
#pragma unroll 1
    for (int s = 0; s <= tiles; ++s) {
      if (s < tiles) {
        const uint32_t b = u & 1u;
        ok = ok && mbar_wait_inl(&ms->k_full[2 * g + b], (u >> 1) & 1u, abort_flag, p.err, tree_site(5)) &&
             mbar_wait_inl(&ms->s_free[g], (u & 1u) ^ 1u, abort_flag, p.err, tree_site(6));
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        tc_fence_after();
        if (leader) {
          // A k-step is a group of 32 elements, whose power of two the product applies.  Both of q's terms are columns.
          const uint64_t ad = k_desc + b * (C::kSlot >> 4);
#pragma unroll 1
          for (int kk = 0; kk < D / 32; ++kk)
            mma_mx_ss(ds, ad + kk * 2, q_desc + kk * 2, idesc_mx_e2m1_e4m3(128, 2 * NR, kk), scales + 4 * b, ones,
                      kk > 0 ? 1u : 0u);
          mma_commit(&ms->s_full[g]);
          mma_commit(&ms->k_empty[2 * g + b]);
        }
        ++u;
      }
      if (s == max(tiles - 1, 0) && leader) mma_commit(&ms->q_empty);  // (without tiles too: the barrier counts both streams)
      if (s > 0) {  // the second product of the tile before
        const uint32_t before = u - (s < tiles ? 2u : 1u);
        ok = ok && mbar_wait_inl(&ms->v16_full[g], before & 1u, abort_flag, p.err, tree_site(12)) &&
             mbar_wait_inl(&ms->p_full[g], before & 1u, abort_flag, p.err, tree_site(3));
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        tc_fence_after();
        const bool far = *static_cast<volatile int*>(&ms->far[g]) != 0;
        if (leader) {
          const uint32_t idesc = far ? kIdescFar : kIdescO;
#pragma unroll 1
          for (int kk = 0; kk < kBN / 16; ++kk)
            mma_bf16_ss(dst, v_desc + kk * 128, p_desc + kk * 128, idesc, (s > 1 || kk > 0) ? 1u : 0u);
          if (far) {  // the second terms
#pragma unroll 1
            for (int kk = 0; kk < kBN / 16; ++kk)
              mma_bf16_ss(dst, v_desc + kk * 128, p_desc + NR / 8 + kk * 128, idesc, 1u);
          }
          mma_commit(&ms->p_free[g]);
        }
      }
    }
  } while (ok && __shfl_sync(0xffffffffu, w.next(p), 0));
  if (leader) {  // the products are done before the end frees the tensor memory
    mma_commit(&ms->drain);
    mbar_wait_drain_inl(&ms->drain, 0, kTreeDrainNs);
  }
}

// R: rows that the softmax works on, of the NR columns of the products.
template <int D, int F, int NR, int R>
__global__ void __launch_bounds__(Cfg<D, F, NR>::kThreads, 1) tree_kernel(const __grid_constant__ TreeParams p) {
  using C = Cfg<D, F, NR>;
  constexpr bool FP8 = C::FP8, FP4 = C::FP4, kWiden = C::kWiden;
  constexpr bool kPg5 = !kWiden && D == 128;  // K/V pages as [row group][half][8 rows][128 bytes]
  constexpr int kSlot = C::kSlot;
  // Rescale once a score exceeds the reference by kLazy; the reference is taken kBase below the maximum.
  constexpr float kLazy = kWiden ? 11.f : 8.f;
  constexpr float kBase = kWiden ? 3.f : 0.f;
  constexpr int kKvLazy = 7;  // widened values stay below 448·2^7
  constexpr int kKvFar = 15;  // value rows that are smaller by more than this need bf16's range
  extern __shared__ uint8_t smem_raw[];
  const uint32_t pad = (1024u - (smem_u32(smem_raw) & 1023u)) & 1023u;
  uint8_t* smem = smem_raw + pad;
  Misc<NR, F>* ms = reinterpret_cast<Misc<NR, F>*>(smem + C::kOffMisc);
  volatile int* abort_flag = &ms->abort_flag;

  const int tid = threadIdx.x;
  const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);  // broadcast: known to be the same in the warp
  const int lane = tid & 31;
  const int part = blockIdx.x;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");  // the joining kernel waits for this grid's end

  if (tid == 0) {
    for (int s = 0; s < C::kRK; ++s) {
      mbar_init(&ms->k_full[s], FP4 ? 4 : 1);
      mbar_init(&ms->k_empty[s], 1);
    }
    for (int s = 0; FP4 && s < C::kRC; ++s) {
      mbar_init(&ms->code_full[s], kCodeArrivals);
      mbar_init(&ms->code_empty[s], 4);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(&ms->ref_full[s][0], 1);
      mbar_init(&ms->ref_full[s][1], 1);
      mbar_init(&ms->v16_full[s], 4);
    }
    for (int s = 0; s < C::kRV; ++s) {
      mbar_init(&ms->v_full[s], FP4 ? kCodeArrivals : 1);
      mbar_init(&ms->v_empty[s], kWiden ? 4 : 1);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(&ms->s_full[s], 1);
      mbar_init(&ms->s_free[s], 128);
      mbar_init(&ms->p_full[s], 128);
      mbar_init(&ms->p_free[s], 1);
    }
    for (int s = 0; s < kScaleRing; ++s) mbar_init(&ms->sc_full[s], 1);
    mbar_init(&ms->q_full, 32);
    mbar_init(&ms->q_empty, FP4 ? 2 : 1);
    mbar_init(&ms->drain, FP4 ? 2 : 1);
    ms->abort_flag = 0;
    fence_barrier_init();
  }
  if (tid < kBadRing * 8) ms->bad[tid >> 3][tid & 7] = 0;
  if (warp == 9) {
    tmem_alloc(&ms->tmem_base, C::kTmemCols);
    tmem_relinquish();
  }
  const TreePart my = find_part<C::kThreads>(p, part, ms->warp_sum, ms->start);
  const uint32_t tmem = ms->tmem_base;

  if (my.count <= 0) {
    // nothing left for this CTA
  } else if (FP4 && warp >= 12) {
    if (warp < 20) {
      reg_dealloc<C::kRegsConvert>();
      if constexpr (FP4) convert_values<D, NR>(p, my, smem, ms, (warp - 12) >> 2);
    } else {
      reg_dealloc<C::kRegsOther>();
      if constexpr (FP4) convert_keys<D, NR>(p, my, smem, ms, tmem);
    }
  } else if (FP4 && warp == 8) {
    reg_dealloc<C::kRegsOther>();
    if constexpr (FP4)
      load_codes<D, C::kRC, kKeyCodes>(p, my, smem + C::kOffCodes, ms->code_full, ms->code_empty, abort_flag, tree_site(1),
                                       [](const TreeWalk&) { return true; });
  } else if (FP4 && warp == 11) {
    reg_dealloc<C::kRegsOther>();
    // The values, and Q of every piece but the first, which the streams load, once the products of the piece before are
    // done with it.
    if constexpr (FP4)
      load_codes<D, C::kRV, kValueCodes>(p, my, smem + C::kOffV, ms->v_full, ms->v_empty, abort_flag, tree_site(2),
                                         [&](const TreeWalk& w) {
        if (w.index == 0) return true;
        if (!__all_sync(0xffffffffu, mbar_wait_inl(&ms->q_empty, (w.index & 1) ^ 1, abort_flag, p.err, tree_site(15))))
          return false;
        load_q<D, F, NR, 32, 2>(p, w, smem + C::kOffQ, ms->f[w.index % kFRing], lane);
        mbar_arrive(&ms->q_full);
        return true;
      });
  } else if (FP4 && (warp == 9 || warp == 10)) {
    reg_dealloc<C::kRegsOther>();
    if constexpr (FP4) issue_products<D, NR>(p, my, smem, ms, tmem, warp - 9);
  } else if (!FP4 && (warp == 8 || warp == 10)) {
    reg_dealloc<C::kRegsOther>();
    // ------------------------------------------- loads of K (warp 8) and V (warp 10)
    const bool is_v = warp == 10;
    if constexpr (!FP4)
      load_pages<D, FP8, kScaleRing>(p, my, is_v, smem + (is_v ? C::kOffV : C::kOffK), is_v ? C::kRV : C::kRK,
                                     is_v ? ms->v_full : ms->k_full, is_v ? ms->v_empty : ms->k_empty, ms->sc_full,
                                     ms->k_scale[0], ms->v_scale[0], abort_flag, tree_site(is_v ? 2 : 1));
  } else if (!FP4 && warp == 9) {
    reg_dealloc<C::kRegsOther>();
    // ------------------------------------------------------------ MMA issuer
    // The whole warp runs the loop, which keeps descriptors warp-uniform, and one elected lane issues.
    constexpr uint32_t kIdescS = FP8 ? idesc_e4m3_f32(128, 2 * NR, false, false)
                                       : idesc_bf16_f32(128, NR, false, false);
    constexpr uint32_t kIdescO = kWiden ? idesc_f16_f32(128, NR, true, true) : idesc_bf16_f32(128, C::kPCols, true, true);
    constexpr uint32_t kIdescFar = idesc_bf16_f32(128, NR, true, true);
    const uint32_t sQ = smem_u32(smem + C::kOffQ), sK = smem_u32(smem + C::kOffK), sP = smem_u32(smem + C::kOffP);
    const uint32_t sV = smem_u32(smem + (kWiden ? C::kOffV16 : C::kOffV));
    const uint64_t q_desc = kWiden && D == 64 ? sdesc_sw64(sQ, 16, 512) : sdesc_sw128(sQ, 16, 1024);
    const bool leader = elect_one_lane();
    Ring<C::kRK> rk;
    Ring<C::kRV> rv;
    uint32_t s_par = 3, p_par = 0;  // parities of s_free and p_full to wait for, a bit per stream
    bool ok = true;
    TreeWalk w;
    w.begin(p, my);
    do {
      // Tile s of the piece belongs to stream s & 1.  Broadcast, like the walk's end below, to keep the loop uniform.
      const int tiles = __shfl_sync(0xffffffffu, w.t1 - w.t0, 0);
      ok = mbar_wait_inl(&ms->q_full, w.index & 1, abort_flag, p.err, tree_site(14));
      // S runs two tiles ahead, so that a stream's next scores are ready when it has stored P̃.
#pragma unroll 1
      for (int s = 0; s < tiles + 2; ++s) {
        const int g = s & 1;
        if (s < tiles) {
          ok = ok && mbar_wait_inl(&ms->k_full[rk.slot], rk.parity, abort_flag, p.err, tree_site(5)) &&
               mbar_wait_inl(&ms->s_free[g], (s_par >> g) & 1u, abort_flag, p.err, tree_site(6));
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          s_par ^= 1u << g;
          tc_fence_after();
          const uint32_t kb = sK + rk.slot * kSlot;
          const uint32_t ds = tmem + g * C::kSCols;
          if (leader) {
            // Descriptors of the k-steps differ from the first ones by their start addresses alone.
            if constexpr (FP8) {
              const uint64_t ad = D == 128 ? sdesc_sw128(kb, 16, 1024) : sdesc_sw64(kb, 16, 512);
#pragma unroll
              for (int kk = 0; kk < D / 32; ++kk)
                mma_e4m3_ss(ds, ad + kk * 2, q_desc + kk * 2, kIdescS, kk > 0 ? 1u : 0u);
            } else {
              const uint64_t ad = sdesc_sw128(kb, 16, kPg5 ? 2048 : 1024);
#pragma unroll
              for (int kk = 0; kk < D / 16; ++kk)
                mma_bf16_ss(ds, ad + (kk >> 2) * 64 + (kk & 3) * 2, q_desc + (kk >> 2) * (NR * 8) + (kk & 3) * 2,
                            kIdescS, kk > 0 ? 1u : 0u);
            }
            mma_commit(&ms->s_full[g]);
            mma_commit(&ms->k_empty[rk.slot]);
            if (s == tiles - 1) mma_commit(&ms->q_empty);
          }
          rk.advance();
        }
        if (s >= 2) {  // the second product of tile s − 2, of the same stream
          ok = ok && mbar_wait_inl(&ms->p_full[g], (p_par >> g) & 1u, abort_flag, p.err, tree_site(3));
          if constexpr (!FP8) ok = ok && mbar_wait_inl(&ms->v_full[rv.slot], rv.parity, abort_flag, p.err, tree_site(4));
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          p_par ^= 1u << g;
          tc_fence_after();
          const uint32_t vb = sV + (FP8 ? g * C::kV16 : rv.slot * kSlot);
          const uint32_t dst = tmem + C::kColO + g * C::kPCols;
          const bool far = FP8 && *static_cast<volatile int*>(&ms->far[g]) != 0;
          if (leader) {
            // A: 16 keys per k-step, the head dim along M in 64-element blocks (D = 64: the one block twice, the upper
            // 64 rows of the result are not read).  B: 16 keys of P̃ᵀ.
            const uint64_t ad = kPg5 ? sdesc_sw128(vb, 1024, 2048) : sdesc_sw128(vb, D == 128 ? kBN * 128 : 0, 1024);
            const uint64_t bd = sdesc_sw128(sP + g * C::kPNext, kPBlock, 1024);
            const uint32_t idesc = far ? kIdescFar : kIdescO;
#pragma unroll
            for (int kk = 0; kk < kBN / 16; ++kk)
              mma_bf16_ss(dst, ad + kk * (kPg5 ? 256 : 128), bd + kk * 128, idesc, (s >= 4 || kk > 0) ? 1u : 0u);
            if (far) {  // the second terms
#pragma unroll 1
              for (int kk = 0; kk < kBN / 16; ++kk)
                mma_bf16_ss(dst, ad + kk * (kPg5 ? 256 : 128), bd + NR / 8 + kk * 128, idesc, 1u);
            }
            mma_commit(&ms->p_free[g]);
            if constexpr (!FP8) mma_commit(&ms->v_empty[rv.slot]);
          }
          rv.advance();
        }
      }
    } while (ok && __shfl_sync(0xffffffffu, w.next(p), 0));
    if (leader) {  // the same for the products, which the end frees the tensor memory of
      mma_commit(&ms->drain);
      mbar_wait_drain_inl(&ms->drain, 0, kTreeDrainNs);
    }
  } else if (warp < 8) {
    reg_alloc<C::kRegsSoftmax>();
    // ----------------------------- softmax: one key per thread, the stream's R rows
    const int g = warp >> 2;
    const int bar = 1 + g;                 // the stream's barrier
    const int kt = tid & 127;              // key in the tile, TMEM lane, head dim of O
    const uint32_t lane_base = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t s_addr = tmem + lane_base + g * C::kSCols;
    const uint32_t o_addr = tmem + lane_base + C::kColO + g * C::kPCols;
    float* nm = ms->nm[g];
    float* corr = ms->corr[g];
    float* red = ms->red[g][0];            // + warp·R
    int64_t* row = ms->row[g];
    int64_t* o_off = ms->o_off[g];
    int* fresh = ms->fresh[g];
    int tile0 = 0;                         // tiles of the pieces before, and those of this stream
    int used = 0;
    bool ok = true;
    TreeWalk w;
    w.begin(p, my);
    load_q<D, F, NR, 256, 4>(p, w, smem + C::kOffQ, ms->f[0], tid);
    named_sync(3, 256);
    if (warp == 0) mbar_arrive(&ms->q_full);
    if constexpr (R < NR) {  // P̃'s columns that no row is worked on for stay zeros
#pragma unroll
      for (int ch = 0; ch < 2 * NR / 8; ++ch)
        if (ch % (NR / 8) >= R / 8)
          *reinterpret_cast<uint4*>(smem + C::kOffP + kt * 128 + (((g * (C::kPNext / 16) + ch) ^ (kt & 7)) << 4)) =
              make_uint4(0, 0, 0, 0);
    }
#pragma unroll 1
    do {
      const int n_tiles = w.t1 - w.t0;
      const int context = w.len - w.drafts;
      const int live = w.drafts * p.G;  // rows that belong to a drafted token
      if (kt < NR) {
        const int t = token_of(p, kt);
        const int h = w.h * p.G + (kt - t * p.G);
        row[kt] = kt < live ? (static_cast<int64_t>(w.b) * p.Hq + h) * p.T + t : -1;
        o_off[kt] = w.b * p.so[0] + h * p.so[1] + static_cast<int64_t>(t) * p.so[2];
        nm[kt] = 0.f;
        fresh[kt] = kt < live;
      }
      named_sync(bar, 128);
      bool unseen = true;  // some row may have seen nothing yet
      float l[R];
#pragma unroll
      for (int n = 0; n < R; ++n) l[n] = 0.f;
      int kv_ref = -1024;
      int done = 0;  // tiles of this piece that this stream has worked on
      const float* f_row = ms->f[w.index % kFRing];
#pragma unroll 1
      for (int i = g; i < n_tiles; i += 2, ++done) {
        const int tile = tile0 + i;
        const int u = used + done;
        const int key = (w.t0 + i) * kBN + kt;
        const bool tail = (w.t0 + i + 1) * kBN > context;  // the tile holds drafted keys or the end
        // Which rows see this key (bit per row); context keys are seen by all.
        uint32_t seen = 0xffffffffu;
        if (tail && key >= context) {
          seen = 0;
          if (key < w.len && live > 0) {
            // Token by token: one byte of the mask stands for G rows.
            const uint8_t* mk = p.mask != nullptr ? p.mask + w.b * p.mask_sb + (key - context) : nullptr;
#pragma unroll 4
            for (int t = 0; t < w.drafts; ++t) {
              const bool on = mk != nullptr ? mk[static_cast<int64_t>(t) * p.T] != 0 : key - context <= t;
              const uint32_t bits = (0xffffffffu >> (32 - p.G)) << (t * p.G);  // its rows
              seen |= on ? bits : 0;
            }
          }
        }
        // E4M3: the powers of two of the key (byte 0 stands for 2^−127, below the normal numbers) and the value row.
        float ks = 1.f;
        int kv = -1024;
        if constexpr (FP8) {
          ok = mbar_wait_inl(&ms->sc_full[tile % kScaleRing], (tile / kScaleRing) & 1, abort_flag, p.err, tree_site(13)) && ok;
          const uint32_t sk = ms->k_scale[tile % kScaleRing][kt];
          ks = sk == 0 ? 5.877471754111438e-39f : __uint_as_float(sk << 23);
          // (A drafted key that no row sees takes no part in the maximum, whatever it holds.)
          if (key < w.len && seen != 0) kv = static_cast<int>(ms->v_scale[tile % kScaleRing][kt]) - 127;
        }
        int code = 0;  // E2M1: the converters say what the tile's widened values are relative to
        if constexpr (FP4) {
          ok = mbar_wait_inl(&ms->ref_full[g][u & 1], (u >> 1) & 1, abort_flag, p.err, tree_site(13)) && ok;
          code = *static_cast<volatile int*>(&ms->ref[g][u & 1]);
        }
        ok = mbar_wait_inl(&ms->s_full[g], u & 1, abort_flag, p.err, tree_site(7)) && ok;
        tc_fence_after();
        // x = score − reference, masked to −∞ where the row does not see the key.  A second time where a reference
        // has moved.
        float x[R];
        bool far = FP4 && (code & 1);  // value rows too far apart for fp16
        bool dead = false;  // a wait of some thread of the stream has failed
#pragma unroll 1
        for (bool again = false;; again = true) {
          // 16 rows at a time; with registers to spare the next ones are on their way from TMEM meanwhile.
          constexpr int kC = R < 16 ? R : 16;
          constexpr int kBuf = R > kC && !FP4 ? 2 : 1;
          uint32_t hi[kBuf][kC], lo[kBuf][kC];
          auto fetch = [&](int c, int to) {
            tmem_ld(s_addr + c, hi[to]);
            if constexpr (kWiden) tmem_ld(s_addr + NR + c, lo[to]);  // the columns of q's second terms
          };
          fetch(0, 0);
#pragma unroll
          for (int c = 0; c < R; c += kC) {
            const int now = (c / kC) % kBuf;
            tmem_wait_ld();
            reg_fence(hi[now]);
            if constexpr (kWiden) reg_fence(lo[now]);
            if (kBuf == 2 && c + kC < R) fetch(c + kC, now ^ 1);
#pragma unroll
            for (int e = 0; e < kC; e += 4) {
              const int n = c + e;
              float4 r4 = make_float4(__uint_as_float(hi[now][e]), __uint_as_float(hi[now][e + 1]),
                                      __uint_as_float(hi[now][e + 2]), __uint_as_float(hi[now][e + 3]));
              float4 f4 = make_float4(p.scale_log2, p.scale_log2, p.scale_log2, p.scale_log2);
              if constexpr (kWiden) {
                ffma2(r4.x, r4.y, __uint_as_float(lo[now][e]), __uint_as_float(lo[now][e + 1]), 0.0625f, 0.0625f, r4.x,
                      r4.y);
                ffma2(r4.z, r4.w, __uint_as_float(lo[now][e + 2]), __uint_as_float(lo[now][e + 3]), 0.0625f, 0.0625f,
                      r4.z, r4.w);
                f4 = *reinterpret_cast<const float4*>(&f_row[n]);
              }
              if constexpr (FP8) {
                fmul2(f4.x, f4.y, f4.x, f4.y, ks, ks);
                fmul2(f4.z, f4.w, f4.z, f4.w, ks, ks);
              }
              const float4 m4 = *reinterpret_cast<const float4*>(&nm[n]);
              ffma2(x[n], x[n + 1], r4.x, r4.y, f4.x, f4.y, m4.x, m4.y);
              ffma2(x[n + 2], x[n + 3], r4.z, r4.w, f4.z, f4.w, m4.z, m4.w);
            }
            if (kBuf == 1 && c + kC < R) fetch(c + kC, 0);
          }
          if (tail) {
#pragma unroll
            for (int n = 0; n < R; ++n)
              if (!((seen >> n) & 1)) x[n] = -INFINITY;
          }
          if (again) break;
          float mx[4] = {x[0], x[1], x[2], x[3]};
#pragma unroll
          for (int n = 4; n < R; n += 8)
#pragma unroll
            for (int e = 0; e < 4; ++e)
              mx[e] = n + 4 + e < R ? fmax3(mx[e], x[n + e], x[(n + 4 + e) % R]) : fmaxf(mx[e], x[n + e]);
          const float top = fmax3(fmaxf(mx[0], mx[1]), mx[2], mx[3]);
          const bool over = unseen || top > kLazy || (FP8 && (kv > kv_ref + kKvLazy || (kv > -126 && kv < kv_ref - kKvFar))) || (FP4 && code >> 1 != kv_ref);
          if (!named_any(bar, 128, over || !ok)) break;
          // A reference moves (the first tile always does): exchange the tile's maxima, rescale ℓ and O.
          if (named_any(bar, 128, !ok)) {
            ok = false;
            dead = true;
            break;
          }
          reduce_cols<R>(x, lane, OpMax(), red + (warp & 3) * R);
          if constexpr (FP8) {
            const int top_kv = __reduce_max_sync(0xffffffffu, kv);
            if (lane == 0) ms->kv_red[g][warp & 3] = top_kv;
          }
          named_sync(bar, 128);
          int kv_new = FP4 ? code >> 1 : kv_ref;
          if constexpr (FP8) {
            const int* kr = ms->kv_red[g];
            kv_new = max(kv_ref, max(max(kr[0], kr[1]), max(kr[2], kr[3])));
            far = named_any(bar, 128, kv > -126 && kv < kv_new - kKvFar);  // (−126: next to nothing, or zeros)
          }
          bool still = false;
          if (kt < R) {
            // Maxima relative to the old reference (0 for a row that has seen nothing).
            const float now = fmaxf(fmaxf(red[kt], red[R + kt]), fmaxf(red[2 * R + kt], red[3 * R + kt]));
            const bool first = fresh[kt] != 0;
            const bool up = now > -INFINITY && (first || now > kBase);
            corr[kt] = !up ? 1.f : first ? 0.f : exp2f(kBase - now);
            if (up) {
              nm[kt] += kBase - now;
              fresh[kt] = 0;
            }
            still = first && !up;
          }
          unseen = named_any(bar, 128, still);
#pragma unroll
          for (int n = 0; n < R; ++n) l[n] *= corr[n];
          if (done > 0) {
            ok = mbar_wait_inl(&ms->p_free[g], (u - 1) & 1, abort_flag, p.err, tree_site(8)) && ok;
            tc_fence_after();
            const float kf = kWiden ? exp2f(static_cast<float>(max(kv_ref - kv_new, -200))) : 1.f;
#pragma unroll 1
            for (int term = 0; term < C::kTerms; ++term) rescale_cols<R>(o_addr + term * NR, corr, kf);
          }
          kv_ref = kv_new;
        }
        if (dead) break;
        tc_fence_before();
        mbar_arrive(&ms->s_free[g]);

        // P̃'s buffer, and E4M3's widened values', are free once the product of the stream's tile before has run.
        if (u > 0) ok = mbar_wait_inl(&ms->p_free[g], (u - 1) & 1, abort_flag, p.err, tree_site(8)) && ok;
        // 16-byte chunks of the key's row, XORed with the key; the stream's begin at `first`.
        uint8_t* prow = smem + C::kOffP + (C::kPNext == kPBlock ? g * kPBlock : 0) + kt * 128;
        const int first = C::kPNext == kPBlock ? 0 : g * (C::kPNext / 16);
#pragma unroll
        for (int ch = 0; ch < R / 8; ++ch) {  // 8 rows per 16-byte chunk
          uint32_t hi[4], lo[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int n = ch * 8 + e * 2;
            x[n] = ex2_approx(x[n]);
            x[n + 1] = ex2_approx(x[n + 1]);
            fadd2(l[n], l[n + 1], l[n], l[n + 1], x[n], x[n + 1]);
            if constexpr (kWiden) {
              hi[e] = pack_f16x2(x[n], x[n + 1]);
            } else {
              split_weights2(x[n], x[n + 1], hi[e], lo[e]);
            }
          }
          *reinterpret_cast<uint4*>(prow + (((first + ch) ^ (kt & 7)) << 4)) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
          if constexpr (!kWiden) {
            const int c2 = first + ch + NR / 8;  // column chunk of the second term
            *reinterpret_cast<uint4*>(prow + ((c2 ^ (kt & 7)) << 4)) =
                make_uint4(lo[0], lo[1], lo[2], lo[3]);
          }
        }
        if (kWiden && far) {  // the weights as two bf16 terms, from what this thread has just stored
#pragma unroll 1
          for (int ch = 0; ch < R / 8; ++ch) {
            uint4* at = reinterpret_cast<uint4*>(prow + (((first + ch) ^ (kt & 7)) << 4));
            uint4 a = *at, d;
            split_f16x2(a.x, a.x, d.x);
            split_f16x2(a.y, a.y, d.y);
            split_f16x2(a.z, a.z, d.z);
            split_f16x2(a.w, a.w, d.w);
            *at = a;
            *reinterpret_cast<uint4*>(prow + (((first + ch + NR / 8) ^ (kt & 7)) << 4)) = d;
          }
        }
        if constexpr (FP8) {  // this key's value row to fp16
          const int slot = tile % C::kRV;
          ok = mbar_wait_inl(&ms->v_full[slot], (tile / C::kRV) & 1, abort_flag, p.err, tree_site(11)) && ok;
          const uint8_t* src = smem + C::kOffV + slot * kSlot + kt * D;
          uint8_t* dst = smem + C::kOffV16 + g * C::kV16 + kt * 128;
          if (kt == 0) ms->far[g] = far;
          const int e = kv - kv_ref;  // the row's power of two, at most 2^kKvLazy
          if (!tail && !far) {
            widen_row<D>(src, dst, kt, power_f16x2(e));
          } else if (far ? widen_row_far<D>(src, dst, kt, e, key >= context, key >= w.len)
                         : widen_row_edge<D>(src, dst, kt, power_f16x2(e), key >= context, key >= w.len)) {
            atomicOr(&ms->bad[w.index % kBadRing][(key - context) >> 5], 1u << ((key - context) & 31));
          }
        }
        if (FP4 && kt == 0) ms->far[g] = far;
        if (!kWiden && tail && key >= context) {
          // This key's value row: zeros past the end, and in place of what a drafted row holds that is not finite.
          const int slot = tile % C::kRV;
          ok = mbar_wait_inl(&ms->v_full[slot], (tile / C::kRV) & 1, abort_flag, p.err, tree_site(9)) && ok;
          uint8_t* vr = smem + C::kOffV + slot * kSlot + (kPg5 ? (kt >> 3) * 2048 + (kt & 7) * 128 : kt * 128);
          const bool bad = clean_value_row<D>(vr, key >= w.len);
          if (bad) atomicOr(&ms->bad[w.index % kBadRing][(key - context) >> 5], 1u << ((key - context) & 31));
        }
        fence_proxy_async_smem();
        tc_fence_before();
        mbar_arrive(&ms->p_full[g]);
        if constexpr (FP8) {
          __syncwarp();
          if (lane == 0) mbar_arrive(&ms->v_empty[tile % C::kRV]);
        }
      }
      tile0 += n_tiles;
      used += done;
      // ------------------------------------------------------------ end of the piece
      // (Its barriers are joined by all threads whatever the waits said.)
      if (done > 0) ok = ok && mbar_wait_inl(&ms->p_free[g], (used - 1) & 1, abort_flag, p.err, tree_site(10));
      reduce_cols<R>(l, lane, OpAdd(), red + (warp & 3) * R);
      tc_fence_before();
      named_sync(3, 256);
      tc_fence_after();
      const bool whole = w.whole();
      const int64_t slot_row = w.slot(p, part) * p.T * p.G;  // first row of the piece's slot
      if (R < NR && kt >= R && kt < NR) ms->scale[g][kt] = 0.f;
      if (kt < R) {
        // Both streams' sums in a fixed order: the same result every time.
        float sums[2], m = -INFINITY, sum = 0.f, mine = 0.f;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float* r4 = ms->red[e][0] + kt;
          sums[e] = (r4[0] + r4[R]) + (r4[2 * R] + r4[3 * R]);
          if (sums[e] != 0.f) m = fmaxf(m, -ms->nm[e][kt]);
        }
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float wgt = sums[e] == 0.f ? 0.f : exp2f(-ms->nm[e][kt] - m);
          sum += sums[e] * wgt;
          if (e == g) mine = wgt;
        }
        if (ok && row[kt] >= 0 && g == 0) {
          if (!whole) {
            p.part_ml[(slot_row + kt) * 2] = m;
            p.part_ml[(slot_row + kt) * 2 + 1] = sum;
          } else if (p.lse != nullptr) {
            p.lse[row[kt]] = sum != 0.f ? (m + log2f(sum)) * 0.6931471805599453f : -INFINITY;
          }
        }
        // What this stream's O is multiplied by, and then by the power of two that its values are relative to (not at
        // once: the product of the two may be too small a number).
        ms->scale[g][kt] = mine * (sum != 0.f ? 1.f / sum : 0.f);
      }
      if (kWiden && kt == 0) ms->kv_scale[g] = exp2f(static_cast<float>(max(kv_ref, -300)));
      if (w.t0 == 0 && tid == 0) p.pieces[w.pair(p)] = w.pieces(part, my.per);
      named_sync(3, 256);
      const uint32_t* bad = ms->bad[w.index % kBadRing];
      // Rows that this stream writes: half of them.
      constexpr int kOut = NR / 2;
      const int c0 = g * kOut;
      if (__all_sync(0xffffffffu, ok) && kt < D) {
        float o[kOut];
#pragma unroll
        for (int q = 0; q < kOut; ++q) o[q] = 0.f;
#pragma unroll 1
        for (int e = 0; e < 2; ++e) {  // streams
#pragma unroll 1
          for (int term = 0; term < C::kTerms; ++term) {
            uint32_t r[kOut];
            tmem_ld(tmem + lane_base + C::kColO + e * C::kPCols + term * NR + c0, r);
            tmem_wait_ld();
            reg_fence(r);
#pragma unroll
            for (int q = 0; q < kOut; ++q) {
              const float k = ms->scale[e][c0 + q];
              if (k == 0.f) continue;  // a stream without keys has left O unwritten
              o[q] += kWiden ? __uint_as_float(r[q]) * k * ms->kv_scale[e] : __uint_as_float(r[q]) * k;
            }
          }
        }
        __nv_bfloat16* out = static_cast<__nv_bfloat16*>(p.o) + kt;
        float* part_o = p.part_o + (slot_row + c0) * D + kt;
#pragma unroll
        for (int q = 0; q < kOut; ++q) {
          if (row[c0 + q] >= 0) {
            if (!whole)
              part_o[q * D] = o[q];
            else
              out[o_off[c0 + q]] = __float2bfloat16_rn(o[q]);
          }
        }
        // What was taken out of drafted value rows goes to the rows that see them.
        for (int u = 0; u < w.drafts; ++u) {
          if (bad[u >> 5] == 0) {
            u |= 31;
            continue;
          }
          if (!((bad[u >> 5] >> (u & 31)) & 1)) continue;
          const float v = taken_out<F>(p, value_row<D>(p, w, u) + kt);
          if (v == 0.f) continue;
#pragma unroll 1
          for (int q = 0; q < kOut; ++q) {
            if (row[c0 + q] < 0 || !token_sees(p, w.b, token_of(p, c0 + q), u)) continue;
            if (!whole)
              part_o[q * D] += v;
            else
              out[o_off[c0 + q]] = __float2bfloat16_rn(__bfloat162float(out[o_off[c0 + q]]) + v);
          }
        }
      }
      tc_fence_before();
      // All have read O and the statistics; any failed wait ends the walk for all.
      ok = !named_any(3, 256, !ok);
      // The flags of three pieces ago: the other stream may still be at the piece before.
      if (tid < 8) ms->bad[(w.index + kBadRing - 3) % kBadRing][tid] = 0;
    } while (ok && w.next(p));
  } else if (!FP4 && warp == 11) {
    reg_dealloc<C::kRegsOther>();
    // ------------------------- Q of every piece but the first, which the streams load
    TreeWalk w;
    w.begin(p, my);
#pragma unroll 1
    while (w.next(p)) {
      // Once the first products of the piece before are done.
      if (!__all_sync(0xffffffffu, mbar_wait_inl(&ms->q_empty, (w.index & 1) ^ 1, abort_flag, p.err, tree_site(15)))) break;
      load_q<D, F, NR, 32, 2>(p, w, smem + C::kOffQ, ms->f[w.index % kFRing], lane);
      mbar_arrive(&ms->q_full);
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 9) {
    tc_fence_after();
    tmem_dealloc(tmem, C::kTmemCols);
  }
}

// Joins the pieces of a cut pair, which hold o/ℓ: weights w = 2^(m − max)·ℓ, O = Σ w·(o/ℓ) / Σ w.  Rows that see
// nothing are written here too.  A thread takes E columns of a row; a warp takes a row, or, where the kernel for many
// rows has stored chunks of four columns for 32 rows side by side (WIDE), those columns of 32 rows.
constexpr int kMergeWarps = 4, kMergeWarpsWide = 8;
template <int D, bool WIDE>
__global__ void __launch_bounds__((WIDE ? kMergeWarpsWide : kMergeWarps) * 32)
    tree_merge_kernel(const __grid_constant__ TreeParams p) {
  constexpr int E = WIDE ? D / kMergeWarpsWide : D / 32;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int rows = p.T * p.G;
  int64_t pair;
  int rr, c0;
  if constexpr (WIDE) {
    const int groups = (rows + 31) >> 5;
    pair = blockIdx.x / groups;
    rr = static_cast<int>(blockIdx.x - pair * groups) * 32 + lane;
    c0 = warp * E;
    if (rr >= rows) return;
  } else {
    const unsigned r = blockIdx.x * kMergeWarps + warp;
    pair = r / rows;
    rr = static_cast<int>(r - pair * rows);
    c0 = lane * E;
    if (pair >= static_cast<int64_t>(p.B) * p.Hkv) return;
  }
  const int b = static_cast<int>(static_cast<unsigned>(pair) / p.Hkv);
  const int t = token_of(p, rr);
  const int h = static_cast<int>(pair - static_cast<int64_t>(b) * p.Hkv) * p.G + rr - t * p.G;
  int len, drafts;
  seq_lengths(p, b, len, drafts);
  __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(p.o) + b * p.so[0] + h * p.so[1] + t * p.so[2] + c0;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  float o[E];
#pragma unroll
  for (int e = 0; e < E; ++e) o[e] = 0.f;
  float m = -INFINITY, l = 0.f;
  if (t < drafts) {
    const int2 pieces = p.pieces[pair];
    if (pieces.y == 1) return;  // not cut: the first kernel has written it
    // A kernel that gave up on a wait may have left none.
    if (pieces.x < 0 || pieces.y < 1 || pieces.y > p.parts - pieces.x) return;
    auto slot = [&](int i) -> int64_t {
      return p.slots_by_pair ? pair + pieces.x + i : 2ll * (pieces.x + i) + (i > 0 ? 0 : 1);
    };
    const float2* ml = reinterpret_cast<const float2*>(p.part_ml);
    const int piece_rows = tree_piece_rows(rows);
    const int first = WIDE ? c0 * 32 - lane * (D - 4) : c0;  // the columns, from row rr's place in [piece_rows, D]
    constexpr int kStep = E < 4 ? E : 4;
    // Four pieces' statistics and rows are on their way at once.
    constexpr int kBatch = 4;
#pragma unroll 1
    for (int i = 0; i < pieces.y; i += kBatch) {
      float2 x[kBatch];
      float v[kBatch][E];
#pragma unroll
      for (int j = 0; j < kBatch; ++j) {
        x[j] = make_float2(-INFINITY, 0.f);
        if (i + j < pieces.y) {
          const int64_t at = slot(i + j) * rows + rr;
          x[j] = ml[at];
          const float* src = p.part_o + (slot(i + j) * piece_rows + rr) * D + first;
#pragma unroll
          for (int e = 0; e < E; e += kStep) {
            if constexpr (kStep == 4) {
              const float4 y = *reinterpret_cast<const float4*>(src + (WIDE ? e * 32 : e));
              v[j][e] = y.x, v[j][e + 1] = y.y, v[j][e + 2] = y.z, v[j][e + 3] = y.w;
            } else {
              const float2 y = *reinterpret_cast<const float2*>(src + e);
              v[j][e] = y.x, v[j][e + 1] = y.y;
            }
          }
        }
      }
      float top = m;
#pragma unroll
      for (int j = 0; j < kBatch; ++j) top = fmaxf(top, x[j].x);
      const float keep = l != 0.f ? exp2f(m - top) : 0.f;
      m = top;
      l *= keep;
#pragma unroll
      for (int e = 0; e < E; ++e) o[e] *= keep;
#pragma unroll
      for (int j = 0; j < kBatch; ++j) {
        if (x[j].y == 0.f) continue;
        const float w = exp2f(x[j].x - top) * x[j].y;
        l += w;
#pragma unroll
        for (int e = 0; e < E; ++e) o[e] += w * v[j][e];
      }
    }
  }
  const float inv = l != 0.f ? 1.f / l : 0.f;
#pragma unroll
  for (int e = 0; e < E; e += 2)
    *reinterpret_cast<uint32_t*>(dst + e) = l != 0.f ? pack_bf16x2(o[e] * inv, o[e + 1] * inv) : 0u;
  if (p.lse != nullptr && c0 == 0)
    p.lse[(static_cast<int64_t>(b) * p.Hq + h) * p.T + t] = l != 0.f ? (m + log2f(l)) * 0.6931471805599453f : -INFINITY;
}

template <int D, bool WIDE>
cudaError_t launch_merge(const TreeParams& p, cudaStream_t s) {
  const int64_t rows = static_cast<int64_t>(p.T) * p.G, pairs = static_cast<int64_t>(p.B) * p.Hkv;
  const int64_t blocks = WIDE ? pairs * ((rows + 31) / 32) : (pairs * rows + kMergeWarps - 1) / kMergeWarps;
  // Its blocks may come up while the first kernel runs; they wait for its end.
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(blocks));
  cfg.blockDim = dim3((WIDE ? kMergeWarpsWide : kMergeWarps) * 32);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, tree_merge_kernel<D, WIDE>, p);
}

template <int D, int F, int NR, int R = NR>
cudaError_t launch_rows(const TreeParams& p, cudaStream_t s) {
  constexpr int kSmem = Cfg<D, F, NR>::kOffMisc + static_cast<int>(sizeof(Misc<NR, F>)) + 1024;
  static_assert(kSmem <= 227 * 1024, "shared memory");
  using M = Misc<NR, F>;
  static_assert(Cfg<D, F, NR>::kOffMisc % 16 == 0 && offsetof(M, nm) % 16 == 0 && offsetof(M, f) % 16 == 0 &&
                    offsetof(M, k_scale) % 16 == 0 && offsetof(M, v_scale) % 16 == 0,
                "16-byte accesses and bulk copies");
  // The register split draws on what the block is launched with, which is the compiled kernel's for good.
  static std::atomic<bool> checked{false};
  cudaError_t e;
  if (!checked.load(std::memory_order_relaxed)) {
    cudaFuncAttributes a;
    e = cudaFuncGetAttributes(&a, tree_kernel<D, F, NR, R>);
    if (e != cudaSuccess) return e;
    if (a.numRegs < Cfg<D, F, NR>::kRegsLaunch) return cudaErrorInvalidConfiguration;
    checked.store(true, std::memory_order_relaxed);
  }
  e = cudaFuncSetAttribute(tree_kernel<D, F, NR, R>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
  if (e != cudaSuccess) return e;
  tree_kernel<D, F, NR, R><<<static_cast<unsigned>(p.parts), Cfg<D, F, NR>::kThreads, kSmem, s>>>(p);
  return cudaGetLastError();
}

template <int D, int F>
cudaError_t launch_d(const TreeParams& p, cudaStream_t s) {
  const int64_t rows = static_cast<int64_t>(p.T) * p.G;
  // By the rows of a pair; 8 sequences of 16384 keys, 8 key/value heads, us with the one and the other:
  //   4 and 16 rows as 16 columns or 32    E4M3 58, 59 | 64, 66    bf16 91, 92 | 91, 93 (head dim 64 54, 55 | 58, 58)
  //                                        E2M1 54, 62 | 71, 76 (head dim 64 47, 53 | 61, 64)
  //   16 and 32 rows here or in the kernel for many rows    E4M3 59, 68 | 76, 78    bf16 92, 95 | 95, 97
  //                                                         E2M1 62, 80 | 85, 87 (head dim 64 53, 66 | 74, 75)
  //   4 rows of which the softmax works on 8 or 16    E2M1 54 | 59 (head dim 64 47 | 51); the others' softmax is no bound
  //   at so few
  // (32 rows are the most that fit here without tiles of rows; 64 columns spilled registers and took 81 us where the
  // other kernel took 69: 8 tokens of 7 heads a group, 16 ragged sequences of up to 8192 bf16 keys.)
  const bool wide = rows > kTreeNarrowRows;
  constexpr int kFew = F == kCacheE2m1 ? 8 : 16;
  cudaError_t e = wide           ? launch_tree_wide(p, D, F, s)
                  : rows <= kFew ? launch_rows<D, F, 16, kFew>(p, s)
                  : rows <= 16   ? launch_rows<D, F, 16>(p, s)
                                 : launch_rows<D, F, 32>(p, s);
  if (e != cudaSuccess) return e;
  return wide ? launch_merge<D, true>(p, s) : launch_merge<D, false>(p, s);
}

}  // namespace

template <int D>
static cudaError_t launch_format(const TreeParams& p, int format, cudaStream_t s) {
  switch (format) {
    case kCacheBf16: return launch_d<D, kCacheBf16>(p, s);
    case kCacheE4m3: return launch_d<D, kCacheE4m3>(p, s);
    case kCacheE2m1: return launch_d<D, kCacheE2m1>(p, s);
  }
  return cudaErrorInvalidValue;
}

cudaError_t launch_decode_tree(const TreeParams& p, int d, int format, cudaStream_t s) {
  if (static_cast<int64_t>(p.B) * p.Hq * p.T >= (1ll << 31) || static_cast<int64_t>(p.parts) * p.row_tiles > 0x7fffffff)
    return cudaErrorInvalidValue;
  return d == 128 ? launch_format<128>(p, format, s) : d == 64 ? launch_format<64>(p, format, s) : cudaErrorInvalidValue;
}

}  // namespace fa

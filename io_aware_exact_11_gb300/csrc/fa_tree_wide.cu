// fa_tree_wide.cu — drafted-token attention for more than 32 query rows per
// (b, key/value head) pair.
//
// With that many rows nothing is padded away by putting them on the matrix rows,
// so this kernel works like the prefill forward: S = Q Kᵀ with 128 query rows on
// the M side, one softmax thread per row, P̃ written over S in tensor memory and
// read from there by O += P̃ V.  Per 128 × 128 scores that reads 96 KB of shared
// memory against 160 KB (and 32 KB of P̃ stored) in the transposed products of the
// kernel for few rows, and a row's maximum needs no other thread: with tiles of 64
// and 128 rows that one took 445 us where this one took 239 (8 sequences of 32768
// E4M3 keys, 8 key/value heads, 256 rows each; 243 to 246 now).
//
// Two streams (warpgroups): with up to 128 rows they share them and take alternate
// key tiles, joined at the end of a piece (TILES = 1); above, a CTA takes two tiles
// of 128 rows over the same keys (TILES = 2), row tiles beyond that being other
// CTAs that work on the same keys at the same time.  The MMA warp alternates: P̃₀V,
// S₀ of the next tile, P̃₁V, S₁.  One commit after a tile's scores says both that they
// are there and that O is stable.
//
// bf16 cache: with shared rows P̃ enters as two bf16 terms, as in the other kernel; with
// two row tiles as one, as in the prefill forward: there the products and exponentials
// are the bound.  E4M3 cache: q enters as hi + lo E4M3 terms into
// one accumulator (exact for elements down to 2⁻¹⁰ of the row's largest, below
// that off by at most 2⁻¹⁸ of it); four converter warps widen V to fp16, each row
// times its power of two relative to a reference that P̃ and O share, and lay out
// the keys' powers of two as floats.  P̃ is fp16, its reference 2^3 below the maximum.
// A tile with value rows further below the reference than 2^15 goes through bf16 (fa_tree.cu).
// E2M1 cache: eight converter warps widen K and V to fp16, each group times its power of two
// relative to a reference: the keys' is their tile's largest group, which multiplies the scores
// in fp32, the values' a running one.  From 2⁻²³ to 2^13 of it that is exact; keys further apart
// are taken each to its own largest group, values go through bf16.  q is fp16, its largest
// element between 2^14 and 2^15: exact down to 2⁻³¹ of that.  P̃ is fp16 as with E4M3.  (Products
// over the codes themselves, as in the kernel for few rows, would take q in two E4M3 terms, twice
// the tensor work at full width.)
//
// The rest (parts, pieces, masks, values in masked places) is as in fa_tree.cu.
//
// Measured on GB300, 8 sequences of 16384 keys, 8 key/value heads of 128 elements (replaying a graph over two caches):
//   64 / 128 / 256 rows, bf16    99 / 105 / 125 us   0.81 / 0.76 of a device copy, 1097 TFLOP/s
//   64 / 128 / 256 rows, E4M3    80 /  84 / 134 us   430 / 813 / 1023 TFLOP/s (32768 keys, 256 rows: 230 us, 1194)
//   64 / 128 / 256 rows, E2M1    88 /  91 / 144 us   390 / 756 / 956 TFLOP/s (32768 keys, 256 rows: 253 us, 1088)
// With two row tiles a step (one tile's P̃V and S, 1024 tensor cycles) takes about 1750 cycles: the issuing
// warp's own instructions, of which it gets one through every dozen cycles beside the softmax warps, and the wait
// for P̃ (S to P̃ is a chain of about 1400 cycles).  E4M3 with shared rows waits for the converters (2400 cycles a
// tile).  With E2M1 the softmax reads
// its scores twice, in rolled loops; with four converter warps for both halves and the scores held in registers the three took
// 131, 135 and 157 us.  Not kept: a second set of eight converter warps for every other tile, which takes registers from the
// softmax (97 us at 64 rows, from 91), and rings and loading warps of their own for the keys' and the values' codes (98).
// A pair boundary costs a CTA 10000 to 15000 cycles (O out, Q in, the first scores).
#include <stddef.h>

#include <atomic>
#include <type_traits>

#include "fa_tree.cuh"

namespace fa {
namespace {

constexpr int kBN = kTreeBN;
constexpr int kRowTile = 128;
constexpr int kMaxRing = 8;
constexpr int kMaxCodeRing = 8;
constexpr int kScaleRing = 16;
constexpr int kTileRing = 8;   // E4M3, E2M1: tiles whose converted scales and references are kept

template <int D, int F, int TILES>
struct Cfg {
  static constexpr bool FP8 = F == kCacheE4m3, FP4 = F == kCacheE2m1;
  static constexpr bool kWiden = FP8 || FP4;  // V, and with E2M1 K too, is widened to fp16
  // Warps: streams 0–3 and 4–7, K loads 8, MMA 9, V loads 10, idle 11; E4M3: converters 12–15; E2M1: all loads 8,
  // converters of keys 12–15 and of values 16–19.
  static constexpr int kThreads = FP4 ? 640 : FP8 ? 512 : 384;
  static constexpr int kRegsLaunch = FP4 ? 96 : FP8 ? 128 : 168;
  static constexpr int kRegsSoftmax = FP4 ? 144 : FP8 ? 200 : 208;
  static constexpr int kRegsOther = kWiden ? 56 : 88;
  static constexpr int kRegsConvert = FP4 ? 64 : FP8 ? kRegsOther : 0;
  static_assert(2 * kRegsSoftmax + kRegsOther + (FP4 ? 2 : 1) * kRegsConvert <= kThreads / 128 * kRegsLaunch,
                "register split");
  static constexpr int kSlot = kBN * D * (FP8 ? 1 : 2);
  static constexpr int kV16 = kWiden ? kBN * D * 2 : 0;
  static constexpr int kQTile = kRowTile * D * 2;        // bf16, fp16 or two E4M3 terms
  static constexpr int kTerms = !kWiden && TILES == 1 ? 2 : 1;  // of P̃
  static constexpr int kFixed = TILES * kQTile + 2 * kV16;
  static constexpr int kMisc = (FP8 ? 13 : FP4 ? 4 : 2) * 1024 + (TILES == 1 ? 4 * 1024 : 0);
  static constexpr int kRoom = 226 * 1024 - kFixed - kMisc;  // 227 KB less the alignment pad
  static constexpr int kRing = kRoom / kSlot < 14 ? kRoom / kSlot : 14;
  static constexpr int kRK = FP4 ? 2 : kRing / 2;
  static constexpr int kRV = FP4 ? 2 : kRing - kRK;
  static constexpr int kOffQ = 0;
  static constexpr int kOffV16 = kOffQ + TILES * kQTile;
  static constexpr int kOffK = kOffV16 + 2 * kV16;
  static constexpr int kOffV = kOffK + kRK * kSlot;
  // E2M1: half tiles of codes in what is left.
  static constexpr int kCodeRoom = (kRoom - kRK * kSlot) / FourBit<D>::kHalf;
  static constexpr int kCodeRing = !FP4 ? 1 : kCodeRoom < kMaxCodeRing ? kCodeRoom : kMaxCodeRing;
  static_assert(!FP4 || kCodeRing >= 3, "codes on their way");
  static constexpr int kOffCodes = kOffV;
  static constexpr int kOffMisc = FP4 ? kOffCodes + kCodeRing * FourBit<D>::kHalf : kOffV + kRV * kSlot;
  static constexpr int kSmem = kOffMisc + kMisc + 1024;
  static constexpr uint32_t kColO = 256;                 // TMEM: S of the streams at 0 and 128, O at 256 and 256 + D
  static_assert(kRK >= 2 && kRV >= 2 && kRV <= kMaxRing && kRV + 4 <= kScaleRing && kSmem <= 227 * 1024, "rings");
  static_assert(kSlot % 1024 == 0 && kQTile % 1024 == 0, "swizzle atoms");
};

struct Bars {
  uint64_t code_full[kMaxCodeRing], code_empty[kMaxCodeRing];  // E2M1
  uint64_t k_full[kMaxRing], k_empty[kMaxRing], v_full[kMaxRing], v_empty[kMaxRing];
  uint64_t s_full[2], p_full[2], v16_full[2], v16_empty[2], ks_full[kTileRing], sc_full[kScaleRing];
  uint64_t q_full, drain;
  uint32_t bad[8][8];       // drafted keys with non-finite values, of up to eight pieces
  long long warp_sum[20];
  TreeWalk walk[2];         // of the streams
  int more[2];
  int start[3];
  uint32_t tmem_base;
  int abort_flag;
};
// TILES = 1 only: statistics of the two streams' rows.
struct Join {
  float m[2][kRowTile], l[2][kRowTile];
  int kv[2];
};
// E4M3 only.
struct Scales {
  alignas(16) uint8_t k_scale[kScaleRing][kBN];
  alignas(16) uint8_t v_scale[kScaleRing][kBN];
  alignas(16) float ks[kTileRing][kBN];  // the keys' powers of two
  int ref[kTileRing];                    // 2·(exponent that the tile's widened values are relative to) + (they are bf16)
  alignas(16) int top[2][4];
  float f[2 * kRowTile];                 // what a row's raw scores are multiplied by
};

// E2M1 only.
struct Refs {
  int ref[kTileRing];   // as with E4M3
  int kref[kTileRing];  // 2·(exponent that the tile's widened keys are relative to), or 1: each to its own, in power
  int range[2][4];      // of keys and values, per warp
  float f[2 * kRowTile];
  alignas(16) uint8_t power[kTileRing][kBN];
};

// Eight elements of a query row, whose other ones the neighbouring kChunks − 1 lanes hold, as fp16 x·2⁻ᵃ; 2⁻ᵃ, which is
// returned as a, brings the row's largest magnitude to between 2^14 and 2^15.  Exact down to 2⁻³¹ of it.
template <int kChunks>
__device__ __forceinline__ int scale_q8(uint4 v, uint4& out) {
  const uint32_t w4[4] = {v.x, v.y, v.z, v.w};
  uint32_t top = 0;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const uint32_t lo = w4[e] << 16 & 0x7fffffffu, hi = w4[e] & 0x7fff0000u;
    if (lo < 0x7f800000u) top = max(top, lo);
    if (hi < 0x7f800000u) top = max(top, hi);
  }
#pragma unroll
  for (int mk = kChunks / 2; mk > 0; mk >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, mk));
  const int a = max(-126, static_cast<int>(top >> 23) - 127 - 14);
  const float inv = __uint_as_float(static_cast<uint32_t>(127 - a) << 23);
  uint32_t o[4];
#pragma unroll
  for (int e = 0; e < 4; ++e)
    o[e] = pack_f16x2(__uint_as_float(w4[e] << 16) * inv, __uint_as_float(w4[e] & 0xffff0000u) * inv);
  out = make_uint4(o[0], o[1], o[2], o[3]);
  return a;
}

// Rows of a tile as a K-major operand (rows that are not there as zeros), by the 128 threads of a stream (TILES = 2)
// or the 256 of both.  E4M3: two terms per element and the factor of the row; E2M1: fp16 and the factor.
template <int D, int F, int NT>
__device__ __forceinline__ void load_q_tile(const TreeParams& p, const TreeWalk& w, uint8_t* q, float* f, int row0,
                                            int id) {
  constexpr int kChunks = D / 8;  // 16-byte chunks of a row
  constexpr int kPer = kRowTile * kChunks / NT;
  // Loads in flight per thread (bf16 with shared rows spills registers with eight).
  constexpr int kBatch = NT == 256 && F != kCacheE4m3 ? 4 : kPer < 8 ? kPer : 8;
  static_assert(kPer % kBatch == 0, "rows of the tile");
  const int live = w.drafts * p.G - row0;
#pragma unroll 1
  for (int i0 = 0; i0 < kPer; i0 += kBatch) {
    uint4 q4[kBatch];
#pragma unroll
    for (int e = 0; e < kBatch; ++e) {
      const int i = (i0 + e) * NT + id;
      const int r = i / kChunks, ch = i % kChunks;
      q4[e] = make_uint4(0, 0, 0, 0);
      if (r < live) {
        const int t = token_of(p, row0 + r);
        q4[e] = *reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p.q) + w.b * p.sq[0] +
                                                (w.h * p.G + row0 + r - t * p.G) * p.sq[1] + t * p.sq[2] + ch * 8);
      }
    }
#pragma unroll
    for (int e8 = 0; e8 < kBatch; ++e8) {
      const int i = (i0 + e8) * NT + id;
      const int r = i / kChunks, ch = i % kChunks;
      const uint4 v = q4[e8];
      if constexpr (F == kCacheE2m1) {
        uint4 x;
        const int a = scale_q8<kChunks>(v, x);
        *reinterpret_cast<uint4*>(q + (ch >> 3) * kRowTile * 128 + r * 128 + (((ch & 7) ^ (r & 7)) << 4)) = x;
        if (ch == 0) f[r] = p.scale_log2 * __uint_as_float(static_cast<uint32_t>(a + 127) << 23);
      } else if constexpr (F == kCacheBf16) {
        *reinterpret_cast<uint4*>(q + (ch >> 3) * kRowTile * 128 + r * 128 + (((ch & 7) ^ (r & 7)) << 4)) = v;
      } else {
        uint2 hi, lo;
        const int a = split_q8<kChunks, 0>(v, hi, lo);
        // Rows of D bytes; chunk of 16 bytes XORed with the row (128-byte rows) or half of it (64-byte rows).
        const int sw = D == 128 ? r & 7 : (r >> 1) & 3;
        uint8_t* dst = q + r * D + (((ch >> 1) ^ sw) << 4) + (ch & 1) * 8;
        *reinterpret_cast<uint2*>(dst) = hi;
        *reinterpret_cast<uint2*>(dst + kRowTile * D) = lo;
        // (Not 0, however small: what a row does not see stands as −∞ when it is multiplied by this.)
        if (ch == 0) f[r] = fmaxf(p.scale_log2 * __uint_as_float(static_cast<uint32_t>(a + 127) << 23), 1e-45f);
      }
    }
  }
  fence_proxy_async_smem();
}

// Multiplies the N columns of this thread's row of O by k.
template <int N>
__device__ __forceinline__ void rescale_row(uint32_t addr, float k) {
#pragma unroll 1
  for (int c = 0; c < N; c += 32) {
    uint32_t r[32];
    tmem_ld32(addr + c, r);
    tmem_wait_ld();
    reg_fence(r);
#pragma unroll
    for (int i = 0; i < 32; ++i) r[i] = __float_as_uint(__uint_as_float(r[i]) * k);
    tmem_st32(addr + c, r);
  }
  tmem_wait_st();
}

// 2^e for e from −127 on (0 below).
__device__ __forceinline__ float power_f32(int e) { return __uint_as_float(static_cast<uint32_t>(max(e, -127) + 127) << 23); }

// E2M1, keys far apart: a row's scores times the keys' own powers of two (byte 0: 2^−127, below the normal numbers).
static __device__ __noinline__ void scale_scores(uint32_t addr, const uint8_t* power) {
#pragma unroll 1
  for (int c = 0; c < kBN; c += 16) {
    uint32_t x[16];
    tmem_ld(addr + c, x);
    tmem_wait_ld();
    reg_fence(x);
    const uint4 b = *reinterpret_cast<const uint4*>(power + c);
    const uint32_t w[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      const uint32_t k = w[e >> 2] >> (8 * (e & 3)) & 0xffu;
      x[e] = __float_as_uint(__uint_as_float(x[e]) * __uint_as_float(k == 0 ? 0x00400000u : k << 23));
    }
    tmem_st(addr + c, x);
  }
  tmem_wait_st();
}

// Which keys of a tile token t sees: all before `context` (a place in the tile, maybe before it) and, up to `end`, the
// drafted ones behind that its row of the mask names.
static __device__ __noinline__ uint4 seen_keys(const uint8_t* row, int t, int context, int end) {
  uint32_t seen[4];
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const int before = context - q * 32;  // context keys among these 32
    seen[q] = before >= 32 ? 0xffffffffu : before > 0 ? (1u << before) - 1 : 0;
  }
#pragma unroll 8
  for (int j = max(0, context); j < end; ++j) {
    const uint32_t on = (row != nullptr ? row[j - context] != 0 : j - context <= t) ? 1u << (j & 31) : 0u;
#pragma unroll
    for (int q = 0; q < 4; ++q) seen[q] |= (j >> 5) == q ? on : 0u;
  }
  return make_uint4(seen[0], seen[1], seen[2], seen[3]);
}

// Turns a row's fp16 weights, as this thread has stored them, into two bf16 terms, the second 64 columns further.
static __device__ __noinline__ void split_weights(uint32_t addr) {
  tmem_wait_st();
#pragma unroll 1
  for (int c = 0; c < 64; c += 8) {
    uint32_t hi[8], lo[8];
    tmem_ld(addr + c, hi);
    tmem_wait_ld();
    reg_fence(hi);
#pragma unroll
    for (int e = 0; e < 8; ++e) split_f16x2(hi[e], hi[e], lo[e]);
    tmem_st(addr + c, hi);
    tmem_st(addr + 64 + c, lo);
  }
  tmem_wait_st();
}

// A key of a tile that holds the end (dead: zeros) or, with a place for its own power of two, of one whose keys lie far apart.
template <int D>
__device__ __noinline__ void widen_keys_edge(const uint8_t* src, uint32_t scales, uint8_t* dst, int r, int ref, bool dead,
                                             uint8_t* power) {
  if (power != nullptr) {
    const int top = exponent_range<D / kE2m1Group>(scales).x;
    *power = static_cast<uint8_t>(top);
    ref = top - 127;
  }
  widen_codes_edge<D>(src, scales, dst, r, ref, false, dead, false);
}

// E2M1: four warps widen the keys' codes and four the values', a row per thread.  The keys' reference goes with their
// tile; the values' is a running one, as with E4M3.  Keys that lie too far apart for fp16 are each taken relative to
// their own largest group, and the softmax multiplies their scores: a key may be seen by some rows only, and to the others
// it must not matter how large it is.  Rows past the end become zeros.
template <int D, int TILES, bool VALUES>
__device__ __forceinline__ void convert_halves(const TreeParams& p, const TreePart& my, uint8_t* smem, Bars* ms, Refs* sc,
                                              int r) {
  using C = Cfg<D, kCacheE2m1, TILES>;
  constexpr int kGroups = D / kE2m1Group;
  constexpr int kBar = VALUES ? 5 : 4;
  volatile int* abort_flag = &ms->abort_flag;
  int base = 0;          // halves of the pieces before
  int used = 0, ref = 0; // tiles of the part that have been widened, and what the last one is relative to
  // As with E4M3, all leave together after a vote on the abort flag.
  bool ok = true;
  TreeWalk w;
  w.begin(p, my);
  do {
    const int context = w.len - w.drafts, tiles = w.t1 - w.t0;
#pragma unroll 1
    for (int i = 0; i < tiles; ++i, ++used) {
      const int at = base + (VALUES ? (i == tiles - 1 ? 2 * i + 1 : 2 * i + 2) : max(2 * i - 1, 0));  // place in the ring's order
      const int slot = at % C::kCodeRing, key = (w.t0 + i) * kBN + r;
      mbar_wait_inl(&ms->code_full[slot], (at / C::kCodeRing) & 1, abort_flag, p.err, tree_site(VALUES ? 0x32 : 0x30));
      __syncwarp();
      const uint8_t* src = smem + C::kOffCodes + slot * FourBit<D>::kHalf;
      const uint8_t* sb = src + FourBit<D>::kCodes + r * kGroups;
      const uint32_t bytes = D == 128 ? *reinterpret_cast<const uint32_t*>(sb) : *reinterpret_cast<const uint16_t*>(sb);
      bool counts = key < w.len;
      if (VALUES && counts && key >= context && p.mask != nullptr)  // a drafted key that no row sees takes no part
        counts = any_token_sees(p.mask + w.b * p.mask_sb + (key - context), w.drafts, p.T);
      bool far = false;
      const bool first = VALUES && i == 0;
      __syncwarp();
      if (named_any(kBar, 128, first || (counts && outside_reference<kGroups>(bytes, ref)) || *abort_flag != 0)) {
        ok = !named_any(kBar, 128, *abort_flag != 0);
        if (!ok) break;
        const int2 range = exponent_range<kGroups>(bytes, counts, kBar, sc->range[VALUES]);
        if (VALUES) {
          if (first || range.x - 127 > ref + kFourLazy) ref = range.x - 127;
          far = range.y - 127 < ref - kFourFar;
        } else if (range.x > 0) {
          ref = range.x - 127;
          far = range.y - 127 < ref - kFourFar;
        }
      }
      if (VALUES) {
        if (r == 0) {
          sc->ref[used % kTileRing] = ref * 2 + (far ? 1 : 0);
          mbar_arrive(&ms->ks_full[used % kTileRing]);
        }
        mbar_wait_inl(&ms->v16_empty[used & 1], ((used >> 1) & 1) ^ 1, abort_flag, p.err, tree_site(0x33));
      } else {
        if (r == 0) sc->kref[used % kTileRing] = far ? 1 : ref * 2;  // (the scores say that it is there)
        mbar_wait_inl(&ms->k_empty[used & 1], ((used >> 1) & 1) ^ 1, abort_flag, p.err, tree_site(0x31));
      }
      __syncwarp();
      uint8_t* dst = smem + (VALUES ? C::kOffV16 : C::kOffK) + (used & 1) * C::kSlot + r * 128;
      if (!far && key - r + kBN <= (VALUES ? context : w.len)) {
        // (Groups at a time 1, 2, 4: 252, 253, 279 us for 256 rows over 8 x 32768 keys, 8 heads.)
        widen_codes<D, 1>(src + r * (D / 2), bytes, dst, r, ref);
      } else if (!VALUES) {
        widen_keys_edge<D>(src + r * (D / 2), bytes, dst, r, ref, !counts, far ? &sc->power[used % kTileRing][r] : nullptr);
      } else if (widen_codes_edge<D>(src + r * (D / 2), bytes, dst, r, ref, key >= context, !counts, far)) {
        atomicOr(&ms->bad[w.index & 7][(key - context) >> 5], 1u << ((key - context) & 31));
      }
      fence_proxy_async_smem();
      __syncwarp();
      if ((r & 31) == 0) {
        mbar_arrive(VALUES ? &ms->v16_full[used & 1] : &ms->k_full[used & 1]);
        mbar_arrive(&ms->code_empty[slot]);
      }
      __syncwarp();
    }
    base += 2 * tiles;
    ok = !named_any(kBar, 128, !ok || *abort_flag != 0);  // the piece's last waits have had none
  } while (ok && w.next(p));
}

template <int D, int F, int TILES>
__global__ void __launch_bounds__(Cfg<D, F, TILES>::kThreads, 1) tree_wide_kernel(const __grid_constant__ TreeParams p) {
  using C = Cfg<D, F, TILES>;
  constexpr bool FP8 = C::FP8, FP4 = C::FP4, kWiden = C::kWiden;
  constexpr bool kPg5 = !kWiden && D == 128;  // K/V pages as [row group][half][8 rows][128 bytes]
  constexpr int kSlot = C::kSlot;
  constexpr float kLazy = 8.f;             // rescale once the maximum exceeds the reference by this …
  constexpr float kBase = kWiden ? 3.f : 0.f; // … the new reference lies this below the maximum
  constexpr int kKvLazy = 7;               // E4M3: widened values stay below 448·2^7
  constexpr int kKvFar = 15;               // value rows that are smaller by more than this need bf16's range
  extern __shared__ uint8_t smem_raw[];
  const uint32_t pad = (1024u - (smem_u32(smem_raw) & 1023u)) & 1023u;
  uint8_t* smem = smem_raw + pad;
  Bars* ms = reinterpret_cast<Bars*>(smem + C::kOffMisc);
  constexpr int kOffScales = (sizeof(Bars) + 15) / 16 * 16;
  using Sc = typename std::conditional<FP4, Refs, Scales>::type;
  constexpr int kOffJoin = kOffScales + (kWiden ? (sizeof(Sc) + 15) / 16 * 16 : 0);
  Sc* sc = reinterpret_cast<Sc*>(smem + C::kOffMisc + kOffScales);  // E4M3 and E2M1 only
  Join* join = reinterpret_cast<Join*>(smem + C::kOffMisc + kOffJoin);
  static_assert(kOffJoin + (TILES == 1 ? sizeof(Join) : 0) <= static_cast<size_t>(C::kMisc), "misc block");
  volatile int* abort_flag = &ms->abort_flag;

  const int tid = threadIdx.x;
  const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);  // broadcast: known to be the same in the warp
  const int lane = tid & 31;
  const int part = blockIdx.y;
  const int row0 = blockIdx.x * kRowTile * TILES;  // row tiles of one part are neighbours: they share its keys in L2
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");  // the joining kernel waits for this grid's end

  if (tid == 0) {
    for (int s = 0; s < C::kRK; ++s) {
      mbar_init(&ms->k_full[s], FP4 ? 4 : 1);
      mbar_init(&ms->k_empty[s], 1);
    }
    for (int s = 0; FP4 && s < C::kCodeRing; ++s) {
      mbar_init(&ms->code_full[s], kCodeArrivals);
      mbar_init(&ms->code_empty[s], 4);
    }
    for (int s = 0; s < C::kRV; ++s) {
      mbar_init(&ms->v_full[s], 1);
      mbar_init(&ms->v_empty[s], FP8 ? 4 : 1);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(&ms->s_full[s], 1);
      mbar_init(&ms->p_full[s], 128);
      mbar_init(&ms->v16_full[s], FP4 ? 4 : 128);
      mbar_init(&ms->v16_empty[s], 1);
    }
    for (int s = 0; s < kScaleRing; ++s) mbar_init(&ms->sc_full[s], 1);
    for (int s = 0; s < kTileRing; ++s) mbar_init(&ms->ks_full[s], FP4 ? 1 : 128);
    mbar_init(&ms->q_full, 256);
    mbar_init(&ms->drain, 1);
    ms->abort_flag = 0;
    fence_barrier_init();
  }
  if (tid < 64) ms->bad[tid >> 3][tid & 7] = 0;
  if (warp == 9) {
    tmem_alloc(&ms->tmem_base, 512);
    tmem_relinquish();
  }
  const TreePart my = find_part<C::kThreads>(p, part, ms->warp_sum, ms->start);
  const uint32_t tmem = ms->tmem_base;

  if (my.count <= 0) {
    // nothing left for this CTA
  } else if (FP4 && warp >= 12) {
    reg_dealloc<C::kRegsConvert>();
    if constexpr (FP4) {
      if (warp < 16)
        convert_halves<D, TILES, false>(p, my, smem, ms, sc, tid & 127);
      else
        convert_halves<D, TILES, true>(p, my, smem, ms, sc, tid & 127);
    }
  } else if (FP4 && warp == 8) {
    reg_dealloc<C::kRegsOther>();
    if constexpr (FP4)
      load_codes<D, C::kCodeRing, kBothHalves>(p, my, smem + C::kOffCodes, ms->code_full, ms->code_empty, abort_flag,
                                               tree_site(0x21), [](const TreeWalk&) { return true; });
  } else if (!FP4 && (warp == 8 || warp == 10)) {
    reg_dealloc<C::kRegsOther>();
    // ------------------------------------------- loads of K (warp 8) and V (warp 10)
    const bool is_v = warp == 10;
    if constexpr (!FP4)
      load_pages<D, FP8, kScaleRing>(p, my, is_v, smem + (is_v ? C::kOffV : C::kOffK), is_v ? C::kRV : C::kRK,
                                     is_v ? ms->v_full : ms->k_full, is_v ? ms->v_empty : ms->k_empty, ms->sc_full,
                                     sc->k_scale[0], sc->v_scale[0], abort_flag, tree_site(is_v ? 0x22 : 0x21));
  } else if (warp == 9) {
    reg_dealloc<C::kRegsOther>();
    // ------------------------------------------------------------ MMA issuer
    // The whole warp runs the loop, which keeps descriptors warp-uniform, and one elected lane issues.
    constexpr uint32_t kIdescS = FP8   ? idesc_e4m3_f32(128, kBN, false, false)
                                 : FP4 ? idesc_f16_f32(128, kBN, false, false)
                                       : idesc_bf16_f32(128, kBN, false, false);
    constexpr uint32_t kIdescFar = idesc_bf16_f32(128, D, false, true);
    constexpr uint32_t kIdescO = kWiden ? idesc_f16_f32(128, D, false, true) : idesc_bf16_f32(128, D, false, true);
    const uint32_t sQ = smem_u32(smem + C::kOffQ), sK = smem_u32(smem + C::kOffK);
    const uint32_t sV = smem_u32(smem + (kWiden ? C::kOffV16 : C::kOffV));
    const bool leader = elect_one_lane();
    Ring<C::kRK> rk;
    Ring<C::kRV> rv;
    int v16 = 0;         // E4M3: the widened tile's place and parity
    uint32_t v16_par = 0;
    int vt = 0;          // E4M3: tile of the part that P̃ is multiplied with
    uint32_t p_par = 0;  // parity of p_full to wait for, a bit per stream
    bool ok = true;
    TreeWalk w;
    w.begin(p, my);
    do {
      // Step s: stream s & 1, tile s (or s / 2).  Broadcast, like the walk's end below, to keep the loop uniform.
      const int steps = __shfl_sync(0xffffffffu, (w.t1 - w.t0) * TILES, 0);
      ok = mbar_wait_inl(&ms->q_full, w.index & 1, abort_flag, p.err, tree_site(0x2e));
#pragma unroll 1
      for (int s = 0; s < steps + 2; ++s) {
        const int g = s & 1;
        const bool first_use = TILES == 1 || g == 0, last_use = TILES == 1 || g == 1;  // of the K or V tile
        const bool scores = s < steps, product = s >= 2;
        // Everything that can be is done before P̃ arrives: what follows is on the streams' critical path, and this
        // warp gets an instruction through every dozen cycles while the softmax warps run.
        if (first_use) {
          if (scores) ok = ok && mbar_wait_inl(&ms->k_full[rk.slot], rk.parity, abort_flag, p.err, tree_site(0x25));
          if (product)
            ok = ok && (kWiden ? mbar_wait_inl(&ms->v16_full[v16], v16_par, abort_flag, p.err, tree_site(0x2f))
                               : mbar_wait_inl(&ms->v_full[rv.slot], rv.parity, abort_flag, p.err, tree_site(0x24)));
        }
        const bool far = kWiden && product && (*static_cast<volatile int*>(&sc->ref[vt % kTileRing]) & 1);
        const uint32_t idesc = far ? kIdescFar : kIdescO;
        const uint32_t ts = tmem + g * kBN;
        const uint32_t to = tmem + C::kColO + g * D;
        const uint32_t vb = sV + (kWiden ? v16 * C::kV16 : rv.slot * kSlot);
        const uint32_t kb = sK + rk.slot * kSlot;
        const uint32_t qb = sQ + (TILES == 1 ? 0 : g * C::kQTile);
        const uint64_t vd = kPg5 ? sdesc_sw128(vb, 1024, 2048) : sdesc_sw128(vb, kBN * 128, 1024);
        const uint64_t qd = FP8 && D == 64 ? sdesc_sw64(qb, 16, 512) : sdesc_sw128(qb, 16, 1024);
        const uint64_t kd = FP8 && D == 64 ? sdesc_sw64(kb, 16, 512) : sdesc_sw128(kb, 16, kPg5 ? 2048 : 1024);
        if (product)
          ok = ok && mbar_wait_inl(&ms->p_full[g], (p_par >> g) & 1u, abort_flag, p.err, tree_site(0x23));
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        tc_fence_after();
        if (product) {  // P̃V of step s − 2, of the same stream
          if (leader) {
#pragma unroll
            for (int term = 0; term < C::kTerms; ++term)
#pragma unroll
              for (int kk = 0; kk < kBN / 16; ++kk)  // A: P̃ over S, 16 keys in 8 columns
                mma_bf16_ts(to, ts + term * 64 + kk * 8, vd + kk * (kPg5 ? 256 : 128), idesc,
                            (s >= 4 || term > 0 || kk > 0) ? 1u : 0u);
            if (kWiden && far) {  // the second terms
#pragma unroll 1
              for (int kk = 0; kk < kBN / 16; ++kk)
                mma_bf16_ts(to, ts + 64 + kk * 8, vd + kk * (kPg5 ? 256 : 128), idesc, 1u);
            }
          }
          p_par ^= 1u << g;
          // With shared rows the value slot is given back at once (after the scores' issue: 1 us of 104 slower); with two
          // row tiles the scores' issue comes first (the other way round 135 instead of 130 us: 256 rows, 8 x 16384 keys).
          if (TILES == 1 && leader) mma_commit(kWiden ? &ms->v16_empty[v16] : &ms->v_empty[rv.slot]);
        }
        if (scores && leader) {  // S over what P̃V has just read: the tensor pipe runs them in this order
          if constexpr (FP8) {
#pragma unroll
            for (int term = 0; term < 2; ++term)
#pragma unroll
              for (int kk = 0; kk < D / 32; ++kk)
                mma_e4m3_ss(ts, qd + term * (kRowTile * D / 16) + kk * 2, kd + kk * 2, kIdescS,
                            (term > 0 || kk > 0) ? 1u : 0u);
          } else {
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk)
              mma_bf16_ss(ts, qd + (kk >> 2) * (kRowTile * 8) + (kk & 3) * 2, kd + (kk >> 2) * (FP4 ? kBN * 8 : 64) + (kk & 3) * 2, kIdescS,
                          kk > 0 ? 1u : 0u);
          }
        }
        if (leader) {
          if (scores || product) mma_commit(&ms->s_full[g]);  // scores, or, where none follow, O of the piece
          if (last_use && scores) mma_commit(&ms->k_empty[rk.slot]);
          if (TILES == 2 && last_use && product) mma_commit(kWiden ? &ms->v16_empty[v16] : &ms->v_empty[rv.slot]);
        }
        if (last_use && scores) rk.advance();
        if (last_use && product) {
          rv.advance();
          ++vt;
          v16 ^= 1;
          v16_par ^= v16 == 0;
        }
      }
    } while (ok && __shfl_sync(0xffffffffu, w.next(p), 0));
    if (leader) {  // the same for the products, which the end frees the tensor memory of
      mma_commit(&ms->drain);
      mbar_wait_drain_inl(&ms->drain, 0, kTreeDrainNs);
    }
  } else if (warp < 8) {
    reg_alloc<C::kRegsSoftmax>();
    // ------------------------------------------------------- softmax: one row per thread
    const int g = warp >> 2;
    const int kt = tid & 127;      // row in the tile, TMEM lane; key in the tile for the value rows' edge
    const int my_row0 = row0 + (TILES == 1 ? 0 : g * kRowTile);
    const uint32_t lane_base = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t s_addr = tmem + lane_base + g * kBN;
    const uint32_t o_addr = tmem + lane_base + C::kColO + g * D;
    int tile0 = 0;                 // tiles of the pieces before
    uint32_t s_par = 0;            // parity of s_full to wait for: scores of each tile, then O of the piece
    bool ok = true;
    const TreeWalk& w = ms->walk[g];
    if (kt == 0) ms->walk[g].begin(p, my);
    named_sync(1 + g, 128);
#pragma unroll 1
    while (true) {
      const int n_tiles = w.t1 - w.t0;
      const int context = w.len - w.drafts;
      const int rr = my_row0 + kt;
      const int t = token_of(p, rr);
      const bool live = rr < w.drafts * p.G;
      const bool busy = __any_sync(0xffffffffu, live);
      const int h = w.h * p.G + (rr - t * p.G);
      // Q of the piece: the stream's tile, or both streams' shares of the one tile.  The products of the piece before
      // that read its place are done: their results have been taken (by both streams, which end a shared piece together).
      if constexpr (TILES == 2)
        load_q_tile<D, F, 128>(p, w, smem + C::kOffQ + g * C::kQTile, kWiden ? sc->f + g * kRowTile : nullptr, my_row0,
                                 kt);
      else
        load_q_tile<D, F, 256>(p, w, smem + C::kOffQ, kWiden ? sc->f : nullptr, my_row0, tid);
      mbar_arrive(&ms->q_full);

      float m_run = -INFINITY, l_run = 0.f;
      int kv_ref = 0;
      int done = 0;  // tiles of this piece that this stream has worked on
#pragma unroll 1
      for (int i = TILES == 1 ? g : 0; i < n_tiles; i += TILES == 1 ? 2 : 1, ++done) {
        const int tile = tile0 + i;
        const int k0 = (w.t0 + i) * kBN;
        const bool tail = k0 + kBN > context;  // the tile holds drafted keys or the end
        uint32_t seen[4];                      // which of its keys this row sees
        if (tail) {
          const uint8_t* row = p.mask != nullptr ? p.mask + w.b * p.mask_sb + static_cast<int64_t>(t) * p.T : nullptr;
          const uint4 s4 = seen_keys(row, t, context - k0, live ? min(kBN, w.len - k0) : 0);
          seen[0] = s4.x, seen[1] = s4.y, seen[2] = s4.z, seen[3] = s4.w;
        }
        if constexpr (kWiden)  // the keys' powers of two, and what the widened tile is relative to
          ok = mbar_wait_inl(&ms->ks_full[tile % kTileRing], (tile / kTileRing) & 1, abort_flag, p.err, tree_site(0x26)) && ok;
        // (P̃V of the stream's tile before has run too: S was issued behind it.)
        ok = mbar_wait_inl(&ms->s_full[g], s_par, abort_flag, p.err, tree_site(0x27)) && ok;
        s_par ^= 1u;
        if (!__all_sync(0xffffffffu, ok)) {
          ok = false;
          break;
        }
        tc_fence_after();
        // A warp without live rows leaves its P̃ as it is: it only reaches its own rows of O, which nobody reads.
        if constexpr (FP4) {
          if (busy) {
            // The scores are read twice, 32 at a time, in loops that are not unrolled: with the converters' code beside it the
            // other formats' way, which holds 128 scores and takes as much code, waited for instructions.
            uint4 see = make_uint4(~0u, ~0u, ~0u, ~0u);
            if (tail) see = make_uint4(seen[0], seen[1], seen[2], seen[3]);
            auto fetch = [&](int c, uint32_t (&x)[32]) {
              tmem_ld32(s_addr + c, x);
              tmem_wait_ld();
              reg_fence(x);
              if (tail) {
#pragma unroll
                for (int e = 0; e < 32; ++e)
                  if (!((see.x >> e) & 1)) x[e] = 0xff800000u;
                see = make_uint4(see.y, see.z, see.w, see.x);
              }
            };
            const int kcode = sc->kref[tile % kTileRing];
            if (kcode & 1) scale_scores(s_addr, sc->power[tile % kTileRing]);
            float top = -INFINITY;
#pragma unroll 1
            for (int c = 0; c < kBN; c += 32) {
              uint32_t x[32];
              fetch(c, x);
              float mx[4] = {top, __uint_as_float(x[29]), __uint_as_float(x[30]), __uint_as_float(x[31])};
#pragma unroll
              for (int e = 0; e < 28; e += 8)
#pragma unroll
                for (int q = 0; q < 4; ++q)
                  mx[q] = fmax3(mx[q], __uint_as_float(x[e + q]), __uint_as_float(x[e + 4 + q < 28 ? e + 4 + q : 28]));
              top = fmax3(fmaxf(mx[0], mx[1]), mx[2], mx[3]);
            }
            // (Not 0, as with E4M3.)
            const float factor =
                fmaxf(sc->f[(TILES == 1 ? 0 : g * kRowTile) + kt] * power_f32(kcode >> 1), 1e-45f);
            const float m_cand = top * factor;
            const bool need = m_cand > m_run + kLazy;
            const float m_new = need ? m_cand - kBase : m_run;
            float corr = need ? ex2_approx(m_run - m_new) : 1.f;
            l_run *= corr;
            const int code = sc->ref[tile % kTileRing];
            const bool moved = done > 0 && code >> 1 != kv_ref;  // the widened values are relative to another exponent
            if (moved) corr *= exp2f(static_cast<float>(max(kv_ref - (code >> 1), -200)));
            kv_ref = code >> 1;
            m_run = m_new;
            if (done > 0 && __any_sync(0xffffffffu, need || moved)) rescale_row<D>(o_addr, corr);
            const float neg = m_new == -INFINITY ? 0.f : -m_new;
            float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 1
            for (int c = 0; c < kBN; c += 32) {
              uint32_t x[32], pk[16];
              fetch(c, x);
#pragma unroll
              for (int e = 0; e < 32; e += 4) {
                float y[4] = {__uint_as_float(x[e]), __uint_as_float(x[e + 1]), __uint_as_float(x[e + 2]),
                              __uint_as_float(x[e + 3])};
                ffma2(y[0], y[1], y[0], y[1], factor, factor, neg, neg);
                ffma2(y[2], y[3], y[2], y[3], factor, factor, neg, neg);
#pragma unroll
                for (int q = 0; q < 4; ++q) y[q] = ex2_approx(y[q]);
                fadd2(sum[0], sum[1], sum[0], sum[1], y[0], y[1]);
                fadd2(sum[2], sum[3], sum[2], sum[3], y[2], y[3]);
                pk[e / 2] = pack_f16x2(y[0], y[1]);
                pk[e / 2 + 1] = pack_f16x2(y[2], y[3]);
              }
              tmem_st(s_addr + c / 2, pk);  // over scores that have been read
            }
            l_run += (sum[0] + sum[1]) + (sum[2] + sum[3]);
            if (code & 1) split_weights(s_addr);
          }
        } else if (busy) {
          float s[kBN];
          {
            uint32_t r0[32], r1[32], r2[32], r3[32];
            tmem_ld32(s_addr, r0);
            tmem_ld32(s_addr + 32, r1);
            tmem_ld32(s_addr + 64, r2);
            tmem_ld32(s_addr + 96, r3);
            tmem_wait_ld();
            reg_fence(r0);
            reg_fence(r1);
            reg_fence(r2);
            reg_fence(r3);
#pragma unroll
            for (int e = 0; e < 32; ++e) {
              s[e] = __uint_as_float(r0[e]);
              s[32 + e] = __uint_as_float(r1[e]);
              s[64 + e] = __uint_as_float(r2[e]);
              s[96 + e] = __uint_as_float(r3[e]);
            }
          }
          float factor = p.scale_log2;
          if constexpr (FP8) {
            factor = sc->f[(TILES == 1 ? 0 : g * kRowTile) + kt];
            const float4* ks = reinterpret_cast<const float4*>(sc->ks[tile % kTileRing]);
#pragma unroll
            for (int e = 0; e < kBN; e += 4) {
              const float4 k4 = ks[e >> 2];
              fmul2(s[e], s[e + 1], s[e], s[e + 1], k4.x, k4.y);
              fmul2(s[e + 2], s[e + 3], s[e + 2], s[e + 3], k4.z, k4.w);
            }
          }
          if (tail) {
#pragma unroll
            for (int e = 0; e < kBN; ++e)
              if (!((seen[e >> 5] >> (e & 31)) & 1)) s[e] = -INFINITY;
          }
          float mx[4] = {s[0], s[1], s[2], s[3]};
#pragma unroll
          for (int e = 4; e + 4 < kBN; e += 8)
#pragma unroll
            for (int q = 0; q < 4; ++q) mx[q] = fmax3(mx[q], s[e + q], s[e + 4 + q]);
#pragma unroll
          for (int q = 0; q < 4; ++q) mx[q] = fmaxf(mx[q], s[kBN - 4 + q]);
          const float m_cand = fmax3(fmaxf(mx[0], mx[1]), mx[2], mx[3]) * factor;
          // A row without a reference takes one; 0 stands in for it while it has seen nothing.
          const bool need = m_cand > m_run + kLazy;
          const float m_new = need ? m_cand - kBase : m_run;
          float corr = need ? ex2_approx(m_run - m_new) : 1.f;
          l_run *= corr;
          bool moved = need;
          bool far = false;  // E4M3: the tile has gone over to bf16
          if constexpr (FP8) {
            const int code = sc->ref[tile % kTileRing];
            const int ref = code >> 1;
            far = code & 1;
            if (done > 0 && ref != kv_ref) {  // the widened values are relative to another exponent
              corr *= exp2f(static_cast<float>(max(kv_ref - ref, -200)));
              moved = true;
            }
            kv_ref = ref;
          }
          m_run = m_new;
          if (done > 0 && __any_sync(0xffffffffu, moved)) rescale_row<D>(o_addr, corr);
          const float neg = m_new == -INFINITY ? 0.f : -m_new;
          float sum[4] = {0.f, 0.f, 0.f, 0.f};
          // Keys whose weights are stored at once (two terms: 16, where 64 spilled registers and took 4 % more).
          constexpr int kPer = C::kTerms == 2 ? 16 : 64;
#pragma unroll
          for (int k = 0; k < kBN; k += kPer) {
            uint32_t pk[kPer / 2], lo[C::kTerms == 2 ? kPer / 2 : 1];
#pragma unroll
            for (int e = 0; e < kPer; e += 4) {
              float* x = s + k + e;
              ffma2(x[0], x[1], x[0], x[1], factor, factor, neg, neg);
              ffma2(x[2], x[3], x[2], x[3], factor, factor, neg, neg);
#pragma unroll
              for (int q = 0; q < 4; ++q) x[q] = ex2_approx(x[q]);
              fadd2(sum[0], sum[1], sum[0], sum[1], x[0], x[1]);
              fadd2(sum[2], sum[3], sum[2], sum[3], x[2], x[3]);
              if constexpr (C::kTerms == 2) {
                split_weights2(x[0], x[1], pk[e / 2], lo[e / 2]);
                split_weights2(x[2], x[3], pk[e / 2 + 1], lo[e / 2 + 1]);
              } else {
                pk[e / 2] = FP8 ? pack_f16x2(x[0], x[1]) : pack_bf16x2(x[0], x[1]);
                pk[e / 2 + 1] = FP8 ? pack_f16x2(x[2], x[3]) : pack_bf16x2(x[2], x[3]);
              }
            }
            tmem_st(s_addr + k / 2, pk);
            if constexpr (C::kTerms == 2) tmem_st(s_addr + 64 + k / 2, lo);
          }
          l_run += (sum[0] + sum[1]) + (sum[2] + sum[3]);
          if (FP8 && far) split_weights(s_addr);
        }
        if (!kWiden && tail && k0 + kt >= context && (TILES == 1 || g == 0)) {
          // Key kt's value row: zeros past the end, and in place of what a drafted row holds that is not finite.
          // (Two row tiles: the first stream does it for both, its product is issued first.)
          const int slot = tile % C::kRV;
          ok = mbar_wait_inl(&ms->v_full[slot], (tile / C::kRV) & 1, abort_flag, p.err, tree_site(0x29)) && ok;
          uint8_t* vr = smem + C::kOffV + slot * kSlot + (kPg5 ? (kt >> 3) * 2048 + (kt & 7) * 128 : kt * 128);
          const int key = k0 + kt;
          const bool bad = clean_value_row<D>(vr, key >= w.len);
          if (bad) atomicOr(&ms->bad[w.index & 7][(key - context) >> 5], 1u << ((key - context) & 31));
          fence_proxy_async_smem();
        }
        __syncwarp();
        tmem_wait_st();
        tc_fence_before();
        mbar_arrive(&ms->p_full[g]);
      }
      tile0 += n_tiles;
      // ------------------------------------------------------------ end of the piece
      if (done > 0) {
        ok = ok && mbar_wait_inl(&ms->s_full[g], s_par, abort_flag, p.err, tree_site(0x2a));
        s_par ^= 1u;
      }
      const bool whole = w.whole();
      const int64_t slot = w.slot(p, part);
      const int64_t slot_row = slot * p.T * p.G + rr;
      float m = l_run != 0.f ? m_run : -INFINITY, sum = l_run;
      float scale[2] = {0.f, 0.f};  // what the streams' O is multiplied by
      if constexpr (TILES == 1) {
        join->m[g][kt] = m;
        join->l[g][kt] = l_run;
        if (kt == 0) join->kv[g] = done > 0 ? kv_ref : -1024;
        tc_fence_before();
        named_sync(3, 256);
        tc_fence_after();
        m = fmaxf(join->m[0][kt], join->m[1][kt]);
        sum = 0.f;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float le = join->l[e][kt];
          scale[e] = le == 0.f ? 0.f : exp2f(join->m[e][kt] - m);
          sum += scale[e] * le;
        }
      } else {
        tc_fence_after();
        scale[g] = 1.f;
      }
      const float inv = sum != 0.f ? 1.f / sum : 0.f;
      // E4M3: times the power of two that the values are relative to, half of it here and half at the end: the whole of it
      // may be too small a number.
      const int half_kv = kWiden ? (TILES == 1 ? max(join->kv[0], join->kv[1]) : kv_ref) >> 1 : 0;
#pragma unroll
      for (int e = 0; e < 2; ++e) scale[e] *= inv * (kWiden ? power_f32((TILES == 1 ? join->kv[e] : kv_ref) - half_kv) : 1.f);
      const bool fine = __all_sync(0xffffffffu, ok);
      if (fine && live && (TILES == 2 || g == 0)) {
        if (!whole) {
          p.part_ml[slot_row * 2] = m;
          p.part_ml[slot_row * 2 + 1] = sum;
        } else if (p.lse != nullptr) {
          p.lse[(static_cast<int64_t>(w.b) * p.Hq + h) * p.T + t] =
              sum != 0.f ? (m + log2f(sum)) * 0.6931471805599453f : -INFINITY;
        }
      }
      if (w.t0 == 0 && blockIdx.x == 0 && tid == 0) p.pieces[w.pair(p)] = w.pieces(part, my.per);
      // The row's columns, or with shared rows this stream's half of them, 32 at a time.
      if (fine) {
        constexpr int kHalf = TILES == 1 ? D / 2 : D;
        const int c0 = TILES == 1 ? g * kHalf : 0;
        __nv_bfloat16* out =
            static_cast<__nv_bfloat16*>(p.o) + w.b * p.so[0] + h * p.so[1] + static_cast<int64_t>(t) * p.so[2];
        // A cut pair's row is stored in chunks of four columns, 32 rows' chunks side by side, in whole lines per warp
        // (row after row each store touched 32 lines, 8000 cycles a piece).
        float* part_o = p.part_o + (slot * tree_piece_rows(p.T * p.G) + rr - lane) * D + lane * 4;
#pragma unroll 1
        for (int c = c0; c < c0 + kHalf; c += 32) {
          float o[32];
#pragma unroll
          for (int e = 0; e < 32; ++e) o[e] = 0.f;
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            if (TILES == 2 && e != g) continue;
            uint32_t r[32];
            tmem_ld32(tmem + lane_base + C::kColO + e * D + c, r);
            tmem_wait_ld();
            reg_fence(r);
            if (scale[e] != 0.f) {  // 0: a stream without keys has left O unwritten
#pragma unroll
              for (int q = 0; q < 32; q += 2)
                ffma2(o[q], o[q + 1], __uint_as_float(r[q]), __uint_as_float(r[q + 1]), scale[e], scale[e], o[q], o[q + 1]);
            }
          }
          if constexpr (kWiden) {
            const float power = power_f32(half_kv);
#pragma unroll
            for (int q = 0; q < 32; q += 2) fmul2(o[q], o[q + 1], o[q], o[q + 1], power, power);
          }
          if (live) {
            if (!whole) {
#pragma unroll
              for (int q = 0; q < 32; q += 4)
                *reinterpret_cast<float4*>(part_o + (c + q) * 32) = make_float4(o[q], o[q + 1], o[q + 2], o[q + 3]);
            } else {
#pragma unroll
              for (int q = 0; q < 32; q += 8)
                *reinterpret_cast<uint4*>(out + c + q) =
                    make_uint4(pack_bf16x2(o[q], o[q + 1]), pack_bf16x2(o[q + 2], o[q + 3]),
                               pack_bf16x2(o[q + 4], o[q + 5]), pack_bf16x2(o[q + 6], o[q + 7]));
            }
          }
        }
        // What was taken out of drafted value rows goes to the rows that see them.
        const uint32_t* bad = ms->bad[w.index & 7];
        for (int u = 0; live && u < w.drafts; ++u) {
          if (bad[u >> 5] == 0) {
            u |= 31;
            continue;
          }
          if (!((bad[u >> 5] >> (u & 31)) & 1) || !token_sees(p, w.b, t, u)) continue;
          const int64_t at = value_row<D>(p, w, u);
          for (int c = c0; c < c0 + kHalf; ++c) {
            const float v = taken_out<F>(p, at + c);
            if (v == 0.f) continue;
            if (!whole)
              part_o[(c & ~3) * 32 + (c & 3)] += v;
            else
              out[c] = __float2bfloat16_rn(__bfloat162float(out[c]) + v);
          }
        }
      }
      tc_fence_before();
      // Any failed wait ends the walk for all; with shared rows both streams have read O and the statistics.
      ok = !named_any(TILES == 1 ? 3 : 1 + g, TILES == 1 ? 256 : 128, !ok);
      // The flags of three pieces ago: the other stream may still be at the piece before.
      if (tid < 8) ms->bad[(w.index + 5) & 7][tid] = 0;
      if (!ok) break;
      if (kt == 0) ms->more[g] = ms->walk[g].next(p);
      named_sync(1 + g, 128);
      if (!ms->more[g]) break;
    }
  } else if (FP8 && warp >= 12) {
    reg_dealloc<C::kRegsOther>();
    if constexpr (FP8) {
    // ------------------------------------ converters: one value row and one key's scale per thread
    const int r = tid - 384;
    int next = 0, ref = 0;  // the tile of the part whose scales come next
    // A wait that fails raises the abort flag, and all leave together, after a vote on it: until then a thread whose wait
    // has failed goes on, since the others wait for it at the vote without a limit.
    bool ok = true;
    auto vote = [&] { ok = !named_any(4, 128, *abort_flag != 0); };
    TreeWalk w;
    w.begin(p, my);
    do {
      const int context = w.len - w.drafts;
      int exponent = 0;  // of this thread's value row, relative to the reference
      bool far_next = false;
      // The scales of tile i of the pair, the n-th of the part: the softmax wants them before the widened values.
      // Slot n % 8 was read for tile n − 8, whose second product the wait for a place to widen into has told the end of.
      auto scales = [&](int i, int n) {
        mbar_wait_inl(&ms->sc_full[n % kScaleRing], (n / kScaleRing) & 1, abort_flag, p.err, tree_site(0x2b));
        const uint32_t kb = sc->k_scale[n % kScaleRing][r];
        const int key = i * kBN + r;
        bool used = key < w.len;
        if (used && key >= context && p.mask != nullptr) {  // a drafted key that no row sees takes no part
          used = any_token_sees(p.mask + w.b * p.mask_sb + (key - context), w.drafts, p.T);
        }
        const int kv = used ? static_cast<int>(sc->v_scale[n % kScaleRing][r]) - 127 : -1024;
        // The largest and the smallest exponent (−126, next to nothing or zeros, does not count), as two halves of a word.
        const int top = __reduce_max_sync(0xffffffffu, kv);
        const int low = __reduce_min_sync(0xffffffffu, kv > -126 ? kv : 2047);
        if (lane == 0) sc->top[n & 1][warp - 12] = ((top + 2048) << 16) | (2048 - low);
        // (Byte 0 stands for 2^−127, below the normal numbers.)
        sc->ks[n % kTileRing][r] = kb == 0 ? 5.877471754111438e-39f : __uint_as_float(kb << 23);
        vote();
        const int4 tp = *reinterpret_cast<const int4*>(sc->top[n & 1]);
        const uint32_t both = __vmaxu2(__vmaxu2(tp.x, tp.y), __vmaxu2(tp.z, tp.w));
        const int most = static_cast<int>(both >> 16) - 2048;
        if (i == w.t0 || most > ref + kKvLazy) ref = most;
        far_next = 2048 - static_cast<int>(both & 0xffffu) < ref - kKvFar;
        if (r == 0) sc->ref[n % kTileRing] = ref * 2 + (far_next ? 1 : 0);
        exponent = kv - ref;
        mbar_arrive(&ms->ks_full[n % kTileRing]);
      };
#pragma unroll 1
      for (int i = w.t0 - 1; i < w.t1; ++i) {
        const int e = exponent;  // at most kKvLazy
        const bool far = far_next;
        const uint32_t f2 = power_f16x2(e);
        const __half2 scale2 = *reinterpret_cast<const __half2*>(&f2);
        if (i + 1 < w.t1) {
          scales(i + 1, next++);
          if (!ok) break;
        }
        if (i < w.t0) continue;  // (the first tile's scales come before its values)
        const int tile = next - (i + 1 < w.t1 ? 2 : 1);
        const int slot = tile % C::kRV;
        mbar_wait_inl(&ms->v_full[slot], (tile / C::kRV) & 1, abort_flag, p.err, tree_site(0x2d));
        mbar_wait_inl(&ms->v16_empty[tile & 1], ((tile >> 1) & 1) ^ 1, abort_flag, p.err, tree_site(0x2c));
        const int key = i * kBN + r;
        const uint8_t* src = smem + C::kOffV + slot * kSlot + r * D;
        uint8_t* dst = smem + C::kOffV16 + (tile & 1) * C::kV16 + r * 128;
        const int sw = D == 128 ? r & 7 : (r >> 1) & 3;
        auto widen = [&](int ch, const uint32_t(&w4)[4]) {
          uint32_t o[8];
#pragma unroll
          for (int q = 0; q < 8; ++q) {
            const uint32_t wide = e4m3x2_to_f16x2(w4[q >> 1] >> (16 * (q & 1)));
            const __half2 x = __hmul2(*reinterpret_cast<const __half2*>(&wide), scale2);
            o[q] = *reinterpret_cast<const uint32_t*>(&x);
          }
          uint8_t* block = dst + (ch >> 2) * kBN * 128;  // 64 elements per 128-byte row
          *reinterpret_cast<uint4*>(block + ((((ch & 3) * 2) ^ (r & 7)) << 4)) = make_uint4(o[0], o[1], o[2], o[3]);
          *reinterpret_cast<uint4*>(block + ((((ch & 3) * 2 + 1) ^ (r & 7)) << 4)) = make_uint4(o[4], o[5], o[6], o[7]);
        };
        if (far) {
          if (widen_row_far<D>(src, dst, r, e, key >= context, key >= w.len))
            atomicOr(&ms->bad[w.index & 7][(key - context) >> 5], 1u << ((key - context) & 31));
        } else if ((i + 1) * kBN <= context) {
          // Two chunks at a time (64, 128 and 256 rows 76, 84, 139 us; four: 79, 86, 140; one: 81, 89, 141).
#pragma unroll 1
          for (int c4 = 0; c4 < D / 16; c4 += 2) {
            uint4 v[2];
#pragma unroll
            for (int q = 0; q < 2; ++q) v[q] = *reinterpret_cast<const uint4*>(src + (((c4 + q) ^ sw) << 4));
#pragma unroll
            for (int q = 0; q < 2; ++q) {
              const uint32_t w4[4] = {v[q].x, v[q].y, v[q].z, v[q].w};
              widen(c4 + q, w4);
            }
          }
        } else {
          // The tile holds drafted keys, whose NaN codes are taken out and flagged, or the end: everything out behind it.
          if (widen_row_edge<D>(src, dst, r, f2, key >= context, key >= w.len))
            atomicOr(&ms->bad[w.index & 7][(key - context) >> 5], 1u << ((key - context) & 31));
        }
        fence_proxy_async_smem();
        mbar_arrive(&ms->v16_full[tile & 1]);
        __syncwarp();
        if (lane == 0) mbar_arrive(&ms->v_empty[slot]);
      }
      vote();  // the piece's last waits have had none
    } while (ok && w.next(p));
    }
  } else {
    reg_dealloc<C::kRegsOther>();  // idle until the end
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 9) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

template <int D, int F, int TILES>
cudaError_t launch(const TreeParams& p, cudaStream_t s) {
  using C = Cfg<D, F, TILES>;
  static_assert(sizeof(Bars) % 8 == 0 && offsetof(Scales, k_scale) % 16 == 0 && offsetof(Scales, v_scale) % 16 == 0 &&
                    offsetof(Scales, ks) % 16 == 0 && C::kOffMisc % 16 == 0,
                "bulk copies and 16-byte accesses");
  // The register split draws on what the block is launched with, which is the compiled kernel's for good.
  static std::atomic<bool> checked{false};
  cudaError_t e;
  if (!checked.load(std::memory_order_relaxed)) {
    cudaFuncAttributes a;
    e = cudaFuncGetAttributes(&a, tree_wide_kernel<D, F, TILES>);
    if (e != cudaSuccess) return e;
    if (a.numRegs < C::kRegsLaunch) return cudaErrorInvalidConfiguration;
    checked.store(true, std::memory_order_relaxed);
  }
  e = cudaFuncSetAttribute(tree_wide_kernel<D, F, TILES>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
  if (e != cudaSuccess) return e;
  tree_wide_kernel<D, F, TILES>
      <<<dim3(static_cast<unsigned>(p.row_tiles), static_cast<unsigned>(p.parts)), C::kThreads, C::kSmem, s>>>(p);
  return cudaGetLastError();
}

// Two row tiles share a CTA's keys where there are more than 128 rows.  Below, the second would be empty: 64 and 128
// rows with shared rows or with two tiles, E4M3 80, 84 | 117, 121 us, bf16 99, 105 | 107, 113, E2M1 88, 91 | 125, 129
// (8 x 16384 keys).
template <int D, int F>
cudaError_t launch_tiles(const TreeParams& p, cudaStream_t s) {
  return p.T * p.G <= kRowTile ? launch<D, F, 1>(p, s) : launch<D, F, 2>(p, s);
}

}  // namespace

int tree_cta_rows(int64_t rows) { return rows <= kRowTile ? kRowTile : 2 * kRowTile; }

template <int D>
static cudaError_t launch_format(const TreeParams& p, int format, cudaStream_t s) {
  switch (format) {
    case kCacheBf16: return launch_tiles<D, kCacheBf16>(p, s);
    case kCacheE4m3: return launch_tiles<D, kCacheE4m3>(p, s);
    case kCacheE2m1: return launch_tiles<D, kCacheE2m1>(p, s);
  }
  return cudaErrorInvalidValue;
}

cudaError_t launch_tree_wide(const TreeParams& p, int d, int format, cudaStream_t s) {
  return d == 128 ? launch_format<128>(p, format, s) : d == 64 ? launch_format<64>(p, format, s) : cudaErrorInvalidValue;
}

}  // namespace fa

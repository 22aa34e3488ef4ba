// fa_tree.cuh — what the kernels of drafted-token attention share: the walk over
// a CTA's part of the key tiles, the slots of cut pairs, and fetching and widening rows of codes.
#pragma once

#include <cuda_fp16.h>

#include "fa_kernels.h"
#include "sm103.cuh"

namespace fa {

constexpr int kTreeBN = 128;                // keys per tile
constexpr uint64_t kTreeDrainNs = 200000000ull;

// Position in a ring of N slots and the parity of its passes.
template <int N>
struct Ring {
  int slot = 0;
  uint32_t parity = 0;
  __device__ __forceinline__ void advance() {
    if (++slot == N) {
      slot = 0;
      parity ^= 1u;
    }
  }
};

__device__ __forceinline__ unsigned int tree_site(unsigned int s) { return (kKernTree << 8) | s; }

// Lengths of sequence b: keys in all and drafted keys among them.  Lengths that
// cannot be are taken as an empty sequence, and false is returned.
__device__ __forceinline__ bool seq_lengths(const TreeParams& p, int b, int& len, int& drafts) {
  len = p.seq_lens[b];
  drafts = p.draft_lens != nullptr ? p.draft_lens[b] : p.T;
  if (p.draft_lens == nullptr && len == 0) drafts = 0;  // an unused batch slot
  const bool fine = drafts >= 0 && drafts <= p.T && len >= drafts && len <= p.max_blocks * p.block_size;
  if (!fine) len = drafts = 0;
  return fine;
}
// Key tiles of a sequence; one without drafted tokens has no rows and needs none.
__device__ __forceinline__ int seq_tiles(int len, int drafts) {
  return drafts > 0 ? (len + kTreeBN - 1) / kTreeBN : 0;
}

__device__ __forceinline__ void report_bad_page(const TreeParams& p) {
  atomicCAS(p.err + 1, 0u, (kKernTree << 8) | kSiteBadBlock);
}

// Row rr of the T·G rows of a pair belongs to token rr / G.
__device__ __forceinline__ int token_of(const TreeParams& p, int rr) {
  return p.G == 1 ? rr : static_cast<int>(__umulhi(static_cast<unsigned>(rr), p.g_magic));
}

// Does token t see drafted key u?
__device__ __forceinline__ bool token_sees(const TreeParams& p, int b, int t, int u) {
  return p.mask != nullptr ? p.mask[b * p.mask_sb + static_cast<int64_t>(t) * p.T + u] != 0 : u <= t;
}

// What few tiles need stands out of line: the kernels' loops are short of instruction cache (inlining the routine for
// far value rows cost the kernel for many rows 6 % on tiles that have none).

// Does any of the first `drafts` tokens see the drafted key whose column of the mask begins at mk?
static __device__ __noinline__ bool any_token_sees(const uint8_t* mk, int drafts, int T) {
  bool sees = false;
#pragma unroll 8
  for (int t = 0; t < drafts; ++t) sees |= mk[static_cast<int64_t>(t) * T] != 0;
  return sees;
}

// 2^e twice as fp16 (e <= 15); far below 1 it fades into fp16's subnormals and out.
__device__ __forceinline__ uint32_t power_f16x2(int e) {
  const uint32_t f = e >= -14 ? static_cast<uint32_t>(e + 15) << 10 : e >= -24 ? 1u << (e + 24) : 0u;
  return f | (f << 16);
}

// Widens one value row of D E4M3 codes to fp16, times the pair of scales.  src: the row in its slot, swizzled as TMA
// wrote it; dst: the row in the first 64-column block of the fp16 tile.  drafted: NaN codes are taken out and reported by
// the result; dead: zeros.
template <int D>
__device__ __noinline__ bool widen_row_edge(const uint8_t* src, uint8_t* dst, int r, uint32_t scale2, bool drafted,
                                            bool dead) {
  const int sw = D == 128 ? r & 7 : (r >> 1) & 3;
  bool bad = false;
#pragma unroll 1
  for (int ch = 0; ch < D / 16; ++ch) {
    const uint4 v = *reinterpret_cast<const uint4*>(src + ((ch ^ sw) << 4));
    uint32_t w[4] = {v.x, v.y, v.z, v.w};
    uint32_t o[8];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      if (drafted) {
#pragma unroll
        for (int q = 0; q < 4; ++q)
          if (((w[e] >> (8 * q)) & 0x7f) == 0x7f) w[e] &= ~(0xffu << (8 * q)), bad = true;
      }
      if (dead) w[e] = 0;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint32_t h = e4m3x2_to_f16x2(w[i >> 1] >> (16 * (i & 1)));
      const __half2 x = __hmul2(*reinterpret_cast<const __half2*>(&h), *reinterpret_cast<const __half2*>(&scale2));
      o[i] = *reinterpret_cast<const uint32_t*>(&x);
    }
    uint8_t* block = dst + (ch >> 2) * kTreeBN * 128;  // 64 elements per 128-byte row
    *reinterpret_cast<uint4*>(block + ((((ch & 3) * 2) ^ (r & 7)) << 4)) = make_uint4(o[0], o[1], o[2], o[3]);
    *reinterpret_cast<uint4*>(block + ((((ch & 3) * 2 + 1) ^ (r & 7)) << 4)) = make_uint4(o[4], o[5], o[6], o[7]);
  }
  return bad && !dead;
}

// Widens one value row of D E4M3 codes times 2^e to bf16, into a tile laid out as the fp16 one: for tiles whose value
// rows lie too far apart for fp16.  drafted: NaN codes are taken out and reported by the result; dead: zeros.
template <int D>
__device__ __noinline__ bool widen_row_far(const uint8_t* src, uint8_t* dst, int r, int e, bool drafted, bool dead) {
  const float f = __uint_as_float(static_cast<uint32_t>(max(e, -126) + 127) << 23);
  const float f2 = e >= -126 ? 1.f : e < -252 ? 0.f : __uint_as_float(static_cast<uint32_t>(e + 126 + 127) << 23);
  const int sw = D == 128 ? r & 7 : (r >> 1) & 3;
  bool bad = false;
#pragma unroll 1
  for (int ch = 0; ch < D / 16; ++ch) {
    const uint4 v = *reinterpret_cast<const uint4*>(src + ((ch ^ sw) << 4));
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    uint32_t o[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      uint32_t c = w[i >> 1] >> (16 * (i & 1)) & 0xffffu;
      if (drafted) {
        if ((c & 0x7fu) == 0x7fu) c &= 0xff00u, bad = true;
        if ((c & 0x7f00u) == 0x7f00u) c &= 0xffu, bad = true;
      }
      if (dead) c = 0;
      const uint32_t h = e4m3x2_to_f16x2(c);
      const float2 x = __half22float2(*reinterpret_cast<const __half2*>(&h));
      o[i] = pack_bf16x2(x.x * f * f2, x.y * f * f2);
    }
    uint8_t* block = dst + (ch >> 2) * kTreeBN * 128;  // 64 elements per 128-byte row
    *reinterpret_cast<uint4*>(block + ((((ch & 3) * 2) ^ (r & 7)) << 4)) = make_uint4(o[0], o[1], o[2], o[3]);
    *reinterpret_cast<uint4*>(block + ((((ch & 3) * 2 + 1) ^ (r & 7)) << 4)) = make_uint4(o[4], o[5], o[6], o[7]);
  }
  return bad && !dead;
}

// A pair of weights p as bf16 terms hi + lo, both positive where p is: an infinite value comes out of two products as
// itself, where a term of the other sign, or zero, would make it NaN.  hi is p·(1 − 2⁻⁸) rounded down (its upper half),
// so lo is between 2⁻⁸ and 2^-6.4 of p and its rounding at most 2⁻⁹ of that: the sum is off by 2⁻¹⁵ p.
__device__ __forceinline__ void split_weights2(float p0, float p1, uint32_t& hi, uint32_t& lo) {
  float a, b;
  fmul2(a, b, p0, p1, 0.99609375f, 0.99609375f);
  hi = __byte_perm(__float_as_uint(a), __float_as_uint(b), 0x7632);
  lo = pack_bf16x2(p0 - __uint_as_float(hi << 16), p1 - __uint_as_float(hi & 0xffff0000u));
}

// A pair of fp16 weights as bf16 terms hi + lo (exact: 11 bits in 8 and 8).
__device__ __forceinline__ void split_f16x2(uint32_t pair, uint32_t& hi, uint32_t& lo) {
  const float2 x = __half22float2(*reinterpret_cast<const __half2*>(&pair));
  hi = pack_bf16x2(x.x, x.y);
  lo = pack_bf16x2(x.x - __uint_as_float(hi << 16), x.y - __uint_as_float(hi & 0xffff0000u));
}

// A CTA's part of the line of key tiles of all (b, key/value head) pairs.
struct TreePart {
  long long per, count;   // tiles per part, and of this one
  int b, h, tile;         // where it begins
};

// Finds it, by all NT threads of the block: sums over the sequences, one block of
// them per thread.  Reports lengths that cannot be.  Contains block barriers.
template <int NT>
__device__ __forceinline__ TreePart find_part(const TreeParams& p, int part, long long* warp_sum, int* start) {
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int per_thread = (p.B + NT - 1) / NT;
  const int b0 = min(p.B, tid * per_thread), b1 = min(p.B, b0 + per_thread);
  long long mine = 0;
#pragma unroll 1
  for (int b = b0; b < b1; ++b) {
    int len, drafts;
    if (!seq_lengths(p, b, len, drafts)) atomicCAS(p.err + 1, 0u, (kKernTree << 8) | kSiteBadLength);
    mine += seq_tiles(len, drafts);
  }
  long long incl = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long x = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += x;
  }
  if (lane == 31) warp_sum[warp] = incl;
  __syncthreads();
  long long before = incl - mine, total = 0;
#pragma unroll 1
  for (int w = 0; w < NT / 32; ++w) {
    if (w < warp) before += warp_sum[w];
    total += warp_sum[w];
  }
  total *= p.Hkv;
  before *= p.Hkv;
  TreePart r;
  r.per = max(2ll, (total + p.parts - 1) / p.parts);  // at least two tiles, one for each stream
  const long long first = part * r.per;
  r.count = min(r.per, total - first);
  if (first >= before && first < before + mine * p.Hkv) {
    long long at = first - before;
#pragma unroll 1
    for (int b = b0; b < b1; ++b) {
      int len, drafts;
      seq_lengths(p, b, len, drafts);
      const int n = seq_tiles(len, drafts);
      if (at < static_cast<long long>(n) * p.Hkv) {  // fits 32 bits: the host checks tiles · Hkv
        start[0] = b;
        start[1] = static_cast<int>(static_cast<unsigned>(at) / static_cast<unsigned>(n));
        start[2] = static_cast<int>(static_cast<unsigned>(at) % static_cast<unsigned>(n));
        break;
      }
      at -= static_cast<long long>(n) * p.Hkv;
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  r.b = start[0];
  r.h = start[1];
  r.tile = start[2];
  return r;
}

// The walk over a part: one pair, or a piece of it, per step.  Plain data, so that
// a warpgroup with no registers to spare keeps it in shared memory.
struct TreeWalk {
  long long left;   // tiles of the part that remain, this piece's excluded
  int b, h, len, drafts, tiles;
  int t0, t1;       // the piece: tiles [t0, t1) of the pair
  int index;        // pieces before this one

  __device__ __forceinline__ void begin(const TreeParams& p, const TreePart& s) {
    b = s.b;
    h = s.h;
    seq_lengths(p, b, len, drafts);
    tiles = seq_tiles(len, drafts);
    t0 = s.tile;
    t1 = static_cast<int>(min(static_cast<long long>(tiles), t0 + s.count));
    left = s.count - (t1 - t0);
    index = 0;
  }
  __device__ __forceinline__ bool next(const TreeParams& p) {
    if (left <= 0) return false;
    if (++h == p.Hkv) {
      h = 0;
      do {
        if (++b >= p.B) return false;
        seq_lengths(p, b, len, drafts);
        tiles = seq_tiles(len, drafts);
      } while (tiles == 0);
    }
    t0 = 0;
    t1 = static_cast<int>(min(static_cast<long long>(tiles), left));
    left -= t1;
    ++index;
    return true;
  }
  __device__ __forceinline__ bool whole() const { return t0 == 0 && t1 == tiles; }
  __device__ __forceinline__ int64_t pair(const TreeParams& p) const { return static_cast<int64_t>(b) * p.Hkv + h; }
  // The slot of a piece of a cut pair: numbered along the line, or two per part (a part has one at each end at most).
  __device__ __forceinline__ int64_t slot(const TreeParams& p, int part) const {
    return p.slots_by_pair ? pair(p) + part : 2ll * part + (t0 > 0 ? 0 : 1);
  }
  // For the joining kernel, at a pair's first piece: its part and how many parts the pair lies in.
  __device__ __forceinline__ int2 pieces(int part, long long per) const {
    const int rest = tiles - (t1 - t0);
    const int step = static_cast<int>(min(per, 1ll << 30));
    return make_int2(part, rest > 0 ? 2 + (rest - 1) / step : 1);
  }
};

// Loads the tiles of a part into a ring, by one warp: K's, or V's and with them both scales' bytes (E4M3).  A page of one
// head is one TMA box; full and empty are the ring's barriers, sc_full those of the scale bytes' own ring, which is longer:
// the slot that V goes to is free, so the tile `ring` before it has been widened, and the scale bytes of the ones before
// that have been read.
template <int D, bool FP8, int kScaleRing>
__device__ __forceinline__ void load_pages(const TreeParams& p, const TreePart& my, bool is_v, uint8_t* dst, int ring,
                                           uint64_t* full, uint64_t* empty, uint64_t* sc_full, uint8_t* k_scale,
                                           uint8_t* v_scale, volatile int* abort_flag, unsigned int site) {
  constexpr bool kPg5 = !FP8 && D == 128;  // pages as [row group][half][8 rows][128 bytes]
  constexpr int kSlot = kTreeBN * D * (FP8 ? 1 : 2);
  const int lane = threadIdx.x & 31;
  const int bshift = 31 - __clz(p.block_size);  // a power of two
  const CUtensorMap* tm = is_v ? &p.tm_v : &p.tm_k;
  dst += lane * p.block_size * (kSlot / kTreeBN);
  if (lane == 0) tma_prefetch_desc(tm);
  const int npt = kTreeBN >> bshift;  // pages per tile
  int slot = 0, sc = 0, issued = 0;
  uint32_t parity = 1;
  bool ok = true;
  TreeWalk w;
  w.begin(p, my);
  do {
    const int pages = (w.len + p.block_size - 1) >> bshift;
    const int32_t* table = p.block_table + static_cast<int64_t>(w.b) * p.max_blocks;
    // The ids of 32 pages at a time, one per lane, loaded one group ahead and checked when they are due.
    int page = w.t0 * npt + lane;
    int id = 0, ahead = page < pages ? table[page] : 0;
    int at = 32;  // the tile's first page in the group
#pragma unroll 1
    for (int i = w.t0; i < w.t1; ++i) {
      if (at == 32) {
        at = 0;
        id = page < pages ? ahead : -1;  // −1: past the end
        if (page < pages && (id < 0 || id >= p.num_blocks)) {
          report_bad_page(p);
          id = 0;
        }
        page += 32;
        ahead = page < pages ? table[page] : 0;
      }
      const int blk = __shfl_sync(0xffffffffu, id, at + lane);
      at += npt;
      ok = __all_sync(0xffffffffu, mbar_wait_inl(&empty[slot], parity, abort_flag, p.err, site));
      if (!ok) break;
      const bool real = lane < npt && blk >= 0;
      const uint32_t n_real = __popc(__ballot_sync(0xffffffffu, real));
      if (lane == 0) {
        mbar_arrive_expect_tx(&full[slot], kSlot);
        if (FP8 && is_v) mbar_arrive_expect_tx(&sc_full[sc], 2 * n_real * p.block_size);
      }
      __syncwarp();
      if (lane < npt) {
        const int row = real ? 0 : p.block_size;  // a row past the page: TMA fills the box with zeros
        const int head = (real ? blk : 0) * p.Hkv + w.h;
        if constexpr (kPg5)
          tma_load_5d(dst + slot * kSlot, tm, &full[slot], 0, 0, 0, row >> 3, head);
        else
          tma_load_4d(dst + slot * kSlot, tm, &full[slot], 0, row, w.h, real ? blk : 0);
        if (FP8 && is_v && real) {
          const int64_t from = static_cast<int64_t>(head) << bshift;
          const int to = sc * kTreeBN + (lane << bshift);
          bulk_load(k_scale + to, p.k_scale + from, p.block_size, &sc_full[sc]);
          bulk_load(v_scale + to, p.v_scale + from, p.block_size, &sc_full[sc]);
        }
      }
      ++issued;
      sc = (sc + 1) % kScaleRing;
      if (++slot == ring) {
        slot = 0;
        parity ^= 1u;
      }
    }
  } while (ok && w.next(p));
  // The copies in flight land before the CTA ends, also where a wait of another warp fails after this one is done.
  if (lane == 0) {
#pragma unroll 1
    for (int n = max(0, issued - ring); n < issued; ++n) {
      mbar_wait_drain_inl(&full[n % ring], (n / ring) & 1, kTreeDrainNs);
      if (FP8 && is_v) mbar_wait_drain_inl(&sc_full[n % kScaleRing], (n / kScaleRing) & 1, kTreeDrainNs);
    }
  }
}

// ---------------------------------------------------------------- a cache in four bits
//
// A page of one head is contiguous: its codes come by one plain bulk copy, its scale bytes by the lanes' asynchronous ones, into
// a ring of half tiles (the keys or the values of 128 rows; in one ring K₀, K₁, V₀, K₂, V₁ … of each piece, the order in which they are used), and
// other warps widen them to fp16, each group times its power of two relative to a reference: from 2⁻²³ to 2^13 of it that
// is exact (the smallest code but zero, 0.5, becomes fp16's smallest step, 2⁻²⁴, and the largest, 6, stays below 65504).
// (Copies of pages without a tensor map: a page of 16 keys is 1 KB of codes and 64 bytes of scales, and the products need
// the codes rearranged anyway.)
constexpr int kFourLazy = 13, kFourFar = 23;

// Whether a row's groups have exponents that a reference does not fit: usually none has, and then it stays.  (NaN, byte 255,
// and next to nothing, 2⁻¹²⁶ and below or zeros, are looked at more closely.)
template <int G>
__device__ __forceinline__ bool outside_reference(uint32_t bytes, int ref) {
  bool outside = false;
#pragma unroll
  for (int j = 0; j < G; ++j) {
    const int e = static_cast<int>(bytes >> (8 * j) & 0xffu) - 127 - ref;
    outside |= static_cast<unsigned>(e + kFourFar) > static_cast<unsigned>(kFourLazy + kFourFar);
  }
  return outside;
}
// The largest and the smallest of G exponent bytes (0 and 255 if there is none).  NaN, and next to nothing for the smallest,
// do not count.
template <int G>
__device__ __forceinline__ int2 exponent_range(uint32_t bytes) {
  int top = 0, low = 255;
#pragma unroll
  for (int j = 0; j < G; ++j) {
    const int e = static_cast<int>(bytes >> (8 * j) & 0xffu);
    if (e != 255) top = max(top, e);
    if (e > 1) low = min(low, e);
  }
  return make_int2(top, low);
}
// The same for the rows of 128 threads that count, by all of them, with barrier `bar`.
template <int G>
__device__ __forceinline__ int2 exponent_range(uint32_t bytes, bool counts, int bar, int* range) {
  const int2 mine = exponent_range<G>(bytes);
  const int top = __reduce_max_sync(0xffffffffu, counts ? mine.x : 0);
  const int low = __reduce_min_sync(0xffffffffu, counts ? mine.y : 255);
  if ((threadIdx.x & 31) == 0) range[(threadIdx.x >> 5) & 3] = top << 8 | (255 - low);
  __syncwarp();
  named_sync(bar, 128);
  int2 r = make_int2(0, 255);
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const int x = range[q];
    r.x = max(r.x, x >> 8);
    r.y = min(r.y, 255 - (x & 0xff));
  }
  return r;
}

template <int D>
struct FourBit {
  static constexpr int kCodes = kTreeBN * D / 2, kScales = kTreeBN * D / kE2m1Group;
  static constexpr int kHalf = kCodes + kScales;  // bytes of a ring's slot
};

// What load_codes fetches: both halves into one ring, in the order above, or the keys or the values alone.
enum CodeParts : int { kBothHalves = 0, kKeyCodes = 1, kValueCodes = 2 };

// Arrivals that a half's barrier waits for: the warp's lanes, as their scales land, and the one that announces the codes.
constexpr int kCodeArrivals = 33;

// Fetches the codes and scales of a part's tiles, by one warp, into a ring of RING halves.  at_piece is called at the start
// of every piece.
template <int D, int RING, CodeParts PARTS, class AtPiece>
__device__ __forceinline__ void load_codes(const TreeParams& p, const TreePart& my, uint8_t* ring, uint64_t* full,
                                           uint64_t* empty, volatile int* abort_flag, unsigned int site,
                                           AtPiece at_piece) {
  constexpr int kRow = D / 2, kRowScales = D / kE2m1Group;
  const int lane = threadIdx.x & 31;
  const int bshift = 31 - __clz(p.block_size);  // a power of two
  const int npt = kTreeBN >> bshift;            // pages per tile
  int slot = 0, issued = 0;
  uint32_t parity = 1;
  bool ok = true;
  // blk: the page of this lane, one of the tile's, or −1 past the end.
  auto half = [&](int blk, int h, bool is_v) {
    ok = mbar_wait_inl(&empty[slot], parity, abort_flag, p.err, site);
    ok = __all_sync(0xffffffffu, ok);
    if (!ok) return;
    const bool real = lane < npt && blk >= 0;
    const uint32_t n_real = __popc(__ballot_sync(0xffffffffu, real));
    if (lane == 0) mbar_arrive_expect_tx(&full[slot], n_real * (kRow << bshift));
    __syncwarp();
    uint8_t* to = ring + slot * FourBit<D>::kHalf;
    if (real) {
      const int64_t row = (static_cast<int64_t>(blk) * p.Hkv + h) << bshift;
      bulk_load(to + ((lane << bshift) * kRow), static_cast<const uint8_t*>(is_v ? p.v_cache : p.k_cache) + row * kRow,
                kRow << bshift, &full[slot]);
    }
    // The scales by sixteen bytes a lane: bulk copies of so little cost as much as those of the codes (64 ragged sequences of
    // up to 8192 keys in pages of 16: 88 us instead of 94).
    const int row0 = lane * (16 / kRowScales);
    const int from = __shfl_sync(0xffffffffu, blk, min(row0 >> bshift, 31));
    if (lane < FourBit<D>::kScales / 16 && from >= 0)
      cp_async16(to + FourBit<D>::kCodes + lane * 16,
                 (is_v ? p.v_scale : p.k_scale) +
                     (((static_cast<int64_t>(from) * p.Hkv + h) << bshift) + (row0 & (p.block_size - 1))) * kRowScales);
    cp_async_arrive(&full[slot]);
    ++issued;
    if (++slot == RING) {
      slot = 0;
      parity ^= 1u;
    }
  };
  TreeWalk w;
  w.begin(p, my);
  do {
    const int pages = (w.len + p.block_size - 1) >> bshift;
    const int32_t* table = p.block_table + static_cast<int64_t>(w.b) * p.max_blocks;
    // The ids of 32 pages at a time, one per lane, loaded one group ahead and checked when they are due.
    int page = w.t0 * npt + lane;
    int id = 0, ahead = page < pages ? table[page] : 0;
    int at = 32;  // the tile's first page in the group
    int before = -1;
    if (!at_piece(w)) break;
#pragma unroll 1
    for (int i = w.t0; i < w.t1 + (PARTS == kBothHalves ? 1 : 0); ++i) {
      int blk = -1;
      if (i < w.t1) {
        if (at == 32) {
          at = 0;
          id = page < pages ? ahead : -1;  // −1: past the end
          if (page < pages && (id < 0 || id >= p.num_blocks)) {
            report_bad_page(p);
            id = 0;
          }
          page += 32;
          ahead = page < pages ? table[page] : 0;
        }
        blk = __shfl_sync(0xffffffffu, id, at + lane);
        at += npt;
        half(blk, w.h, PARTS == kValueCodes);
      }
      if (PARTS == kBothHalves && ok && i > w.t0) half(before, w.h, true);
      if (!ok) break;
      before = blk;
    }
  } while (ok && w.next(p));
  // The copies in flight land before the CTA ends.
  if (lane == 0) {
#pragma unroll 1
    for (int n = max(0, issued - RING); n < issued; ++n) mbar_wait_drain_inl(&full[n % RING], (n / RING) & 1, kTreeDrainNs);
  }
}

// A row's group g of 32 codes to its places in a 16-bit tile of rows of 128 bytes (64 columns), r: the row.
template <class Convert>
__device__ __forceinline__ void widen_group(uint4 c, uint8_t* dst, int r, int g, Convert convert) {
  const uint32_t w[4] = {c.x, c.y, c.z, c.w};
  uint8_t* block = dst + (g >> 1) * kTreeBN * 128;
#pragma unroll
  for (int j = 0; j < 4; ++j)
    *reinterpret_cast<uint4*>(block + ((((g & 1) * 4 + j) ^ (r & 7)) << 4)) = convert(w[j]);
}
// Eight codes to fp16, times the pair of scales.
__device__ __forceinline__ uint4 widen_e2m1x8(uint32_t w, uint32_t scale2) {
  uint32_t o[4];
  e2m1x8_to_f16(w, o);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __half2 x = __hmul2(*reinterpret_cast<const __half2*>(&o[i]), *reinterpret_cast<const __half2*>(&scale2));
    o[i] = *reinterpret_cast<const uint32_t*>(&x);
  }
  return make_uint4(o[0], o[1], o[2], o[3]);
}
// The group a thread takes at step j: rows of 64 bytes lie four to a pass over the banks, so neighbouring pairs of rows
// begin with different groups.
template <int D>
__device__ __forceinline__ int group_at(int j, int r) {
  return D == 128 ? (j + (r >> 1)) & 3 : j;
}

// Widens one row of E2M1 codes to fp16, each group times its power of two relative to 2^ref.
// src: the row's codes, scales: its bytes.  A larger body saves waits and costs instruction fetches, which all warps' roles
// compete for, so how many groups are unrolled is the caller's choice.
template <int D, int UNROLL>
__device__ __forceinline__ void widen_codes(const uint8_t* src, uint32_t scales, uint8_t* dst, int r, int ref) {
  // Rows are 128 bytes long and begin at multiples of that: the swizzle takes one operation a store.
  const uint32_t to = smem_u32(dst) ^ ((r & 7) << 4);
#pragma unroll UNROLL
  for (int j = 0; j < D / kE2m1Group; ++j) {
    const int g = group_at<D>(j, r);
    const uint4 c = *reinterpret_cast<const uint4*>(src + g * 16);
    const int s = static_cast<int>(scales >> (8 * g) & 0xffu), e = s - 127 - ref;
    uint32_t scale2 = static_cast<uint32_t>(e + 15) * 0x04000400u;  // 2^e twice, a normal number but for …
    if (static_cast<unsigned>(e + 14) > 29u || s == 255) scale2 = s == 255 ? 0x7e007e00u : power_f16x2(e);
    const uint32_t at = (to + (g >> 1) * (kTreeBN * 128)) ^ ((g & 1) << 6), w[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
    for (int q = 0; q < 4; ++q) st_shared16(at ^ (q << 4), widen_e2m1x8(w[q], scale2));
  }
}
// The same out of line for tiles that hold drafted keys (whose NaN groups are taken out and reported by the result), the
// end (dead: zeros), or, far, value groups that lie too far apart for fp16 and go to bf16.
template <int D>
__device__ __noinline__ bool widen_codes_edge(const uint8_t* src, uint32_t scales, uint8_t* dst, int r, int ref,
                                              bool drafted, bool dead, bool far) {
  bool bad = false;
#pragma unroll 1
  for (int g = 0; g < D / kE2m1Group; ++g) {
    uint4 c = *reinterpret_cast<const uint4*>(src + g * 16);
    uint32_t s = scales >> (8 * g) & 0xffu;
    const bool out = drafted && s == 255;
    bad |= out;
    if (out || dead) {
      c = make_uint4(0, 0, 0, 0);
      s = 127;
    }
    const int e = out || dead ? 0 : static_cast<int>(s) - 127 - ref;
    if (far) {
      // 2^e in two factors, as it may be too small a number by itself.
      const float f = s == 255 ? __uint_as_float(0x7fffffffu) : __uint_as_float(static_cast<uint32_t>(max(e, -126) + 127) << 23);
      const float f2 = e >= -126 ? 1.f : e < -252 ? 0.f : __uint_as_float(static_cast<uint32_t>(e + 126 + 127) << 23);
      widen_group(c, dst, r, g, [&](uint32_t w) {
        uint32_t o[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t h = e2m1x2_to_f16x2(w >> (8 * i));
          const float2 x = __half22float2(*reinterpret_cast<const __half2*>(&h));
          o[i] = pack_bf16x2(x.x * f * f2, x.y * f * f2);
        }
        return make_uint4(o[0], o[1], o[2], o[3]);
      });
    } else {
      const uint32_t scale2 = s == 255 ? 0x7e007e00u : power_f16x2(e);
      widen_group(c, dst, r, g, [&](uint32_t w) { return widen_e2m1x8(w, scale2); });
    }
  }
  return bad && !dead;
}

// Eight elements of a query row, whose other ones the neighbouring kChunks − 1 lanes hold, as E4M3 terms
// x·2⁻ᵃ = hi + lo·2^−kLow; 2⁻ᵃ, which is returned as a, brings the row's largest magnitude to at most 448.
template <int kChunks, int kLow>
__device__ __forceinline__ int split_q8(uint4 v, uint2& hi, uint2& lo) {
  const uint32_t w4[4] = {v.x, v.y, v.z, v.w};
  float x[8];
  uint32_t top = 0;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    x[e] = __uint_as_float(e & 1 ? w4[e >> 1] & 0xffff0000u : w4[e >> 1] << 16);
    const uint32_t a = __float_as_uint(x[e]) & 0x7fffffffu;
    if (a < 0x7f800000u) top = max(top, a);
    else x[e] = __uint_as_float(0x7fffffffu);
  }
#pragma unroll
  for (int mk = kChunks / 2; mk > 0; mk >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, mk));
  const int a = max(-126, static_cast<int>(top >> 23) - 135 + ((top & 0x7fffffu) > 0x600000u ? 1 : 0));
  const float inv = __uint_as_float(static_cast<uint32_t>(127 - a) << 23);
  constexpr float kUp = 1 << kLow;
  uint32_t h2[2] = {0, 0}, l2[2] = {0, 0};
#pragma unroll
  for (int e = 0; e < 8; e += 2) {
    const float y0 = x[e] * inv, y1 = x[e + 1] * inv;
    const uint32_t h = pack_e4m3x2(y0, y1);
    const uint32_t back = e4m3x2_to_f16x2(h);
    const float2 z = __half22float2(*reinterpret_cast<const __half2*>(&back));
    h2[e >> 2] |= h << ((e & 2) * 8);
    l2[e >> 2] |= pack_e4m3x2((y0 - z.x) * kUp, (y1 - z.y) * kUp) << ((e & 2) * 8);
  }
  hi = make_uint2(h2[0], h2[1]);
  lo = make_uint2(l2[0], l2[1]);
  return a;
}

// Takes what is not finite out of a drafted key's bf16 value row where it lies (in pieces of 128 bytes), and says whether
// there was any; a row past the end becomes zeros.
template <int D>
__device__ __forceinline__ bool clean_value_row(uint8_t* row, bool past_end) {
  bool bad = false;
#pragma unroll 2
  for (int ch = 0; ch < D / 8; ++ch) {
    uint4* at = reinterpret_cast<uint4*>(row + (ch >> 3) * 1024 + (ch & 7) * 16);
    uint32_t v4[4] = {0, 0, 0, 0};
    if (!past_end) {
      const uint4 v = *at;
      v4[0] = v.x, v4[1] = v.y, v4[2] = v.z, v4[3] = v.w;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if ((v4[e] & 0x7f80u) == 0x7f80u) v4[e] &= 0xffff0000u, bad = true;
        if ((v4[e] & 0x7f800000u) == 0x7f800000u) v4[e] &= 0xffffu, bad = true;
      }
    }
    *at = make_uint4(v4[0], v4[1], v4[2], v4[3]);
  }
  return bad;
}

// Where drafted key u's value row of the walk's pair lies in the cache, for what was taken out of it: to be added to the
// rows that see it (a page id that is none was read as page 0).
template <int D>
__device__ __forceinline__ int64_t value_row(const TreeParams& p, const TreeWalk& w, int u) {
  const int bshift = 31 - __clz(p.block_size), key = w.len - w.drafts + u;
  int blk = p.block_table[static_cast<int64_t>(w.b) * p.max_blocks + (key >> bshift)];
  if (blk < 0 || blk >= p.num_blocks) blk = 0;
  return (((static_cast<int64_t>(blk) * p.Hkv + w.h) << bshift) + (key & (p.block_size - 1))) * D;
}
// The element there if it is not finite, else 0.
template <int F>
__device__ __forceinline__ float taken_out(const TreeParams& p, int64_t at) {
  if (F == kCacheE2m1) return p.v_scale[at / kE2m1Group] == 255 ? NAN : 0.f;
  if (F == kCacheE4m3) return (static_cast<const uint8_t*>(p.v_cache)[at] & 0x7f) == 0x7f ? NAN : 0.f;
  const float v = __bfloat162float(static_cast<const __nv_bfloat16*>(p.v_cache)[at]);
  return fabsf(v) <= 3.4028234663852886e38f ? 0.f : v;
}

// True on one lane of a converged warp.
__device__ __forceinline__ bool elect_one_lane() {
  uint32_t pred = 0;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(pred));
  return pred != 0;
}

}  // namespace fa

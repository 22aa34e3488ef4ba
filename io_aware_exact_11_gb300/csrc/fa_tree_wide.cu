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
//
// The rest (parts, pieces, masks, values in masked places) is as in fa_tree.cu.
//
// Measured on GB300, 8 sequences of 16384 keys, 8 key/value heads of 128 elements (replaying a graph over two caches):
//   64 / 128 / 256 rows, bf16    98 / 104 / 125 us   0.82 / 0.77 of a device copy, 1100 TFLOP/s
//   64 / 128 / 256 rows, E4M3    76 /  84 / 140 us   452 / 818 / 982 TFLOP/s
// With two row tiles a step (one tile's P̃V and S, 1024 tensor cycles) takes about 1750 cycles: the issuing
// warp's own instructions, of which it gets one through every dozen cycles beside the softmax warps, and the wait
// for P̃ (S to P̃ is a chain of about 1400 cycles).  E4M3 with shared rows waits for the converters (2400 cycles a
// tile).  A pair boundary costs a CTA 10000 to 15000 cycles (O out, Q in, the first scores).
#include <stddef.h>

#include <atomic>

#include "fa_tree.cuh"

namespace fa {
namespace {

constexpr int kBN = kTreeBN;
constexpr int kRowTile = 128;
constexpr int kMaxRing = 8;
constexpr int kScaleRing = 16;
constexpr int kTileRing = 8;   // E4M3: tiles whose converted scales are kept

template <int D, bool FP8, int TILES>
struct Cfg {
  // Warps: streams 0–3 and 4–7, K loads 8, MMA 9, V loads 10, idle 11; E4M3: converters 12–15.
  static constexpr int kThreads = FP8 ? 512 : 384;
  static constexpr int kRegsLaunch = FP8 ? 128 : 168;
  static constexpr int kRegsSoftmax = FP8 ? 200 : 208;
  static constexpr int kRegsOther = FP8 ? 56 : 88;
  static_assert(2 * kRegsSoftmax + (FP8 ? 2 : 1) * kRegsOther <= (FP8 ? 4 : 3) * kRegsLaunch, "register split");
  static constexpr int kSlot = kBN * D * (FP8 ? 1 : 2);
  static constexpr int kV16 = FP8 ? kBN * D * 2 : 0;
  static constexpr int kQTile = kRowTile * D * 2;        // bf16, or two E4M3 terms
  static constexpr int kTerms = !FP8 && TILES == 1 ? 2 : 1;  // of P̃
  static constexpr int kFixed = TILES * kQTile + 2 * kV16;
  static constexpr int kMisc = (FP8 ? 13 : 2) * 1024 + (TILES == 1 ? 4 * 1024 : 0);
  static constexpr int kRoom = 226 * 1024 - kFixed - kMisc;  // 227 KB less the alignment pad
  static constexpr int kRing = kRoom / kSlot < 14 ? kRoom / kSlot : 14;
  static constexpr int kRK = kRing / 2;
  static constexpr int kRV = kRing - kRK;
  static constexpr int kOffQ = 0;
  static constexpr int kOffV16 = kOffQ + TILES * kQTile;
  static constexpr int kOffK = kOffV16 + 2 * kV16;
  static constexpr int kOffV = kOffK + kRK * kSlot;
  static constexpr int kOffMisc = kOffV + kRV * kSlot;
  static constexpr int kSmem = kOffMisc + kMisc + 1024;
  static constexpr uint32_t kColO = 256;                 // TMEM: S of the streams at 0 and 128, O at 256 and 256 + D
  static_assert(kRK >= 2 && kRV >= 2 && kRV <= kMaxRing && kRV + 4 <= kScaleRing && kSmem <= 227 * 1024, "rings");
  static_assert(kSlot % 1024 == 0 && kQTile % 1024 == 0, "swizzle atoms");
};

struct Bars {
  uint64_t k_full[kMaxRing], k_empty[kMaxRing], v_full[kMaxRing], v_empty[kMaxRing];
  uint64_t s_full[2], p_full[2], v16_full[2], v16_empty[2], ks_full[kTileRing], sc_full[kScaleRing];
  uint64_t q_full, drain;
  uint32_t bad[8][8];       // drafted keys with non-finite values, of up to eight pieces
  long long warp_sum[16];
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

// Rows of a tile as a K-major operand (rows that are not there as zeros), by the 128 threads of a stream (TILES = 2)
// or the 256 of both.  E4M3: two terms per element and the factor of the row.
template <int D, bool FP8, int NT>
__device__ __forceinline__ void load_q_tile(const TreeParams& p, const TreeWalk& w, uint8_t* q, float* f, int row0,
                                            int id) {
  constexpr int kChunks = D / 8;  // 16-byte chunks of a row
  constexpr int kPer = kRowTile * kChunks / NT;
  // Loads in flight per thread (bf16 with shared rows spills registers with eight).
  constexpr int kBatch = NT == 256 && !FP8 ? 4 : kPer < 8 ? kPer : 8;
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
      if constexpr (!FP8) {
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

template <int D, bool FP8, int TILES>
__global__ void __launch_bounds__(Cfg<D, FP8, TILES>::kThreads, 1) tree_wide_kernel(const __grid_constant__ TreeParams p) {
  using C = Cfg<D, FP8, TILES>;
  constexpr bool kPg5 = !FP8 && D == 128;  // K/V pages as [row group][half][8 rows][128 bytes]
  constexpr int kSlot = C::kSlot;
  constexpr float kLazy = 8.f;             // rescale once the maximum exceeds the reference by this …
  constexpr float kBase = FP8 ? 3.f : 0.f; // … the new reference lies this below the maximum
  constexpr int kKvLazy = 7;               // E4M3: widened values stay below 448·2^7
  constexpr int kKvFar = 15;               // value rows that are smaller by more than this need bf16's range
  extern __shared__ uint8_t smem_raw[];
  const uint32_t pad = (1024u - (smem_u32(smem_raw) & 1023u)) & 1023u;
  uint8_t* smem = smem_raw + pad;
  Bars* ms = reinterpret_cast<Bars*>(smem + C::kOffMisc);
  constexpr int kOffScales = (sizeof(Bars) + 15) / 16 * 16;
  constexpr int kOffJoin = kOffScales + (FP8 ? (sizeof(Scales) + 15) / 16 * 16 : 0);
  Scales* sc = reinterpret_cast<Scales*>(smem + C::kOffMisc + kOffScales);  // E4M3 only
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
      mbar_init(&ms->k_full[s], 1);
      mbar_init(&ms->k_empty[s], 1);
    }
    for (int s = 0; s < C::kRV; ++s) {
      mbar_init(&ms->v_full[s], 1);
      mbar_init(&ms->v_empty[s], FP8 ? 4 : 1);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(&ms->s_full[s], 1);
      mbar_init(&ms->p_full[s], 128);
      mbar_init(&ms->v16_full[s], 128);
      mbar_init(&ms->v16_empty[s], 1);
    }
    for (int s = 0; s < kScaleRing; ++s) mbar_init(&ms->sc_full[s], 1);
    for (int s = 0; s < kTileRing; ++s) mbar_init(&ms->ks_full[s], 128);
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
  } else if (warp == 8 || warp == 10) {
    reg_dealloc<C::kRegsOther>();
    // ------------------------------------------- loads of K (warp 8) and V (warp 10)
    const bool is_v = warp == 10;
    load_pages<D, FP8, kScaleRing>(p, my, is_v, smem + (is_v ? C::kOffV : C::kOffK), is_v ? C::kRV : C::kRK,
                                   is_v ? ms->v_full : ms->k_full, is_v ? ms->v_empty : ms->k_empty, ms->sc_full,
                                   sc->k_scale[0], sc->v_scale[0], abort_flag, tree_site(is_v ? 0x22 : 0x21));
  } else if (warp == 9) {
    reg_dealloc<C::kRegsOther>();
    // ------------------------------------------------------------ MMA issuer
    // The whole warp runs the loop, which keeps descriptors warp-uniform, and one elected lane issues.
    constexpr uint32_t kIdescS = FP8 ? idesc_e4m3_f32(128, kBN, false, false) : idesc_bf16_f32(128, kBN, false, false);
    constexpr uint32_t kIdescFar = idesc_bf16_f32(128, D, false, true);
    constexpr uint32_t kIdescO = FP8 ? idesc_f16_f32(128, D, false, true) : idesc_bf16_f32(128, D, false, true);
    const uint32_t sQ = smem_u32(smem + C::kOffQ), sK = smem_u32(smem + C::kOffK);
    const uint32_t sV = smem_u32(smem + (FP8 ? C::kOffV16 : C::kOffV));
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
            ok = ok && (FP8 ? mbar_wait_inl(&ms->v16_full[v16], v16_par, abort_flag, p.err, tree_site(0x2f))
                            : mbar_wait_inl(&ms->v_full[rv.slot], rv.parity, abort_flag, p.err, tree_site(0x24)));
        }
        const bool far = FP8 && product && (*static_cast<volatile int*>(&sc->ref[vt % kTileRing]) & 1);
        const uint32_t idesc = far ? kIdescFar : kIdescO;
        const uint32_t ts = tmem + g * kBN;
        const uint32_t to = tmem + C::kColO + g * D;
        const uint32_t vb = sV + (FP8 ? v16 * C::kV16 : rv.slot * kSlot);
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
            if (FP8 && far) {  // the second terms
#pragma unroll 1
              for (int kk = 0; kk < kBN / 16; ++kk)
                mma_bf16_ts(to, ts + 64 + kk * 8, vd + kk * (kPg5 ? 256 : 128), idesc, 1u);
            }
          }
          p_par ^= 1u << g;
          // With shared rows the value slot is given back at once (after the scores' issue: 1 us of 104 slower); with two
          // row tiles the scores' issue comes first (the other way round 135 instead of 130 us: 256 rows, 8 x 16384 keys).
          if (TILES == 1 && leader) mma_commit(FP8 ? &ms->v16_empty[v16] : &ms->v_empty[rv.slot]);
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
              mma_bf16_ss(ts, qd + (kk >> 2) * (kRowTile * 8) + (kk & 3) * 2, kd + (kk >> 2) * 64 + (kk & 3) * 2, kIdescS,
                          kk > 0 ? 1u : 0u);
          }
        }
        if (leader) {
          if (scores || product) mma_commit(&ms->s_full[g]);  // scores, or, where none follow, O of the piece
          if (last_use && scores) mma_commit(&ms->k_empty[rk.slot]);
          if (TILES == 2 && last_use && product) mma_commit(FP8 ? &ms->v16_empty[v16] : &ms->v_empty[rv.slot]);
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
        load_q_tile<D, FP8, 128>(p, w, smem + C::kOffQ + g * C::kQTile, FP8 ? sc->f + g * kRowTile : nullptr, my_row0,
                                 kt);
      else
        load_q_tile<D, FP8, 256>(p, w, smem + C::kOffQ, FP8 ? sc->f : nullptr, my_row0, tid);
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
        if constexpr (FP8)  // the keys' powers of two
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
        if (busy) {
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
        if (!FP8 && tail && k0 + kt >= context && (TILES == 1 || g == 0)) {
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
      const int half_kv = FP8 ? (TILES == 1 ? max(join->kv[0], join->kv[1]) : kv_ref) >> 1 : 0;
#pragma unroll
      for (int e = 0; e < 2; ++e) scale[e] *= inv * (FP8 ? power_f32((TILES == 1 ? join->kv[e] : kv_ref) - half_kv) : 1.f);
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
          if constexpr (FP8) {
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
            const float v = taken_out<FP8>(p, at + c);
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

template <int D, bool FP8, int TILES>
cudaError_t launch(const TreeParams& p, cudaStream_t s) {
  using C = Cfg<D, FP8, TILES>;
  static_assert(sizeof(Bars) % 8 == 0 && offsetof(Scales, k_scale) % 16 == 0 && offsetof(Scales, v_scale) % 16 == 0 &&
                    offsetof(Scales, ks) % 16 == 0 && C::kOffMisc % 16 == 0,
                "bulk copies and 16-byte accesses");
  // The register split draws on what the block is launched with, which is the compiled kernel's for good.
  static std::atomic<bool> checked{false};
  cudaError_t e;
  if (!checked.load(std::memory_order_relaxed)) {
    cudaFuncAttributes a;
    e = cudaFuncGetAttributes(&a, tree_wide_kernel<D, FP8, TILES>);
    if (e != cudaSuccess) return e;
    if (a.numRegs < C::kRegsLaunch) return cudaErrorInvalidConfiguration;
    checked.store(true, std::memory_order_relaxed);
  }
  e = cudaFuncSetAttribute(tree_wide_kernel<D, FP8, TILES>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
  if (e != cudaSuccess) return e;
  tree_wide_kernel<D, FP8, TILES>
      <<<dim3(static_cast<unsigned>(p.row_tiles), static_cast<unsigned>(p.parts)), C::kThreads, C::kSmem, s>>>(p);
  return cudaGetLastError();
}

// Two row tiles share a CTA's keys where there are more than 128 rows.  Below, the second would be empty: 64 and 128
// rows with shared rows or with two tiles, E4M3 76, 84 | 114, 121 us, bf16 98, 103 | 103, 109 us (8 x 16384 keys).
template <int D, bool FP8>
cudaError_t launch_tiles(const TreeParams& p, cudaStream_t s) {
  return p.T * p.G <= kRowTile ? launch<D, FP8, 1>(p, s) : launch<D, FP8, 2>(p, s);
}

}  // namespace

int tree_cta_rows(int64_t rows) { return rows <= kRowTile ? kRowTile : 2 * kRowTile; }

cudaError_t launch_tree_wide(const TreeParams& p, int d, bool fp8, cudaStream_t s) {
  if (d == 128) return fp8 ? launch_tiles<128, true>(p, s) : launch_tiles<128, false>(p, s);
  if (d == 64) return fp8 ? launch_tiles<64, true>(p, s) : launch_tiles<64, false>(p, s);
  return cudaErrorInvalidValue;
}

}  // namespace fa

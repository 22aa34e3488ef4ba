// fa_pages.cu — the paged cache's pages and rows moved about: rows of a sequence
// brought together, pages copied, and pages shared among sequences, freed and
// reserved.
//
// Rows.  The i-th row kept of a sequence goes from position keep[i] to first + i,
// in place.  With keep[i] ≥ first + i no row is written before all that read it
// have: the place first + i is read for rows j with keep[j] = first + i ≥ first + j,
// that is j ≤ i.  So a block that walks over the rows in chunks, and has read a chunk
// (and some of those after it) before it writes any of it, needs no second copy and no
// order among the rows of a chunk.  Blocks share a sequence by heads and by columns of
// 64 bytes, which never meet; by rows only within a cluster, whose barrier they pass
// together at every chunk.
//
// Pages.  holders[p] counts the sequences whose table names page p; 0 is free.
// Sharing a sequence's pages adds one to each, freeing takes one away, and who is to
// write into a page that others hold too gets one of its own (if the sequence has tokens
// in it, the caller copies its contents).  All results are those of one sequence after
// the other in the order given, with free pages handed out by rising number, whatever
// order the blocks run in: counts are sums of whole numbers, and which sequence gets
// which page follows from prefix sums, not from atomics.  A page that c sequences are
// about to write into and r hold is given up by all of them but the last, and by the last
// too if r > c: when its turn comes, r − (c − 1) sequences still hold it.
//
// Bound: copies and moves by device memory, each byte read and written once; the
// tables by the launches and the chains of dependent loads (length → table → count).
//
// Reserving takes three kernels: free pages per segment and missing pages per sequence
// (a block per segment, a warp per sequence), prefix sums over both (one block), and the
// hand-out, in which every free page finds its sequence by a search in the prefix
// sums: no list of free pages is kept or written.  Pages are shared up to the one that
// holds a sequence's last token, unless a length was set back without giving up what lay
// behind it, and those reserved before have no gaps, unless the caller left some.  Where a
// table names such pages, the middle kernel takes the sequences in turn.
#include "fa_kernels.h"
#include "sm103.cuh"

namespace fa {
namespace {

constexpr int kThreads = 256;
constexpr unsigned int kNowhere = 0xffffffffu;  // of a row that stays

__device__ __forceinline__ void report(unsigned int* err, unsigned int what) {
  atomicCAS(err + 1, 0u, (kKernPages << 8) | what);
}

// ------------------------------------------------------------------ rows and pages

__device__ __forceinline__ uint32_t cluster_blocks() {
  uint32_t n;
  asm("mov.u32 %0, %%cluster_nctaid.x;" : "=r"(n));
  return n;
}
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_ctaid.x;" : "=r"(r));
  return r;
}
// Barrier of all threads of the cluster; what each read or wrote before it comes before what the others do behind it.
__device__ __forceinline__ void cluster_sync() {
  asm volatile(
      "barrier.cluster.arrive.release;\n\t"
      "barrier.cluster.wait.acquire;" ::: "memory");
}

__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// A chunk is U passes of the block over rows, of which kDeep are on their way, and kSteps chunks make a plan.  (Deeper rings
// and longer plans leave room for fewer blocks: with 4 and 8 of two passes the E4M3 rows below take 50 us as now, those in bf16
// 79 instead of 75, and twice as many E4M3 rows 81 instead of 75.)
template <int LANES, int U>
struct Plan {
  static constexpr int kStep = kThreads / LANES * U, kDeep = U == 2 ? 3 : 2, kSteps = U == 2 ? 6 : 5, kPlan = kSteps * kStep;
  static_assert(kSteps - (kDeep - 1) > 3, "a barrier between a plan's places and the first look at them");
  static constexpr int kSmem = kDeep * U * kThreads * 16 + 2 * kPlan * 8;
};

// Moves LANES 16-byte columns of the rows kept of one sequence and head, keys or values.  SB: bytes of a row's scales,
// moved by the blocks of the first columns.  Of every chunk the blocks of a cluster take equal shares.
//
// 8 sequences of 16384 tokens, 8 heads, d = 128, 6000 rows kept of each: 75 us in bf16 (5.2 TB/s of reads and writes), 50 in
// E4M3, 36 in E2M1.  Bound by the latency from a chunk's reads to its barrier while the SMs have two blocks each, and by
// device memory beyond that.
template <int RB, int SB, int LANES, int U>
__global__ void __launch_bounds__(kThreads, 4) cache_compact_kernel(const __grid_constant__ MoveParams p) {
  constexpr int kCols = RB / (16 * LANES);
  constexpr int kRows = kThreads / LANES;  // a pass of the block
  using P = Plan<LANES, U>;
  constexpr int kStep = P::kStep, kDeep = P::kDeep, NP = P::kPlan / kThreads;
  const int lane = threadIdx.x % LANES, r = threadIdx.x / LANES;
  const int cl = static_cast<int>(cluster_blocks()), q = static_cast<int>(cluster_rank());
  const int64_t group = blockIdx.x / cl;
  const int part = static_cast<int>(group % (2 * kCols));
  const int64_t pair = group / (2 * kCols);
  const int b = static_cast<int>(pair / p.Hkv), h = static_cast<int>(pair - static_cast<int64_t>(b) * p.Hkv);
  const int col = part >> 1, which = part & 1;
  const bool scales = SB > 0 && col == 0;
  uint8_t* const cache = p.cache[which] + (col * LANES + lane) * 16;
  uint8_t* const scale = p.scale[which];
  const int shift = 31 - __clz(p.block_size);  // a power of two
  const int room = p.max_blocks << shift;
  const int first = p.first[b], n = p.keep_lens != nullptr ? p.keep_lens[b] : p.N;
  if (n < 0 || n > p.N || first < 0 || first > room - n) {
    if (threadIdx.x == 0) report(p.err, kSiteBadLength);
    return;
  }
  const int* keep = p.keep + b * p.keep_sb;
  const int* table = p.block_table + static_cast<int64_t>(b) * p.max_blocks;
  // A row that is moved takes three loads, each of which gives the next one's address: its position, its pages and itself.
  // The first two are made for a plan of several chunks at a time, while the chunks of the plan before are moved (between
  // those 81 and 56 us instead of 76 and 52 for the bf16 and E4M3 rows above).  The rows go through shared memory: a barrier waits for all loads into
  // registers before it, so only asynchronous copies can be on their way across it (through registers 102 us, and 177 with
  // the positions and pages loaded beside the rows).
  extern __shared__ uint4 ring[];                                             // [kDeep][U][kThreads]
  uint2* const plans = reinterpret_cast<uint2*>(ring + kDeep * U * kThreads);  // of two plans, the places (page · page size +
                                                                              // row in it) that a row comes from and goes to
  const int mask = p.block_size - 1;
  auto row = [&](unsigned int place) -> int64_t {
    return ((static_cast<int64_t>(place >> shift) * p.Hkv + h) << shift) + (place & mask);
  };
  auto barrier = [&] {
    if (cl > 1)
      cluster_sync();
    else
      __syncthreads();
  };
  // Of every cl chunks this block takes the q-th: the i-th row of its k-th plan is row_at(k, i) of those kept.
  auto row_at = [&](int k, int i) {
    return static_cast<int64_t>(k) * P::kPlan * cl + static_cast<int64_t>(i / kStep * cl + q) * kStep + i % kStep;
  };
  const int steps = static_cast<int>((n + static_cast<int64_t>(kStep) * cl - 1) / (static_cast<int64_t>(kStep) * cl));
  int t[NP], x[NP], y[NP];
  uint32_t s[NP];
  auto positions = [&](int k) {
#pragma unroll
    for (int j = 0; j < NP; ++j) {
      const int64_t i = row_at(k, j * kThreads + threadIdx.x);
      t[j] = i < n ? keep[i] : -1;
    }
  };
  auto pages = [&](int k) {
#pragma unroll
    for (int j = 0; j < NP; ++j) {
      const int64_t i = row_at(k, j * kThreads + threadIdx.x), to = first + i;
      x[j] = y[j] = 0;
      if (i >= n) continue;
      if (t[j] < to || t[j] >= room) {
        report(p.err, kSiteBadLength);
        t[j] = -1;
      } else if (t[j] == to) {
        t[j] = -1;
      } else {
        x[j] = table[t[j] >> shift];
        y[j] = table[to >> shift];
      }
    }
  };
  auto places = [&](int k) {
#pragma unroll
    for (int j = 0; j < NP; ++j) {
      const int i = j * kThreads + threadIdx.x;
      uint2 e = make_uint2(kNowhere, 0);
      if (t[j] >= 0) {
        if (x[j] < 0 || x[j] >= p.num_blocks || y[j] < 0 || y[j] >= p.num_blocks)
          report(p.err, kSiteBadBlock);
        else
          e = make_uint2((static_cast<unsigned int>(x[j]) << shift) + (t[j] & mask),
                         (static_cast<unsigned int>(y[j]) << shift) + static_cast<unsigned int>((first + row_at(k, i)) & mask));
      }
      plans[(k & 1) * P::kPlan + i] = e;
      if (scales && e.x != kNowhere) {
        const int64_t from = row(e.x);
        if constexpr (SB == 1) s[j] = scale[from];
        if constexpr (SB == 2) s[j] = reinterpret_cast<const uint16_t*>(scale)[from];
        if constexpr (SB == 4) s[j] = reinterpret_cast<const uint32_t*>(scale)[from];
      }
    }
  };
  auto move_scales = [&](int k) {
#pragma unroll
    for (int j = 0; SB > 0 && j < NP; ++j) {
      if (!scales) break;
      const uint2 e = plans[(k & 1) * P::kPlan + j * kThreads + threadIdx.x];
      if (e.x == kNowhere) continue;
      const int64_t to = row(e.y);
      if constexpr (SB == 1) scale[to] = static_cast<uint8_t>(s[j]);
      if constexpr (SB == 2) reinterpret_cast<uint16_t*>(scale)[to] = static_cast<uint16_t>(s[j]);
      if constexpr (SB == 4) reinterpret_cast<uint32_t*>(scale)[to] = s[j];
    }
  };
  auto place = [&](int step, int u) {
    return plans[(step / P::kSteps & 1) * P::kPlan + step % P::kSteps * kStep + u * kRows + r];
  };
  auto load = [&](int slot, int step) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const unsigned int from = step < steps ? place(step, u).x : kNowhere;
      if (from != kNowhere) cp_async16(&ring[(slot * U + u) * kThreads + threadIdx.x], cache + row(from) * RB);
    }
    cp_async_commit();
  };
  positions(0);
  pages(0);
  places(0);
  barrier();  // the plan's places are there, and its scales have been read
  move_scales(0);
#pragma unroll
  for (int k = 0; k < kDeep - 1; ++k) load(k, k);
  int slot = 0;
#pragma unroll 1
  for (int step = 0; step < steps; ++step) {
    load(slot == 0 ? kDeep - 1 : slot - 1, step + kDeep - 1);
    cp_async_wait<kDeep - 1>();
    barrier();  // all of the chunk that is stored now has been read
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const uint2 e = place(step, u);
      if (e.x != kNowhere) *reinterpret_cast<uint4*>(cache + row(e.y) * RB) = ring[(slot * U + u) * kThreads + threadIdx.x];
    }
    slot = slot == kDeep - 1 ? 0 : slot + 1;
    // The next plan: its places are written where the plan before lay, two chunks before the first one looks there.
    const int next = step / P::kSteps + 1;
    if (next * P::kSteps < steps) {
      const int phase = step % P::kSteps;
      if (phase == 0) positions(next);
      if (phase == 1) pages(next);
      if (phase == 2) places(next);
      if (phase == 3) move_scales(next);  // (a barrier after they have been read)
    }
  }
}

// Whole pages: block (piece, pair of pages), 16 bytes a thread and pass, keys then values.
constexpr int kCopyPass = 4;
__global__ void __launch_bounds__(kThreads) cache_copy_kernel(const __grid_constant__ MoveParams p, int64_t page_bytes,
                                                              int scale_bytes) {
  const int src = p.src[blockIdx.y], dst = p.dst[blockIdx.y];
  if (src == -1 && dst == -1) return;
  if (src < 0 || src >= p.num_blocks || dst < 0 || dst >= p.num_blocks) {
    if (threadIdx.x == 0) report(p.err, kSiteBadBlock);
    return;
  }
  if (src == dst) return;
  const int64_t words = page_bytes / 16;
  uint4 x[2][kCopyPass];
  const int64_t w0 = static_cast<int64_t>(blockIdx.x) * kThreads * kCopyPass + threadIdx.x;
#pragma unroll
  for (int j = 0; j < 2; ++j)
#pragma unroll
    for (int u = 0; u < kCopyPass; ++u)
      if (w0 + u * kThreads < words)
        x[j][u] = reinterpret_cast<const uint4*>(p.cache[j] + src * page_bytes)[w0 + u * kThreads];
#pragma unroll
  for (int j = 0; j < 2; ++j)
#pragma unroll
    for (int u = 0; u < kCopyPass; ++u)
      if (w0 + u * kThreads < words) reinterpret_cast<uint4*>(p.cache[j] + dst * page_bytes)[w0 + u * kThreads] = x[j][u];
  if (scale_bytes > 0) {  // a multiple of 16: block_size is
    const int64_t at = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x;
    const int64_t step = static_cast<int64_t>(gridDim.x) * kThreads;
    for (int64_t w = at; w < scale_bytes / 16; w += step)
#pragma unroll
      for (int j = 0; j < 2; ++j)
        reinterpret_cast<uint4*>(p.scale[j] + static_cast<int64_t>(dst) * scale_bytes)[w] =
            reinterpret_cast<const uint4*>(p.scale[j] + static_cast<int64_t>(src) * scale_bytes)[w];
  }
}

// ------------------------------------------------------------------ shared and freed

// Is x among list[0 … n)?  By all threads of the block, which get the answer.
__device__ __forceinline__ bool among(const int* list, int n, int x) {
  bool found = false;
  for (int j = threadIdx.x; j < n; j += kThreads) found |= list[j] == x;
  return __syncthreads_or(found);
}

// A block per pair (src, dst): dst, which holds nothing, takes src's pages.
__global__ void __launch_bounds__(kThreads) pages_fork_kernel(const __grid_constant__ PageParams p) {
  const int src = p.src[blockIdx.x], dst = p.dst[blockIdx.x];
  const int shift = 31 - __clz(p.block_size);  // a power of two
  bool fine = src >= 0 && src < p.B && dst >= 0 && dst < p.B;
  // A sequence that two pairs fill, or that is filled and read, would depend on the order: the first pair to fill it
  // counts, and no pair reads one that is filled.
  fine = !among(p.dst, blockIdx.x, dst) && fine;
  fine = !among(p.dst, p.n, src) && fine;
  if (!fine) {
    if (threadIdx.x == 0) report(p.err, kSiteBadSequence);
    return;
  }
  const int len = p.seq_lens[src];
  const int* from = p.block_table + static_cast<int64_t>(src) * p.max_blocks;
  int* to = p.block_table + static_cast<int64_t>(dst) * p.max_blocks;
  bool holds = p.seq_lens[dst] != 0;
  for (int j = threadIdx.x; j < p.max_blocks; j += kThreads) holds |= to[j] >= 0;
  holds = __syncthreads_or(holds);
  const bool fits = len >= 0 && len <= static_cast<int64_t>(p.max_blocks) << shift;
  if (holds || !fits) {
    if (threadIdx.x == 0) report(p.err, holds ? kSiteBadSequence : kSiteBadLength);
    return;
  }
  const int used = (len + p.block_size - 1) >> shift;
  for (int j = threadIdx.x; j < used; j += kThreads) {
    const int page = from[j];
    if (page >= 0 && page < p.num_blocks)
      atomicAdd(p.holders + page, 1);
    else
      report(p.err, kSiteBadBlock);
    to[j] = page;
  }
  for (int j = used + threadIdx.x; j < p.max_blocks; j += kThreads) to[j] = -1;
  if (threadIdx.x == 0) p.seq_lens[dst] = len;
}

// A block per sequence: its pages behind the first lens[i] tokens (all, without lens) lose a holder.
__global__ void __launch_bounds__(kThreads) pages_free_kernel(const __grid_constant__ PageParams p) {
  const int b = p.src[blockIdx.x];
  const int keep = p.lens != nullptr ? p.lens[blockIdx.x] : 0;
  const int shift = 31 - __clz(p.block_size);  // a power of two
  const bool twice = among(p.src, blockIdx.x, b);  // the first entry of a sequence counts
  if (b < 0 || b >= p.B || twice || keep < 0) {
    if (threadIdx.x == 0) report(p.err, keep < 0 ? kSiteBadLength : kSiteBadSequence);
    return;
  }
  int len = p.seq_lens[b];
  const int64_t room = static_cast<int64_t>(p.max_blocks) << shift;
  if (len < 0 || len > room) {
    if (threadIdx.x == 0) report(p.err, kSiteBadLength);
    len = len < 0 ? 0 : static_cast<int>(room);
  }
  __syncthreads();  // all have read the length
  len = min(len, keep);
  int* table = p.block_table + static_cast<int64_t>(b) * p.max_blocks;
  for (int j = static_cast<int>((static_cast<int64_t>(len) + p.block_size - 1) >> shift) + threadIdx.x; j < p.max_blocks;
       j += kThreads) {
    const int page = table[j];
    if (page == -1) continue;
    table[j] = -1;
    if (page < 0 || page >= p.num_blocks) {
      report(p.err, kSiteBadBlock);
    } else if (atomicSub(p.holders + page, 1) <= 0) {
      atomicAdd(p.holders + page, 1);  // nobody was said to hold it
      report(p.err, kSiteBadHolders);
    }
  }
  if (threadIdx.x == 0) p.seq_lens[b] = len;
}

// ------------------------------------------------------------------------ reserved

// Exclusive prefix sum over the block's threads, and the sum of all.
template <int NT>
__device__ __forceinline__ int block_prefix(int mine, int* warp_sum, int& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int incl = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int x = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += x;
  }
  __syncthreads();  // of the call before
  if (lane == 31) warp_sum[warp] = incl;
  __syncthreads();
  int before = 0;
  total = 0;
#pragma unroll
  for (int w = 0; w < NT / 32; ++w) {
    const int x = warp_sum[w];
    before += w < warp ? x : 0;
    total += x;
  }
  return before + incl - mine;
}

// The free ones among four neighbouring pages, a bit each.
__device__ __forceinline__ uint32_t free_pages(const PageParams& p, int page0) {
  uint32_t bits = 0;
  if (page0 + 4 <= p.num_blocks && (reinterpret_cast<uintptr_t>(p.holders) & 15u) == 0) {
    const int4 x = *reinterpret_cast<const int4*>(p.holders + page0);
    bits = (x.x == 0 ? 1u : 0u) | (x.y == 0 ? 2u : 0u) | (x.z == 0 ? 4u : 0u) | (x.w == 0 ? 8u : 0u);
  } else {
    for (int q = 0; q < 4 && page0 + q < p.num_blocks; ++q) bits |= p.holders[page0 + q] == 0 ? 1u << q : 0u;
  }
  return bits;
}

// Free pages of a segment, or what each of eight sequences misses.
static_assert(kPageSegment == kThreads * 4, "4 pages a thread");
__global__ void __launch_bounds__(kThreads) pages_count_kernel(const __grid_constant__ PageParams p, int segments) {
  __shared__ int warp_sum[kThreads / 32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (static_cast<int>(blockIdx.x) < segments) {
    int total;
    block_prefix<kThreads>(__popc(free_pages(p, blockIdx.x * kPageSegment + threadIdx.x * 4)), warp_sum, total);
    if (threadIdx.x == 0) p.seg[blockIdx.x] = total;
    return;
  }
  const int b = (blockIdx.x - segments) * (kThreads / 32) + warp;
  if (b >= p.B) return;
  const int shift = 31 - __clz(p.block_size);  // a power of two
  const int len = p.seq_lens[b], more = p.lens[b];
  const int64_t room = static_cast<int64_t>(p.max_blocks) << shift;
  const bool fine = len >= 0 && more >= 0 && static_cast<int64_t>(len) + more <= room;
  int last = -1, from = 0, want = fine ? 0 : -1;  // −1: cannot be served
  if (!fine) {
    if (lane == 0) report(p.err, kSiteBadLength);
  } else if (more > 0) {
    const int* table = p.block_table + static_cast<int64_t>(b) * p.max_blocks;
    const int lo = len >> shift;  // the next token's entry
    const int have = static_cast<int>((static_cast<int64_t>(len) + p.block_size - 1) >> shift);
    const int need = static_cast<int>((static_cast<int64_t>(len) + more + p.block_size - 1) >> shift);
    // Mostly pages reserved before come first, and behind them the table is empty.
    bool bad = false, unheld = false, in_turn = false;
    from = need;
    auto look = [&](int j, int page) {
      const int held = page >= 0 && page < p.num_blocks ? p.holders[page] : 1;
      bad |= page >= p.num_blocks || (j < have && page < 0);
      unheld |= held < 1;
      const uint32_t missing = __ballot_sync(0xffffffffu, j < need && page < 0);
      if (missing != 0 && from == need) from = j - lane + __ffs(missing) - 1;
      in_turn |= (j >= have && held > 1) || (page >= 0 && j > from);
    };
    const int first = lo + lane < need ? table[lo + lane] : -1;
    if (lo < have) last = __shfl_sync(0xffffffffu, first, 0);
    look(lo + lane, first);
    // (Every 32 looked at by themselves, 18 us instead of 15 for 8 x 2048 entries.)
    constexpr int U = 16;
#pragma unroll 1
    for (int j0 = lo + 32; j0 < need; j0 += 32 * U) {
      int page[U], all = -1;
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int j = j0 + u * 32 + lane;
        page[u] = j < need ? table[j] : -1;
      }
#pragma unroll
      for (int u = 0; u < U; ++u) all &= page[u];
      if (__all_sync(0xffffffffu, all < 0)) {
        from = min(from, j0);
      } else {
#pragma unroll
        for (int u = 0; u < U; ++u) look(j0 + u * 32 + lane, page[u]);
      }
    }
    bad = __any_sync(0xffffffffu, bad);
    unheld = __any_sync(0xffffffffu, unheld);
    want = need - from;
    if (bad || unheld) {
      if (lane == 0) report(p.err, bad ? kSiteBadBlock : kSiteBadHolders);
      last = want = -1;
    } else if (__any_sync(0xffffffffu, in_turn)) {
      from = ~have;  // its turn will tell how many pages it needs, and where
    }
  }
  if (lane == 0) {
    p.last[b] = last;
    p.from[b] = from;
    p.want[b] = want;
  }
}

// One sequence after the other, by all threads of the scanning block: where tables name pages behind their sequences' tokens that
// others hold too, how many a sequence needs depends on what those before it have given up; and where entries are missing
// between others, which those are has to be told to the hand-out.  Entries that are to get a page
// become −2 − (their place among the sequence's), by which the hand-out finds them.  Some 2.7 us a sequence, all of it
// latency: a state that a call leaves behind it for good.
constexpr int kScanThreads = 1024;
static __device__ __noinline__ void reserve_in_turn(const PageParams& p, int frees, int* warp_sum) {
  const int tid = threadIdx.x;
  const int shift = 31 - __clz(p.block_size);  // a power of two
  int at = 0;         // pages given so far
  bool cut = false;   // there were too few for somebody
#pragma unroll 1
  for (int b = 0; b < p.B; ++b) {
    const int want = p.want[b], more = p.lens[b], last = p.last[b], from = p.from[b];
    int* const table = p.block_table + static_cast<int64_t>(b) * p.max_blocks;
    const int need =
        from < 0 ? static_cast<int>((static_cast<int64_t>(p.seq_lens[b]) + more + p.block_size - 1) >> shift) : 0;
    bool served = want >= 0 && (more == 0 || !cut);
    int copy = -1, mine = 0;
    if (served && more > 0) {
      if (last >= 0 && p.holders[last] > 1) copy = last;
      mine = want;
      if (from < 0) {
        int needs = 0;
        for (int j = ~from + tid; j < need; j += kScanThreads) needs += table[j] < 0 || p.holders[table[j]] > 1 ? 1 : 0;
        block_prefix<kScanThreads>(needs, warp_sum, mine);
      }
      mine += copy >= 0 ? 1 : 0;
      served = mine <= frees - at;
      cut = !served;
    }
    __syncthreads();  // all have read what changes now
    if (tid == 0) {
      p.granted[b] = served ? 1 : 0;
      p.copy_src[b] = served ? copy : -1;
      p.copy_dst[b] = -1;
      p.want[b] = at;
      if (served && copy >= 0) atomicSub(p.holders + copy, 1);
    }
    if (served) {
      int before = 0;
#pragma unroll 1
      for (int j0 = ~from; from < 0 && j0 < need; j0 += kScanThreads) {
        const int j = j0 + tid;
        const int page = j < need ? table[j] : -1;
        const bool needs = j < need && (page < 0 || p.holders[page] > 1);
        int total;
        const int place = before + block_prefix<kScanThreads>(needs ? 1 : 0, warp_sum, total);
        if (needs) {
          if (page >= 0) atomicSub(p.holders + page, 1);
          table[j] = -2 - place;
        }
        before += total;
      }
      at += mine;
    }
    __syncthreads();
  }
  if (tid == 0) *p.total = at;
  // A page that is copied loses this holder where the copy is handed out.
  for (int b = tid; b < p.B; b += kScanThreads)
    if (p.copy_src[b] >= 0) atomicAdd(p.holders + p.copy_src[b], 1);
}

// Prefix sums over segments and sequences, and who is served.  512 sequences that all write into shared pages: 13 us, most of
// it every thread's count over all sequences' last pages (19 us with one page a load and a search that ends early).
constexpr int kMaxSequences = 4096;
__global__ void __launch_bounds__(kScanThreads) pages_scan_kernel(const __grid_constant__ PageParams p, int segments) {
  __shared__ __align__(16) int last_of[kMaxSequences];
  __shared__ int warp_sum[kScanThreads / 32];
  __shared__ int first_short;
  const int tid = threadIdx.x;
  const int quads = (p.B + 3) / 4;
  bool in_turn = false;
  for (int b = tid; b < 4 * quads; b += kScanThreads) {
    last_of[b] = b < p.B ? p.last[b] : -1;
    in_turn |= b < p.B && p.from[b] < 0;
  }
  if (tid == 0) first_short = p.B;
  int frees = 0;
  for (int s0 = 0; s0 < segments; s0 += kScanThreads) {
    const int s = s0 + tid;
    int total;
    const int before = frees + block_prefix<kScanThreads>(s < segments ? p.seg[s] : 0, warp_sum, total);
    if (s < segments) p.seg[s] = before;
    frees += total;
  }
  if (__syncthreads_or(in_turn)) {
    reserve_in_turn(p, frees, warp_sum);
    return;
  }
  int given = 0;
  for (int b0 = 0; b0 < p.B; b0 += kScanThreads) {
    const int b = b0 + tid;
    bool copies = false;
    int want = 0;
    if (b < p.B) {
      want = p.want[b];
      const int page = last_of[b];
      const int held = page >= 0 ? p.holders[page] : 0;
      if (held > 1) {
        // Does a later one write there?  Else, how many do before?
        int before = 0;
        bool later = false;
        const int4* last4 = reinterpret_cast<const int4*>(last_of);
#pragma unroll 4
        for (int q = 0; q < b / 4; ++q) {
          const int4 x = last4[q];
          before += (x.x == page) + (x.y == page) + (x.z == page) + (x.w == page);
        }
        for (int j = b / 4 * 4; j < b; ++j) before += last_of[j] == page;
        for (int j = b + 1; j < (b / 4 + 1) * 4; ++j) later = later || last_of[j] == page;
#pragma unroll 4
        for (int q = b / 4 + 1; q < quads; ++q) {
          const int4 x = last4[q];
          later = later || x.x == page || x.y == page || x.z == page || x.w == page;
        }
        copies = later || held - before > 1;
      }
    }
    const int mine = max(want, 0) + (copies ? 1 : 0);
    int total;
    const int at = given + block_prefix<kScanThreads>(mine, warp_sum, total);
    // From the first one that finds too few pages on, nobody with tokens to come is served: a later one may count on
    // the copy that an earlier one did not get.  (Sums stay below 2^31: the host bounds B · max_blocks.)
    if (mine > 0 && at + mine > frees) atomicMin(&first_short, b);
    __syncthreads();
    if (b < p.B) {
      const bool served = want >= 0 && (b < first_short || p.lens[b] == 0);
      p.granted[b] = served ? 1 : 0;
      p.copy_src[b] = served && copies ? last_of[b] : -1;
      p.copy_dst[b] = -1;
      p.want[b] = at;
      if (b == first_short) *p.total = at;
    }
    given += total;
    __syncthreads();
  }
  if (tid == 0 && first_short == p.B) *p.total = given;
}

// A block per segment: its free pages, as long as pages are handed out, go to their sequences.  The free ones are listed
// first, so that every thread has at most four searches, with their loads on the way together: 7 us for 2000 pages, against
// 18 with segments of 4096 pages and 16 neighbouring pages a thread.
__global__ void __launch_bounds__(kThreads) pages_hand_out_kernel(const __grid_constant__ PageParams p) {
  __shared__ int warp_sum[kThreads / 32];
  __shared__ uint16_t list[kPageSegment];
  __shared__ int begin_of[kMaxSequences];
  const int total = *p.total, before = p.seg[blockIdx.x];
  if (before >= total) return;
  for (int b = threadIdx.x; b < p.B; b += kThreads) begin_of[b] = p.want[b];
  uint32_t bits = free_pages(p, blockIdx.x * kPageSegment + threadIdx.x * 4);
  int sum;
  int place = block_prefix<kThreads>(__popc(bits), warp_sum, sum);
  for (; bits != 0; bits &= bits - 1) list[place++] = static_cast<uint16_t>(threadIdx.x * 4 + __ffs(bits) - 1);
  __syncthreads();
  const int shift = 31 - __clz(p.block_size);  // a power of two
  const int n = min(sum, total - before);
  constexpr int U = kPageSegment / kThreads;
  int seq[U], shared[U], from[U], len[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int at = u * kThreads + threadIdx.x;
    if (at >= n) continue;
    int lo = 0, hi = p.B;  // the last sequence that begins at or before this page's place
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (begin_of[mid] <= before + at)
        lo = mid;
      else
        hi = mid;
    }
    seq[u] = lo;
    shared[u] = p.copy_src[lo];
    from[u] = p.from[lo];
    len[u] = p.seq_lens[lo];
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int at = u * kThreads + threadIdx.x;
    if (at >= n) continue;
    const int page = blockIdx.x * kPageSegment + list[at];
    const int i = before + at - begin_of[seq[u]] - (shared[u] >= 0 ? 1 : 0);
    int* table = p.block_table + static_cast<int64_t>(seq[u]) * p.max_blocks;
    p.holders[page] = 1;
    if (i < 0) {
      table[len[u] >> shift] = page;
      p.copy_dst[seq[u]] = page;
      atomicSub(p.holders + shared[u], 1);
    } else if (from[u] >= 0) {
      table[from[u] + i] = page;
    } else {  // (others of the sequence's entries are filled meanwhile, with pages: no other becomes what is looked for)
      const volatile int* entry = table;
      int j = ~from[u] + i;
      while (j < p.max_blocks && entry[j] != -2 - i) ++j;
      if (j < p.max_blocks) table[j] = page;
    }
  }
}

template <int RB, int SB>
cudaError_t launch_compact(const MoveParams& p, cudaStream_t s) {
  // Columns of 64 bytes (32-byte rows: 32): four lanes hold a row's part (one lane, 16 bytes: 120 us instead of 50 for the E4M3
  // rows above, 173 instead of 75 for bf16).  Blocks that do not fill the SMs are clusters that share the rows: one sequence of
  // 32768 tokens, 2 heads, 12000 rows kept, E4M3, 8 blocks: 22 us, 67 without clusters; the E2M1 rows above, 128 blocks: 36 and
  // 48.  A cluster's barrier costs more than a block's, so where the SMs have a block each there are none: the 256 blocks of the
  // E4M3 rows take 54 us in pairs and 50 alone.
  constexpr int kLanes = RB >= 64 ? 4 : RB / 16;
  constexpr int kRows = kThreads / kLanes;
  const int64_t blocks = static_cast<int64_t>(p.B) * p.Hkv * 2 * (RB / (16 * kLanes));
  int cl = 1;
  if (blocks < 152) {
    while (cl < 8 && blocks * cl < 304 && cl * 2 * kRows < p.N) cl *= 2;
  }
  if (blocks * cl > 0x7fffffff) return cudaErrorInvalidValue;
  cudaLaunchAttribute attr = {};
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = cl;
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(blocks * cl));
  cfg.blockDim = dim3(kThreads);
  cfg.stream = s;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  // Chunks of four passes where clusters wait for one another at each (two: 26 and 40 us instead of 22 and 36, the one sequence
  // and the E2M1 rows above), of two otherwise (four: the E4M3 rows above 48 us instead of 50, but twice as many 91 instead of 75,
  // and those in bf16 81 instead of 75).
  auto launch = [&](auto* kernel, int smem) {
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    cfg.dynamicSmemBytes = smem;
    return cudaLaunchKernelEx(&cfg, kernel, p);
  };
  return cl > 1 ? launch(cache_compact_kernel<RB, SB, kLanes, 4>, Plan<kLanes, 4>::kSmem)
                : launch(cache_compact_kernel<RB, SB, kLanes, 2>, Plan<kLanes, 2>::kSmem);
}

}  // namespace

cudaError_t launch_cache_compact(const MoveParams& p, int d, int format, cudaStream_t s) {
  if (d == 128) {
    if (format == kCacheBf16) return launch_compact<256, 0>(p, s);
    if (format == kCacheE4m3) return launch_compact<128, 1>(p, s);
    if (format == kCacheE2m1) return launch_compact<64, 4>(p, s);
  } else if (d == 64) {
    if (format == kCacheBf16) return launch_compact<128, 0>(p, s);
    if (format == kCacheE4m3) return launch_compact<64, 1>(p, s);
    if (format == kCacheE2m1) return launch_compact<32, 2>(p, s);
  }
  return cudaErrorInvalidValue;
}

cudaError_t launch_cache_copy(const MoveParams& p, int d, int format, int n, cudaStream_t s) {
  const int64_t rows = static_cast<int64_t>(p.Hkv) * p.block_size;
  const int64_t page = rows * cache_row_bytes(d, format);
  const int64_t pieces = (page / 16 + kThreads * kCopyPass - 1) / (kThreads * kCopyPass);
  if (pieces > 0x7fffffff || n > 65535) return cudaErrorInvalidValue;
  cache_copy_kernel<<<dim3(static_cast<unsigned>(pieces), n), kThreads, 0, s>>>(
      p, page, static_cast<int>(rows * cache_row_scales(d, format)));
  return cudaGetLastError();
}

cudaError_t launch_pages_fork(const PageParams& p, cudaStream_t s) {
  pages_fork_kernel<<<p.n, kThreads, 0, s>>>(p);
  return cudaGetLastError();
}

cudaError_t launch_pages_free(const PageParams& p, cudaStream_t s) {
  pages_free_kernel<<<p.n, kThreads, 0, s>>>(p);
  return cudaGetLastError();
}

cudaError_t launch_pages_reserve(const PageParams& p, cudaStream_t s) {
  const int segments = static_cast<int>((static_cast<int64_t>(p.num_blocks) + kPageSegment - 1) / kPageSegment);
  const int counts = segments + (p.B + kThreads / 32 - 1) / (kThreads / 32);
  if (p.B > kMaxSequences) return cudaErrorInvalidValue;
  pages_count_kernel<<<counts, kThreads, 0, s>>>(p, segments);
  pages_scan_kernel<<<1, kScanThreads, 0, s>>>(p, segments);
  pages_hand_out_kernel<<<segments, kThreads, 0, s>>>(p);
  return cudaGetLastError();
}

}  // namespace fa

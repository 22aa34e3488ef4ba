// fa_cache.cu — writing keys and values into the paged cache and reading them
// back as contiguous rows.
//
// Formats.  bf16: rows are copied.  E4M3: a row x of one head is held as codes
// c_i = rn(x_i·2⁻ᵏ) and one byte k + 127, where k is the smallest whole number
// with max|x_i| ≤ 448·2ᵏ (448 is E4M3's largest value), but at least −126.
// The power of two makes x·2⁻ᵏ and c·2ᵏ exact, so the rounding to E4M3 (at most
// half a step, 2⁻⁴ relative) is the only one, and reading back into bf16 adds
// none.  A finer scale would not make it smaller: it would only shift the
// values within their binades.  Infinities and NaN do not count for the
// maximum and become the NaN code.
//
// Bound: device memory.  Writing: 2·(2d) bytes read and 2·(d + 1) written per
// token and head (bf16: 2·2d); d/8 lanes hold one row, 16 bytes of it each, and
// the row maximum is log2(d/8) lane exchanges, so a row never leaves registers.
//
// Measured on GB300 (d = 128): gathering 4 sequences of 32768 E4M3 keys, 8 heads: 124 us,
// 6.5 TB/s, 0.97 of a device copy; writing 8 ragged sequences of up to 8192 tokens as
// E4M3, 4 heads: 31 us, 5.1 TB/s, 0.77 (it quantises on the way); a token for each of 64
// sequences: the launch (11 us a call from Python).
#include <cuda_fp16.h>

#include <type_traits>

#include "fa_kernels.h"
#include "sm103.cuh"

namespace fa {
namespace {

constexpr int kThreads = 128;

__device__ __forceinline__ void report(unsigned int* err, unsigned int what) {
  atomicCAS(err + 1, 0u, (kKernCache << 8) | what);
}

// The page of logical key t, or −1 (and a report) if the table's entry is no page.
__device__ __forceinline__ int page_of(const CacheParams& p, int b, int t) {
  const int shift = 31 - __clz(p.block_size);  // a power of two
  const int blk = p.block_table[static_cast<int64_t>(b) * p.max_blocks + (t >> shift)];
  if (blk >= 0 && blk < p.num_blocks) return blk;
  report(p.err, kSiteBadBlock);
  return -1;
}

// The larger one of each of two 16-bit halves.
__device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b) { return __vmaxu2(a, b); }

// Quantises 8 elements of a key's row and 8 of its value's; the lanes of the rows (8 or 16 neighbours) hold the rest.
// Magnitudes order like their bits, so a maximum is taken over 16-bit halves, and both rows' go through the lane
// exchanges in one word.
template <int D>
__device__ __forceinline__ void quantise8(uint4 k, uint4 v, uint2& kc, uint2& vc, int& ke, int& ve) {
  uint32_t w[2][4] = {{k.x, k.y, k.z, k.w}, {v.x, v.y, v.z, v.w}};
  auto row_max = [](const uint32_t(&x)[2][4]) -> uint32_t {  // the key row's in the lower half
    uint32_t t[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) t[j] = max2(max2(x[j][0], x[j][1]), max2(x[j][2], x[j][3]));
    uint32_t top = __byte_perm(max2(t[0], t[0] >> 16), max2(t[1], t[1] << 16), 0x7610);
#pragma unroll
    for (int m = D / 16; m > 0; m >>= 1) top = max2(top, __shfl_xor_sync(0xffffffffu, top, m));
    return top;
  };
  uint32_t mag[2][4];
#pragma unroll
  for (int j = 0; j < 2; ++j)
#pragma unroll
    for (int i = 0; i < 4; ++i) mag[j][i] = w[j][i] & 0x7fff7fffu;
  uint32_t top = row_max(mag);
  if (__any_sync(0xffffffffu, (top & 0xffffu) >= 0x7f80u || top >= 0x7f800000u)) {
    // Infinities and NaN somewhere in the warp's rows: they do not count for the maximum and become NaN.
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if ((w[j][i] & 0x7f80u) == 0x7f80u) w[j][i] |= 0x7fffu, mag[j][i] &= 0xffff0000u;
        if ((w[j][i] & 0x7f800000u) == 0x7f800000u) w[j][i] |= 0x7fff0000u, mag[j][i] &= 0xffffu;
      }
    top = row_max(mag);
  }
  // A maximum is 1.f·2^(e−127) with 7 bits of f; 448 = 1.75·2^8, so k = e − 127 − 8, one more when 1.f exceeds 1.75.
  auto exponent = [](uint32_t t) { return max(-126, static_cast<int>(t >> 7) - 135 + ((t & 0x7fu) > 0x60u ? 1 : 0)); };
  ke = exponent(top & 0xffffu);
  ve = exponent(top >> 16);
  uint32_t c[2][4];
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const float inv = __uint_as_float(static_cast<uint32_t>(127 - (j == 0 ? ke : ve)) << 23);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float lo, hi;
      fmul2(lo, hi, __uint_as_float(w[j][i] << 16), __uint_as_float(w[j][i] & 0xffff0000u), inv, inv);
      c[j][i] = pack_e4m3x2(lo, hi);
    }
  }
  kc = make_uint2(c[0][0] | (c[0][1] << 16), c[0][2] | (c[0][3] << 16));
  vc = make_uint2(c[1][0] | (c[1][1] << 16), c[1][2] | (c[1][3] << 16));
}

// Item (b, group of R tokens, h), h fastest: 8 or 16 lanes for the R rows.
template <int D, int R>
struct Item {
  static constexpr int kLanes = D / 8;
  int b, n0, h, lane8;
  bool in;
  __device__ __forceinline__ explicit Item(const CacheParams& p) {
    const int64_t id = (static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x) / kLanes;
    lane8 = threadIdx.x % kLanes;
    const int groups = (p.N + R - 1) / R;
    const int64_t tok = id / p.Hkv;
    h = static_cast<int>(id - tok * p.Hkv);
    b = static_cast<int>(tok / groups);
    n0 = static_cast<int>(tok - static_cast<int64_t>(b) * groups) * R;
    in = b < p.B;
  }
};

template <int D, bool FP8, int R>
__global__ void __launch_bounds__(kThreads) cache_append_kernel(const __grid_constant__ CacheParams p) {
  const Item<D, R> it(p);
  const int shift = 31 - __clz(p.block_size);  // a power of two
  int len = 0;
  int64_t start = 0;
  if (it.in) {
    start = p.start[it.b];
    len = p.lens != nullptr ? p.lens[it.b] : p.N;
    if (len < 0 || len > p.N) {
      report(p.err, kSiteBadLength);
      len = 0;
    }
  }
  // The rows are on their way while their slots are looked up.
  uint4 kr[R], vr[R];
  const int count = min(R, len - it.n0);  // rows of this item that are written
  const __nv_bfloat16* kp = static_cast<const __nv_bfloat16*>(p.k_rows) + it.b * p.sk[0] + it.h * p.sk[1] +
                            it.n0 * p.sk[2] + it.lane8 * 8;
  const __nv_bfloat16* vp = static_cast<const __nv_bfloat16*>(p.v_rows) + it.b * p.sv[0] + it.h * p.sv[1] +
                            it.n0 * p.sv[2] + it.lane8 * 8;
#pragma unroll
  for (int r = 0; r < R; ++r) {
    kr[r] = vr[r] = make_uint4(0, 0, 0, 0);
    if (r < count) {
      kr[r] = *reinterpret_cast<const uint4*>(kp + r * p.sk[2]);
      vr[r] = *reinterpret_cast<const uint4*>(vp + r * p.sv[2]);
    }
  }
  // The usual item's tokens lie in one page: its rows follow one another.
  const int64_t t0 = start + it.n0;
  const int64_t room = static_cast<int64_t>(p.max_blocks) * p.block_size;
  const bool together = count == R && t0 >= 0 && t0 + R <= room && t0 >> shift == (t0 + R - 1) >> shift;
  int64_t row[R];
#pragma unroll
  for (int r = 0; r < R; ++r) row[r] = -1;
  if (together) {
    const int t = static_cast<int>(t0);
    const int blk = page_of(p, it.b, t);
    if (blk >= 0) row[0] = ((static_cast<int64_t>(blk) * p.Hkv + it.h) << shift) + (t & (p.block_size - 1));
  } else if (count > 0) {
    if (t0 < 0 || t0 + count > room) report(p.err, kSiteBadLength);
    int page = -1, blk = -1;  // the page of the token before and where it lies
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const int t = static_cast<int>(t0) + r;
      if (r < count && t0 + r >= 0 && t0 + r < room) {
        if (t >> shift != page) {
          page = t >> shift;
          blk = page_of(p, it.b, t);
        }
        if (blk >= 0) row[r] = ((static_cast<int64_t>(blk) * p.Hkv + it.h) << shift) + (t & (p.block_size - 1));
      }
    }
  }
  using Out = typename std::conditional<FP8, uint2, uint4>::type;  // 8 elements
  Out kc[R], vc[R];
  int ke[R], ve[R];
#pragma unroll
  for (int r = 0; r < R; ++r) {
    if constexpr (FP8) {
      quantise8<D>(kr[r], vr[r], kc[r], vc[r], ke[r], ve[r]);
    } else {
      kc[r] = kr[r];
      vc[r] = vr[r];
    }
  }
  auto scales = [&](int64_t at, int r) {
    if (FP8 && it.lane8 == 0) {
      p.k_scale[at] = static_cast<uint8_t>(ke[r] + 127);
      p.v_scale[at] = static_cast<uint8_t>(ve[r] + 127);
    }
  };
  Out* const k_out = static_cast<Out*>(p.k_cache) + it.lane8;
  Out* const v_out = static_cast<Out*>(p.v_cache) + it.lane8;
  if (together) {
    if (row[0] >= 0) {
      Out* kd = k_out + row[0] * (D / 8);
      Out* vd = v_out + row[0] * (D / 8);
#pragma unroll
      for (int r = 0; r < R; ++r) {
        kd[r * (D / 8)] = kc[r];
        vd[r * (D / 8)] = vc[r];
      }
      if (R == 4 && FP8 && (row[0] & 3) == 0) {  // four scale bytes at once
        if (it.lane8 == 0) {
          auto four = [](const int(&e)[R]) {
            return static_cast<uint32_t>((e[0] + 127) | (e[1 % R] + 127) << 8 | (e[2 % R] + 127) << 16) |
                   static_cast<uint32_t>(e[3 % R] + 127) << 24;
          };
          *reinterpret_cast<uint32_t*>(p.k_scale + row[0]) = four(ke);
          *reinterpret_cast<uint32_t*>(p.v_scale + row[0]) = four(ve);
        }
      } else {
#pragma unroll
        for (int r = 0; r < R; ++r) scales(row[0] + r, r);
      }
    }
  } else {
#pragma unroll
    for (int r = 0; r < R; ++r)
      if (row[r] >= 0) {
        k_out[row[r] * (D / 8)] = kc[r];
        v_out[row[r] * (D / 8)] = vc[r];
        scales(row[r], r);
      }
  }
}

// Eight codes times 2^(s−127) as bf16.
__device__ __forceinline__ uint4 dequantise8(uint2 c, uint32_t s) {
  const uint32_t w[2] = {c.x, c.y};
  uint32_t out[4];
  // 2^(s−127) is a normal number for s ≥ 1; s = 0 stands for 2^−127, half the smallest normal one.
  const float f = s == 0 ? 5.877471754111438e-39f : __uint_as_float(s << 23);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t h = e4m3x2_to_f16x2(w[i >> 1] >> (16 * (i & 1)));
    const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&h));
    out[i] = pack_bf16x2(v.x * f, v.y * f);
  }
  return make_uint4(out[0], out[1], out[2], out[3]);
}

template <int D, bool FP8, int R>
__global__ void __launch_bounds__(kThreads) cache_gather_kernel(const __grid_constant__ CacheParams p) {
  const Item<D, R> it(p);
  if (!it.in) return;
  int len = p.lens[it.b];
  if (len < 0 || len > static_cast<int64_t>(p.max_blocks) * p.block_size) {
    report(p.err, kSiteBadLength);
    len = 0;
  }
  using Raw = typename std::conditional<FP8, uint2, uint4>::type;  // 8 elements
  Raw kr[R], vr[R];
  uint32_t ks[R], vs[R];
  bool live[R];
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const int n = it.n0 + r;
    kr[r] = vr[r] = Raw{};
    ks[r] = vs[r] = 127;
    const int blk = n < len && n < p.N ? page_of(p, it.b, n) : -1;
    live[r] = blk >= 0;
    if (live[r]) {
      const int64_t row = (static_cast<int64_t>(blk) * p.Hkv + it.h) * p.block_size + (n & (p.block_size - 1));
      kr[r] = reinterpret_cast<const Raw*>(p.k_cache)[row * (D / 8) + it.lane8];
      vr[r] = reinterpret_cast<const Raw*>(p.v_cache)[row * (D / 8) + it.lane8];
      if constexpr (FP8) {
        ks[r] = p.k_scale[row];
        vs[r] = p.v_scale[row];
      }
    }
  }
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const int n = it.n0 + r;
    if (n >= p.N) break;
    uint4 k8, v8;
    if constexpr (FP8) {
      k8 = dequantise8(kr[r], ks[r]);
      v8 = dequantise8(vr[r], vs[r]);
    } else {
      k8 = kr[r];
      v8 = vr[r];
    }
    *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.k_rows) + it.b * p.sk[0] + it.h * p.sk[1] + n * p.sk[2] +
                              it.lane8 * 8) = k8;
    *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.v_rows) + it.b * p.sv[0] + it.h * p.sv[1] + n * p.sv[2] +
                              it.lane8 * 8) = v8;
  }
}

template <bool APPEND, int D, bool FP8, int R>
cudaError_t launch_r(const CacheParams& p, cudaStream_t stream) {
  const int64_t items = static_cast<int64_t>(p.B) * ((p.N + R - 1) / R) * p.Hkv;
  const int64_t blocks = (items * (D / 8) + kThreads - 1) / kThreads;
  if (blocks > 0x7fffffff) return cudaErrorInvalidValue;
  if (APPEND)
    cache_append_kernel<D, FP8, R><<<static_cast<unsigned>(blocks), kThreads, 0, stream>>>(p);
  else
    cache_gather_kernel<D, FP8, R><<<static_cast<unsigned>(blocks), kThreads, 0, stream>>>(p);
  return cudaGetLastError();
}

// Four tokens per thread once one per thread would fill the machine several times over: the look-up of their slots
// and the loads of their rows then overlap, where one per thread spends its life on that chain of loads; below, more
// threads with shorter chains are quicker.  One, two and four, replaying a graph, d = 128, us:
//   writing E4M3, 4 heads   8 x 512 tokens 4.8, 4.7, 5.1   8 x 2048 11.9, 10.6, 11.1   8 x 8192 39.0, 32.2, 31.6
//   reading E4M3            8 x 512 5.0, 4.9, 5.0   8 x 2048 12.2, 10.8, 10.8   4 x 32768, 8 heads 146, 122, 122
//   bf16                    8 x 8192, 4 heads, writing 41.2, 41.4, 41.3 and reading 43.5, 42.0, 42.2
// The rule turns to four between the second and the third size (4 x 152 x 2048 threads of one token).
template <bool APPEND, int D, bool FP8>
cudaError_t launch_d(const CacheParams& p, cudaStream_t stream) {
  const int64_t threads = static_cast<int64_t>(p.B) * p.N * p.Hkv * (D / 8);
  return p.N >= 4 && threads >= 4ll * 152 * 2048 ? launch_r<APPEND, D, FP8, 4>(p, stream)
                                                 : launch_r<APPEND, D, FP8, 1>(p, stream);
}

template <bool APPEND>
cudaError_t launch(const CacheParams& p, int d, bool fp8, cudaStream_t stream) {
  if (d == 128) return fp8 ? launch_d<APPEND, 128, true>(p, stream) : launch_d<APPEND, 128, false>(p, stream);
  if (d == 64) return fp8 ? launch_d<APPEND, 64, true>(p, stream) : launch_d<APPEND, 64, false>(p, stream);
  return cudaErrorInvalidValue;
}

}  // namespace

cudaError_t launch_cache_append(const CacheParams& p, int d, bool fp8, cudaStream_t s) {
  return launch<true>(p, d, fp8, s);
}
cudaError_t launch_cache_gather(const CacheParams& p, int d, bool fp8, cudaStream_t s) {
  return launch<false>(p, d, fp8, s);
}

}  // namespace fa

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
#include <cuda_fp16.h>

#include "fa_kernels.h"
#include "sm103.cuh"

namespace fa {
namespace {

constexpr int kThreads = 256;

__device__ __forceinline__ void report(unsigned int* err, unsigned int what) {
  atomicCAS(err + 1, 0u, (kKernCache << 8) | what);
}

// The page of logical key t, or −1 (and a report) if the table's entry is no page.
__device__ __forceinline__ int page_of(const CacheParams& p, int b, int t) {
  const int blk = p.block_table[static_cast<int64_t>(b) * p.max_blocks + t / p.block_size];
  if (blk >= 0 && blk < p.num_blocks) return blk;
  report(p.err, kSiteBadBlock);
  return -1;
}

// Writes 8 elements of a row; the lanes of the row (8 or 16 neighbours) hold the rest of it.
template <int D>
__device__ __forceinline__ void quantise_row(uint4 raw, uint8_t* codes, uint8_t* scale, int64_t row, int lane8,
                                             bool live) {
  const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
  float x[8];
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(w[i] << 16);
    x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t a = __float_as_uint(x[i]) & 0x7fffffffu;
    if (a < 0x7f800000u) top = max(top, a);  // magnitudes order like their bits
  }
#pragma unroll
  for (int m = D / 16; m > 0; m >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, m));
  // top = 1.f·2^(e−127); 448 = 1.75·2^8, so k = e − 127 − 8, one more when 1.f exceeds 1.75.
  const int k = max(-126, static_cast<int>(top >> 23) - 135 + ((top & 0x7fffffu) > 0x600000u ? 1 : 0));
  const float inv = __uint_as_float(static_cast<uint32_t>(127 - k) << 23);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const bool finite = (__float_as_uint(x[i]) & 0x7fffffffu) < 0x7f800000u;
    x[i] = finite ? x[i] * inv : __uint_as_float(0x7fffffffu);
  }
  if (!live) return;
  uint2 out;
  out.x = pack_e4m3x2(x[0], x[1]) | (pack_e4m3x2(x[2], x[3]) << 16);
  out.y = pack_e4m3x2(x[4], x[5]) | (pack_e4m3x2(x[6], x[7]) << 16);
  *reinterpret_cast<uint2*>(codes + row * D + lane8 * 8) = out;
  if (lane8 == 0) scale[row] = static_cast<uint8_t>(k + 127);
}

template <int D, bool FP8>
__global__ void __launch_bounds__(kThreads) cache_append_kernel(const __grid_constant__ CacheParams p) {
  constexpr int kLanes = D / 8;
  const int64_t id = (static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x) / kLanes;  // (b, n, h), h fastest
  const int lane8 = threadIdx.x % kLanes;
  const int64_t tok = id / p.Hkv;
  const int h = static_cast<int>(id - tok * p.Hkv);
  const int b = static_cast<int>(tok / p.N);
  const int n = static_cast<int>(tok - static_cast<int64_t>(b) * p.N);
  bool live = b < p.B;
  int64_t row = 0;
  if (live) {
    int len = p.N;
    if (p.lens != nullptr) {
      len = p.lens[b];
      if (len < 0 || len > p.N) {
        report(p.err, kSiteBadLength);
        len = 0;
      }
    }
    live = n < len;
    if (live) {
      const int64_t t = static_cast<int64_t>(p.start[b]) + n;
      if (t < 0 || t >= static_cast<int64_t>(p.max_blocks) * p.block_size) {
        report(p.err, kSiteBadLength);
        live = false;
      } else {
        const int blk = page_of(p, b, static_cast<int>(t));
        live = blk >= 0;
        row = (static_cast<int64_t>(blk) * p.Hkv + h) * p.block_size + t % p.block_size;
      }
    }
  }
  uint4 kr = make_uint4(0, 0, 0, 0), vr = kr;
  if (live) {
    kr = *reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p.k_rows) + b * p.sk[0] + h * p.sk[1] +
                                         n * p.sk[2] + lane8 * 8);
    vr = *reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p.v_rows) + b * p.sv[0] + h * p.sv[1] +
                                         n * p.sv[2] + lane8 * 8);
  }
  if (FP8) {
    quantise_row<D>(kr, static_cast<uint8_t*>(p.k_cache), p.k_scale, row, lane8, live);
    quantise_row<D>(vr, static_cast<uint8_t*>(p.v_cache), p.v_scale, row, lane8, live);
  } else if (live) {
    *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.k_cache) + row * D + lane8 * 8) = kr;
    *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.v_cache) + row * D + lane8 * 8) = vr;
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

template <int D, bool FP8>
__global__ void __launch_bounds__(kThreads) cache_gather_kernel(const __grid_constant__ CacheParams p) {
  constexpr int kLanes = D / 8;
  const int64_t id = (static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x) / kLanes;  // (b, h, n), n fastest
  const int lane8 = threadIdx.x % kLanes;
  const int64_t bh = id / p.N;
  const int n = static_cast<int>(id - bh * p.N);
  const int b = static_cast<int>(bh / p.Hkv);
  const int h = static_cast<int>(bh - static_cast<int64_t>(b) * p.Hkv);
  if (b >= p.B) return;
  int len = p.lens[b];
  if (len < 0 || len > static_cast<int64_t>(p.max_blocks) * p.block_size) {
    report(p.err, kSiteBadLength);
    len = 0;
  }
  uint4 kr = make_uint4(0, 0, 0, 0), vr = kr;
  const int blk = n < len ? page_of(p, b, n) : -1;
  if (blk >= 0) {
    const int64_t row = (static_cast<int64_t>(blk) * p.Hkv + h) * p.block_size + n % p.block_size;
    if (FP8) {
      const uint2 kc = *reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(p.k_cache) + row * D + lane8 * 8);
      const uint2 vc = *reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(p.v_cache) + row * D + lane8 * 8);
      kr = dequantise8(kc, p.k_scale[row]);
      vr = dequantise8(vc, p.v_scale[row]);
    } else {
      kr = *reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p.k_cache) + row * D + lane8 * 8);
      vr = *reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p.v_cache) + row * D + lane8 * 8);
    }
  }
  *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.k_rows) + b * p.sk[0] + h * p.sk[1] + n * p.sk[2] +
                            lane8 * 8) = kr;
  *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.v_rows) + b * p.sv[0] + h * p.sv[1] + n * p.sv[2] +
                            lane8 * 8) = vr;
}

template <bool APPEND, int D, bool FP8>
cudaError_t launch_d(const CacheParams& p, cudaStream_t stream) {
  const int64_t rows = static_cast<int64_t>(p.B) * p.N * p.Hkv;
  const int64_t blocks = (rows * (D / 8) + kThreads - 1) / kThreads;
  if (blocks > 0x7fffffff) return cudaErrorInvalidValue;
  if (APPEND)
    cache_append_kernel<D, FP8><<<static_cast<unsigned>(blocks), kThreads, 0, stream>>>(p);
  else
    cache_gather_kernel<D, FP8><<<static_cast<unsigned>(blocks), kThreads, 0, stream>>>(p);
  return cudaGetLastError();
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

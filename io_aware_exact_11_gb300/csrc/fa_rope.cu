// fa_rope.cu — rotary positions of q and k, and the gradient (the transposed
// rotation).
//
// Pair i of a head at position p turns by the angle θ = p·w_i:
//   y₁ = μ(x₁ cos θ − x₂ sin θ),  y₂ = μ(x₂ cos θ + x₁ sin θ),
// with pairs (i, i + r/2) or (2i, 2i + 1) of the first r elements.  The
// gradient turns back by −θ with the same μ.
//
// Angles.  θ/2π = p·(w_i/2π) is only needed modulo 1 and p is a whole number,
// so w_i/2π is held as a 64-bit fraction of a turn, rounded from 192 bits of 1/2π, and
// p times it is one 64-bit product that wraps exactly where whole turns drop out.  Far
// positions lose nothing: the error is at most p·2⁻⁶⁵ turns for the float64 w_i given, where
// a float32 product would be off by p·2⁻²⁴ radians.  Of the product the upper 32
// bits are kept (2⁻³² turns, 1.5e-9 rad) and rounded to float32, half turns in
// [−1, 1): 2⁻²⁵ of them, π·2⁻²⁵ rad at most.  sincospif adds its own 2 ulp.
//
// Bound: device memory, q and k read once and written once.  A thread owns one
// 16-byte column of one token and walks over heads with it, so that the sines
// are computed once for all of them and kept in registers; with few tokens
// there are few heads per thread (the launcher splits them until the grid fills
// the machine).
//
// Measured on GB300: the gradients of 16 + 16 heads of 128 elements at 2 x 8192 tokens, bf16: 49 us, 5.5 TB/s,
// 0.82 of a device copy; one token: the launch (17 us a call from Python).
#include "fa_kernels.h"
#include "sm103.cuh"

namespace fa {
namespace {

constexpr int kThreads = 128;
constexpr int kHeadsInFlight = 2;  // heads a thread loads before it turns them

template <typename T>
__device__ __forceinline__ float to_f32(T x);
template <>
__device__ __forceinline__ float to_f32<float>(float x) { return x; }
template <>
__device__ __forceinline__ float to_f32<__nv_bfloat16>(__nv_bfloat16 x) { return __bfloat162float(x); }
template <typename T>
__device__ __forceinline__ T from_f32(float x);
template <>
__device__ __forceinline__ float from_f32<float>(float x) { return x; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float x) { return __float2bfloat16_rn(x); }

// V elements moved as one access where V·sizeof(T) is 16 bytes.
template <typename T, int V>
struct alignas(sizeof(T) * V == 16 ? 16 : alignof(T)) Vec {
  T x[V];
};

// HALF: a column is V pairs, two vectors r/2 apart.  INTER: one vector of V/2 pairs.
template <typename T, int V, bool INTER>
__global__ void __launch_bounds__(kThreads, 8) rope_kernel(const __grid_constant__ RopeParams p) {
  constexpr int kPairs = INTER ? V / 2 : V;
  // The frequencies by (pair of a column, column), copied by one lane per warp: a constant that differs between the
  // lanes is fetched once for each of them.
  __shared__ uint64_t turns[128];
  for (int i = threadIdx.x >> 5; i < p.rot / 2; i += kThreads / 32)
    if ((threadIdx.x & 31) == 0) turns[i % kPairs * p.rot_cols + i / kPairs] = p.turns[i];
  __syncthreads();
  const int64_t item = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x;
  const int cols = p.rot_cols + p.copy_cols;
  const int64_t tok = item / cols;
  const int col = static_cast<int>(item - tok * cols);
  if (tok >= static_cast<int64_t>(p.B) * p.N) return;
  const int b = static_cast<int>(tok / p.N);
  const int n = static_cast<int>(tok - static_cast<int64_t>(b) * p.N);
  // The block's heads are q's or k's.
  const bool is_k = static_cast<int>(blockIdx.y) >= p.q_groups;
  const int h0 = (blockIdx.y - (is_k ? p.q_groups : 0)) * p.heads_per_thread;
  const int heads = min(p.heads_per_thread, (is_k ? p.Hk : p.Hq) - h0);

  const bool turn = col < p.rot_cols;
  const int e0 = turn ? col * V : p.rot + (col - p.rot_cols) * V;  // first element of the column
  const int64_t* ss = is_k ? p.sk : p.sq;
  const int64_t* ds = is_k ? p.sko : p.sqo;
  const T* src = static_cast<const T*>(is_k ? p.k : p.q) + b * ss[0] + h0 * ss[1] + n * ss[2] + e0;
  T* dst = static_cast<T*>(is_k ? p.k_out : p.q_out) + b * ds[0] + h0 * ds[1] + n * ds[2] + e0;
  const int64_t src_h = ss[1], dst_h = ds[1];
  const int half = p.rot >> 1;
  Vec<T, V> a[kHeadsInFlight], c[kHeadsInFlight];
  auto load = [&](int h) {
#pragma unroll
    for (int u = 0; u < kHeadsInFlight; ++u) {
      if (h + u < heads) {
        a[u] = *reinterpret_cast<const Vec<T, V>*>(src);
        if (!INTER && turn) c[u] = *reinterpret_cast<const Vec<T, V>*>(src + half);
      }
      src += src_h;
    }
  };
  load(0);  // on their way while the angles are worked out

  float cs[kPairs], sn[kPairs];
  if (turn) {
    const int64_t pos = p.position0 + (p.positions != nullptr ? p.positions[b * p.pos_stride_b + n] : n);
#pragma unroll
    for (int i = 0; i < kPairs; ++i) {
      const uint64_t t = static_cast<uint64_t>(pos) * turns[i * p.rot_cols + col];
      const float half_turns = static_cast<float>(static_cast<int32_t>(t >> 32)) * 4.656612873077393e-10f;  // 2^-31
      sincospif(half_turns, &sn[i], &cs[i]);
      cs[i] *= p.magnitude;
      sn[i] *= p.sign * p.magnitude;
    }
  }

  for (int h = 0; h < heads; h += kHeadsInFlight) {
    if (h > 0) load(h);
#pragma unroll
    for (int u = 0; u < kHeadsInFlight; ++u) {
      if (h + u < heads) {
        if (turn) {
#pragma unroll
          for (int i = 0; i < kPairs; ++i) {
            T& t1 = INTER ? a[u].x[2 * i] : a[u].x[i];
            T& t2 = INTER ? a[u].x[(2 * i + 1) % V] : c[u].x[i];
            const float x1 = to_f32<T>(t1), x2 = to_f32<T>(t2);
            t1 = from_f32<T>(x1 * cs[i] - x2 * sn[i]);  // rounded once, on the way out
            t2 = from_f32<T>(x2 * cs[i] + x1 * sn[i]);
          }
          if (!INTER) *reinterpret_cast<Vec<T, V>*>(dst + half) = c[u];
        }
        *reinterpret_cast<Vec<T, V>*>(dst) = a[u];
      }
      dst += dst_h;
    }
  }
}

template <typename T, int V, bool INTER>
cudaError_t launch_v(RopeParams p, bool in_place, cudaStream_t stream) {
  p.rot_cols = (INTER ? p.rot : p.rot / 2) / V;
  p.copy_cols = in_place ? 0 : (p.d - p.rot) / V;
  const int64_t items = static_cast<int64_t>(p.B) * p.N * (p.rot_cols + p.copy_cols);
  const int64_t blocks = (items + kThreads - 1) / kThreads;
  if (blocks > 0x7fffffff) return cudaErrorInvalidValue;
  // Heads per thread: all of a tensor's when the tokens alone give every SM about 1024 threads, fewer (down to one)
  // when they do not.  All heads, this rule and one head a thread, replaying
  // a graph: one token of 28 + 4 heads 16, 9, 9 us; 2 x 8192 tokens of 16 + 16 heads 51, 51, 105 us.
  const int most = p.Hq > p.Hk ? p.Hq : p.Hk;
  int per = most;
  while (per > 1 && blocks * ((p.Hq + per - 1) / per + (p.Hk + per - 1) / per) < 152 * 8) per = (per + 1) / 2;
  p.heads_per_thread = per;
  p.q_groups = (p.Hq + per - 1) / per;
  const int groups = p.q_groups + (p.Hk + per - 1) / per;
  rope_kernel<T, V, INTER><<<dim3(static_cast<unsigned>(blocks), groups), kThreads, 0, stream>>>(p);
  return cudaGetLastError();
}

template <typename T>
cudaError_t launch_t(const RopeParams& p, bool inter, bool in_place, cudaStream_t stream) {
  constexpr int V = 16 / sizeof(T);
  // 16-byte columns where every pointer, stride and the head's parts allow them.
  auto al = [](const void* x) { return (reinterpret_cast<uintptr_t>(x) & 15u) == 0; };
  bool wide = al(p.q) && al(p.k) && al(p.q_out) && al(p.k_out) && (inter ? p.rot : p.rot / 2) % V == 0 &&
              (p.d - p.rot) % V == 0;
  for (int i = 0; i < 3; ++i)
    wide = wide && p.sq[i] % V == 0 && p.sk[i] % V == 0 && p.sqo[i] % V == 0 && p.sko[i] % V == 0;
  if (wide) return inter ? launch_v<T, V, true>(p, in_place, stream) : launch_v<T, V, false>(p, in_place, stream);
  if (!inter) return launch_v<T, 1, false>(p, in_place, stream);
  return launch_v<T, 2, true>(p, in_place, stream);  // d and r are even, and so is the rest
}

}  // namespace

cudaError_t launch_rope(const RopeParams& p, bool fp32, bool inter, bool in_place, cudaStream_t stream) {
  return fp32 ? launch_t<float>(p, inter, in_place, stream) : launch_t<__nv_bfloat16>(p, inter, in_place, stream);
}

}  // namespace fa

// fa_rope.cu — rotary positions of q and k, and the gradient (the transposed
// rotation).
//
// Pair i of a head at position p turns by the angle θ = p·w_i:
//   y₁ = μ(x₁ cos θ − x₂ sin θ),  y₂ = μ(x₂ cos θ + x₁ sin θ),
// with pairs (i, i + r/2) or (2i, 2i + 1) of the first r elements.  The
// gradient turns back by −θ with the same μ.
//
// Angles.  θ/2π = p·(w_i/2π) is only needed modulo 1 and p is a whole number,
// so w_i/2π is held as a 64-bit fraction of a turn and p times it is one 64-bit
// product that wraps exactly where whole turns drop out.  Far positions lose
// nothing: the error is p·2⁻⁶⁴ turns (plus the float64 rounding of w_i), where
// a float32 product would be off by p·2⁻²⁴ radians.  sincospif of the signed
// fraction then has float32 accuracy.
//
// Bound: device memory, q and k read once and written once.  A thread owns one
// 16-byte column of one token and walks over heads with it, so that the sines
// are computed once for all of them and kept in registers; with few tokens
// there are few heads per thread (the launcher splits them until the grid fills
// the machine).
#include "fa_kernels.h"
#include "sm103.cuh"

namespace fa {
namespace {

constexpr int kThreads = 128;
constexpr int kHeadsInFlight = 4;  // loads outstanding per thread before the first use

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
__global__ void __launch_bounds__(kThreads) rope_kernel(const __grid_constant__ RopeParams p) {
  constexpr int kPairs = INTER ? V / 2 : V;
  const int64_t item = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x;
  const int cols = p.rot_cols + p.copy_cols;
  const int64_t tok = item / cols;
  const int col = static_cast<int>(item - tok * cols);
  if (tok >= static_cast<int64_t>(p.B) * p.N) return;
  const int b = static_cast<int>(tok / p.N);
  const int n = static_cast<int>(tok - static_cast<int64_t>(b) * p.N);
  const int heads = p.Hq + p.Hk;
  const int h0 = blockIdx.y * p.heads_per_thread;
  const int h1 = min(heads, h0 + p.heads_per_thread);

  const bool turn = col < p.rot_cols;
  const int e0 = turn ? col * V : p.rot + (col - p.rot_cols) * V;  // first element of the column
  float cs[kPairs], sn[kPairs];
  if (turn) {
    const int64_t pos = p.position0 + (p.positions != nullptr ? p.positions[b * p.pos_stride_b + n] : n);
#pragma unroll
    for (int i = 0; i < kPairs; ++i) {
      const uint64_t t = static_cast<uint64_t>(pos) * p.turns[col * kPairs + i];
      const float half_turns = static_cast<float>(static_cast<int64_t>(t)) * 1.0842021724855044e-19f;  // 2^-63
      sincospif(half_turns, &sn[i], &cs[i]);
      cs[i] *= p.magnitude;
      sn[i] *= p.sign * p.magnitude;
    }
  }

  const T* q = static_cast<const T*>(p.q) + b * p.sq[0] + n * p.sq[2] + e0;
  const T* k = static_cast<const T*>(p.k) + b * p.sk[0] + n * p.sk[2] + e0;
  T* qo = static_cast<T*>(p.q_out) + b * p.sqo[0] + n * p.sqo[2] + e0;
  T* ko = static_cast<T*>(p.k_out) + b * p.sko[0] + n * p.sko[2] + e0;
  const int half = p.rot >> 1;
  for (int h = h0; h < h1; h += kHeadsInFlight) {
    Vec<T, V> a[kHeadsInFlight], c[kHeadsInFlight];
#pragma unroll
    for (int u = 0; u < kHeadsInFlight; ++u) {
      if (h + u < h1) {
        const T* src = h + u < p.Hq ? q + (h + u) * p.sq[1] : k + (h + u - p.Hq) * p.sk[1];
        a[u] = *reinterpret_cast<const Vec<T, V>*>(src);
        if (!INTER && turn) c[u] = *reinterpret_cast<const Vec<T, V>*>(src + half);
      }
    }
#pragma unroll
    for (int u = 0; u < kHeadsInFlight; ++u) {
      if (h + u < h1) {
        T* dst = h + u < p.Hq ? qo + (h + u) * p.sqo[1] : ko + (h + u - p.Hq) * p.sko[1];
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
  const int heads = p.Hq + p.Hk;
  // Heads per thread: all of them when the tokens alone give every SM about
  // 1024 threads, fewer (down to one) when they do not.
  int groups = 1;
  while (groups < heads && blocks * groups < 152 * 8) groups *= 2;
  p.heads_per_thread = (heads + groups - 1) / groups;
  groups = (heads + p.heads_per_thread - 1) / p.heads_per_thread;
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

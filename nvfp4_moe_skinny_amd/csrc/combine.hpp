// combine.hpp - the routing-weighted sum of expert outputs per token row:
//   out[m] = bf16( sum_j w[m][j] y[m k + j] (+ shared[m]) (+ residual[m]) )
// in j order, then the shared term, then the residual, FP32, one rounding at
// the end. A pair of weight 0 adds nothing, whatever its y row holds (a pair
// whose expert lives elsewhere has no y).
// Bound: memory (k y rows read per row written; M = 4096, k = 8, H = 2048, BF16,
// 168 MB: 30 us, 5.5 TB/s; M = 16 in FP32, 1.3 MB: 3.2 us, a launch and one round
// trip). Four outputs a thread, 8 or 16 bytes a load, all k loads in flight.
#pragma once

#include "common.hpp"

namespace nvfp4moe {

constexpr int kCombineThreads = 256;

__device__ __forceinline__ float combine_f32(float v) { return v; }
__device__ __forceinline__ float combine_f32(uint16_t v) { return bf16_to_f32(v); }

// V consecutive elements, V * sizeof(T) bytes aligned to the same.
template <typename T, int V>
struct alignas(sizeof(T) * V) Pack {
  T v[V];
};

// One thread per V outputs of a row.
template <typename T, int V, int KMAX>
__global__ void __launch_bounds__(kCombineThreads) combine_kernel(
    const T* __restrict__ y, const float* __restrict__ w, const T* __restrict__ shared,
    const uint16_t* __restrict__ residual, int64_t units, int per_row, int k, int64_t H,
    uint16_t* __restrict__ out) {
  const int64_t u = (int64_t)blockIdx.x * kCombineThreads + threadIdx.x;
  if (u >= units) return;
  const int64_t m = u / per_row;
  const int64_t n = (u - m * per_row) * V;
  Pack<T, V> yv[KMAX];
  float wv[KMAX];
#pragma unroll
  for (int j = 0; j < KMAX; ++j) {
    const int jj = j < k ? j : k - 1;  // past k: the last row again, with weight 0
    yv[j] = *reinterpret_cast<const Pack<T, V>*>(y + (m * k + jj) * H + n);
    wv[j] = w[m * k + jj];
  }
  // without a shared expert or a residual: some row's place, not added
  const Pack<T, V> sv = *reinterpret_cast<const Pack<T, V>*>((shared ? shared : y) + m * H + n);
  Pack<uint16_t, V> rv = {};
  if (residual) rv = *reinterpret_cast<const Pack<uint16_t, V>*>(residual + m * H + n);
  Pack<uint16_t, V> o;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    float acc = 0.0f;
#pragma unroll
    for (int j = 0; j < KMAX; ++j) {
      const float t = fmaf(wv[j], combine_f32(yv[j].v[i]), acc);
      acc = j < k && wv[j] != 0.0f ? t : acc;
    }
    if (shared) acc += combine_f32(sv.v[i]);
    if (residual) acc += bf16_to_f32(rv.v[i]);
    o.v[i] = f32_to_bf16_rne(acc);
  }
  *reinterpret_cast<Pack<uint16_t, V>*>(out + m * H + n) = o;
}

}  // namespace nvfp4moe

// block8.hpp - BF16 / FP32 values -> E4M3 codes with one FP32 scale per block
// of 128: rows (1 x 128 blocks, activations) and weights (128 x 128 blocks).
//
// a = max(amax of the block, 2^-117); scale = a / 448; code = E4M3 nearest to
// v * (448 / a), ties to even. Both quotients are correctly rounded FP32
// divisions, one each per block; the product is one FP32 rounding. The floor
// keeps the scale a normal number and 448 / a finite (2^-117 / 448 = 2^-125.8,
// 448 * 2^117 = 2^125.8). |v| <= a gives |v * (448 / a)| <= 448 (1 + 2^-22),
// which rounds to at most 448, so the conversion never meets its overflow
// behaviour. A block that holds an infinity or a NaN gets a non-finite scale
// and NaN codes (magnitude bits order like values, NaN above infinity), so
// whatever is multiplied with that row comes out NaN.
#pragma once

#include "common.hpp"

namespace nvfp4moe {

constexpr int kBlock8 = 128;
constexpr float kBlock8Max = 448.0f;
constexpr float kBlock8AmaxMin = 0x1p-117f;

__host__ __device__ constexpr int64_t blocks128(int64_t n) { return (n + kBlock8 - 1) / kBlock8; }

// Four values -> four E4M3 codes (RNE), value 0 in the low byte.
__device__ __forceinline__ uint32_t e4m3_pack4(float a, float b, float c, float d) {
  int w = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
  return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(c, d, w, true);
}

// amax of a block (as magnitude bits) -> its scale and the factor onto codes.
__device__ __forceinline__ void block8_scale(uint32_t amax_bits, float& scale, float& factor) {
  float a = __uint_as_float(amax_bits);
  a = a < kBlock8AmaxMin ? kBlock8AmaxMin : a;  // a NaN stays
  scale = a / kBlock8Max;
  factor = kBlock8Max / a;
}

// Eight consecutive elements as FP32.
template <typename T>
struct Eight;
template <>
struct Eight<uint16_t> {  // BF16 bits
  uint4 v;
  __device__ __forceinline__ void load(const uint16_t* p) { v = *reinterpret_cast<const uint4*>(p); }
  __device__ __forceinline__ void get(float (&f)[8]) const {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = __uint_as_float(u4_get(v, i) << 16);
      f[2 * i + 1] = __uint_as_float(u4_get(v, i) & 0xFFFF0000u);
    }
  }
};
template <>
struct Eight<float> {
  float4 a, b;
  __device__ __forceinline__ void load(const float* p) {
    a = reinterpret_cast<const float4*>(p)[0];
    b = reinterpret_cast<const float4*>(p)[1];
  }
  __device__ __forceinline__ void get(float (&f)[8]) const {
    f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
    f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
  }
};

__device__ __forceinline__ uint32_t amax_bits8(const float (&f)[8]) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(f[i]) & 0x7FFFFFFFu);
  return m;
}

// Maximum over the lane's row of 16 lanes, in every lane of it.
__device__ __forceinline__ uint32_t row16_max(uint32_t v) {
  v = max(v, dpp_u32(v, kDppQuadXor1));
  v = max(v, dpp_u32(v, kDppQuadXor2));
  v = max(v, dpp_u32(v, kDppRowRor4));
  return max(v, dpp_u32(v, kDppRowRor8));
}

// silu(a) * b with the full-precision exponential and a correctly rounded
// quotient: the fast forms (2^-22 or so of the value) moved a few codes in a
// million across an E4M3 rounding boundary, and the pass is bound by memory.
__device__ __forceinline__ float silu_mul(float a, float b) { return a / (1.0f + expf(-a)) * b; }

constexpr int kQuantRowsThreads = 256;

// One 128-block per 16 lanes, eight elements per lane (16 bytes of BF16), held
// in registers between the maximum, found by row rotations among the 16 lanes,
// and the codes: one pass over the data, no LDS, no barrier. A block of 256
// threads takes 16 consecutive blocks of the row-major order. Bound: memory for
// many rows (swiglu, M = 8192, K = 512, 21 MB: 7.8 us, 2.7 TB/s, of which a
// launch and one round trip take 2.2, the time of M = 4).
template <typename T, bool SWIGLU>
__global__ void __launch_bounds__(kQuantRowsThreads) fp8_quantize_rows_kernel(
    const T* __restrict__ x, int64_t M, int K, int64_t ldx, int KB, uint8_t* __restrict__ codes,
    float* __restrict__ scales) {
  const int64_t unit = (int64_t)blockIdx.x * (kQuantRowsThreads / 16) + (threadIdx.x >> 4);
  const int64_t m = unit / KB;
  if (m >= M) return;  // whole 16-lane groups
  const int b = (int)(unit - m * KB);
  const int col = b * kBlock8 + 8 * (threadIdx.x & 15);
  float f[8] = {0, 0, 0, 0, 0, 0, 0, 0};
  if (col < K) {
    Eight<T> v;
    v.load(x + m * ldx + col);
    v.get(f);
    if constexpr (SWIGLU) {
      Eight<T> u;
      float g[8];
      u.load(x + m * ldx + K + col);
      u.get(g);
#pragma unroll
      for (int i = 0; i < 8; ++i) f[i] = silu_mul(f[i], g[i]);
    }
  }
  float s, r;
  block8_scale(row16_max(amax_bits8(f)), s, r);
  if (col < K) {
    uint2 c;
    c.x = e4m3_pack4(f[0] * r, f[1] * r, f[2] * r, f[3] * r);
    c.y = e4m3_pack4(f[4] * r, f[5] * r, f[6] * r, f[7] * r);
    *reinterpret_cast<uint2*>(codes + m * K + col) = c;
  }
  if ((threadIdx.x & 15) == 0) scales[(int64_t)b * M + m] = s;
}

constexpr int kQuantBlocksThreads = 256;

// One 128 x 128 block per workgroup: 16 lanes per row, 16 rows at a time, the
// block held in registers between the maximum and the codes, so each element is
// read once. Bound: memory (256 x [1024][2048] BF16, 1.6 GB: 298 us, 5.4 TB/s;
// [2048][4096], 25 MB: 6.6 us).
template <typename T>
__global__ void __launch_bounds__(kQuantBlocksThreads) fp8_quantize_blocks_kernel(
    const T* __restrict__ x, int64_t N, int K, int NB, int KB, uint8_t* __restrict__ codes,
    float* __restrict__ scales) {
  __shared__ uint32_t wmax[kQuantBlocksThreads / 64];
  const int64_t blk = blockIdx.x;
  const int kb = (int)(blk % KB);
  const int64_t gn = blk / KB;
  const int nb = (int)(gn % NB);
  const int64_t g = gn / NB;
  const int col = kb * kBlock8 + 8 * (threadIdx.x & 15);
  const int64_t row0 = (int64_t)nb * kBlock8 + (threadIdx.x >> 4);
  const bool in_col = col < K;
  Eight<T> v[8];
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int64_t n = row0 + 16 * i;
    // past the matrix: the block's first element group again (no new maximum)
    const int64_t rn = n < N ? n : (int64_t)nb * kBlock8;
    const int rc = in_col ? col : kb * kBlock8;
    v[i].load(x + (g * N + rn) * K + rc);
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    float f[8];
    v[i].get(f);
    m = max(m, amax_bits8(f));
  }
  m = wave_max_u32(m);
  if ((threadIdx.x & 63) == 0) wmax[threadIdx.x >> 6] = m;
  __syncthreads();
  m = max(max(wmax[0], wmax[1]), max(wmax[2], wmax[3]));
  float s, r;
  block8_scale(m, s, r);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int64_t n = row0 + 16 * i;
    float f[8];
    v[i].get(f);
    uint2 c;
    c.x = e4m3_pack4(f[0] * r, f[1] * r, f[2] * r, f[3] * r);
    c.y = e4m3_pack4(f[4] * r, f[5] * r, f[6] * r, f[7] * r);
    if (in_col && n < N) *reinterpret_cast<uint2*>(codes + (g * N + n) * K + col) = c;
  }
  if (threadIdx.x == 0) scales[blk] = s;
}

}  // namespace nvfp4moe

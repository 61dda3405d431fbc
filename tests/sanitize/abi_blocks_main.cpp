// abi_blocks_main.cpp - the host-side validation of the block-scaled and
// grouped calls under AddressSanitizer and UndefinedBehaviorSanitizer
// (tests/test_sanitizers_blocks.py): every call is rejected, or has no rows,
// before any launch, so no GPU is needed.
#include <cstdio>
#include <cstring>

#include "nvfp4moe.h"

#define EXPECT(call, code)                                                        \
  do {                                                                            \
    const long long got = (long long)(call);                                      \
    if (got != (code)) {                                                          \
      std::printf("FAIL %s: %lld (%s)\n", #call, got, nvfp4moe_last_error_detail()); \
      return 1;                                                                   \
    }                                                                             \
  } while (0)

int main() {
  void* f = reinterpret_cast<void*>(4096);
  void* odd = reinterpret_cast<void*>(4100);
  auto u8 = static_cast<uint8_t*>(f);
  auto u16 = static_cast<uint16_t*>(f);
  auto f32 = static_cast<float*>(f);
  auto i32 = static_cast<int32_t*>(f);
  const int64_t big = (int64_t)1 << 62, low = -big - big;
  const int32_t BF = NVFP4MOE_BF16, F32 = NVFP4MOE_F32;
  const int32_t shape = NVFP4MOE_ERR_BAD_SHAPE, unsup = NVFP4MOE_ERR_UNSUPPORTED,
                null = NVFP4MOE_ERR_NULL_ARG;

  for (int64_t v : {big, low, (int64_t)1 << 33, (int64_t)-1}) {
    const int64_t bad = v < 0 ? shape : unsup;
    EXPECT(fp8_quantize_rows(f, BF, v, 128, 128, 0, u8, f32, nullptr), bad);
    EXPECT(fp8_quantize_blocks(f, BF, v, 128, 128, u8, f32, nullptr), bad);
    EXPECT(fp8_quantize_blocks(f, BF, 1, v, 128, u8, f32, nullptr), bad);
    EXPECT(fp8_block_gemm(u8, f32, v, 128, u8, f32, 128, f, BF, 128, nullptr), bad);
    EXPECT(fp8_block_gemm(u8, f32, 4, 128, u8, f32, v, f, BF, 128, nullptr), bad);
    EXPECT(moe_combine(f, F32, f32, nullptr, nullptr, v, 8, 128, u16, nullptr), bad);
    EXPECT(moe_combine(f, F32, f32, nullptr, nullptr, 4, 8, v, u16, nullptr), bad);
  }
  for (int64_t K : {(int64_t)0, (int64_t)-16, low}) {
    EXPECT(fp8_quantize_rows(f, BF, 4, K, 128, 1, u8, f32, nullptr), shape);
    EXPECT(fp8_block_gemm(u8, f32, 4, K, u8, f32, 128, f, BF, 128, nullptr), shape);
  }
  for (int64_t K : {(int64_t)24, (int64_t)65552, big}) {
    EXPECT(fp8_quantize_rows(f, BF, 4, K, big, 0, u8, f32, nullptr), unsup);
    EXPECT(fp8_quantize_blocks(f, BF, 1, 4, K, u8, f32, nullptr), unsup);
  }
  for (int64_t ld : {(int64_t)0, low, (int64_t)127, big}) {
    EXPECT(fp8_quantize_rows(f, BF, 4, 128, ld, 0, u8, f32, nullptr), shape);
    EXPECT(fp8_block_gemm(u8, f32, 4, 128, u8, f32, 128, f, BF, ld, nullptr), shape);
  }
  EXPECT(fp8_quantize_blocks(f, BF, ((int64_t)1 << 31) - 1, (int64_t)1 << 20, 65536, u8, f32,
                             nullptr),
         unsup);
  EXPECT(fp8_block_gemm(u8, f32, (int64_t)1 << 24, 128, u8, f32, (int64_t)1 << 20, f, BF,
                        (int64_t)1 << 20, nullptr),
         unsup);
  // more lanes than a launch holds
  EXPECT(fp8_quantize_rows(f, BF, (int64_t)1 << 20, 65536, 65536, 0, u8, f32, nullptr), unsup);
  EXPECT(fp8_quantize_blocks(f, BF, 1 << 12, 128 * 64, 128 * 64, u8, f32, nullptr), unsup);
  EXPECT(moe_combine(f, F32, f32, nullptr, nullptr, (int64_t)1 << 16, 1, ((int64_t)1 << 15) + 1,
                     u16, nullptr),
         unsup);
  EXPECT(fp8_quantize_rows(odd, BF, 4, 128, 128, 0, u8, f32, nullptr), unsup);
  EXPECT(fp8_quantize_rows(nullptr, BF, 4, 128, 128, 0, u8, f32, nullptr), null);
  EXPECT(fp8_quantize_rows(nullptr, BF, 0, 128, 128, 0, nullptr, nullptr, nullptr), NVFP4MOE_OK);
  EXPECT(fp8_block_gemm(u8, nullptr, 4, 128, u8, f32, 128, f, BF, 128, nullptr), null);

  moe_grouped_args a;
  std::memset(&a, 0, sizeof(a));
  EXPECT(moe_grouped_gemm(nullptr, nullptr), null);
  a.x = a.w = f;
  a.x_scales = a.w_scales = f32;
  a.pairs = a.active = a.active_offsets = a.n_active = i32;
  a.y = f;
  a.ldy = a.N = 128;
  a.R = 32;
  a.x_rows = 4;
  a.pairs_per_row = 8;
  a.E = 16;
  a.K = 128;
  a.type = NVFP4MOE_FP8;
  a.y_type = BF;
  int64_t* const sizes[] = {&a.R, &a.x_rows, &a.pairs_per_row, &a.E, &a.N, &a.K, &a.ldy};
  for (int64_t* s : sizes) {
    const int64_t was = *s;
    for (int64_t v : {big, low, (int64_t)-1}) {
      *s = v;
      const int32_t st = moe_grouped_gemm(&a, nullptr);
      if (st != shape && st != unsup) {
        std::printf("FAIL size %d = %lld: %d\n", (int)(s - &a.ldy), (long long)v, (int)st);
        return 1;
      }
    }
    *s = was;
  }
  a.type = 7;
  EXPECT(moe_grouped_gemm(&a, nullptr), shape);
  a.type = NVFP4MOE_FP8;
  a.x = odd;
  EXPECT(moe_grouped_gemm(&a, nullptr), unsup);
  a.x = f;
  a.x_scales = nullptr;
  EXPECT(moe_grouped_gemm(&a, nullptr), null);
  a.R = 0;
  EXPECT(moe_grouped_gemm(&a, nullptr), NVFP4MOE_OK);
  std::printf("ok\n");
  return 0;
}

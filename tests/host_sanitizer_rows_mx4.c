/*
 * Host-side checks of the rows-in-expert-order and MX4 calls for the
 * AddressSanitizer / UndefinedBehaviorSanitizer build of the library
 * (tests/test_host_sanitizer_rows_mx4.py).  Every call here returns before any
 * kernel launch.  The pointers are stand-ins that the host code checks for NULL
 * and alignment but never dereferences.
 */
#include <limits.h>
#include <stdint.h>
#include <stdio.h>
#include <string.h>

#include "moe_lora.h"

static int failures = 0;

#define EXPECT(cond)                                                   \
  do {                                                                 \
    if (!(cond)) {                                                     \
      fprintf(stderr, "FAILED line %d: %s\n", __LINE__, #cond);       \
      ++failures;                                                      \
    }                                                                  \
  } while (0)

#define REFUSED(call)                                                                \
  do {                                                                               \
    const int st_ = (call);                                                          \
    EXPECT(st_ == MOE_LORA_ERR_INVALID || st_ == MOE_LORA_ERR_UNSUPPORTED ||         \
           st_ == MOE_LORA_ERR_WORKSPACE);                                           \
  } while (0)

static void* fake(uintptr_t i) { return (void*)(uintptr_t)(4096 * (i + 1)); }

static const int32_t kInts[] = {INT32_MIN, INT32_MIN + 1, -1, 0, 1, 16, 1 << 24, (1 << 30) - 1,
                                1 << 30, INT32_MAX - 1, INT32_MAX};
static const int64_t kLongs[] = {INT64_MIN, -1, 0, 1, INT32_MAX, (int64_t)INT32_MAX + 1,
                                 (int64_t)1 << 40, INT64_MAX};
enum { kNumInts = sizeof(kInts) / sizeof(kInts[0]), kNumLongs = sizeof(kLongs) / sizeof(kLongs[0]) };

/* y, rows and the layout are missing, so that no size is launched; only the empty ones succeed */
static void check_rows(void) {
  for (int t = 0; t < kNumInts; ++t)
    for (int k = 0; k < kNumInts; ++k)
      for (int h = 0; h < kNumInts; ++h)
        for (int r = 0; r < kNumLongs; ++r)
          for (int dt = -1; dt < 6; ++dt) {
            const int32_t T = kInts[t], K = kInts[k], H = kInts[h];
            const int64_t R = kLongs[r];
            int st = moe_lora_permute(T, K, H, dt, R, NULL, NULL, NULL, NULL, NULL, NULL);
            EXPECT(st != MOE_LORA_OK || (T == 0 && R == 0));
            st = moe_lora_unpermute(T, K, H, dt, dt, R, NULL, NULL, NULL, NULL, NULL);
            EXPECT(st != MOE_LORA_OK || T == 0);
            st = moe_lora_permute_backward(T, K, H, dt, dt, R, NULL, NULL, NULL, NULL);
            EXPECT(st != MOE_LORA_OK || T == 0);
            st = moe_lora_unpermute_backward(T, K, H, dt, dt, R, NULL, NULL, NULL, NULL, NULL, NULL,
                                             NULL, NULL, NULL);
            EXPECT(st != MOE_LORA_OK || (T == 0 && R == 0));
            REFUSED(moe_lora_align_pair_rows(T, K, H, 0, 16, NULL, NULL, NULL, NULL, NULL, NULL, NULL,
                                             NULL, NULL, NULL, 0, NULL));
          }
}

static void check_mx4(void) {
  for (int r = 0; r < kNumLongs; ++r)
    for (int c = 0; c < kNumInts; ++c)
      for (int dt = -1; dt < 6; ++dt) {
        const int64_t R = kLongs[r];
        int st = moe_lora_mx4_quantize(R, kInts[c], dt, NULL, NULL, NULL, NULL, NULL);
        EXPECT(st != MOE_LORA_OK || R == 0);
        st = moe_lora_mx4_dequantize(R, kInts[c], dt, NULL, NULL, NULL, NULL);
        EXPECT(st != MOE_LORA_OK || R == 0);
      }
}

static moe_lora_mx4_gemm_args gemm_args(int64_t M, int32_t N, int32_t K, int32_t E, int32_t bm) {
  moe_lora_mx4_gemm_args a;
  memset(&a, 0, sizeof(a));
  a.struct_size = sizeof(a);
  a.x_dtype = MOE_LORA_MX4;
  a.out_dtype = MOE_LORA_BF16;
  a.num_rows = M; a.out_features = N; a.in_features = K; a.num_experts = E; a.block_m = bm;
  a.x = fake(0); a.w = (const uint8_t*)fake(2);
  a.w_scale = (const uint8_t*)fake(3); a.tile_expert = (const int32_t*)fake(4); a.out = fake(5);
  return a;   /* x_scale is missing */
}

static void check_gemm(void) {
  EXPECT(moe_lora_mx4_gemm(NULL, NULL) == MOE_LORA_ERR_INVALID);
  for (int m = 0; m < kNumLongs; ++m)
    for (int n = 0; n < kNumInts; ++n)
      for (int k = 0; k < kNumInts; ++k)
        for (int b = 0; b < kNumInts; ++b)
          for (int silu = 0; silu < 2; ++silu) {
            moe_lora_mx4_gemm_args a = gemm_args(kLongs[m], kInts[n], kInts[k], kInts[b], kInts[b]);
            a.silu_mul = silu;
            int st = moe_lora_mx4_gemm(&a, NULL);
            EXPECT(st != MOE_LORA_OK || kLongs[m] == 0);
            a.tile_expert = NULL;
            a.num_experts = 1;
            st = moe_lora_mx4_gemm(&a, NULL);
            EXPECT(st != MOE_LORA_OK || kLongs[m] == 0);
          }
  const int32_t blocks[] = {16, 32, 48, 64, 96, 128, 144, 192, 256};
  for (int i = 0; i < 9; ++i)
    for (int64_t rows = blocks[i]; rows < (int64_t)1 << 31; rows *= 3)
      for (int32_t n = 16; n <= 1 << 24; n *= 4) {
        moe_lora_mx4_gemm_args a = gemm_args(rows, n, 32, 4, blocks[i]);
        const int64_t counted = (rows + 15) / 16 * ((n + 63) / 64);
        const int64_t groups = rows / 16 < 32 || blocks[i] % 32 == 0 ? 0 : (rows + 255) / 256 * 16;
        const int fits = counted < (1 << 24) && groups * ((n + 63) / 64) < (1 << 24);
        EXPECT(moe_lora_mx4_gemm(&a, NULL) ==
               (fits ? MOE_LORA_ERR_INVALID : MOE_LORA_ERR_UNSUPPORTED));
      }
}

int main(void) {
  check_rows();
  check_mx4();
  check_gemm();
  if (failures) {
    fprintf(stderr, "%d host checks failed\n", failures);
    return 1;
  }
  printf("all host checks passed\n");
  return 0;
}

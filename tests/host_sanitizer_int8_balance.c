/*
 * Host-side checks of the 8-bit integer, norm and balance-loss calls for the
 * AddressSanitizer / UndefinedBehaviorSanitizer build of the library
 * (tests/test_host_sanitizer_int8_balance.py).  Every call here returns before any
 * kernel launch.  The pointers are stand-ins that the host code checks for NULL
 * and alignment but never dereferences.
 */
#include <limits.h>
#include <math.h>
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

static void* fake(uintptr_t i) { return (void*)(uintptr_t)(4096 * (i + 1)); }

static const int32_t kInts[] = {INT32_MIN, INT32_MIN + 1, -1, 0, 1, 16, 256, 257, 1024, 16384, 131056, 1 << 24,
                                1 << 30, INT32_MAX - 1, INT32_MAX};
static const int64_t kLongs[] = {INT64_MIN, -1, 0, 1, 256, INT32_MAX, (int64_t)INT32_MAX + 1,
                                 (int64_t)1 << 40, INT64_MAX};
enum { kNumInts = sizeof(kInts) / sizeof(kInts[0]), kNumLongs = sizeof(kLongs) / sizeof(kLongs[0]) };

/* an output is missing, so that no size is launched; only the empty ones succeed */
static void check_rows(void) {
  for (int r = 0; r < kNumLongs; ++r)
    for (int c = 0; c < kNumInts; ++c)
      for (int dt = -1; dt < 6; ++dt) {
        const int64_t R = kLongs[r];
        int st = moe_lora_int8_quantize(R, kInts[c], dt, fake(0), NULL, (int8_t*)fake(1), NULL, NULL);
        EXPECT(st != MOE_LORA_OK || R == 0);
        st = moe_lora_int8_dequantize(R, kInts[c], dt, (int8_t*)fake(0), (float*)fake(1), NULL, NULL);
        EXPECT(st != MOE_LORA_OK || R == 0);
        st = moe_lora_rms_norm_quantize(R, kInts[c], dt, dt, dt, 1e-6, fake(0), NULL, fake(1), (int8_t*)fake(2),
                                        NULL, NULL, NULL, NULL);
        EXPECT(st != MOE_LORA_OK || R == 0);
      }
  const double eps[] = {-1.0, -0.0, 0.0, 1e-6, 3e38, 1e300, INFINITY, -INFINITY, NAN};
  for (int i = 0; i < 9; ++i) {
    const int st = moe_lora_rms_norm_quantize(0, 64, 0, 0, 0, eps[i], NULL, NULL, NULL, NULL, NULL, NULL, NULL, NULL);
    EXPECT((st == MOE_LORA_OK) == (eps[i] >= 0.0 && eps[i] <= 3e38));
  }
}

static moe_lora_int8_gemm_args gemm_args(int64_t M, int32_t N, int32_t K, int32_t E, int32_t bm) {
  moe_lora_int8_gemm_args a;
  memset(&a, 0, sizeof(a));
  a.struct_size = sizeof(a);
  a.out_dtype = MOE_LORA_BF16;
  a.num_rows = M; a.out_features = N; a.in_features = K; a.num_experts = E; a.block_m = bm;
  a.x = (const int8_t*)fake(0); a.x_scale = (const float*)fake(1); a.w = (const int8_t*)fake(2);
  a.tile_expert = (const int32_t*)fake(4); a.out = fake(5);
  return a;   /* w_scale is missing */
}

static void check_gemm(void) {
  EXPECT(moe_lora_int8_gemm(NULL, NULL) == MOE_LORA_ERR_INVALID);
  for (int m = 0; m < kNumLongs; ++m)
    for (int n = 0; n < kNumInts; ++n)
      for (int k = 0; k < kNumInts; ++k)
        for (int b = 0; b < kNumInts; ++b) {
          moe_lora_int8_gemm_args a = gemm_args(kLongs[m], kInts[n], kInts[k], kInts[b], kInts[b]);
          EXPECT(moe_lora_int8_gemm(&a, NULL) != MOE_LORA_OK || kLongs[m] == 0);
          a.silu_mul = 1;
          a.sorted_pair_ids = (const int32_t*)fake(6);
          a.num_pairs = kInts[k]; a.top_k = kInts[n]; a.num_tokens = kLongs[m];
          EXPECT(moe_lora_int8_gemm(&a, NULL) != MOE_LORA_OK || kLongs[m] == 0);
          a = gemm_args(kLongs[m], kInts[n], kInts[k], 1, kInts[b]);
          a.tile_expert = NULL;
          EXPECT(moe_lora_int8_gemm(&a, NULL) != MOE_LORA_OK || kLongs[m] == 0);
        }
}

static void check_balance(void) {
  for (int t = 0; t < kNumInts; ++t)
    for (int e = 0; e < kNumInts; ++e) {
      const int32_t T = kInts[t], E = kInts[e];
      const size_t need = moe_lora_balance_loss_workspace_bytes(T, E);
      EXPECT(need < ((size_t)1 << 32));
      for (int k = 0; k < kNumInts; ++k)
        for (int dt = -1; dt < 6; ++dt) {
          EXPECT(moe_lora_balance_loss(T, E, kInts[k], dt, fake(0), (int32_t*)fake(1), NULL, (float*)fake(2),
                                       (int32_t*)fake(3), (float*)fake(4), NULL, fake(5), need, NULL) !=
                 MOE_LORA_OK);   /* num_valid is missing */
          const int st = moe_lora_balance_loss_backward(T, E, kInts[k], dt, dt, fake(0), NULL, (int32_t*)fake(1),
                                                        (int32_t*)fake(2), NULL, NULL, NULL);
          EXPECT(st != MOE_LORA_OK || T == 0);
        }
    }
}

int main(void) {
  check_rows();
  check_gemm();
  check_balance();
  if (failures) {
    fprintf(stderr, "%d host checks failed\n", failures);
    return 1;
  }
  printf("all host checks passed\n");
  return 0;
}

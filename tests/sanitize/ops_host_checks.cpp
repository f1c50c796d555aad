// Host-side checks of the operators around the loss (norm, AdamW, sampling): their argument
// checks, workspace queries and the AdamW plan, built with AddressSanitizer and
// UndefinedBehaviorSanitizer on the host code.  No call reaches a kernel launch.
#include <limits.h>
#include <math.h>
#include <stdint.h>
#include <stdio.h>
#include <stdlib.h>
#include <string.h>

#include "grpo.h"

static int g_fail = 0;
#define CHECK(cond)                                                            \
  do {                                                                         \
    if (!(cond)) {                                                             \
      fprintf(stderr, "%s:%d: check failed: %s\n", __FILE__, __LINE__, #cond); \
      ++g_fail;                                                                \
    }                                                                          \
  } while (0)

static void* const FAKE = (void*)0x1000;   // never dereferenced

static void workspaces() {
  const int64_t sizes[] = {INT64_MIN, -1, 0, 1, 7, 255, 4096, 4097, 16385, 151936, 1 << 20, (1 << 20) + 1,
                           1 << 24, (1 << 24) + 1, INT32_MAX, (int64_t)INT32_MAX + 1, INT64_MAX};
  for (int64_t a : sizes)
    for (int64_t b : sizes) {
      for (int dt = -1; dt <= 3; ++dt) {
        const size_t n = grpo_norm_workspace_bytes(a, b, dt);
        CHECK((n != 0) == (a > 0 && a <= INT32_MAX && b > 0 && b <= (1 << 24) && (dt == 0 || dt == 1)));
      }
      const size_t s = grpo_sample_workspace_bytes(a, b);
      CHECK((s != 0) == (a > 0 && a <= (1 << 20) && b > 0 && b <= (1 << 20)));
      CHECK(s < (size_t)1 << 31);        // rows go in batches
    }
}

static void plans() {
  const int counts[] = {0, 1, 2, 63, 64, 65, 1000};
  for (int count : counts) {
    const size_t need = grpo_adamw_plan_bytes(count);
    // exactly the bytes asked for, so that a write past them is seen
    char* image = (char*)malloc(need);
    grpo_adamw_tensor* t = (grpo_adamw_tensor*)calloc(count + 1, sizeof *t);
    for (int bits = 8; bits <= 32; bits += 24)
      for (int master = 0; master < 2; ++master) {
        for (int i = 0; i < count; ++i) {
          const uintptr_t at = (uintptr_t)(count - i) << 32;     // downwards: the check sorts
          t[i] = grpo_adamw_tensor{(void*)at,
                                   (void*)(at + (1 << 26)),
                                   master ? (float*)(at + (2 << 26)) : nullptr,
                                   (void*)(at + (3 << 26)),
                                   (void*)(at + (4 << 26)),
                                   bits == 8 ? (float*)(at + (5ull << 26)) : nullptr,
                                   bits == 8 ? (float*)(at + (6ull << 26)) : nullptr,
                                   (int64_t)i * 997 % 100003};
        }
        CHECK(grpo_adamw_plan(t, count, GRPO_BF16, GRPO_F32, bits, image, need) == GRPO_OK);
        if (count > 2) {
          const grpo_adamw_tensor keep = t[2];
          t[2].exp_avg = t[1].exp_avg;
          CHECK(grpo_adamw_plan(t, count, GRPO_BF16, GRPO_F32, bits, image, need) == GRPO_ERR_INVALID_ARG);
          t[2] = keep;
          t[2].n = INT64_MAX;
          CHECK(grpo_adamw_plan(t, count, GRPO_BF16, GRPO_F32, bits, image, need) == GRPO_ERR_INVALID_ARG);
          t[2].n = (int64_t)1 << 48;      // 2^36 chunks
          CHECK(grpo_adamw_plan(t, count, GRPO_BF16, GRPO_F32, bits, image, need) != GRPO_OK);
          t[2] = keep;
        }
        CHECK(grpo_adamw_plan(t, count, GRPO_BF16, GRPO_F32, bits, image, need - 1) == GRPO_ERR_WORKSPACE);
      }
    grpo_adamw_opts o{};
    o.beta1 = 0.9;
    o.beta2 = 0.999;
    o.step = 0;
    CHECK(grpo_adamw_plan(t, 0, GRPO_BF16, GRPO_F32, 8, image, need) == GRPO_OK);
    CHECK(grpo_adamw(image, nullptr, &o, nullptr) == GRPO_ERR_INVALID_ARG);
    o.step = INT64_MAX;
    CHECK(grpo_adamw(image, nullptr, &o, nullptr) == GRPO_OK);       // an empty plan launches nothing
    free(image);
    free(t);
  }
  CHECK(grpo_adamw_plan_bytes(INT64_MIN) == 0);
  CHECK(grpo_adamw_plan_bytes(INT64_MAX) == 0);
  CHECK(grpo_moment_values(FAKE, (float*)FAKE, INT64_MAX, 0, (float*)FAKE, nullptr) == GRPO_ERR_UNSUPPORTED);
}

static void rejected_calls() {
  float f = 0.f;
  CHECK(grpo_norm_fwd(FAKE, FAKE, nullptr, INT64_MAX, INT64_MAX, 0, 0, 1e-5f, FAKE, &f, &f, nullptr) ==
        GRPO_ERR_UNSUPPORTED);
  CHECK(grpo_norm_fwd(FAKE, FAKE, nullptr, 4, 4, 0, 0, -1.f, FAKE, &f, &f, nullptr) == GRPO_ERR_INVALID_ARG);
  CHECK(grpo_norm_bwd(FAKE, FAKE, FAKE, nullptr, &f, 4, 4, 0, GRPO_NORM_LAYER, 0, FAKE, &f, &f, FAKE, 1 << 20,
                      nullptr) == GRPO_ERR_INVALID_ARG);
  CHECK(grpo_norm_bwd(FAKE, FAKE, FAKE, &f, &f, INT32_MAX, 1 << 24, 0, GRPO_NORM_RMS, 1, FAKE, &f, &f, FAKE, 0,
                      nullptr) == GRPO_ERR_WORKSPACE);
  int32_t token;
  grpo_sample_opts o{};
  CHECK(grpo_sample(FAKE, 0, 4, 100, INT64_MIN, &f, &o, &token, &f, FAKE, 1 << 20, nullptr) ==
        GRPO_ERR_INVALID_ARG);
  CHECK(grpo_sample(FAKE, 0, INT64_MAX, 100, 100, &f, &o, &token, &f, FAKE, 1 << 20, nullptr) ==
        GRPO_ERR_UNSUPPORTED);
  o.top_k = INT_MIN;
  CHECK(grpo_sample(FAKE, 0, 4, 100, 100, &f, &o, &token, &f, FAKE, 1 << 20, nullptr) == GRPO_ERR_INVALID_ARG);
  o.top_k = 0;
  o.temperature = NAN;
  CHECK(grpo_sample(FAKE, 0, 4, 100, 100, &f, &o, &token, &f, FAKE, 1 << 20, nullptr) == GRPO_ERR_INVALID_ARG);
  CHECK(grpo_sample(FAKE, 0, 4, 100, 100, &f, nullptr, &token, &f, FAKE, 16, nullptr) == GRPO_ERR_WORKSPACE);
}

int main() {
  workspaces();
  plans();
  rejected_calls();
  if (g_fail) {
    fprintf(stderr, "%d check(s) failed\n", g_fail);
    return 1;
  }
  printf("host checks passed\n");
  return 0;
}

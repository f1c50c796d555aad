// Host-side checks of the losses over given log-probabilities and of the gradients' norm: argument
// checks, workspace queries and the gradient plan, built with AddressSanitizer and
// UndefinedBehaviorSanitizer on the host code.  No call reaches a kernel launch.
#include <float.h>
#include <limits.h>
#include <math.h>
#include <stdint.h>
#include <stdio.h>
#include <stdlib.h>

#include "grpo.h"

static int g_fail = 0;
#define CHECK(cond)                                                            \
  do {                                                                         \
    if (!(cond)) {                                                             \
      fprintf(stderr, "%s:%d: check failed: %s\n", __FILE__, __LINE__, #cond); \
      ++g_fail;                                                                \
    }                                                                          \
  } while (0)

static void* const FAKE2 = (void*)0x100000;
static void* const FAKE = (void*)0x1000;   // never dereferenced

static void workspaces() {
  const int64_t sizes[] = {INT64_MIN, -1, 0, 1, 2, 7, 255, 1024, 1025, 4097, 20480, 1 << 20, 1 << 30, (1 << 30) + 1,
                           INT32_MAX, (int64_t)INT32_MAX + 1, (int64_t)1 << 33, INT64_MAX};
  for (int64_t a : sizes)
    for (int64_t b : sizes)
      for (int per = 1; per <= 2; ++per) {
        const size_t n = per == 1 ? grpo_clip_loss_workspace_bytes(a, b) : grpo_pref_loss_workspace_bytes(a, b);
        const bool fits = a > 0 && b > 0 && (__int128)a * b * per <= INT32_MAX;
        CHECK((n != 0) == fits);
        CHECK(n < (size_t)1 << 31);
      }
}

static void plans() {
  const int counts[] = {0, 1, 2, 63, 64, 65, 1000};
  for (int count : counts) {
    const size_t need = grpo_grad_plan_bytes(count);
    // exactly the bytes asked for, so that a write past them is seen
    char* image = (char*)malloc(need);
    grpo_grad_tensor* t = (grpo_grad_tensor*)calloc(count + 1, sizeof *t);
    for (int i = 0; i < count; ++i)   // downwards: the check sorts
      t[i] = grpo_grad_tensor{(void*)((uintptr_t)(count - i) << 32), (int64_t)i * 997 % 100003, i % 2, 0};
    CHECK(grpo_grad_plan(t, count, image, need) == GRPO_OK);
    CHECK(grpo_grad_plan(t, count, image, need - 1) == GRPO_ERR_WORKSPACE);
    if (count > 2) {
      const grpo_grad_tensor keep = t[2];
      t[2].grad = t[1].grad;
      CHECK(grpo_grad_plan(t, count, image, need) == GRPO_ERR_INVALID_ARG);
      t[2] = keep;
      const int64_t bad[] = {-1, INT64_MAX, INT64_MIN, ((int64_t)1 << 48) + 1};
      for (int64_t n : bad) {
        t[2].n = n;
        CHECK(grpo_grad_plan(t, count, image, need) == GRPO_ERR_INVALID_ARG);
      }
      t[2].n = (int64_t)1 << 48;      // 2^35 chunks
      CHECK(grpo_grad_plan(t, count, image, need) == GRPO_ERR_UNSUPPORTED);
    }
    CHECK(grpo_grad_plan(t, 0, image, need) == GRPO_OK);
    CHECK(grpo_grad_clip(image, nullptr, (float*)FAKE, nullptr) == GRPO_OK);
    CHECK(grpo_grad_norm(image, nullptr, 0, NAN, (float*)FAKE, (float*)FAKE, FAKE, 1 << 20, nullptr) ==
          GRPO_ERR_INVALID_ARG);
    free(image);
    free(t);
  }
  CHECK(grpo_grad_plan_bytes(INT64_MIN) == 0);
  CHECK(grpo_grad_plan_bytes(INT64_MAX) == 0);
}

static void rejected_calls() {
  float f = 0.f;
  uint8_t m = 1;
  int32_t y = 0;
  grpo_clip_opts c{};
  CHECK(grpo_clip_loss_fwd(&f, nullptr, nullptr, &m, &f, INT64_MAX, INT64_MAX, &c, &f, &f, &f, FAKE, 1 << 20, nullptr) ==
        GRPO_ERR_UNSUPPORTED);
  c.beta = 1.0;
  CHECK(grpo_clip_loss_fwd(&f, &f, nullptr, &m, &f, 4, 4, &c, &f, &f, &f, FAKE, 1 << 20, nullptr) == GRPO_ERR_INVALID_ARG);
  c.beta = DBL_MAX;
  CHECK(grpo_clip_loss_bwd(&f, &f, &f, &m, &f, &f, nullptr, 4, 4, &c, &f, nullptr) == GRPO_ERR_INVALID_ARG);
  CHECK(grpo_clip_loss_bwd(&f, &f, &f, &m, &f, &f, nullptr, INT64_MIN, 4, nullptr, &f, nullptr) == GRPO_ERR_INVALID_ARG);
  grpo_pref_opts p{};
  CHECK(grpo_pref_loss_fwd(&f, &f, &m, 4, 4, &p, &f, &f, &f, FAKE, 1 << 20, nullptr) == GRPO_ERR_INVALID_ARG);
  p.beta = 0.1;
  CHECK(grpo_pref_loss_fwd(&f, &f, &m, INT64_MAX, INT64_MAX, &p, &f, &f, &f, FAKE, 1 << 20, nullptr) ==
        GRPO_ERR_UNSUPPORTED);
  CHECK(grpo_pref_loss_fwd(&f, &f, &m, 4, 4, &p, &f, &f, &f, FAKE, 0, nullptr) == GRPO_ERR_WORKSPACE);
  CHECK(grpo_pref_loss_bwd(&m, &f, nullptr, INT64_MAX, 1, &f, nullptr) == GRPO_ERR_UNSUPPORTED);
  CHECK(grpo_logprobs_fwd(FAKE, FAKE, &y, INT64_MAX, 16, 32, GRPO_BF16, 8, nullptr, &f, &f, FAKE, 1 << 20, nullptr) ==
        GRPO_ERR_UNSUPPORTED);
  CHECK(grpo_logprobs_bwd(FAKE, FAKE, &y, &f, &f, &f, 8, 16, 32, GRPO_BF16, 8, nullptr, 0, GRPO_F32, FAKE2, nullptr, FAKE, 64,
                          nullptr) == GRPO_ERR_WORKSPACE);
  CHECK(grpo_logprobs_bwd(FAKE, FAKE, &y, &f, &f, &f, 8, 16, 32, GRPO_BF16, 8, nullptr, 0, GRPO_F32, nullptr, FAKE, FAKE, 1 << 30,
                          nullptr) == GRPO_ERR_INVALID_ARG);
  CHECK(grpo_logprobs_bwd(FAKE, FAKE, &y, &f, &f, &f, 8, 16, 32, GRPO_FP8_E4M3, 8, nullptr, 0, GRPO_F32, FAKE, &f, FAKE,
                          1 << 20, nullptr) == GRPO_ERR_INVALID_ARG);
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

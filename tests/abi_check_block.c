/*
 * Host-side checks of the operators around the long convolution, compiled as C and
 * linked against the library's host code built with AddressSanitizer and
 * UndefinedBehaviorSanitizer (any finding aborts): the size queries over boundary
 * and extreme arguments against the ranges the header states. Nothing here
 * reaches the GPU.
 */
#include <limits.h>
#include <stdio.h>

#include "hyena.h"

static int failures = 0;

static void expect(int got, int want, const char *what, long long a, long long b, long long c, long long d) {
  if (got != want) {
    fprintf(stderr, "%s(%lld, %lld, %lld, %lld): %d, expected %d\n", what, a, b, c, d, got, want);
    ++failures;
  }
}

static const int kSizes[] = {INT_MIN, -64, -1, 0, 1, 2, 7, 8, 12, 64, 72, 1000, 4096, 8192, 8200, 1 << 16, (1 << 16) + 8,
                             1 << 20, (1 << 20) + 1, 1 << 24, (1 << 24) + 8, INT_MAX - 7, INT_MAX};
#define N ((int)(sizeof(kSizes) / sizeof(kSizes[0])))

static int in(long long x, long long lo, long long hi) { return x >= lo && x <= hi; }

int main(void) {
  for (int i = 0; i < N; ++i)
    for (int j = 0; j < N; ++j)
      for (int k = 0; k < N; ++k) {
        const long long a = kSizes[i], b = kSizes[j], c = kSizes[k];
        for (int dt = -1; dt <= 2; ++dt) {
          const int dt_ok = dt == 0 || dt == 1;
          /* B, L, D (the product of two 2^24 and one 2^16 stays below 2^64) */
          const int glr = dt_ok && in(a, 1, 1 << 20) && in(b, 1, 1 << 24) && in(c, 8, 1 << 16) && c % 8 == 0 &&
                          a * c < (1LL << 31) && a * c <= ((1LL << 40) - 1) / b;
          expect(hyena_glr_workspace_bytes((int)a, (int)b, (int)c, dt) > 0, glr, "glr", a, b, c, dt);
          expect(hyena_glr_bwd_workspace_bytes((int)a, (int)b, (int)c, dt) > 0, glr, "glr_bwd", a, b, c, dt);
          /* M, D, F */
          const int ffn = dt_ok && in(a, 1, 1 << 24) && in(b, 8, 1 << 16) && b % 8 == 0 && in(c, 8, 1 << 16) && c % 8 == 0;
          expect(hyena_ffn_workspace_bytes((int)a, (int)b, (int)c, dt) > 0, ffn, "ffn", a, b, c, dt);
          expect(hyena_ffn_bwd_workspace_bytes((int)a, (int)b, (int)c, dt) > 0, ffn, "ffn_bwd", a, b, c, dt);
          /* B, S, C; every size as G */
          for (int l = 0; l < N; ++l) {
            const long long g = kSizes[l];
            const int gn = dt_ok && in(a, 1, 1 << 24) && in(b, 1, 1 << 24) && in(c, 8, 8192) && c % 8 == 0 && in(g, 1, c) &&
                           c % (g > 0 ? g : 1) == 0 && a * c < (1LL << 31) && a * c <= ((1LL << 40) - 1) / b;
            expect(hyena_group_norm_workspace_bytes((int)a, (int)b, (int)c, (int)g, dt) > 0, gn, "group_norm", a, b, c, g);
            expect(hyena_group_norm_bwd_workspace_bytes((int)a, (int)b, (int)c, (int)g, dt) > 0, gn, "group_norm_bwd", a, b,
                   c, g);
          }
        }
      }
  if (failures) {
    fprintf(stderr, "%d expectation(s) failed\n", failures);
    return 1;
  }
  printf("abi_check_block: all expectations hold\n");
  return 0;
}

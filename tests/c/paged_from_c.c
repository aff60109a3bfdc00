/* A plain C99 caller of attn_paged.h: the host functions and calls that are
 * refused before any GPU work.  Exits nonzero if a check fails. */
#include <math.h>
#include <stdint.h>
#include <stdio.h>
#include <string.h>

#include "attn_paged.h"

static int fails = 0;

static void expect(const char* what, attn_status got, attn_status want) {
  if (got != want) {
    printf("%s: got %d (%s), want %d\n", what, (int)got, attn_status_string(got), (int)want);
    ++fails;
  }
}

int main(void) {
  attn_rope_freq f;
  double w[4];
  uint64_t steps[4];
  memset(&f, 0, sizeof f);
  f.rot_dim = 8;
  f.base = 16.0;
  expect("frequencies", attn_rope_freqs(&f, w), ATTN_OK);
  if (fabs(w[1] - 0.5) > 1e-15 || fabs(w[3] - 0.125) > 1e-15) {
    printf("frequencies: %g %g\n", w[1], w[3]);
    ++fails;
  }
  expect("steps", attn_rope_steps(w, 4, steps), ATTN_OK);
  if (fabs((double)steps[0] / 18446744073709551616.0 - 0.15915494309189535) > 1e-15) ++fails;
  f.scaling = ATTN_ROPE_SCALE_BY_PARTS;
  f.factor = 2.0;
  expect("by parts without a length", attn_rope_freqs(&f, w), ATTN_ERR_INVALID_ARG);

  attn_paged_cache c;
  memset(&c, 0, sizeof c);
  c.page_size = 16;
  c.Hkv = 1;
  c.Dqk = c.Dv = 96;
  expect("head dim 96", attn_paged_decode(&c, 0, NULL, NULL, NAN, NULL, NULL, NULL, 0, NULL), ATTN_ERR_UNSUPPORTED);
  c.Dqk = c.Dv = 64;
  expect("no sequences", attn_paged_decode(&c, 0, NULL, NULL, NAN, NULL, NULL, NULL, 0, NULL), ATTN_OK);
  expect("no new tokens", attn_paged_append(&c, NULL, NULL, NULL), ATTN_ERR_INVALID_ARG);
  expect("rotation of nothing given", attn_rope(1, 1, 64, NULL, NULL, 1, NULL, NULL, NULL, 0, 0, NULL),
         ATTN_ERR_INVALID_ARG);
  if (strcmp(attn_status_string(ATTN_ERR_PAGE), "unknown status") == 0) ++fails;
  printf("%d\n", fails);
  return fails != 0;
}

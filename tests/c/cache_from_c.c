/* A plain C99 caller of attn_cache.h: calls that are empty or refused before
 * any GPU work.  Exits nonzero if a check fails. */
#include <math.h>
#include <stdio.h>
#include <string.h>

#include "attn_cache.h"

static int fails = 0;

static void expect(const char* what, attn_status got, attn_status want) {
  if (got != want) {
    printf("%s: got %d (%s), want %d\n", what, (int)got, attn_status_string(got), (int)want);
    ++fails;
  }
}

int main(void) {
  attn_paged_cache4 c;
  attn_paged_cache d;
  attn_paged_weight w;
  attn_paged_eviction e;
  memset(&c, 0, sizeof c);
  memset(&d, 0, sizeof d);
  memset(&w, 0, sizeof w);
  memset(&e, 0, sizeof e);
  c.page_size = d.page_size = 16;
  c.Hkv = d.Hkv = 1;
  c.Dqk = c.Dv = d.Dqk = d.Dv = 96;
  expect("head dim 96", attn_paged_decode4(&c, 0, NULL, NULL, NAN, NULL, NULL, NULL, 0, NULL), ATTN_ERR_UNSUPPORTED);
  c.Dqk = c.Dv = d.Dqk = d.Dv = 64;
  expect("no sequences", attn_paged_decode4_f16(&c, 0, NULL, NULL, NAN, NULL, NULL, NULL, 0, NULL), ATTN_OK);
  expect("no new tokens", attn_paged_append4(&c, NULL, NULL, NULL), ATTN_ERR_INVALID_ARG);
  expect("nothing to gather", attn_paged_gather4(&c, 0, NULL, NULL, NULL, NULL, NULL, NULL), ATTN_OK);
  expect("nothing to gather", attn_paged_gather(&d, 0, NULL, NULL, NULL, NULL, NULL, NULL), ATTN_OK);
  expect("weights of nothing", attn_paged_weights(&d, 0, NULL, NULL, NAN, &w, NULL), ATTN_OK);
  w.decay = 2.0f;
  expect("decay 2", attn_paged_weights4(&c, 0, NULL, NULL, NAN, &w, NULL), ATTN_ERR_INVALID_ARG);
  expect("eviction from nothing", attn_paged_evict4(&c, &e, NULL, 0, NULL), ATTN_OK);
  e.sinks = -1;
  expect("sinks -1", attn_paged_evict(&d, &e, NULL, 0, NULL), ATTN_ERR_INVALID_ARG);
  if (attn_paged_evict_workspace(2, 3, 4, 5) != 2 * 3 * 4 * 5 * 8) ++fails;
  if (attn_paged_decode4_workspace(NULL, 1) != 0) ++fails;
  printf("%d\n", fails);
  return fails != 0;
}

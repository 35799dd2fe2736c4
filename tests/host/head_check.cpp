// The deal of dX's tiles to workgroups, as k_head_dx walks it: every step of
// every tile exactly once, parts in places of their own inside the workspace,
// every part that the join reads written; and the workspace layouts.
#include <algorithm>
#include <cstdio>
#include <set>
#include <vector>

#include "head_plan.h"

using namespace qn;

static int fail(const char* what, int a, int b, int c) {
  std::printf("%s: wgs %d tiles %d steps %d\n", what, a, b, c);
  return 1;
}

static int check_deal(int wgs, int tiles, int steps) {
  const HeadDeal d = head_deal(wgs, tiles, steps);
  std::vector<int> seen((size_t)tiles * steps, 0);
  std::set<int> slots;
  const int whole = tiles / wgs, per = wgs / 8;
  int64_t most = 0;
  for (int b = 0; b < wgs; ++b) {
    const int xcd = b & 7, in = b >> 3;
    const int h0 = d.rest * xcd / 8, h1 = d.rest * (xcd + 1) / 8;
    const bool is_head = in < h1 - h0;
    const int e = xcd * per - h0 + in - (h1 - h0);
    int64_t at = 0, end = 0, work = 0;
    if (d.extra > 0 && !is_head && e < d.extra) {
      if (e < 0) return fail("extra", wgs, tiles, steps);
      at = head_tail_first(d, e);
      end = head_tail_first(d, e + 1);
    }
    for (int seg = 0;; ++seg) {
      int tile, s0 = 0, s1 = d.steps, slot = -1;
      if (seg < whole) {
        tile = seg * wgs + xcd * per + in;
      } else if (is_head) {
        if (seg > whole) break;
        tile = whole * wgs + h0 + in;
        s1 = d.head;
        if (d.extra > 0) slot = h0 + in;
      } else {
        if (at >= end) break;
        const int tail = d.steps - d.head, t = (int)(at / tail);
        s0 = d.head + (int)(at - (int64_t)t * tail);
        s1 = (int)std::min<int64_t>(d.steps, s0 + (end - at));
        at += s1 - s0;
        tile = whole * wgs + t;
        slot = d.rest + t + e;
        if (e < head_tail_owner(d, (int64_t)t * tail) ||
            e > head_tail_owner(d, (int64_t)(t + 1) * tail - 1))
          return fail("owner", wgs, tiles, steps);
      }
      if (slot >= 0 && (!slots.insert(slot).second || slot >= head_parts(d) || slot >= 2 * wgs))
        return fail("slot", wgs, tiles, steps);
      if (tile >= tiles || s1 <= s0) return fail("tile", wgs, tiles, steps);
      for (int s = s0; s < s1; ++s) seen[(size_t)tile * steps + s]++;
      work += s1 - s0;
    }
    most = std::max(most, work);
  }
  for (int v : seen)
    if (v != 1) return fail("step", wgs, tiles, steps);
  if (d.extra > 0) {
    const int tail = d.steps - d.head;
    for (int t = 0; t < d.rest; ++t) {
      if (slots.count(t) == 0) return fail("head", wgs, tiles, steps);
      for (int e = head_tail_owner(d, (int64_t)t * tail);
           e <= head_tail_owner(d, (int64_t)(t + 1) * tail - 1); ++e)
        if (slots.count(d.rest + t + e) == 0) return fail("part", wgs, tiles, steps);
    }
    // nobody has more than its share, 10/8 of it where tails are kept in step, or the
    // smallest part
    const int64_t share = cdiv((int64_t)d.rest * steps, wgs);
    if (most > (int64_t)whole * steps +
                   std::max<int64_t>(2 * HEAD_PART, d.each > 0 ? share * 10 / 8 + 2 : share))
      return fail("share", wgs, tiles, steps);
    if (d.extra > wgs - d.rest) return fail("extra", wgs, tiles, steps);
  }
  return 0;
}

int main() {
  for (int wgs : {256, 512})
    for (int tiles : {0, 1, 2, 7, 8, 31, 32, 100, 128, 176, 200, 204, 205, 255, 256, 257, 300, 409,
                      410, 432, 511, 512, 513, 700})
      for (int steps : {1, 2, 8, 9, 16, 31, 64, 100, 500, 2004})
        if (check_deal(wgs, tiles, steps)) return 1;
  for (int64_t rows : {0, 1, 32, 33, 129, 300, 4096, 100000})
    for (int64_t dim : {8, 64, 1000, 8192})
      for (int64_t vocab : {1, 255, 257, 32000, 128256, 1 << 20}) {
        const HeadFwdPlan f = head_fwd_plan(rows, dim, vocab);
        if (f.slices * HEAD_SLICE < vocab || f.mp < rows || f.total < f.sums) return 1;
        for (int need = 1; need < 4; ++need) {
          const HeadBwdPlan b = head_bwd_plan(rows, dim, vocab, need & 1, need & 2);
          // the pieces cover the vocabulary, and none is empty
          if (b.vp % 256 != 0 || b.pieces * b.vp < vocab || (b.pieces - 1) * b.vp >= vocab) return 1;
          if (b.g + size_t(b.mp) * b.vp * 2 > b.xs || b.total < b.part) return 1;
          // byte offsets inside a block of G and a step of the weight fit 31 bits
          if (b.vp * 256 * 2 > (int64_t(1) << 31) || dim * 256 * 2 > (int64_t(1) << 31)) return 1;
        }
      }
  std::puts("ok");
  return 0;
}

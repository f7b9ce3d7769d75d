// attend_plan.cuh -- how the dense attention's work is cut into one equal share per CTA.
//
// A unit is a request (prompts), or a group's shared prefix, or what a request has of its own
// (shared prefixes).  For each KV head it has one item per kTile * 2 query rows, and an item is
// the pass of its rows over its keys in tiles of kKeys.  All items stand in one line, a unit's
// heads one after the other and a head's items in order, each as long as its cost; CTA c of n
// takes the c-th of n equal lengths of the line.  A cut inside an item falls on the nearest key
// tile and both neighbours compute it alike, so every tile has one owner, every CTA ends within
// a tile's cost of the others, and a CTA has at most one item that began before it.
//
// What a single token attends to by itself (a decode row's own pages) is too little work for a
// row tile and bound by the bytes of its keys: it stands in a second line, in pages, that is cut
// into one share per warp.  The CTAs are dealt between the two lines by their lengths.
#pragma once

#include <stdint.h>

namespace vt {

constexpr int kTile = 128;  // query rows of one accumulator tile; an item has two
constexpr int kKeys = 128;  // keys of one step

// Costs, in keys times what a key costs, which is the same for an item of one row tile and one of
// two.  A step of 128 keys takes ~3200 cycles with two and 2400-2900 with one, by a fit over whole
// calls: nothing runs beside the chain of a single tile.  Yet shares cut with 3/4 of the cost for
// one tile are the slower ones (387 us with equal costs, 393 so for the packed prompts, 908 and 934
// for the chunks, 193 and 201 for the prefix groups, 519 and 553 for the document; cold inputs).
constexpr int kCostKey = 4;
constexpr int kCostItem = 256;      // loading q, filling the pipeline, writing out: two steps
constexpr int64_t kMinShare = 4 * kKeys * kCostKey;  // no CTA takes less than four key tiles

// The second line: pages of a request's own, for each KV head, and what an item of them costs
// beyond (its query, its result).
constexpr int kWarps = 12;        // of a CTA, each with a share
constexpr int kOwnItem = 2;       // pages
constexpr int kMinPages = 4;      // no warp takes less
// A page of one head in the costs of the first line: one value for every shape.  Measured (us, cold
// inputs) with 20 / 30 / 45 / 60 / 80, at 128 dims: 128 requests on five prefixes of 12800 tokens
// with 100-4096 own, 32/8 heads 223 / 207 / 221 / 248 / 291; 256 on one of 65536 with 17-300 own,
// 32/8 heads 406 / 306 / 315 / 315 / 315, 48/8 heads 604 / 512 / 459 / 494 / 495, 64/8 heads
// 834 / 603 / 585 / 575 / 588.  At 64 dims, where a step costs nearly as much and a page half, the
// best is lower: the five prefixes 141 / 156 / 180 / 208 / 248 (32/8 heads), the document
// 403 / 408 / 410 / 420 / 426 (48/8).
constexpr int kOwnPage = 45;

struct Unit {
  int tok0, n;     // its query tokens (0: no items)
  int vis0;        // keys that the first token sees; each further one sees `step` more
  int step;        // 1: causal, 0: all see all
  int kv_len;      // keys there are, from page `page0` of table row `row`
  int page0, row;
  bool bad;        // a bad length: no keys, empty rows
};

#define VT_HD __host__ __device__ __forceinline__

// A decode row's own pages, and the cost of one head's item of them in the second line.
VT_HD int own_pages(const Unit& u) { return (u.kv_len + 15) / 16; }
VT_HD int64_t own_cost(const Unit& u) { return u.kv_len > 0 ? own_pages(u) + kOwnItem : 0; }
VT_HD int own_cut(int64_t x, int pages) { return x <= 0 ? 0 : x < pages ? (int)x : pages; }

// Items of one head; tpt: tokens of a row tile.
VT_HD int unit_items(const Unit& u, int tpt) { return (u.n + 2 * tpt - 1) / (2 * tpt); }

// Keys that item t has to look at.
VT_HD int item_keys(const Unit& u, int tpt, int t) {
  if (!u.step) return u.vis0;
  const int last = (t + 1) * 2 * tpt;
  return u.vis0 + (last < u.n ? last : u.n) - 1;
}

// What a key costs in item t.
VT_HD int item_weight(const Unit&, int, int) { return kCostKey; }

VT_HD int64_t item_cost(const Unit& u, int tpt, int t) {
  return (int64_t)item_weight(u, tpt, t) * (kCostItem + item_keys(u, tpt, t));
}

// Cost of a head's items before t <= unit_items; all but the last item have two full tiles.
VT_HD int64_t cost_before(const Unit& u, int tpt, int t) {
  const int n = unit_items(u, tpt);
  if (t <= 0) return 0;
  const int64_t f = t < n ? t : n - 1;
  int64_t keys = f * u.vis0;
  if (u.step) keys += 2 * (int64_t)tpt * (f * (f + 1) / 2) - f;
  const int64_t c = kCostKey * (f * kCostItem + keys);
  return t < n ? c : c + item_cost(u, tpt, n - 1);
}

// Key tiles before cost x of an item.
VT_HD int cut_tile(int64_t x, int64_t cost, int weight, int n_tiles) {
  if (x <= 0) return 0;
  if (x >= cost) return n_tiles;
  const int64_t t = (x / weight + kKeys / 2) / kKeys;
  return t < n_tiles ? (int)t : n_tiles;
}

// The CTA from which on the second line is worked on; `tiles` and `pages`: the lines' lengths.
VT_HD int first_own(int64_t tiles, int64_t pages, int ctas) {
  if (pages == 0) return ctas;
  if (tiles == 0) return 0;
  const double own = (double)pages * kOwnPage;
  const int n = (int)(own / ((double)tiles + own) * ctas + 0.5);
  return ctas - (n < 1 ? 1 : n > ctas - 1 ? ctas - 1 : n);
}

// Those (of `most`) that share a line of length `total`, no share less than `least`.
VT_HD int share_count(int64_t total, int most, int64_t least) {
  const int64_t n = total / least;
  return n < 1 ? 1 : n < most ? (int)n : most;
}
// A line and its n equal shares; the c-th begins at floor(total c / n).
struct Line {
  int64_t total, base;  // base = total / n
  double inv;           // n / total
  int n, rem;           // rem = total % n
};
VT_HD Line make_line(int64_t total, int most, int64_t least) {
  Line x;
  x.total = total;
  x.n = share_count(total, most, least);
  x.base = total / x.n;
  x.rem = (int)(total - x.base * x.n);
  x.inv = total > 0 ? (double)x.n / (double)total : 0.0;
  return x;
}
// (rem c < n^2, and n is at most 12 per SM: far inside 32 bits)
VT_HD int64_t share_begin(const Line& x, int c) {
  return x.base * c + (unsigned)x.rem * (unsigned)c / (unsigned)x.n;
}
// The share that position x < total is in.
VT_HD int share_of(const Line& x, int64_t pos) {
  int c = (int)((double)pos * x.inv);
  c = c < 0 ? 0 : c >= x.n ? x.n - 1 : c;
  while (c > 0 && share_begin(x, c) > pos) --c;
  while (c + 1 < x.n && share_begin(x, c + 1) <= pos) ++c;
  return c;
}

}  // namespace vt

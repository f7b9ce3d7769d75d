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
// There are two such lines, and the CTAs are dealt between them by their lengths.  Units of one
// row tile (decode, drafted tokens, a prefix that few share) read their keys once for few rows:
// they are bound by bytes, what they need is many of those in flight, and nearly all shared memory
// of their CTAs goes to them.  All others need room for two tiles of queries and for results.
#pragma once

#include <stdint.h>

namespace vt {

constexpr int kTile = 128;  // query rows of one accumulator tile; an item has two
constexpr int kKeys = 128;  // keys of one step

// Costs, in keys times a weight.  An item of one row tile takes less than one of two, but not
// half: its keys are loaded all the same.
constexpr int kCostTwo = 4, kCostOne = 3, kCostNarrow = 3;
constexpr int kCostItem = 256;      // loading q, filling the pipeline, writing out
constexpr int kCostItemNarrow = 128;
constexpr int64_t kMinShare = 4 * kKeys * kCostTwo;  // no CTA takes less than four key tiles

struct Unit {
  int tok0, n;     // its query tokens (0: no items)
  int vis0;        // keys that the first token sees; each further one sees `step` more
  int step;        // 1: causal, 0: all see all
  int kv_len;      // keys there are, from page `page0` of table row `row`
  int page0, row;
  bool bad;        // a bad length: no keys, empty rows
  bool narrow;
};

#define VT_HD __host__ __device__ __forceinline__

// Items of one head; tpt: tokens of a row tile.
VT_HD int unit_items(const Unit& u, int tpt) { return (u.n + 2 * tpt - 1) / (2 * tpt); }

// Keys that item t has to look at.
VT_HD int item_keys(const Unit& u, int tpt, int t) {
  if (!u.step) return u.vis0;
  const int last = (t + 1) * 2 * tpt;
  return u.vis0 + (last < u.n ? last : u.n) - 1;
}

VT_HD int item_weight(const Unit& u, int tpt, int t) {
  return u.narrow ? kCostNarrow : u.n - t * 2 * tpt > tpt ? kCostTwo : kCostOne;
}

VT_HD int64_t item_cost(const Unit& u, int tpt, int t) {
  return (int64_t)item_weight(u, tpt, t) *
         ((u.narrow ? kCostItemNarrow : kCostItem) + item_keys(u, tpt, t));
}

// Cost of a head's items before t <= unit_items; all but the last item have two full tiles.
VT_HD int64_t cost_before(const Unit& u, int tpt, int t) {
  const int n = unit_items(u, tpt);
  if (t <= 0) return 0;
  const int64_t f = t < n ? t : n - 1;
  int64_t keys = f * u.vis0;
  if (u.step) keys += 2 * (int64_t)tpt * (f * (f + 1) / 2) - f;
  const int64_t c = kCostTwo * (f * kCostItem + keys);
  return t < n ? c : c + item_cost(u, tpt, n - 1);
}

// Key tiles before cost x of an item.
VT_HD int cut_tile(int64_t x, int64_t cost, int weight, int n_tiles) {
  if (x <= 0) return 0;
  if (x >= cost) return n_tiles;
  const int64_t t = (x / weight + kKeys / 2) / kKeys;
  return t < n_tiles ? (int)t : n_tiles;
}

// The CTAs from which on the narrow line is worked on.
VT_HD int first_narrow(int64_t wide, int64_t narrow, int ctas) {
  if (narrow == 0) return ctas;
  if (wide == 0) return 0;
  const int n = (int)((double)narrow / (double)(wide + narrow) * ctas + 0.5);
  return ctas - (n < 1 ? 1 : n > ctas - 1 ? ctas - 1 : n);
}

// CTAs that share a line of length `total`, and where the c-th share begins.
VT_HD int share_count(int64_t total, int ctas) {
  const int64_t n = total / kMinShare;
  return n < 1 ? 1 : n < ctas ? (int)n : ctas;
}
VT_HD int64_t share_begin(int64_t total, int n, int c) {
  return total / n * c + total % n * c / n;
}
// The share that position x < total is in.
VT_HD int share_of(int64_t total, int n, int64_t x) {
  int c = (int)((double)x / (double)total * n);
  c = c < 0 ? 0 : c >= n ? n - 1 : c;
  while (c > 0 && share_begin(total, n, c) > x) --c;
  while (c + 1 < n && share_begin(total, n, c + 1) <= x) ++c;
  return c;
}

}  // namespace vt

// How the decode kernels over the 8-bit and the 4-bit pool lay units over CTAs, and the
// checks of their calls' arguments: host side.  (Times are the 8-bit kernel's.)
#pragma once

#include <algorithm>
#include <cstring>
#include <vector>

#include "common.h"
#include "split_units.cuh"
#include "unit_walk.cuh"

namespace pa {
namespace split {

// What a kernel's CTAs and units cost, in pages.
struct Rules {
  int segment_charge;     // charged per unit start
  int whole_pages;        // units this short are not split while SMs are idle
  int min_pages;          // per CTA at least, where units are split
  int long_pages;         // a launch of this many per SM runs on long_grid_pct of the SMs
  int long_grid_pct;
  int two_parts_pages;    // worth what a CTA loses with parts of two units
  int whole_extra_pages;  // beyond an equal share, for units kept whole
  int unit_charge;        // that a whole unit costs beside its own
  int snap_pages;         // how far a CTA's end moves to a unit's border
};

// For units of one length, a grid (at least 80% of `grid`) that divides them, or
// that they divide: no CTA has parts of two units.  0 if there is none.
inline int even_grid(int count, int grid) {
  for (int g = grid; g * 5 >= grid * 4; --g)
    if (count % g == 0 || g % count == 0) return g;
  return 0;
}

// Pages that each CTA has at most if no CTA takes parts of two units (the fewest
// for which the units' CTAs fit the grid), or 0 where that is more than
// two_parts_pages above an equal share.  A CTA with a part of a split unit before
// another segment is ~5 us behind the others: a table row, q, an arrival and its
// fence lie between the two.  (Against equal shares: 7 ragged requests in 5 tiles
// 24.9 -> 23.6 us, 20,000 tokens in 3 tiles 15.7 -> 14.5, 9,000 and 800 tokens 12.3
// -> 10.5, 3 x 54,748 in 4 tiles unchanged; 200 KB or 300 KB did as well but for 12
// x 9,000 in 3 tiles, 26.0 -> 25.4.)
inline int pages_alone(const int32_t* pages, size_t n, long long sum, int count, int grid,
                       const Rules& rules) {
  if (count > grid) return 0;
  auto fits = [&](long long most) {
    long long ctas = 0;
    for (size_t i = 0; i < n; ++i) ctas += (pages[i] + most - 1) / most;
    return ctas <= grid;
  };
  long long lo = (sum + grid - 1) / grid, hi = sum / grid + rules.two_parts_pages;
  if (!fits(hi)) return 0;
  while (lo < hi) {
    const long long mid = (lo + hi) / 2;
    if (fits(mid)) hi = mid;
    else lo = mid + 1;
  }
  return (int)lo;
}

// Cuts a launch's units into CTAs.  A unit on one CTA costs a step per two
// pages (0.5-0.65 us); a unit on several costs partials and their merge, about
// 2 us more.
inline void cut_pages(const Unit* units, const int32_t* pages, size_t n, long long total, int sms,
                      int heads, const Rules& rules, std::vector<int32_t>* starts) {
  int count = 0, most = 0, least = 1 << 30;   // units with pages
  long long sum = 0;
  for (size_t i = 0; i < n; ++i) {
    if (pages[i] == 0) continue;
    ++count;
    sum += pages[i];
    most = std::max(most, pages[i]);
    least = std::min(least, pages[i]);
  }
  starts->reserve(sms + 1);
  if (count == 0) {
    starts->assign({0, 1});
    return;
  }
  if (count <= sms && most <= rules.whole_pages) {
    for (size_t i = 0; i < n; ++i)
      if (pages[i] != 0) starts->push_back(starts->empty() ? 0 : units[i].page_first);
    starts->push_back(static_cast<int32_t>(total));
    return;
  }
  int grid = sum >= (long long)rules.long_pages * sms
                 ? sms * rules.long_grid_pct / 100
                 : (int)std::min<long long>(sms, sum / rules.min_pages);
  grid = std::max(grid, 1);
  // As the bf16 kernel's: the CTAs at the same offset of each kv head's block
  // of units stream the same pages at the same time.
  if (grid >= heads) grid -= grid % heads;
  const int alone = most == least ? 0 : pages_alone(pages, n, sum, count, grid, rules);
  if (alone > 0) {
    for (size_t i = 0; i < n; ++i) {
      const int parts = (pages[i] + alone - 1) / alone;
      for (int k = 0; k < parts; ++k)
        starts->push_back(starts->empty() ? 0 : units[i].page_first +
                                                    (int)((long long)pages[i] * k / parts));
    }
    starts->push_back(static_cast<int32_t>(total));
    return;
  }
  if (const int even = most == least ? even_grid(count, grid) : 0) grid = even;
  starts->push_back(0);
  int at = 0;
  size_t i = 0;
  for (int k = 1; k < grid; ++k) {
    int to = at + ((int)total - at) / (grid - k + 1);
    // the unit that holds the border, if one does
    while (i < n && (pages[i] == 0 || units[i].page_first + pages[i] <= to)) ++i;
    if (i < n && to > units[i].page_first) {
      const int lo = units[i].page_first, hi = lo + pages[i];
      if (to - lo <= rules.snap_pages && to - lo <= hi - to && lo > at) to = lo;
      else if (hi - to <= rules.snap_pages) to = hi;
    }
    if (to <= at) continue;
    starts->push_back(to);
    at = to;
  }
  if (total > at) starts->push_back(static_cast<int32_t>(total));
}

// Adds CTAs that have no pages where units without pages (padded requests, tiles
// behind a request's end) outnumber the CTAs: those are dealt out to all CTAs, a
// warp each (4 requests of 700 tokens and 252 without any: 8.1 us, 24.8 without
// these CTAs; 1 and 63: 7.6, 21.2).
inline void deal_empty(size_t empty, int sms, std::vector<int32_t>* starts) {
  const size_t ctas = std::min<size_t>(sms, empty);
  if (starts->size() < ctas + 1) starts->resize(ctas + 1, starts->back());
}

inline void cut(const Unit* units, const int32_t* pages, size_t n, long long total, int sms,
                int heads, const Rules& rules, std::vector<int32_t>* starts) {
  cut_pages(units, pages, n, total, sms, heads, rules, starts);
  deal_empty(std::count(pages, pages + n, 0), sms, starts);
}

// Lays a launch's units out anew so that every CTA has whole ones, the longest
// first dealt to the CTA with the least, where that comes within whole_extra_pages
// of equal shares: no unit is split, and nothing merged.  A CTA takes its
// shortest first, so that launches end in long streams.  (Shortest / longest
// first, and equal shares: 64 requests of up to 2,500 tokens 32.9 / 33.6 / 35.6
// us, at 256 dims 29.8 / 29.7 / 33.5, 256 of up to 600 33.9 / 37.6 / 37.1, 120 of
// up to 2,000 with 2 kv heads 14.5 / 14.9 / 19.3.  Giving each kv head CTAs of its
// own, which then read the same pages at the same time, made no difference; with
// 400 KB for the pages beyond a share 42 of up to 4,000 took 34.4 us instead of 32.0, with 3.2
// MB nothing changed.)
// Linear in the units: a sort by counting, and CTAs kept in lists by their load
// (the least load only grows).  Returns the order of the units that have pages, or
// nothing if they stay as they are.
inline std::vector<int> pack(Plan* plan, Launch* L, int sms, const Rules& rules) {
  const int32_t* pages = plan->pages.data() + L->u0;
  Unit* units = plan->units.data() + L->u0;
  const int n = (int)L->n;
  long long sum = 0;
  int count = 0, most = 0, least = 1 << 30;   // units with pages
  for (int i = 0; i < n; ++i) {
    if (pages[i] == 0) continue;
    ++count;
    sum += pages[i];
    most = std::max(most, pages[i]);
    least = std::min(least, pages[i]);
  }
  const int grid = sum >= (long long)rules.long_pages * sms ? sms * rules.long_grid_pct / 100 : sms;
  if (count <= grid) return {};
  // (Units of one length stay in an even grid: 64 x 2,048 tokens 42.9 us, 43.9 dealt
  // out; 180 x 1,000 60.5 and 62.4.  Without one, 50 x 1,000 23.4 and 22.5.)
  if (most == least && even_grid(count, grid)) return {};
  // Loads are pages and a few more per unit.
  const long long limit =
      (sum + (long long)rules.unit_charge * count) / grid + rules.whole_extra_pages;
  if (most + rules.unit_charge > limit || limit > 1 << 20) return {};
  // Units by their pages, and CTAs by their loads: heads of lists.
  std::vector<int> of_pages(most + 1, -1), of_load(limit + 1, -1), next_unit(n), next_cta(grid),
      first(grid, -1);
  for (int i = n - 1; i >= 0; --i) {
    next_unit[i] = of_pages[pages[i]];
    of_pages[pages[i]] = i;
  }
  for (int k = 0; k < grid; ++k) next_cta[k] = k + 1 < grid ? k + 1 : -1;
  of_load[0] = 0;
  int load = 0;
  for (int p = most; p > 0; --p) {
    for (int i = of_pages[p]; i >= 0;) {
      while (of_load[load] < 0) ++load;
      const int k = of_load[load], to = load + p + rules.unit_charge, next = next_unit[i];
      if (to > limit) return {};
      of_load[load] = next_cta[k];
      next_cta[k] = of_load[to];
      of_load[to] = k;
      next_unit[i] = first[k];   // the CTA's last comes first
      first[k] = i;
      i = next;
    }
  }
  std::vector<int> order;
  order.reserve(count);
  L->starts.clear();
  int32_t at = 0;
  for (int k = 0; k < grid; ++k) {
    L->starts.push_back(at);
    for (int i = first[k]; i >= 0; i = next_unit[i]) {
      order.push_back(i);
      units[i].page_first = at;
      units[i].n_parts = 1;
      units[i].first_cta = static_cast<uint8_t>(k);
      at += pages[i];
    }
  }
  L->starts.push_back(at);
  deal_empty(n - count, sms, &L->starts);
  L->grid = (int)L->starts.size() - 1;
  return order;
}

// A launch's units and CTAs into a kernel's parameters.
template <class Prm>
void fill_units(const Plan& plan, const Launch& L, const std::vector<int>& order, Prm* prm) {
  prm->n_units = static_cast<int>(L.n);
  prm->grid = L.grid;
  // Units without pages go last: every role walks its CTA's units, and skipping
  // one costs it ~0.2 us (4 requests of 700 tokens and 252 without any: 64.5 us
  // with the others among them).
  DevUnit* to = prm->units;
  auto add = [&](const Unit& u) {
    *to++ = {u.page_first, u.bt, u.tok_start, u.tok_end, u.g, u.part_base, u.n_parts, u.first_cta};
  };
  for (int i : order) add(plan.units[L.u0 + i]);
  for (size_t i = L.u0; order.empty() && i < L.u0 + L.n; ++i)
    if (plan.pages[i] != 0) add(plan.units[i]);
  prm->n_full = static_cast<int>(to - prm->units);
  for (size_t i = L.u0; i < L.u0 + L.n && to < prm->units + L.n; ++i)
    if (plan.pages[i] == 0) add(plan.units[i]);
  std::memcpy(prm->starts, L.starts.data(), L.starts.size() * sizeof(int32_t));
  for (int k = 0, u = 0; k < L.grid; ++k) {
    // the last unit that starts at or before the CTA's first page
    while (u + 1 < prm->n_full && prm->units[u + 1].page_first <= L.starts[k]) ++u;
    prm->first_unit[k] = static_cast<int16_t>(u);
  }
}

// The arguments that both kernels' calls have.
inline int check_decode(const void* q, const void* pool, const void* scales, int64_t pool_pages,
                        int64_t most_pages, const int32_t* page_table, int max_pages,
                        const int32_t* tiles, int B, int T, int Hq, int Hkv, int D,
                        const float* out, const float* lse, const float* merged_out,
                        const float* merged_lse, const void* workspace, size_t ws_bytes) {
  if (D != 128 && D != 256)
    return fail(PA_ERR_UNSUPPORTED, "head_dim %d not built (supported: 128, 256)", D);
  PA_REQUIRE(Hkv >= 1 && Hq >= Hkv && Hq % Hkv == 0,
             "n_q_heads (%d) must be a positive multiple of n_kv_heads (%d)", Hq, Hkv);
  if (Hq / Hkv > kMaxG)
    return fail(PA_ERR_UNSUPPORTED, "group size %d above the supported %d", Hq / Hkv, kMaxG);
  PA_REQUIRE(q && pool && scales && page_table && tiles && out && lse && workspace,
             "null pointer argument");
  PA_REQUIRE(max_pages >= 1 && pool_pages >= 1, "max_pages and pool_pages must be >= 1");
  auto aligned = [](const void* ptr, int n) { return reinterpret_cast<uintptr_t>(ptr) % n == 0; };
  PA_REQUIRE(aligned(q, 16), "q must be 16-byte aligned");
  PA_REQUIRE(aligned(pool, 16), "pool must be 16-byte aligned");
  PA_REQUIRE(aligned(scales, 16), "scales must be 16-byte aligned");
  PA_REQUIRE(aligned(out, 16), "out must be 16-byte aligned");
  PA_REQUIRE(aligned(workspace, 256), "workspace must be 256-byte aligned");
  PA_REQUIRE((merged_out == nullptr) == (merged_lse == nullptr),
             "merged_out and merged_lse go together");
  PA_REQUIRE(aligned(merged_out, 16), "merged_out must be 16-byte aligned");
  PA_REQUIRE(pool_pages < most_pages, "pool too large for 32-bit coordinates");
  PA_REQUIRE((long long)B * T * Hq < (1ll << 31), "output too large");
  const size_t need = workspace_bytes(B, T, Hkv, D);
  PA_REQUIRE(ws_bytes >= need, "workspace of %zu bytes is smaller than the %zu needed", ws_bytes,
             need);
  const long long max_tok = (long long)max_pages * kPage;
  for (long long i = 0; i < (long long)B * T; ++i) {
    const int s = tiles[2 * i], e = tiles[2 * i + 1];
    PA_REQUIRE(s >= 0 && s <= e && e <= max_tok,
               "tile %lld of request %lld is [%d, %d), outside [0, %lld]", i % T, i / T, s, e,
               max_tok);
  }
  return PA_OK;
}

}  // namespace split
}  // namespace pa

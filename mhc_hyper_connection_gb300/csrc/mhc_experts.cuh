// mhc_experts.cuh -- the plan of routed tokens as the host lays it out and the
// kernels read it (include/mhc_route.h, mhc_experts.h).
#pragma once

#include <stdint.h>

namespace mhc {

constexpr int kMostExperts = 1024, kMostChoices = 32, kMostGroups = 32;
constexpr int kPlanHead = 64;            // int32 words before the counts; [1] rows with padding, [2] tiles
constexpr int kPlanPad = 16;             // an expert's rows begin at a multiple: one step of a product's depth
constexpr int kPlanBand = 8;             // tiles of one expert that share a tile of its weights one after the other

// Where the parts of a plan lie, in int32 words from its start.
struct PlanLayout {
  int64_t slots, cap_rows, cap_tiles;
  int width;                             // most rows of a tile
  int64_t counts, starts, table, places, rows, scratch, total;
};

// Slots up to which a single block sorts them alone, and those that else one block of the
// counting and placing kernels takes: 32 a warp or, from 2^17 on, what leaves 128 blocks to
// sum over.
constexpr int kPlanAlone = 2048;
inline int64_t plan_chunk(int64_t slots) { return 1024 * ((slots + (1 << 17) - 1) >> 17); }

inline PlanLayout plan_layout(int64_t T, int64_t k, int64_t E) {
  PlanLayout l;
  auto up = [](int64_t v) { return (v + 63) & ~int64_t(63); };
  l.slots = T * k;
  const int64_t active = E < l.slots ? E : l.slots;
  l.cap_rows = l.slots + (kPlanPad - 1) * active;
  // Tiles hold up to four times an expert's share: most experts then are one tile,
  // and the ring keeps short stages where there are few tokens.
  int64_t w = (4 * l.slots + E - 1) / (E > 0 ? E : 1);
  w = (w + 31) & ~int64_t(31);
  l.width = (int)(w < 32 ? 32 : w > 256 ? 256 : w);
  l.cap_tiles = l.slots / l.width + active;
  l.counts = kPlanHead;
  l.starts = l.counts + up(E);
  l.table = l.starts + up(E + 1);
  l.places = l.table + up(8 * l.cap_tiles);
  l.rows = l.places + up(l.slots);
  l.scratch = l.rows + up(l.cap_rows);
  const int64_t blocks = l.slots > kPlanAlone ? (l.slots + plan_chunk(l.slots) - 1) / plan_chunk(l.slots) : 0;
  l.total = l.scratch + up(blocks * E);
  return l;
}

// A plan on the device.  Table entry i (two int4): {expert, first entry of its band,
// entries of the band, first row of the band}, {rows of the band, rows of a tile, how many
// of the band's first tiles have 32 more}.
// What is read from it is held inside these bounds, so a buffer that no plan was
// written to gives wrong numbers and nothing worse.
struct PlanView {
  int *head, *counts, *starts, *places, *rows, *scratch;
  int4* table;
  int width, E, slots, cap_rows, cap_tiles;
};
inline PlanView plan_view(const PlanLayout& l, int64_t E, void* plan) {
  int* p = static_cast<int*>(plan);
  return {p, p + l.counts, p + l.starts, p + l.places, p + l.rows, p + l.scratch, reinterpret_cast<int4*>(p + l.table), l.width,
          (int)E, (int)l.slots, (int)l.cap_rows, (int)l.cap_tiles};
}

}  // namespace mhc

// How the tiles of a symmetric product (TileMode kSym) are cut up.  Host code
// without HIP, so that every size's plan can be looked at on any machine.
#pragma once

#include <stddef.h>
#include <stdint.h>

namespace mi355gemm {
namespace tune {

// The tile shape, and what is cut into ranges of K: `whole` tiles, then `rest`
// of them in `splits` ranges of `per` slabs of 64 (the last may be shorter, but
// none has fewer than two).
struct SymPlan {
  int shape = -1, bm = 0;
  uint32_t whole = 0, rest = 0;
  int splits = 1, per = 0;
  size_t sum_bytes() const { return (size_t)rest * splits * bm * bm * sizeof(float); }
};

// kSym's: the time of a slab and of a tile's end in microseconds, from launches of
// each shape.
struct SymShape {
  int bm, per_cu;
  double slab, alone, end;   // alone: tiles do not outnumber the CUs
};
constexpr SymShape kSymShapes[] = {
    {256, 1, 1.5, 1.5, 10.},
    {128, 2, 0.92, 0.6, 4.},
    {192, 1, 1.0, 1.0, 6.},
};

// For M x M over `slabs` slabs of K, `batch` matrices, on `cus` CUs (the cost of a
// plan; it is right on any number of them).
inline SymPlan plan_sym(int M, int slabs, int batch, int cus) {
  SymPlan best;
  double best_cost = 0;
  auto consider = [&](int i, int64_t tiles, int64_t whole, int splits) {
    const SymShape& s = kSymShapes[i];
    const int64_t slots = (int64_t)s.per_cu * cus, rest = tiles - whole;
    const int per = (slabs + splits - 1) / splits;
    splits = (slabs + per - 1) / per;
    // (no range of one slab: two work items behind each other are three slabs at least,
    // as the kernel's stream of copies wants them)
    if (rest && slabs - (splits - 1) * per < 2) return;
    if (rest * splits >= (int64_t(1) << 31)) return;
    double cost = 0;
    if (whole)
      cost += (double)((whole + slots - 1) / slots) *
              (slabs * (whole <= cus ? s.alone : s.slab) + s.end);
    if (rest) {
      const int64_t items = rest * splits;
      cost += (double)((items + slots - 1) / slots) *
                  (per * (items <= cus ? s.alone : s.slab) + 3.) +
              (double)items * s.bm * s.bm * 8 * 2.5e-7 + 6.;
    }
    if (best.shape < 0 || cost < best_cost) {
      best = SymPlan{i, s.bm, (uint32_t)whole, (uint32_t)rest, splits, per};
      best_cost = cost;
    }
  };
  for (int i = 0; i < 3; ++i) {
    const SymShape& s = kSymShapes[i];
    if (M < s.bm) continue;
    const int64_t t = (M + s.bm - 1) / s.bm, tiles = t * (t + 1) / 2 * batch;
    const int64_t slots = (int64_t)s.per_cu * cus, whole = tiles / slots * slots;
    consider(i, tiles, tiles, 1);
    if (whole == tiles) continue;
    for (int splits = 2; splits <= 64 && 2 * splits <= slabs; ++splits) {
      consider(i, tiles, whole, splits);
      if ((tiles - whole) * splits >= 2 * slots) break;
    }
  }
  return best;
}

}  // namespace tune
}  // namespace mi355gemm

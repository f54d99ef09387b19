// Tile-kernel instances of an orthogonalised update (TileModes kSym and kMul).
#include "hgemm_shapes.hpp"
#include "tune.hpp"

namespace mi355gemm {
namespace tune {

using hshape::BK;
constexpr int GM = 8;

namespace {

// Tile-times as in hgemm_shapes.hpp; `each` tiles of a matrix.
struct Shape {
  int bm, bn, per_cu;
  int64_t time, time_alone;
};
template <typename F>
int choose(const Shape* s, int n, int M, int N, int batch, int cus, F each) {
  int best = -1;
  int64_t best_cost = 0;
  for (int i = 0; i < n; ++i) {
    if (M < s[i].bm || N < s[i].bn) continue;
    const int64_t tiles = each(s[i]) * batch, slots = (int64_t)s[i].per_cu * cus;
    const int64_t cost = (tiles + slots - 1) / slots * (tiles <= cus ? s[i].time_alone : s[i].time);
    if (best < 0 || cost < best_cost) {
      best = i;
      best_cost = cost;
    }
  }
  return best;
}

constexpr Shape kSymShapes[] = {
    {256, 256, 1, 256 * 256, 256 * 256},
    {128, 128, 2, 2 * 128 * 128 * 6 / 5, 128 * 128 * 8 / 5},
    {192, 192, 1, 192 * 192 * 6 / 5, 192 * 192 * 6 / 5},
};
constexpr Shape kMulShapes[] = {
    {256, 256, 1, 256 * 256, 256 * 256},
    {128, 128, 2, 2 * 128 * 128 * 6 / 5, 128 * 128 * 8 / 5},
    {192, 256, 1, 192 * 256 * 11 / 10, 192 * 256 * 11 / 10},
};

}  // namespace

hipError_t launch_sym_tiles(const Args16& a, const OrthoExtra& x, int batch, int cus,
                            hipStream_t stream) {
  using hgemm::kSym;
  auto each = [&](const Shape& s) {
    const int64_t t = (a.M + s.bm - 1) / s.bm;
    return t * (t + 1) / 2;
  };
  switch (choose(kSymShapes, 3, a.M, a.N, batch, cus, each)) {
    case 0:
      return hgemm::launch_ortho<256, 256, BK, 4, 2, GM, 1, 2, 0, kSym>(a, x, batch, cus, stream);
    case 1:
      return hgemm::launch_ortho<128, 128, BK, 2, 2, GM, 0, 0, 0, kSym>(a, x, batch, 2 * cus,
                                                                       stream);
    case 2:
      return hgemm::launch_ortho<192, 192, BK, 4, 2, GM, 1, 0, 0, kSym>(a, x, batch, cus, stream);
    default:
      return hipErrorInvalidValue;
  }
}

hipError_t launch_mul_tiles(const Args16& a, const OrthoExtra& x, bool a_kmajor, int batch, int cus,
                            hipStream_t stream) {
  using hgemm::kMul;
  auto each = [&](const Shape& s) {
    return (int64_t)((a.M + s.bm - 1) / s.bm) * ((a.N + s.bn - 1) / s.bn);
  };
  if (a_kmajor) {
    if (choose(kMulShapes, 2, a.M, a.N, batch, cus, each) == 0)
      return hgemm::launch_ortho<256, 256, BK, 4, 2, GM, 1, 2, 2, kMul>(a, x, batch, cus, stream);
    return hgemm::launch_ortho<128, 128, BK, 2, 2, GM, 0, 0, 2, kMul>(a, x, batch, 2 * cus, stream);
  }
  switch (choose(kMulShapes, 3, a.M, a.N, batch, cus, each)) {
    case 0:
      return hgemm::launch_ortho<256, 256, BK, 4, 2, GM, 1, 2, 1, kMul>(a, x, batch, cus, stream);
    case 1:
      return hgemm::launch_ortho<128, 128, BK, 2, 2, GM, 0, 0, 1, kMul>(a, x, batch, 2 * cus,
                                                                       stream);
    case 2:
      return hgemm::launch_ortho<192, 256, BK, 4, 2, GM, 1, 2, 1, kMul>(a, x, batch, cus, stream);
    default:
      return hipErrorInvalidValue;
  }
}

}  // namespace tune
}  // namespace mi355gemm

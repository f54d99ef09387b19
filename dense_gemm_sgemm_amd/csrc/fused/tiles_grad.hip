// Tile-kernel instances of the gradient products: dW = d^T * X (TileMode
// kGradW: d K-major, X transposed beforehand) and dX = d * W (kGradX: W
// K-major).  The K-major operand is read in place through the transposing LDS
// reads; with both operands K-major the tiles spill and took a third more time
// (16384 x 2 x 4096 over 4096 rows bf16: 1240 against 969 us).
#include "fused.hpp"
#include "hgemm_shapes.hpp"

namespace mi355gemm {
namespace fused {

using hshape::BK;
constexpr int GM = 4;   // tile rows of a group: 4 against 8 measured 2 % faster here

// dX has the third one too, for rows that fill it and no others (3800 x 4096 x
// 1500 bf16, all gradients: 242 against 289 us; 1500 x 11008 x 4096: 581
// against 601); a K-major A has tiles of a power of two.
static constexpr Shape kShapes[] = {
    {256, 256, 1, 256 * 256, 256 * 256},
    {128, 128, 2, 2 * 128 * 128 * 6 / 5, 128 * 128 * 8 / 5},
    {192, 256, 1, 0, 0},   // (plan_grad_x has its own times)
};

template <int FMT>
static hipError_t grad_w(const Args16& a, const FusedExtra& x, int cus, hipStream_t stream) {
  using hgemm::kGradW;
  switch (choose_shape(kShapes, 2, a.M, a.N, x.parts, cus)) {
    case 0:
      return hgemm::launch_fused<256, 256, BK, 4, 2, GM, 1, 2, FMT, 2, kGradW>(a, x, cus, stream);
    case 1:
      return hgemm::launch_fused<128, 128, BK, 2, 2, GM, 0, 0, FMT, 2, kGradW>(a, x, 2 * cus,
                                                                              stream);
    default:
      return hipErrorInvalidValue;
  }
}

template <int FMT>
static hipError_t grad_x(const Args16& a, const FusedExtra& x, int shape, int cus,
                         hipStream_t stream) {
  using hgemm::kGradX;
  if (shape == 0)
    return hgemm::launch_fused<256, 256, BK, 4, 2, GM, 1, 2, FMT, 1, kGradX>(a, x, cus, stream);
  if (shape == 2)
    return hgemm::launch_fused<192, 256, BK, 4, 2, GM, 1, 2, FMT, 1, kGradX>(a, x, cus, stream);
  return hgemm::launch_fused<128, 128, BK, 2, 2, GM, 0, 0, FMT, 1, kGradX>(a, x, 2 * cus, stream);
}

// Few tiles over a long K (all of N, or a piece of it): K is cut into ranges
// that fill the chip.  The time in microseconds of `rounds` of work items, a
// slab of a 256 x 256 tile taking 1.5 (192 x 256: 1.2; two 128 x 128 tiles on a
// CU 0.92, one alone 0.6, as in the cost model of the plain tiles), 3 to store a
// tile, and the ranges' sums written and read at 5 bytes a picosecond.
GradXPlan plan_grad_x(int M, int N, int slabs, bool sums) {
  GradXPlan best;
  double best_cost = 0;
  for (int i = 0; i < 3; ++i) {
    if (M < kShapes[i].bm || N < kShapes[i].bn) continue;
    const int64_t tiles = (int64_t)((M + kShapes[i].bm - 1) / kShapes[i].bm) *
                          ((N + kShapes[i].bn - 1) / kShapes[i].bn);
    for (int want = 1; want <= 64 && want * 4 <= std::max(slabs, 4); ++want) {
      const int per = (slabs + want - 1) / want, splits = (slabs + per - 1) / per;
      const int64_t items = tiles * splits, slots = kShapes[i].per_cu * kPlanCus;
      const double slab = i == 0 ? 1.5 : i == 2 ? 1.2 : items <= kPlanCus ? 0.6 : 0.92;
      double cost = (double)((items + slots - 1) / slots) * (per * slab + 3.0);
      if (splits > 1 || sums) cost += (double)splits * M * N * 8 * 2e-7 + 4.0;
      if (best.splits == 0 || cost < best_cost) {
        best = GradXPlan{i, splits, per};
        best_cost = cost;
      }
      if (items >= 2 * slots) break;
    }
  }
  return best;
}

hipError_t launch_grad_w(const Args16& a, const FusedExtra& x, int cus, hipStream_t stream) {
  return a.fmt == kFmtBF16 ? grad_w<kFmtBF16>(a, x, cus, stream)
                           : grad_w<kFmtF16>(a, x, cus, stream);
}

hipError_t launch_grad_x(const Args16& a, const FusedExtra& x, const GradXPlan& plan, int cus,
                         hipStream_t stream) {
  FusedExtra y = x;
  y.splits = plan.splits;
  y.per = plan.per;
  return a.fmt == kFmtBF16 ? grad_x<kFmtBF16>(a, y, plan.shape, cus, stream)
                           : grad_x<kFmtF16>(a, y, plan.shape, cus, stream);
}

}  // namespace fused
}  // namespace mi355gemm

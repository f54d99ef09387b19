// Tile-kernel instances of the gradient products: dW = d^T * X (TileMode
// kGradW, both operands K-major) and dX = d * W (kGradX, W K-major), read in
// place through the transposing LDS reads.
#include "fused.hpp"
#include "hgemm_shapes.hpp"

namespace mi355gemm {
namespace fused {

using namespace hshape;

static constexpr Shape kShapesW[] = {
    {256, 224, 1, 256 * 224, 256 * 224},   // 256 x 256 spills with both operands transposed
    {128, 128, 2, 2 * 128 * 128 * 6 / 5, 128 * 128 * 8 / 5},
};
static constexpr Shape kShapesX[] = {
    {256, 256, 1, 256 * 256, 256 * 256},
    {128, 128, 2, 2 * 128 * 128 * 6 / 5, 128 * 128 * 8 / 5},
};

template <int FMT>
static hipError_t grad_w(const Args16& a, const FusedExtra& x, int cus, hipStream_t stream) {
  using hgemm::kGradW;
  switch (choose_shape(kShapesW, 2, a.M, a.N, x.parts, cus)) {
    case 0:
      return hgemm::launch_fused<256, 224, BK, 4, 2, GM, 1, 0, FMT, 3, kGradW>(a, x, cus, stream);
    case 1:
      return hgemm::launch_fused<128, 128, BK, 2, 2, GM, 0, 0, FMT, 3, kGradW>(a, x, 2 * cus,
                                                                              stream);
    default:
      return hipErrorInvalidValue;
  }
}

template <int FMT>
static hipError_t grad_x(const Args16& a, const FusedExtra& x, int cus, hipStream_t stream) {
  using hgemm::kGradX;
  switch (choose_shape(kShapesX, 2, a.M, a.N, 1, cus)) {
    case 0:
      return hgemm::launch_fused<256, 256, BK, 4, 2, GM, 1, 2, FMT, 1, kGradX>(a, x, cus, stream);
    case 1:
      return hgemm::launch_fused<128, 128, BK, 2, 2, GM, 0, 0, FMT, 1, kGradX>(a, x, 2 * cus,
                                                                              stream);
    default:
      return hipErrorInvalidValue;
  }
}

hipError_t launch_grad_w(const Args16& a, const FusedExtra& x, int cus, hipStream_t stream) {
  return a.fmt == kFmtBF16 ? grad_w<kFmtBF16>(a, x, cus, stream)
                           : grad_w<kFmtF16>(a, x, cus, stream);
}

hipError_t launch_grad_x(const Args16& a, const FusedExtra& x, int cus, hipStream_t stream) {
  return a.fmt == kFmtBF16 ? grad_x<kFmtBF16>(a, x, cus, stream)
                           : grad_x<kFmtF16>(a, x, cus, stream);
}

}  // namespace fused
}  // namespace mi355gemm

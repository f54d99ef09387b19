// Tile-kernel instances of the gated product (TileMode kGated): a tile's B
// rows are 16-row blocks of Wg and Wu in turn, so a 256 x 256 tile makes
// 256 x 128 outputs from 256 x 128 columns of each product.
#include "fused.hpp"
#include "hgemm_shapes.hpp"

namespace mi355gemm {
namespace fused {

using namespace hshape;

// Output tiles of 256 x 128, 128 x 64 (two workgroups per CU), 128 x 96 and
// 192 x 128; the tile-times of the plain product's tiles of twice the width.
// The last is for rows that fill its tiles and no others (1500 x 11008 x 4096
// bf16: 258 against 292 us; 759 x 14344 x 4096: 178 against 197); without its
// 11 / 10 it would take products of many rounds from the first (2725 x 10657 x
// 4096: 425 against 391).
static constexpr Shape kShapes[] = {
    {256, 128, 1, 256 * 256, 256 * 256},
    {128, 64, 2, 2 * 128 * 128 * 6 / 5, 128 * 128 * 8 / 5},
    {128, 96, 1, 128 * 192 * 4 / 3, 128 * 192 * 4 / 3},
    {192, 128, 1, 192 * 256 * 11 / 10, 192 * 256 * 11 / 10},
};

template <int FMT>
static hipError_t launch_fmt(const Args16& a, const FusedExtra& x, int cus, hipStream_t stream) {
  using hgemm::kGated;
  switch (choose_shape(kShapes, 4, a.M, a.N, 1, cus)) {
    case 0:
      return hgemm::launch_fused<256, 256, BK, 4, 2, GM, 1, 2, FMT, 0, kGated>(a, x, cus, stream);
    case 1:
      return hgemm::launch_fused<128, 128, BK, 2, 2, GM, 0, 0, FMT, 0, kGated>(a, x, 2 * cus,
                                                                              stream);
    case 2:
      return hgemm::launch_fused<128, 192, BK, 2, 2, GM, 0, 0, FMT, 0, kGated>(a, x, cus, stream);
    case 3:
      return hgemm::launch_fused<192, 256, BK, 4, 2, GM, 1, 2, FMT, 0, kGated>(a, x, cus, stream);
    default:
      return hipErrorInvalidValue;
  }
}

hipError_t launch_gated_tiles(const Args16& a, const FusedExtra& x, int cus, hipStream_t stream) {
  return a.fmt == kFmtBF16 ? launch_fmt<kFmtBF16>(a, x, cus, stream)
                           : launch_fmt<kFmtF16>(a, x, cus, stream);
}

}  // namespace fused
}  // namespace mi355gemm

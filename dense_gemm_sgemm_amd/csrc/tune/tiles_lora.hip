// Tile-kernel instances of a product with adapters (TileMode kLora): A * B^T,
// and with B K-major for the gradient of X.  bf16, 4096^3, 8 adapters of 32 ranks in
// segments: 109 us (60 % of the matrix cores' time), K-major 113 with one of 16.
#include "hgemm_shapes.hpp"
#include "tune.hpp"

namespace mi355gemm {
namespace tune {

using hshape::BK;

namespace {

constexpr int GM = 8;
// (tile-times, as of the products in the other operators' tiles)
constexpr fused::Shape kShapes[] = {
    {256, 256, 1, 256 * 256, 256 * 256},
    {128, 128, 2, 2 * 128 * 128 * 6 / 5, 128 * 128 * 8 / 5},
    {192, 256, 1, 192 * 256 * 11 / 10, 192 * 256 * 11 / 10},
};

// (W: K-major, over whole slabs of 64: no code for a last one that is none)
template <int FMT, int LAY, int W>
hipError_t launch(const Args16& a, const LoraExtra& x, int cus, hipStream_t stream) {
  switch (fused::choose_shape(kShapes, 3, a.M, a.N, 1, cus)) {
    case 0:
      return hgemm::launch_lora<256, 256, BK, 4, 2, GM, 1, 2 + W, FMT, LAY>(a, x, cus, stream);
    case 1:
      return hgemm::launch_lora<128, 128, BK, 2, 2, GM, 0, W, FMT, LAY>(a, x, 2 * cus, stream);
    case 2:
      return hgemm::launch_lora<192, 256, BK, 4, 2, GM, 1, 2 + W, FMT, LAY>(a, x, cus, stream);
    default:
      return hipErrorInvalidValue;
  }
}

}  // namespace

hipError_t launch_lora_tiles(const Args16& a, const LoraExtra& x, bool kmajor, int cus,
                             hipStream_t stream) {
  if (!kmajor)
    return a.fmt == kFmtBF16 ? launch<kFmtBF16, 0, 0>(a, x, cus, stream)
                             : launch<kFmtF16, 0, 0>(a, x, cus, stream);
  if (a.K % BK == 0)
    return a.fmt == kFmtBF16 ? launch<kFmtBF16, 1, 4>(a, x, cus, stream)
                             : launch<kFmtF16, 1, 4>(a, x, cus, stream);
  return a.fmt == kFmtBF16 ? launch<kFmtBF16, 1, 0>(a, x, cus, stream)
                           : launch<kFmtF16, 1, 0>(a, x, cus, stream);
}

}  // namespace tune
}  // namespace mi355gemm

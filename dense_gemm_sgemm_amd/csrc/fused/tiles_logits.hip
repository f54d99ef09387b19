// Tile-kernel instances that turn logits X * W^T into softmax statistics
// (TileMode kLse) or their gradients (kDlogit) while they are in registers.
#include "fused.hpp"
#include "hgemm_shapes.hpp"

namespace mi355gemm {
namespace fused {

using namespace hshape;

// The last one is for rows that fill its tiles and no others (370 x 32000 x
// 4096 bf16, forward: 113 against 126 us; 333 x 50001 x 2048: 106 against 111;
// 11 / 10 as for the gated product), and for K from kLongK: the shorter, the
// more its longer epilogue counts (333 x 50001 x 768, with gradients: 204
// against 200 us; 827 x 20904 x 256, forward: 24.8 against 23.4).
constexpr int kLongK = 1024;
static constexpr Shape kShapes[] = {
    {256, 256, 1, 256 * 256, 256 * 256},
    {128, 128, 2, 2 * 128 * 128 * 6 / 5, 128 * 128 * 8 / 5},
    {192, 256, 1, 192 * 256 * 11 / 10, 192 * 256 * 11 / 10},
};

// The shape is chosen for the chip's 256 CUs: the statistics' workspace is
// sized by it before a device is asked.
static int shape_of(int M, int N, int K) {
  return choose_shape(kShapes, K >= kLongK ? 3 : 2, M, N, 1, kPlanCus);
}

template <int FMT, int MODE>
static hipError_t launch_fmt(const Args16& a, const FusedExtra& x, int cus, hipStream_t stream) {
  switch (shape_of(a.M, a.N, a.K)) {
    case 0:
      return hgemm::launch_fused<256, 256, BK, 4, 2, GM, 1, 2, FMT, 0, MODE>(a, x, cus, stream);
    case 1:
      return hgemm::launch_fused<128, 128, BK, 2, 2, GM, 0, 0, FMT, 0, MODE>(a, x, 2 * cus, stream);
    case 2:
      return hgemm::launch_fused<192, 256, BK, 4, 2, GM, 1, 2, FMT, 0, MODE>(a, x, cus, stream);
    default:
      return hipErrorInvalidValue;
  }
}

hipError_t launch_lse_tiles(const Args16& a, const FusedExtra& x, int cus, hipStream_t stream) {
  return a.fmt == kFmtBF16 ? launch_fmt<kFmtBF16, hgemm::kLse>(a, x, cus, stream)
                           : launch_fmt<kFmtF16, hgemm::kLse>(a, x, cus, stream);
}

// All shapes have two wave columns.
int lse_chunks(int M, int N, int K) {
  const int i = shape_of(pad_rows(M), pad_rows(N), pad_k(K));
  return (pad_rows(N) + kShapes[i].bn - 1) / kShapes[i].bn * 2;
}

hipError_t launch_dlogit_tiles(const Args16& a, const FusedExtra& x, int cus, hipStream_t stream) {
  return a.fmt == kFmtBF16 ? launch_fmt<kFmtBF16, hgemm::kDlogit>(a, x, cus, stream)
                           : launch_fmt<kFmtF16, hgemm::kDlogit>(a, x, cus, stream);
}

}  // namespace fused
}  // namespace mi355gemm

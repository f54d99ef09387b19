// Declarations shared by the operators of fine tuning (libmi355tune.so).
#pragma once

#include "fused/fused.hpp"
#include "mi355tune.h"

namespace mi355gemm {
namespace tune {

using fused::Mat;
using hgemm::OrthoExtra;

// Products of an orthogonalised update over `batch` matrices (tiles_ortho.hip):
// kSym, and kMul with the second operand K-major or (a_kmajor) the first one.
hipError_t launch_sym_tiles(const Args16& a, const OrthoExtra& x, int batch, int cus,
                            hipStream_t stream);
hipError_t launch_mul_tiles(const Args16& a, const OrthoExtra& x, bool a_kmajor, int batch, int cus,
                            hipStream_t stream);

}  // namespace tune
}  // namespace mi355gemm

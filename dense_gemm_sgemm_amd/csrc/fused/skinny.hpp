// What the kernels for few rows of X share (decode steps: M <= 64 rows a
// workgroup, the weights streamed from HBM once).
//
// A workgroup owns 16 weight rows (outputs n) and all of K, which its waves
// share out.  Weights go from memory to registers, X through a copy in LDS that
// is each wave's own (XStage below: no barrier) or, for the fewest rows of
// gemm_w4, the workgroup's (one barrier before the products); the sums of the
// waves are added through LDS at the end.  A wave multiplies with v_mfma_f32_16x16x32: X rows are the first
// operand (lane l: row l % 16, k = 8 (l / 16) .. + 7 of a step's 32), weight
// rows the second (lane l: row n0 + l % 16, the same k), so a lane's four
// accumulators are rows 4 (l / 16) .. + 3 of X against its one weight row.
// Any one-to-one choice of the 32 k of a step does, as long as both operands
// make the same.  MT = 1, 2 or 4 blocks of 16 X rows.
#pragma once

#include "fused.hpp"

namespace mi355gemm {
namespace fused {
namespace skinny {

typedef _Float16 h8 __attribute__((ext_vector_type(8)));
typedef float f4 __attribute__((ext_vector_type(4)));
using hgemm::mfma16;

// k .. k + 7 of an X row (TAIL: zeros past K).  Rows start at any 2-byte
// address.
template <bool TAIL>
__device__ __forceinline__ h8 load_x(const half_t* row, int k, int K) {
  h8 v = {};
  if (!TAIL || k <= K - 8) {
    __builtin_memcpy(&v, row + k, 16);
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (k < K - e) v[e] = row[k + e];
  }
  return v;
}

// A wave's own copy in LDS of KB values of its X rows.  Read straight into the
// fragments' layout, X costs 16 rows x 64 bytes an instruction, and a CU took
// such loads at one per 50-80 cycles: with 16 rows of X and 4-bit weights they
// were half the time.  Here a load instruction covers whole lines (KB = 64: 8
// rows x 128 bytes), one stage ahead in registers, and the fragments come from
// LDS.  Rows are 16 bytes longer than their data, so that 16 of them start in
// different banks.  Only the one wave uses the copy: LDS serves a wave's
// accesses in order, so no barrier is needed.
template <int MT, int KB>
struct XStage {
  static constexpr int kPitch = 2 * KB + 16, kPieces = KB / 8, kRows = 64 / kPieces;
  static constexpr int kLoads = 16 * MT / kRows;
  static constexpr int kBytes = 16 * MT * kPitch;
  h8 v[kLoads];

  // Rows from m0 (past M the last one again, unstored), columns from k.
  template <bool TAIL>
  __device__ __forceinline__ void load(const half_t* X, int64_t ldx, int m0, int M, int k, int K,
                                       int lane) {
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const int m = m0 + i * kRows + lane / kPieces;
      v[i] = load_x<TAIL>(X + (m < M ? m : M - 1) * ldx, k + lane % kPieces * 8, K);
    }
  }
  template <typename F>
  __device__ __forceinline__ void store(unsigned char* buf, int lane, F order) const {
    asm volatile("" ::: "memory");
#pragma unroll
    for (int i = 0; i < kLoads; ++i)
      *(h8*)(buf + (i * kRows + lane / kPieces) * kPitch + lane % kPieces * 16) = order(v[i]);
    asm volatile("" ::: "memory");
    __builtin_amdgcn_wave_barrier();
  }
  // Row 16 t + r, values k .. k + 7 of the stage.
  __device__ __forceinline__ static h8 read(const unsigned char* buf, int t, int r, int k) {
    return *(const h8*)(buf + (16 * t + r) * kPitch + 2 * k);
  }
};

// Adds the waves' sums (Q f4 of each lane) in the order of the waves; the
// result is complete in wave 0.
template <int Q>
__device__ __forceinline__ void add_waves(f4 (&acc)[Q], float* lds, int wave, int lane, int waves) {
  f4* part = reinterpret_cast<f4*>(lds);
  if (wave > 0) {
#pragma unroll
    for (int q = 0; q < Q; ++q) part[((wave - 1) * Q + q) * 64 + lane] = acc[q];
  }
  __syncthreads();
  if (wave > 0) return;
  for (int w = 0; w + 1 < waves; ++w)
#pragma unroll
    for (int q = 0; q < Q; ++q) acc[q] += part[(w * Q + q) * 64 + lane];
}

// Waves of a workgroup that share `pieces` of K: four, or eight while they have
// two pieces each (one to multiply, one in flight) and the launch has less than
// 32 waves a CU; fewer where there are fewer pieces.
inline int waves_for(int64_t workgroups, int pieces, int most, int cus) {
  int waves = 4;
  while (waves < most && 4 * waves <= pieces && workgroups * waves < 32 * (int64_t)cus) waves *= 2;
  while (waves > 1 && waves > pieces) waves /= 2;
  return waves;
}

}  // namespace skinny
}  // namespace fused
}  // namespace mi355gemm

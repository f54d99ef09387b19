// Declarations shared by the fused operators (libmi355fused.so).
#pragma once

#include <algorithm>

#include "device.hpp"
#include "hgemm_tile.hpp"
#include "internal.h"
#include "mi355fused.h"

namespace mi355gemm {
namespace fused {

using hgemm::FusedExtra;

// A 16-bit matrix as a caller gave it.
struct Mat {
  const half_t* p = nullptr;
  int64_t ld = 0;
};

// The tile kernels read operands of at least kMinRows rows and kMinK columns
// in whole 16-byte pieces.  What is not so is first copied, padded with
// zeros, into the workspace.
constexpr int kMinRows = 128, kMinK = 128;
inline int pad_rows(int rows) { return rows < kMinRows ? kMinRows : rows; }
// (whole slabs of zeros rather than the fewest: no K tail)
inline int pad_k(int K) { return K < kMinK ? kMinK : K % 8 == 0 ? K : (int)round_up(K, 64); }
// Rows of the copies, of d and of transposed operands start at whole 128-byte
// lines: a copy instruction of the tiles takes 8 rows x 128 bytes, which on
// rows at other addresses is 16 lines instead of 8 (5000 x 3001 over K = 1537,
// copied to rows of 1544 and of 1600 values: 109 and 100 us in all).
inline int64_t line_ld(int64_t cols) { return round_up(cols, 64); }
inline bool needs_copy(const void* p, int64_t ld, int rows, int K) {
  return rows < kMinRows || K < kMinK || K % 8 != 0 || !aligned16(p) || ld % 8 != 0 ||
         ld >= (int64_t(1) << 28);
}
// Rows of the reduction of dW = d^T X: whole slabs.
inline int pad_slabs(int M) { return (int)round_up(pad_rows(M), 64); }
inline size_t copy_bytes(int rows, int K) {
  return round256((size_t)pad_rows(rows) * line_ld(pad_k(K)) * 2);
}

// Up to three padded copies in one launch: dst[r][c] (ld a multiple of 8,
// cols_p % 8 == 0) for r < rows_p, c < cols_p, zero outside the source.
struct PadJob {
  const half_t* src = nullptr;
  half_t* dst = nullptr;
  int64_t lds = 0, ldd = 0;
  int rows = 0, cols = 0, rows_p = 0, cols_p = 0;
};
struct PadJobs {
  PadJob job[3];
  int64_t blocks[3] = {0, 0, 0};   // blocks up to and including each job's
  int count = 0;
  // Adds the copy of m ([rows][K]) to dst (add: if it needs one); returns the
  // matrix the kernels read and advances dst past the copy.
  Mat add(Mat m, int rows, int K, char*& dst);
  Mat copy(Mat m, int rows, int K, char*& dst);
};
hipError_t launch_pad(const PadJobs& jobs, hipStream_t stream);

// A transposition for the gradients of weights: dst[c][r] = src[r][c], rows of
// dst `ldd` (a multiple of 8) apart; its rows_p x cols_p extent (in the
// source's orientation, rows_p a multiple of 64) is written, zero outside the
// source.  A wave takes 64 x 64: lane (i, j) = (l / 8, l % 8) the 8 x 8 block
// at rows 8 i, columns 8 j, eight row pieces of 16 bytes turned in registers.
struct Transpose {
  const half_t* src;
  half_t* dst;
  int64_t lds, ldd;
  int rows, cols, rows_p, cols_p;
  // rows to leave out (zeros, whatever they hold): those with this target
  const long long* targets = nullptr;
  long long ignore = 0;
  int64_t tiles() const { return (int64_t)(rows_p / 64) * ((cols_p + 63) / 64); }
};

__device__ __forceinline__ void transpose_tile(const Transpose& p, int64_t tile, int lane) {
  typedef _Float16 h8 __attribute__((ext_vector_type(8)));
  typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
  const int tiles_c = (p.cols_p + 63) / 64;
  if (tile >= (int64_t)(p.rows_p / 64) * tiles_c) return;
  const int r0 = (int)(tile / tiles_c) * 64 + 8 * (lane >> 3);
  const int c0 = (int)(tile % tiles_c) * 64 + 8 * (lane & 7);
  u32x4 x[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    h8 v = {};
    if (r0 + e < p.rows && c0 < p.cols &&
        (p.targets == nullptr || p.targets[r0 + e] != p.ignore)) {
      const half_t* s = p.src + (int64_t)(r0 + e) * p.lds + c0;
      if (c0 + 8 <= p.cols) {
        __builtin_memcpy(&v, s, 16);
      } else {
#pragma unroll
        for (int k = 0; k < 8; ++k)
          if (c0 + k < p.cols) v[k] = s[k];
      }
    }
    x[e] = __builtin_bit_cast(u32x4, v);
  }
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const int sh = 16 * (k & 1);
    u32x4 w;
#pragma unroll
    for (int q = 0; q < 4; ++q)
      w[q] = ((x[2 * q][k >> 1] >> sh) & 0xFFFFu) | (((x[2 * q + 1][k >> 1] >> sh) & 0xFFFFu) << 16);
    if (c0 + k < p.cols_p) *(u32x4*)(p.dst + (int64_t)(c0 + k) * p.ldd + r0) = w;
  }
}

// The tile-kernel launchers (tiles_*.hip); a.fmt selects the format.
hipError_t launch_gated_tiles(const Args16& a, const FusedExtra& x, int cus, hipStream_t stream);
hipError_t launch_grad_w(const Args16& a, const FusedExtra& x, int cus, hipStream_t stream);
// kGradX: the tile shape and the ranges of K (splits == 1: none) for an M x N
// result over `slabs` slabs of 64, made for the chip's 256 CUs since the
// workspace is sized before a device is asked.  sums: fp32 sums are kept
// anyway (K comes in pieces).
constexpr int kPlanCus = 256;
struct GradXPlan {
  int shape = 0, splits = 0, per = 0;
};
GradXPlan plan_grad_x(int M, int N, int slabs, bool sums);
hipError_t launch_grad_x(const Args16& a, const FusedExtra& x, const GradXPlan& plan, int cus,
                         hipStream_t stream);
// out = the sums of x.sum's ranges, scaled and rounded.
hipError_t launch_sums(int fmt, const FusedExtra& x, int splits, half_t* out, int64_t ldo, int M,
                       int N, hipStream_t stream);
hipError_t launch_lse_tiles(const Args16& a, const FusedExtra& x, int cus, hipStream_t stream);
hipError_t launch_dlogit_tiles(const Args16& a, const FusedExtra& x, int cus, hipStream_t stream);
// The gated product where by_rows says so, operands as they are (no copies).
hipError_t launch_gated_rows(const Args16& a, const FusedExtra& x, int cus, hipStream_t stream);
// Wave columns of the kLse tiles for X [M][K] and W [N][K]: partial results of a row.
int lse_chunks(int M, int N, int K);

// Cost model of hgemm_shapes.hpp for the ragged form over M x N outputs whose
// tiles are (bm, bn, workgroups per CU, tile-time); returns the cheapest index.
struct Shape {
  int bm, bn, per_cu;
  int64_t time, time_alone;   // alone: tiles do not outnumber the CUs
};
inline int choose_shape(const Shape* s, int n, int M, int N, int tiles_mul, int cus) {
  int best = -1;
  int64_t best_cost = 0;
  for (int i = 0; i < n; ++i) {
    if (M < s[i].bm || N < s[i].bn) continue;
    const int64_t tiles = (int64_t)((M + s[i].bm - 1) / s[i].bm) * tiles_mul *
                          ((N + s[i].bn - 1) / s[i].bn);
    const int64_t slots = (int64_t)s[i].per_cu * cus;
    const int64_t cost = (tiles + slots - 1) / slots * (tiles <= cus ? s[i].time_alone : s[i].time);
    if (best < 0 || cost < best_cost) {
      best = i;
      best_cost = cost;
    }
  }
  return best;
}

// Sizes are limited so that rows made here (d of two parts, transposed X) keep
// the tiles' 32-bit lane offsets (rows of 2^28 elements at most, seven of which
// are 2^32 - 2^29 bytes) and padded sizes stay ints.
constexpr int kMaxSize = 1 << 27;
inline int check_sizes(int M, int N, int K) {
  if (M < 0 || N < 0 || K < 0) return GEMM_ERR_NEGATIVE_DIM;
  return M > kMaxSize || N > kMaxSize || K > kMaxSize ? GEMM_ERR_BAD_ARG : GEMM_OK;
}
inline bool bad_type(int type) { return type != GEMM_TYPE_F16 && type != GEMM_TYPE_BF16; }
inline bool bad_act(int act) {
  return act != GEMM_ACT_NONE && act != GEMM_ACT_RELU && act != GEMM_ACT_SILU;
}
inline bool bad_ld(int ld, int64_t cols) { return ld < (cols > 1 ? cols : 1); }

}  // namespace fused
}  // namespace mi355gemm

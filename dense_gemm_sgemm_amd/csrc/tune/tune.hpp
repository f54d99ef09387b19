// Declarations shared by the operators of fine tuning (libmi355tune.so).
#pragma once

#include "fused/fused.hpp"
#include "mi355tune.h"
#include "sym_plan.hpp"

namespace mi355gemm {
namespace tune {

using fused::Mat;
using hgemm::LoraExtra;
using hgemm::OrthoExtra;

// Products of an orthogonalised update over `batch` matrices (tiles_ortho.hip):
// kSym, and kMul with the second operand K-major or (a_kmajor) the first one.
// x.sum: room for the plan's sums, which are joined and stored here too.
hipError_t launch_sym_tiles(const Args16& a, const OrthoExtra& x, const SymPlan& plan, int batch,
                            int cus, hipStream_t stream);
hipError_t launch_mul_tiles(const Args16& a, const OrthoExtra& x, bool a_kmajor, int batch, int cus,
                            hipStream_t stream);

// ---- Low-rank adapters.
//
// A row's product with its adapter's first factor, t[m][r] = sum_k X[m][k]
// A_a[r][k], is needed as an operand of the matrix cores.  Rounded to the type
// it would carry an error of its own as large as the output's; so it is kept
// in two 16-bit values, hi + lo, against the same values of the other factor:
// 16 ranks are the 32 k of one instruction.  Both are stored times a power of
// two for the row's block of 16 ranks that brings the largest of them to 2^13
// .. 2^14, so that neither leaves binary16's normal range; the factor that
// undoes it, times the adapter's scale, is applied to the block's sums in fp32.
//
// hi is cut off, not rounded, and neither is zero for a value that is not: both
// then have the value's sign, and an infinity that they meet in the other factor
// gives one infinity, not a NaN.  What stands for such a zero is binary16's least
// value, 2^-37 of the block's largest, and in bf16 2^-73 of it.
//
//   t2      : [M][ld2], for each block 16 hi values, then 16 lo
//   factor  : float [M][blocks]
// Rows without an adapter are left as they were: what reads t2 or the factors
// drops the sums of rows that are not the adapter's, whatever they are.
constexpr int kMaxRank = 1024;
__host__ __device__ inline int rank_blocks(int R) { return (R + 15) / 16; }
__host__ __device__ inline int64_t rank_ld2(int R) { return 32 * (int64_t)rank_blocks(R); }

// v = hi + lo but for 2^-15 (bf16) or 2^-21 (fp16) of it, |v| < 2^14 (or not
// finite), as above.
template <int FMT>
__device__ __forceinline__ void split_value(float v, half_t& hi, half_t& lo) {
  const half_t least = f32_to_word<FMT>(copysignf(FMT == kFmtF16 ? 0x1p-24f : 0x1p-60f, v));
  auto zero = [](half_t w) { return (__builtin_bit_cast(uint16_t, w) & 0x7FFF) == 0; };
  hi = f32_to_word<FMT>(v);
  uint16_t bits = __builtin_bit_cast(uint16_t, hi);
  if (fabsf(word_to_f32<FMT>(hi)) > fabsf(v)) --bits;   // towards zero
  hi = __builtin_bit_cast(half_t, bits);
  lo = fabsf(v) < __builtin_inff() ? f32_to_word<FMT>(v - word_to_f32<FMT>(hi)) : hi;
  if (v != 0.f && zero(hi)) hi = least;
  if (v != 0.f && zero(lo)) lo = least;
}
// 2^(13 - floor(log2 top)) and its inverse, within what fp32 holds.
__device__ __forceinline__ void scale_for(float top, float& up, float& down) {
  const int e = top == 0.f ? 13 : (int)(__float_as_uint(fmaxf(top, 0x1p-100f)) >> 23) - 127;
  up = __uint_as_float((uint32_t)(127 + 13 - e) << 23);
  down = __uint_as_float((uint32_t)(127 - 13 + e) << 23);
}

struct ShrinkArgs {
  const half_t* X;     // [M][ldx]
  const half_t* A;     // [S][R][lda], matrices stride_a apart
  int64_t ldx, lda, stride_a;
  const long long* ids;
  const float* scales;   // [S] or null
  half_t* t2;            // or null, with factor
  float* factor;
  int64_t ld2;
  float* t32;            // [M][ldt] or null: the sums themselves
  int64_t ldt;
  int M, K, R, S;
  int slots = 1;   // (set by the launcher)
};
hipError_t launch_shrink(int fmt, const ShrinkArgs& p, hipStream_t stream);

// The adapters' part beside a product of few rows (lora_rows.hip), operands as
// they are; x as for the tiles but for B, whose ranks may be any number.  `sums`:
// the product is there already, in `ranges` fp32 sums [M][ld_sum] behind each
// other.
struct RowSums {
  const float* sum = nullptr;
  int64_t ld_sum = 0;
  int ranges = 0;
};
hipError_t launch_lora_rows(const Args16& a, const LoraExtra& x, const RowSums& sums, int cus,
                            hipStream_t stream);
// dC W for few rows, in ranges of N (lora_dx.hip).
struct DxPlan {
  int splits = 0, per = 0;
  int64_t ld = 0;
  size_t bytes = 0;
};
DxPlan plan_dx(int M, int N, int K);
hipError_t launch_dx(int fmt, const half_t* dC, int64_t lddc, const half_t* W, int64_t ldw, int M,
                     int N, int K, const DxPlan& plan, float* sum, hipStream_t stream);
// C = A B^T (kmajor: A B) with the adapters' part.
hipError_t launch_lora_tiles(const Args16& a, const LoraExtra& x, bool kmajor, int cus,
                             hipStream_t stream);

// ---- Gradients of the adapters (lora_grad.hip).
//
// dA_a[r][k] = sum_m dt[m][r] X[m][k] over the rows of adapter a, and dB alike
// with dC and t: sums over rows, which lie in any order.  The rows are listed
// adapter by adapter, each adapter's list filled up to whole steps of 32 with
// -1, so that a matrix-core step of 32 rows belongs to one adapter.
struct GroupArgs {
  const long long* ids;
  int M, S;
  int* first;          // [S + 1] an adapter's first step, and the number of all
  int* rows;           // [32 * steps]
  int* step_adapter;   // [steps], -1 past the last one
  int steps;           // as many as there can be
};
inline int max_steps(int M, int S) { return (int)(((int64_t)M + 31) / 32 + std::min(M, S)); }
constexpr int kHistogram = 2048;   // adapters that one workgroup counts
// Each adapter's rows are found among all M: what a call may ask for.  2^40 is 2^30
// turns of a workgroup of 1024, half a second.
inline bool can_list(int M, int S) { return (int64_t)M * std::min(M, S) <= int64_t(1) << 40; }

// One of the two gradients: `left` [rows][ld_left] fp32 (dt or t) times `right`
// [rows][ld_right] 16-bit (X or dC).
struct GradJob {
  const float* left = nullptr;
  int64_t ld_left = 0;
  const half_t* right = nullptr;
  int64_t ld_right = 0;
  int cols = 0;             // of right
  half_t* out = nullptr;    // null: not asked for
  int64_t ldo = 0, stride_o = 0;
  int transposed = 0;       // out[a][col][rank] (dB) instead of out[a][rank][col]
  half_t* pack = nullptr;   // left's ranks in list order, [hi, lo][padded][32 * steps]
  float* step_factor = nullptr;   // [steps]
  float* partial = nullptr;
  int blocks = 0;           // of 128 columns
};
struct GradArgs {
  GroupArgs g;
  GradJob job[2];
  const float* scales;      // [S] or null
  int R, padded;            // ranks, and in whole groups of 16
  int groups;               // of 16 * RB ranks
  int chunks, chunk_steps;  // the steps are cut into chunks, each a workgroup's
  bool by_adapter;          // how partial sums are numbered
};
struct GradPlan {
  int steps, rb, groups, chunks, chunk_steps, padded;
  bool by_adapter;
  size_t pack, partial[2];   // bytes of one job's
};
GradPlan plan_grad(int M, int N, int K, int R, int S);
hipError_t launch_adapter_grads(int fmt, const GradArgs& p, const GradPlan& plan,
                                hipStream_t stream);

// dst[l][o][i] = src[l][i][o] for i < inner (zeros up to inner_p, a multiple of
// 8) and o < outer, in `count` matrices.
struct TurnArgs {
  const half_t* src;
  half_t* dst;
  int64_t lds, stride_s, ldd, stride_d;
  int inner, inner_p, outer, count;
};
// The lists (group: or null) and up to two stacks, in one launch.
hipError_t launch_lists(const GroupArgs* group, const TurnArgs* turns, int count,
                        hipStream_t stream);
// dst[l][r][0 .. cols_p) = src[l][r][0 .. cols), zeros past cols (cols_p a
// multiple of 8, rows of dst cols_p apart).
struct WidenArgs {
  const half_t* src;
  half_t* dst;
  int64_t lds, stride_s;
  int rows, cols, cols_p, count;
};
hipError_t launch_widen(const WidenArgs& p, hipStream_t stream);
// The last 64 of K columns (K % 64 != 0) of src [rows][lds] for the tiles: dst
// [rows_p][64], zeros for those of a slab of 64 before the last and past `rows`.
struct TailArgs {
  const half_t* src;
  half_t* dst;
  int64_t lds;
  int rows, rows_p, K;
};
hipError_t launch_tail(const TailArgs& p, hipStream_t stream);

// A lane's 8 x 8 block of 16-bit values with rows and columns exchanged.
__device__ __forceinline__ void turn8(hgemm::h8 (&v)[8]) {
  typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
  u32x4 x[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) x[e] = __builtin_bit_cast(u32x4, v[e]);
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    u32x4 w;
#pragma unroll
    for (int q = 0; q < 4; ++q)   // bytes of {second, first}: the low or the high halves
      w[q] = __builtin_amdgcn_perm(x[2 * q + 1][k >> 1], x[2 * q][k >> 1],
                                   k & 1 ? 0x07060302u : 0x05040100u);
    v[k] = __builtin_bit_cast(hgemm::h8, w);
  }
}

// The four waves' sums, 16 rows at a time, in the order of the waves; complete in
// wave 0.
template <int RB>
__device__ __forceinline__ void add_up(hgemm::f4 (&acc)[RB][8], hgemm::f4* lds, int wave, int lane) {
#pragma unroll
  for (int q = 0; q < RB; ++q) {
    __syncthreads();
    if (wave > 0) {
#pragma unroll
      for (int e = 0; e < 8; ++e) lds[((wave - 1) * 8 + e) * 64 + lane] = acc[q][e];
    }
    __syncthreads();
    if (wave == 0) {
      for (int w = 0; w + 1 < 4; ++w)
#pragma unroll
        for (int e = 0; e < 8; ++e) acc[q][e] += lds[(w * 8 + e) * 64 + lane];
    }
  }
}

// Row m's adapter: its number, -1 for none, -2 for one that does not exist.
__device__ __forceinline__ int adapter_of(const long long* ids, int64_t m, int S) {
  const long long id = ids[m];
  return id < 0 ? -1 : id >= S ? -2 : (int)id;
}

}  // namespace tune
}  // namespace mi355gemm

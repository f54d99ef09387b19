// Shared by the forms of gemm_ortho: ortho.hip, on the tile kernel,
// ortho_small.hip, for a shorter side of up to 64, and ortho_mid.hip between them.
#pragma once

#include "tune.hpp"

namespace mi355gemm {
namespace tune {
namespace ortho {

typedef _Float16 h8 __attribute__((ext_vector_type(8)));
constexpr int kThreads = 256;
constexpr int kScaleX = 12, kScaleA = 10;   // powers of two of what is stored
constexpr int kNormBlocks = 256;            // partial sums of a matrix, at most
constexpr int kSplitSteps = 3;              // iterates 0 .. 2 are held in two values
enum { kF32 = -1 };                         // beside GEMM_TYPE_F16 and GEMM_TYPE_BF16

__device__ __forceinline__ float load_one(const void* g, int64_t i, int type) {
  if (type == kF32) return static_cast<const float*>(g)[i];
  const half_t w = static_cast<const half_t*>(g)[i];
  return type == GEMM_TYPE_BF16 ? word_to_f32<kFmtBF16>(w) : word_to_f32<kFmtF16>(w);
}

// Eight values of a row at columns c .., zeros past n; any alignment.
__device__ __forceinline__ void load8(const void* g, int64_t row, int c, int n, int type,
                                      float (&v)[8]) {
  if (c + 8 <= n) {
    if (type == kF32) {
      __builtin_memcpy(v, static_cast<const float*>(g) + row + c, 32);
    } else {
      h8 w;
      __builtin_memcpy(&w, static_cast<const half_t*>(g) + row + c, 16);
#pragma unroll
      for (int e = 0; e < 8; ++e)
        v[e] = type == GEMM_TYPE_BF16 ? word_to_f32<kFmtBF16>(w[e]) : word_to_f32<kFmtF16>(w[e]);
    }
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = c + e < n ? load_one(g, row + c + e, type) : 0.f;
  }
}

struct StartArgs {
  const void* G;
  int64_t ldg, stride_g;
  int type, m, n, L, blocks;   // blocks: partial sums of a matrix
  double* sums;                // [L][blocks]
  float* coef;                 // [L][4] (Growth)
  double eps;
  float next, next_most;       // of Growth at step 0
  half_t *hi, *lo;             // [L][sp][tp]
  int64_t stride_x, tiles;     // tiles: 64 x 64 ones of a matrix (transposed start)
  int sp, tp;
};

// The power of two a matrix is stored with and what is left of 1 / (|G| + eps):
// |G| = f 2^e with f in [0.5, 1), X0 = G 2^-e, rho = 2^e / (|G| + eps).
__device__ __forceinline__ void start_of(const StartArgs& p, int64_t l, double& up, double& rho) {
  double s = 0.;
  for (int i = threadIdx.x & 63; i < p.blocks; i += 64) s += p.sums[l * p.blocks + i];
#pragma unroll
  for (int k = 32; k >= 1; k /= 2) s += __shfl_xor(s, k);
  const double norm = sqrt(s);
  int e = 0;
  if (norm > 0. && norm < __builtin_inf()) (void)frexp(norm, &e);
  up = ldexp(1., kScaleX - e);
  rho = norm > 0. ? ldexp(1., e) / (norm + p.eps) : 1.;
  // an infinite or NaN norm: every value of the result is NaN
  if (!(norm < __builtin_inf())) up = rho = __builtin_nan("");
}

__device__ __forceinline__ void put_coef(const StartArgs& p, int64_t l, double rho) {
  // step 0 sees X0, which is the normalised matrix / rho (under 2^-190 the result is
  // zero in any type)
  float* own = p.coef + 4 * l;
  const float small = rho > 0. && rho < hgemm::kSmall ? (float)fmax(rho * 0x1p64, 0x1p-126)
                                                      : __builtin_inff();
  const float given[4] = {0.f, 0.f, 0.f, small};
  const double back = 1. / hgemm::growth_rate(given, p.next, p.next_most);
  own[0] = (float)(rho * rho * rho * rho * rho * back);
  own[1] = (float)(rho * rho * rho * back);
  own[2] = (float)(rho * back);
  own[3] = small;
}
// The factors of step k, and of the result (k = steps).
inline hgemm::Growth growth_of(const float* coef, const float* coeffs, int k, int steps) {
  hgemm::Growth g;
  g.coef = coef;
  g.first = k == 0;
  double now = 0x1p-64, most = now;
  for (int i = 0; i <= k; ++i) {
    if (i == k) {
      g.now = (float)now;
      g.most = (float)most;
      if (k == steps) break;
    }
    constexpr double s2 = (double)hgemm::kSmall * hgemm::kSmall;
    const float* f = coeffs + 3 * i;
    // (coefficients of next to nothing: by something, so that it can be divided by)
    const double grows =
        fmax(fabs((double)f[0]) + fabs((double)f[1]) * s2 + fabs((double)f[2]) * s2 * s2, 0x1p-10);
    now *= grows;
    most = fmax(most, now);
    if (i == k) {
      g.next = (float)now;
      g.next_most = (float)most;
      g.inverse = (float)(1. / grows);
    }
  }
  return g;
}

// A shorter side of up to kSmallSide (ortho_small.hip).
constexpr int kSmallSide = 64, kMaxSlabs = 16;
struct SmallPlan {
  int side, slabs, slab;   // the padded side, and the slabs that the longer one is cut into
  size_t x, gram;          // bytes of an iterate's hi (or lo) values, of partial products
  size_t total() const { return 4 * x + 2 * gram; }
};
SmallPlan plan_small(int L, int s, int t);
struct SmallOut {
  void* O;
  int64_t ldo, stride_o;
  int type;
};
// Eight values of the result's row m < m_end, columns n .. (those below n_end).
__device__ __forceinline__ void store_out8(const SmallOut& o, int64_t l, int m, int n, int m_end,
                                           int n_end, const float (&v)[8]) {
  if (m >= m_end || n >= n_end) return;
  const int64_t at = l * o.stride_o + (int64_t)m * o.ldo + n;
  if (o.type == kF32) {
    float* d = static_cast<float*>(o.O) + at;
    if (n + 8 <= n_end) {
      __builtin_memcpy(d, v, 32);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (n + e < n_end) d[e] = v[e];
    }
    return;
  }
  h8 w;
#pragma unroll
  for (int e = 0; e < 8; ++e)
    w[e] = o.type == GEMM_TYPE_BF16 ? f32_to_word<kFmtBF16>(v[e]) : f32_to_word<kFmtF16>(v[e]);
  half_t* d = static_cast<half_t*>(o.O) + at;
  if (n + 8 <= n_end) {
    __builtin_memcpy(d, &w, 16);
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (n + e < n_end) d[e] = w[e];
  }
}
// Everything after the norms; st's hi, lo and tiles are not used.
hipError_t launch_small(const StartArgs& st, const SmallPlan& p, int steps, const float* coeffs,
                        const SmallOut& out, char* ws, hipStream_t stream);

// Middling sizes (ortho_mid.hip).
struct MidPlan {
  int sp, tp, splits, per;
  size_t x, a, sum;        // bytes of a buffer: hi (or lo) of an iterate, of A or C; sums
  size_t total() const { return 8 * x + 4 * a + sum; }
};
MidPlan plan_mid(int L, int s, int t);
hipError_t launch_mid(const StartArgs& st, const MidPlan& p, int steps, const float* coeffs,
                      const SmallOut& out, char* ws, hipStream_t stream);

}  // namespace ortho
}  // namespace tune
}  // namespace mi355gemm

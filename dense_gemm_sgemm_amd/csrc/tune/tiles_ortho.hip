// Tile-kernel instances of an orthogonalised update (TileModes kSym and kMul):
// bound by the matrix cores.  4096^3: half of a symmetric product on 192 x 192
// tiles 77 us (253 tiles for 256 CUs; 50 % busy), C X on 256 x 256 112 us (62 %).
#include "hgemm_shapes.hpp"
#include "tune.hpp"

namespace mi355gemm {
namespace tune {

using hshape::BK;
constexpr int GM = 8;

namespace {

// Tile-times as in hgemm_shapes.hpp; `each` tiles of a matrix.
struct Shape {
  int bm, bn, per_cu;
  int64_t time, time_alone;
};
template <typename F>
int choose(const Shape* s, int n, int M, int N, int batch, int cus, F each) {
  int best = -1;
  int64_t best_cost = 0;
  for (int i = 0; i < n; ++i) {
    if (M < s[i].bm || N < s[i].bn) continue;
    const int64_t tiles = each(s[i]) * batch, slots = (int64_t)s[i].per_cu * cus;
    const int64_t cost = (tiles + slots - 1) / slots * (tiles <= cus ? s[i].time_alone : s[i].time);
    if (best < 0 || cost < best_cost) {
      best = i;
      best_cost = cost;
    }
  }
  return best;
}

constexpr Shape kMulShapes[] = {
    {256, 256, 1, 256 * 256, 256 * 256},
    {128, 128, 2, 2 * 128 * 128 * 6 / 5, 128 * 128 * 8 / 5},
    {192, 256, 1, 192 * 256 * 11 / 10, 192 * 256 * 11 / 10},
};

typedef float f4 __attribute__((ext_vector_type(4)));
typedef _Float16 h4 __attribute__((ext_vector_type(4)));

struct JoinArgs {
  OrthoExtra x;
  int64_t ld;
  int M, bm, blocks;   // blocks: of 64 rows of a tile
};

// The ranges of the tiles that were cut: a workgroup adds up 64 x 64 of a tile
// in order and stores it on both sides of the diagonal, the other one through
// LDS (rows of 65 floats).  What kSym's own end does with alpha * acc.
__global__ __launch_bounds__(256) void join_kernel(JoinArgs p, int64_t base) {
  __shared__ float turned[64][65];
  const OrthoExtra& x = p.x;
  const int64_t id = base + blockIdx.x;
  const int sub = p.blocks * p.blocks;
  const uint32_t rest = (uint32_t)(id / sub), tile = x.whole + rest;
  const int bi = (int)(id % sub) / p.blocks, bj = (int)(id % sub) % p.blocks;
  const int l = (int)(tile / x.tiles_each), i = (int)(tile % x.tiles_each);
  int tm = (int)((sqrtf(8.f * (float)i + 1.f) - 1.f) * 0.5f);
  while (tm * (tm + 1) / 2 > i) --tm;
  while ((tm + 1) * (tm + 2) / 2 <= i) ++tm;
  const int tn = i - tm * (tm + 1) / 2;
  const int m_tile = min(tm * p.bm, p.M - p.bm), n_tile = min(tn * p.bm, p.M - p.bm);
  const int m0 = m_tile + 64 * bi, n0 = n_tile + 64 * bj;
  // (blocks of an earlier tile, and those above the diagonal: by the other ones)
  if (m0 < tm * p.bm || n0 < tn * p.bm || n0 > m0) return;
  float beta = x.beta, gamma = x.gamma, alpha = 1.f;
  if (x.growth.coef) {
    float fb, fa;
    hgemm::growth_factors(x.growth, x.growth.coef + 4 * l, alpha, fb, fa);
    beta *= fb;
    gamma *= fa;
  }
  const int64_t stride = (int64_t)x.rest * p.bm * p.bm;
  const float* src = x.sum + (int64_t)rest * p.bm * p.bm + (int64_t)(64 * bi) * p.bm + 64 * bj;
  const int64_t at = l * x.stride_c;
  f4 v[4];
  const int c = 4 * (threadIdx.x & 15), r = threadIdx.x >> 4;
#pragma unroll
  for (int u = 0; u < 4; ++u) v[u] = f4{0.f, 0.f, 0.f, 0.f};
  for (int s = 0; s < x.splits; ++s)
#pragma unroll
    for (int u = 0; u < 4; ++u) v[u] += *(const f4*)(src + s * stride + (r + 16 * u) * p.bm + c);
  auto put = [&](int row, int col, f4 w) {
    h4 hi, lo;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      hi[e] = (half_t)w[e];
      lo[e] = (half_t)(w[e] - (float)hi[e]);
    }
    const int64_t q = at + (int64_t)row * p.ld + col;
    *(h4*)(x.hi + q) = hi;
    if (x.lo) *(h4*)(x.lo + q) = lo;
  };
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    const int m = m0 + r + 16 * u, n = n0 + c;
    v[u] *= alpha;
    if (x.q_hi) {
      const int64_t q = at + (int64_t)m * p.ld + n;
      const h4 qh = *(const h4*)(x.q_hi + q);
      h4 ql = {};
      if (x.q_lo) ql = *(const h4*)(x.q_lo + q);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        v[u][e] += beta * ((float)qh[e] + (float)ql[e]);
        if (m == n + e) v[u][e] += gamma;
      }
    }
    put(m, n, v[u]);
#pragma unroll
    for (int e = 0; e < 4; ++e) turned[c + e][r + 16 * u] = v[u][e];
  }
  if (m0 == n0) return;
  __syncthreads();
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    const int row = r + 16 * u;
    put(n0 + row, m0 + c,
        f4{turned[row][c], turned[row][c + 1], turned[row][c + 2], turned[row][c + 3]});
  }
}

}  // namespace

hipError_t launch_sym_tiles(const Args16& a, const OrthoExtra& x, const SymPlan& plan, int batch,
                            int cus, hipStream_t stream) {
  using hgemm::kSym;
  OrthoExtra y = x;
  y.whole = plan.whole;
  y.rest = plan.rest;
  y.splits = plan.splits;
  y.per = plan.per;
  hipError_t e = hipErrorInvalidValue;
  switch (plan.shape) {
    case 0:
      e = hgemm::launch_ortho<256, 256, BK, 4, 2, GM, 1, 2, 0, kSym>(a, y, batch, cus, stream);
      break;
    case 1:
      e = hgemm::launch_ortho<128, 128, BK, 2, 2, GM, 0, 0, 0, kSym>(a, y, batch, 2 * cus, stream);
      break;
    case 2:
      e = hgemm::launch_ortho<192, 192, BK, 4, 2, GM, 1, 0, 0, kSym>(a, y, batch, cus, stream);
      break;
  }
  if (e != hipSuccess || plan.rest == 0) return e;
  const int64_t t = (a.M + plan.bm - 1) / plan.bm;
  y.tiles_each = (uint32_t)(t * (t + 1) / 2);
  const JoinArgs j{y, a.ldc, a.M, plan.bm, plan.bm / 64};
  return launch_tiles((const void*)join_kernel, j, (int64_t)plan.rest * j.blocks * j.blocks, 256, 0,
                      stream);
}

hipError_t launch_mul_tiles(const Args16& a, const OrthoExtra& x, bool a_kmajor, int batch, int cus,
                            hipStream_t stream) {
  using hgemm::kMul;
  auto each = [&](const Shape& s) {
    return (int64_t)((a.M + s.bm - 1) / s.bm) * ((a.N + s.bn - 1) / s.bn);
  };
  if (a_kmajor) {
    if (choose(kMulShapes, 2, a.M, a.N, batch, cus, each) == 0)
      return hgemm::launch_ortho<256, 256, BK, 4, 2, GM, 1, 2, 2, kMul>(a, x, batch, cus, stream);
    return hgemm::launch_ortho<128, 128, BK, 2, 2, GM, 0, 0, 2, kMul>(a, x, batch, 2 * cus, stream);
  }
  switch (choose(kMulShapes, 3, a.M, a.N, batch, cus, each)) {
    case 0:
      return hgemm::launch_ortho<256, 256, BK, 4, 2, GM, 1, 2, 1, kMul>(a, x, batch, cus, stream);
    case 1:
      return hgemm::launch_ortho<128, 128, BK, 2, 2, GM, 0, 0, 1, kMul>(a, x, batch, 2 * cus,
                                                                       stream);
    case 2:
      return hgemm::launch_ortho<192, 256, BK, 4, 2, GM, 1, 2, 1, kMul>(a, x, batch, cus, stream);
    default:
      return hipErrorInvalidValue;
  }
}

}  // namespace tune
}  // namespace mi355gemm

// gemm_ortho for matrices of middling size: a step of the tile kernel's launches
// is mostly its beginning and end there (9 us of 12 for a 200 x 256 matrix),
// so these are 64 x 64 tiles with short code.
//
// All three products are of rows with rows: beside X [s][t] its transpose [t][s]
// is kept, A and C are symmetric.  Everything is in two binary16 values with
// three products for one, as in ortho_small.hip.  A workgroup's four waves take
// 32 x 32 of a tile each; slabs of 64 of K go through registers into two LDS
// stages, one slab ahead.  The tile's values then go to LDS in fp32 and from
// there, rounded, to both places they are kept in, in whole 16-byte pieces.
//
// X X^T over a long side is cut into ranges whose fp32 sums a second kernel adds.
#include "ortho.hpp"

namespace mi355gemm {
namespace tune {
namespace ortho {
namespace {

using hgemm::f4;
constexpr int BT = 64, kPitch = BT + 8;            // a slab row in LDS, 16-bit values
constexpr int kMat = BT * kPitch;                  // values of one operand's slab
constexpr int kOutPitch = BT + 4;                  // fp32

struct Two {
  half_t* hi;
  half_t* lo;
};
struct MidArgs {
  Two a, b;                    // rows of the product's two sides
  int64_t lda, ldb, stride_a, stride_b;
  int slabs, cols;             // of 64 each: K, and the tiles across a matrix
  int sym, tiles;              // sym: tiles on and below the diagonal
  int splits, per;             // ranges of K (1: none)
  float* sum;                  // [matrix][range][tile][64][64]
  // out = alpha acc + beta q + gamma [m == n], times the matrix's own factors (the
  // last one: factor), to `to` and turned to `turned`
  Two to, turned, q;
  int64_t ldt, ldtt, stride_t;
  float alpha, beta, gamma;
  hgemm::Growth growth;
  // the last one: rounded to the result instead, turned or not
  SmallOut out;
  int last, tall, m_end, n_end;   // (of the result as it lies)
};

__device__ __forceinline__ void tile_of(const MidArgs& p, int i, int& tm, int& tn) {
  if (!p.sym) {
    tm = i / p.cols;
    tn = i - tm * p.cols;
    return;
  }
  tm = (int)((sqrtf(8.f * (float)i + 1.f) - 1.f) * 0.5f);
  while (tm * (tm + 1) / 2 > i) --tm;
  while ((tm + 1) * (tm + 2) / 2 <= i) ++tm;
  tn = i - tm * (tm + 1) / 2;
}

// Eight values of a tile's row (or column) in fp32, to hi and lo.
__device__ __forceinline__ void put8(Two to, int64_t at, const float (&v)[8]) {
  h8 hi, lo;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    hi[e] = (half_t)v[e];
    lo[e] = (half_t)(v[e] - (float)hi[e]);
  }
  *(h8*)(to.hi + at) = hi;
  *(h8*)(to.lo + at) = lo;
}

// A tile whose sums lie in `t` [64][kOutPitch], to where it is kept.
__device__ __forceinline__ void finish_tile(const MidArgs& p, float* t, int64_t l, int tm, int tn) {
  const int row = threadIdx.x >> 2, c0 = (threadIdx.x & 3) * 16;
  const int m0 = tm * BT, n0 = tn * BT;
  float alpha = p.alpha, beta = p.beta, gamma = p.gamma;
  if (p.last) {
    alpha *= hgemm::growth_rate(p.growth.coef + 4 * l, p.growth.now, p.growth.most);
  } else if (p.growth.coef) {
    float fc, fb, fa;
    hgemm::growth_factors(p.growth, p.growth.coef + 4 * l, fc, fb, fa);
    alpha *= fc;
    beta *= fb;
    gamma *= fa;
  }
  __syncthreads();
  if (!p.last || !p.tall) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int c = c0 + 8 * h;
      float v[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = alpha * t[row * kOutPitch + c + e];
      const int64_t at = l * p.stride_t + (int64_t)(m0 + row) * p.ldt + n0 + c;
      if (p.q.hi) {
        const h8 qh = *(const h8*)(p.q.hi + at), ql = *(const h8*)(p.q.lo + at);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          v[e] += beta * ((float)qh[e] + (float)ql[e]);
          if (m0 + row == n0 + c + e) v[e] += gamma;
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) t[row * kOutPitch + c + e] = v[e];
      }
      if (p.last) {
        store_out8(p.out, l, m0 + row, n0 + c, p.m_end, p.n_end, v);
      } else {
        put8(p.to, at, v);
      }
    }
  }
  if (p.last ? !p.tall : p.sym && tm == tn) return;
  if (p.q.hi) __syncthreads();
  const float again = p.q.hi ? 1.f : alpha;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int c = c0 + 8 * h;
    float v[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = again * t[(c + e) * kOutPitch + row];
    if (p.last)
      store_out8(p.out, l, n0 + row, m0 + c, p.m_end, p.n_end, v);
    else
      put8(p.turned, l * p.stride_t + (int64_t)(n0 + row) * p.ldtt + m0 + c, v);
  }
}

__global__ __launch_bounds__(kThreads) void mid_kernel(MidArgs p, int64_t base) {
  __shared__ __attribute__((aligned(16))) half_t lds[2][4][kMat];   // stage; a hi, a lo, b hi, b lo
  static_assert(BT * kOutPitch * 4 <= 4 * kMat * 2, "the tile takes a stage's place");
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int g = lane >> 4, r = lane & 15, wm = (wave >> 1) * 32, wn = (wave & 1) * 32;
  int64_t id = base + blockIdx.x;
  const int tile = (int)(id % p.tiles);
  id /= p.tiles;
  const int range = (int)(id % p.splits);
  const int64_t l = id / p.splits;
  int tm, tn;
  tile_of(p, tile, tm, tn);
  const int s0 = range * p.per, s1 = s0 + p.per < p.slabs ? s0 + p.per : p.slabs;

  // a thread's two pieces of each operand's slab: rows i, i + 32 at columns 8 j
  const int i = threadIdx.x >> 3, j = threadIdx.x & 7;
  const half_t* src[4];
  src[0] = p.a.hi + l * p.stride_a + (int64_t)(tm * BT + i) * p.lda + 8 * j;
  src[1] = p.a.lo + (src[0] - p.a.hi);
  src[2] = p.b.hi + l * p.stride_b + (int64_t)(tn * BT + i) * p.ldb + 8 * j;
  src[3] = p.b.lo + (src[2] - p.b.hi);
  h8 v[4][2];
  auto load = [&](int s) __attribute__((always_inline)) {
#pragma unroll
    for (int q = 0; q < 4; ++q)
#pragma unroll
      for (int h = 0; h < 2; ++h)
        v[q][h] = *(const h8*)(src[q] + (int64_t)s * BT + h * 32 * (q < 2 ? p.lda : p.ldb));
  };
  auto store = [&](int stage) __attribute__((always_inline)) {
#pragma unroll
    for (int q = 0; q < 4; ++q)
#pragma unroll
      for (int h = 0; h < 2; ++h) *(h8*)(lds[stage][q] + (i + 32 * h) * kPitch + 8 * j) = v[q][h];
  };
  f4 acc[2][2];
#pragma unroll
  for (int x = 0; x < 2; ++x)
#pragma unroll
    for (int y = 0; y < 2; ++y) acc[x][y] = f4{0.f, 0.f, 0.f, 0.f};
  load(s0);
  store(0);
  __syncthreads();
  for (int s = s0; s < s1; ++s) {
    const int stage = (s - s0) & 1;
    if (s + 1 < s1) load(s + 1);
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      h8 f[4][2];
#pragma unroll
      for (int q = 0; q < 4; ++q)
#pragma unroll
        for (int x = 0; x < 2; ++x)
          f[q][x] = *(const h8*)(lds[stage][q] + ((q < 2 ? wm : wn) + 16 * x + r) * kPitch + 32 * k +
                                 8 * g);
#pragma unroll
      for (int x = 0; x < 2; ++x)
#pragma unroll
        for (int y = 0; y < 2; ++y) {
          // b first: a lane gets four columns of one row
          acc[x][y] = hgemm::mfma16<kFmtF16>(f[2][y], f[0][x], acc[x][y]);
          acc[x][y] = hgemm::mfma16<kFmtF16>(f[3][y], f[0][x], acc[x][y]);
          acc[x][y] = hgemm::mfma16<kFmtF16>(f[2][y], f[1][x], acc[x][y]);
        }
    }
    if (s + 1 < s1) store(1 - stage);
    __syncthreads();
  }
  float* t = reinterpret_cast<float*>(&lds[0][0][0]);
  int pitch = kOutPitch;
  if (p.splits > 1) {
    t = p.sum + ((l * p.splits + range) * p.tiles + tile) * (BT * BT);
    pitch = BT;
  }
#pragma unroll
  for (int x = 0; x < 2; ++x)
#pragma unroll
    for (int y = 0; y < 2; ++y)
      *(f4*)(t + (wm + 16 * x + r) * pitch + wn + 16 * y + 4 * g) = acc[x][y];
  if (p.splits == 1) finish_tile(p, t, l, tm, tn);
}

// The ranges of a tile, added in order.
__global__ __launch_bounds__(kThreads) void mid_join_kernel(MidArgs p, int64_t base) {
  __shared__ __attribute__((aligned(16))) float t[BT * kOutPitch];
  const int64_t id = base + blockIdx.x, l = id / p.tiles;
  const int tile = (int)(id % p.tiles);
  int tm, tn;
  tile_of(p, tile, tm, tn);
  const float* src = p.sum + (l * p.splits * p.tiles + tile) * (BT * BT);
  const int c = 4 * (threadIdx.x & 15), r = threadIdx.x >> 4;
  f4 v[4];
#pragma unroll
  for (int u = 0; u < 4; ++u) v[u] = f4{0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
  for (int s = 0; s < p.splits; ++s)
#pragma unroll
    for (int u = 0; u < 4; ++u)
      v[u] += *(const f4*)(src + (int64_t)s * p.tiles * (BT * BT) + (r + 16 * u) * BT + c);
#pragma unroll
  for (int u = 0; u < 4; ++u) *(f4*)(t + (r + 16 * u) * kOutPitch + c) = v[u];
  finish_tile(p, t, l, tm, tn);
}

// X0 and its transpose from G, a 64 x 64 tile a workgroup.
__global__ __launch_bounds__(kThreads) void mid_start_kernel(StartArgs st, MidArgs p, int64_t base) {
  __shared__ __attribute__((aligned(16))) float t[BT * kOutPitch];
  const int64_t id = base + blockIdx.x, l = id / p.tiles;
  const int tile = (int)(id % p.tiles), tm = tile / p.cols, tn = tile % p.cols;   // of X
  double up, rho;
  start_of(st, l, up, rho);
  if (tile == 0 && threadIdx.x == 0) put_coef(st, l, rho);
  const char* G = static_cast<const char*>(st.G) + l * st.stride_g * (st.type == kF32 ? 4 : 2);
  const bool tall = st.m > st.n;
  const int r0 = (tall ? tn : tm) * BT, c0 = (tall ? tm : tn) * BT;   // in G
  const int row = threadIdx.x >> 2;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int c = (threadIdx.x & 3) * 16 + 8 * h;
    float v[8] = {};
    if (r0 + row < st.m && c0 + c < st.n)
      load8(G, (int64_t)(r0 + row) * st.ldg, c0 + c, st.n, st.type, v);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float x = (float)((double)v[e] * up);
      t[tall ? (c + e) * kOutPitch + row : row * kOutPitch + c + e] = x;
    }
  }
  finish_tile(p, t, l, tm, tn);
}

}  // namespace

MidPlan plan_mid(int L, int s, int t) {
  MidPlan p;
  p.sp = (int)round_up(s, BT);
  p.tp = (int)round_up(t, BT);
  const int rows = p.sp / BT, tiles = rows * (rows + 1) / 2, slabs = p.tp / BT;
  // ranges of about eight slabs while the launch is small
  const int64_t most = std::max<int64_t>(1, 1024 / ((int64_t)tiles * L));
  p.splits = slabs <= 12 ? 1 : (int)std::min<int64_t>(most, (slabs + 7) / 8);
  p.per = (slabs + p.splits - 1) / p.splits;
  p.splits = (slabs + p.per - 1) / p.per;
  p.x = round256((size_t)L * p.sp * p.tp * 2);
  p.a = round256((size_t)L * p.sp * p.sp * 2);
  p.sum = p.splits > 1 ? (size_t)L * p.splits * tiles * BT * BT * sizeof(float) : 0;
  return p;
}

hipError_t launch_mid(const StartArgs& st, const MidPlan& p, int steps, const float* coeffs,
                      const SmallOut& out, char* ws, hipStream_t stream) {
  auto two = [&](size_t bytes) {
    const Two t{reinterpret_cast<half_t*>(ws), reinterpret_cast<half_t*>(ws + bytes)};
    ws += 2 * bytes;
    return t;
  };
  Two x[2], xt[2];
  for (int i = 0; i < 2; ++i) {
    x[i] = two(p.x);
    xt[i] = two(p.x);
  }
  const Two a = two(p.a), c = two(p.a);
  float* sum = reinterpret_cast<float*>(ws);
  const int rows = p.sp / BT, cols = p.tp / BT, half = rows * (rows + 1) / 2;
  const int64_t stride_x = (int64_t)p.sp * p.tp, stride_a = (int64_t)p.sp * p.sp;
  MidArgs m{};
  m.cols = cols;
  m.tiles = rows * cols;
  m.splits = 1;
  m.alpha = 1.f;
  m.to = x[0];
  m.turned = xt[0];
  m.ldt = p.tp;
  m.ldtt = p.sp;
  m.stride_t = stride_x;
  {
    constexpr int64_t kMax = int64_t(1) << 20;
    const int64_t tiles = (int64_t)st.L * m.tiles;
    for (int64_t base = 0; base < tiles; base += kMax) {
      StartArgs s = st;
      int64_t b = base;
      void* args[] = {&s, &m, &b};
      const hipError_t e = hipLaunchKernel((const void*)mid_start_kernel,
                                           dim3((unsigned)std::min(kMax, tiles - base)),
                                           dim3(kThreads), args, 0, stream);
      if (e != hipSuccess) return e;
    }
  }
  auto launch = [&](const MidArgs& k) {
    hipError_t e = launch_tiles((const void*)mid_kernel, k, (int64_t)st.L * k.tiles * k.splits,
                                kThreads, 0, stream);
    if (e == hipSuccess && k.splits > 1)
      e = launch_tiles((const void*)mid_join_kernel, k, (int64_t)st.L * k.tiles, kThreads, 0, stream);
    return e;
  };
  const bool tall = st.m > st.n;
  for (int k = 0; k < steps; ++k) {
    const int i = k & 1;
    const float* f = coeffs + 3 * k;
    m = MidArgs{};
    m.a = m.b = x[i];
    m.lda = m.ldb = p.tp;
    m.stride_a = m.stride_b = stride_x;
    m.slabs = cols;
    m.cols = rows;
    m.sym = 1;
    m.tiles = half;
    m.splits = p.splits;
    m.per = p.per;
    m.sum = sum;
    m.to = m.turned = a;
    m.ldt = m.ldtt = p.sp;
    m.stride_t = stride_a;
    m.alpha = ldexpf(1.f, kScaleA - 2 * kScaleX);
    hipError_t e = launch(m);
    if (e != hipSuccess) return e;
    m.a = m.b = m.q = a;
    m.lda = m.ldb = p.sp;
    m.stride_a = m.stride_b = stride_a;
    m.slabs = m.per = rows;
    m.splits = 1;
    m.to = m.turned = c;
    m.alpha = ldexpf(f[2], -kScaleA);
    m.beta = f[1];
    m.gamma = ldexpf(f[0], kScaleA);
    m.growth = growth_of(st.coef, coeffs, k, steps);
    e = launch(m);
    if (e != hipSuccess) return e;
    m = MidArgs{};
    m.a = c;
    m.b = xt[i];
    m.lda = m.ldb = p.sp;
    m.stride_a = stride_a;
    m.stride_b = stride_x;
    m.slabs = m.per = rows;
    m.cols = cols;
    m.tiles = rows * cols;
    m.splits = 1;
    m.to = x[1 - i];
    m.turned = xt[1 - i];
    m.ldt = p.tp;
    m.ldtt = p.sp;
    m.stride_t = stride_x;
    m.last = k + 1 == steps;
    if (m.last) m.growth = growth_of(st.coef, coeffs, steps, steps);
    m.alpha = ldexpf(1.f, -kScaleA - (m.last ? kScaleX : 0));
    m.out = out;
    m.tall = tall;
    m.m_end = st.m;
    m.n_end = st.n;
    e = launch(m);
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace ortho
}  // namespace tune
}  // namespace mi355gemm

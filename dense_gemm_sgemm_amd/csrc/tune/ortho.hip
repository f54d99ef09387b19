// gemm_ortho: an update orthogonalised by Newton-Schulz products.  C entry
// points and the kernels that make the first iterate; the products are modes
// of the tile kernel (kSym, kMul).
//
// The iterate is kept with its shorter side s as rows, [s][t], zero past the
// matrix in whole slabs of 64 (zero rows and columns stay zero).  A step is
//     A = X X^T            (kSym: half of it is computed, both halves stored)
//     C = a I + b A + c A^2   (kSym)
//     X = C X              (kMul, X read K-major; the last step of a tall
//                           matrix makes X^T C instead, so nothing is transposed)
// in binary16 on the matrix cores with fp32 sums.  Values are stored times
// powers of two (X 2^12, A and C 2^10), which puts the whole range they can
// have into binary16's normal one.
//
// Precision.  What a step adds to X must stay small beside the smallest part
// of X that counts, and a strong direction has it buried: X rounded to 11 bits
// carries noise of 2^-12 of the strong directions' size in every direction,
// and the first steps multiply what is small by 3.4 each.  So the first
// iterate is the input times a power of two, exact for 16-bit inputs (the
// rest of 1 / (|G| + eps) goes into the steps' coefficients, see Growth), and up to
// the third one an iterate is two binary16 values, hi + lo, whose products
// are added up: with momentum whose four strongest directions are 100 times
// the rest in the Frobenius norm, the result is off by 0.11 % instead of 2.4 %
// (bfloat16 throughout: 19 %).  Rounding A and C only turns the strong
// directions by that much.  Outputs in bfloat16 (steps of 0.4 %) take that;
// binary16 and fp32 outputs take two values for X, A and C throughout and
// three products for each one.
#define MI355TUNE_BUILDING 1
#include "ortho.hpp"

namespace mi355gemm {
namespace tune {
namespace {

using namespace ortho;

// Sums of squares, in 64 bits: the squares of fp32 values neither overflow nor
// vanish there, and their sum is as good as exact.  Bound by HBM.
__global__ __launch_bounds__(kThreads) void norm_kernel(StartArgs p, int64_t base) {
  __shared__ double part[kThreads / 64];
  const int64_t block = base + blockIdx.x;
  const int64_t l = block / p.blocks;
  const int b = (int)(block % p.blocks);
  const int chunks = (p.n + 7) / 8;
  const int64_t pieces = (int64_t)p.m * chunks;
  const char* g = static_cast<const char*>(p.G) + l * p.stride_g * (p.type == kF32 ? 4 : 2);
  double s = 0.;
  for (int64_t t = (int64_t)b * kThreads + threadIdx.x; t < pieces;
       t += (int64_t)p.blocks * kThreads) {
    const int64_t row = t / chunks;
    float v[8];
    load8(g, row * p.ldg, (int)(t - row * chunks) * 8, p.n, p.type, v);
#pragma unroll
    for (int e = 0; e < 8; ++e) s += (double)v[e] * (double)v[e];
  }
#pragma unroll
  for (int k = 32; k >= 1; k /= 2) s += __shfl_xor(s, k);
  if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = s;
  __syncthreads();
  if (threadIdx.x != 0) return;
  for (int w = 1; w < kThreads / 64; ++w) s += part[w];
  p.sums[block] = s;
}

__device__ __forceinline__ void put_start(const StartArgs& p, int64_t at, const float (&v)[8],
                                          double up) {
  h8 hi, lo;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const float x = (float)((double)v[e] * up);
    hi[e] = (half_t)x;
    lo[e] = (half_t)(x - (float)hi[e]);
  }
  *(h8*)(p.hi + at) = hi;
  if (p.lo) *(h8*)(p.lo + at) = lo;
}

// X0 as it lies: a thread 8 columns.  Bound by HBM.
__global__ __launch_bounds__(kThreads) void start_kernel(StartArgs p, int64_t base) {
  const int chunks = p.tp / 8;
  const int64_t per = ((int64_t)p.sp * chunks + kThreads - 1) / kThreads;   // workgroups a matrix
  const int64_t l = (base + blockIdx.x) / per, b = (base + blockIdx.x) % per;
  double up, rho;
  start_of(p, l, up, rho);
  if (b == 0 && threadIdx.x == 0) put_coef(p, l, rho);
  const int64_t t = b * kThreads + threadIdx.x;
  if (t >= (int64_t)p.sp * chunks) return;
  const int64_t row = t / chunks;
  const int c = (int)(t - row * chunks) * 8;
  float v[8] = {};
  if (row < p.m && c < p.n)
    load8(static_cast<const char*>(p.G) + l * p.stride_g * (p.type == kF32 ? 4 : 2), row * p.ldg, c,
          p.n, p.type, v);
  put_start(p, l * p.stride_x + row * p.tp + c, v, up);
}

// X0 transposed (more rows than columns): a workgroup a 64 x 64 tile through
// LDS, rows of 65 floats.
__global__ __launch_bounds__(kThreads) void start_t_kernel(StartArgs p, int64_t base) {
  __shared__ float tile[64][65];
  const int64_t l = (base + blockIdx.x) / p.tiles, b = (base + blockIdx.x) % p.tiles;
  double up, rho;
  start_of(p, l, up, rho);
  if (b == 0 && threadIdx.x == 0) put_coef(p, l, rho);
  const int tiles_c = p.sp / 64;
  const int r0 = (int)(b / tiles_c) * 64, c0 = (int)(b % tiles_c) * 64;   // in G
  const char* g = static_cast<const char*>(p.G) + l * p.stride_g * (p.type == kF32 ? 4 : 2);
  for (int t = threadIdx.x; t < 64 * 8; t += kThreads) {
    const int row = t / 8, c = t % 8 * 8;
    float v[8] = {};
    if (r0 + row < p.m && c0 + c < p.n) load8(g, (int64_t)(r0 + row) * p.ldg, c0 + c, p.n, p.type, v);
#pragma unroll
    for (int e = 0; e < 8; ++e) tile[row][c + e] = v[e];
  }
  __syncthreads();
  for (int t = threadIdx.x; t < 64 * 8; t += kThreads) {
    const int row = t / 8, c = t % 8 * 8;   // of X0
    float v[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = tile[c + e][row];
    put_start(p, l * p.stride_x + (int64_t)(c0 + row) * p.tp + r0 + c, v, up);
  }
}

// The workspace: two iterates, A and C (hi, and lo where it is held), the sums
// of squares and the first step's factors.
struct Plan {
  int s, t, sp, tp, blocks;
  bool tall, fine;       // fine: two values throughout
  bool x_lo, x0_lo;      // iterates, the first one, have a second value
  size_t x, a, sums, coef;   // bytes of one buffer
  int x_count, a_count;
  size_t cut;            // fp32 sums of tiles whose K is cut into ranges
  bool small, mid;
  SmallPlan few;
  MidPlan between;
  size_t total() const {
    return sums + coef +
           (small ? few.total() : mid ? between.total() : x_count * x + a_count * a + cut);
  }
};

// The parts of a step's products (see `parts` below) depend on which iterates
// are held in two values: iterate i, of `steps` steps.
bool held(const Plan& p, int i, int steps) {
  // (an iterate that only the last step reads needs no second value)
  return p.fine ? i > 0 || p.x0_lo : i + 1 < steps && i < kSplitSteps && (i > 0 || p.x0_lo);
}
// X X^T and A^2 of a step, planned for kPlanCus CUs: the workspace is sized before
// a device is asked.
SymPlan plan_gram(const Plan& p, int L, bool lo) {
  return plan_sym(p.sp, (p.fine && lo ? 3 : 1) * (p.tp / 64), L, fused::kPlanCus);
}
SymPlan plan_square(const Plan& p, int L) {
  return plan_sym(p.sp, (p.fine ? 3 : 1) * (p.sp / 64), L, fused::kPlanCus);
}

// The short tiles of ortho_mid.hip, where the tile kernel's launches would be
// mostly their beginning and end; they do three products for one throughout, so
// they are worth it for twice as much where the others would too (bf16, fp16; us
// on short and large tiles: 128 x 128 92 and 132, 92 and 190; 256 x 4096 163 and
// 310, 164 and 431; four of 512 x 1024 243 and 253, 242 and 337; sixteen of 384 x
// 512 297 and 217, 297 and 374; 1024 x 1024 264 and 315, 263 and 440; 1024 x 2048
// 354 and 322, 353 and 457; four of 768 x 1024 420 and 291, 420 and 424).
bool by_mid(bool fine, int L, int s, int t) {
  const int64_t size = (int64_t)L * s * t;
  return s <= 1024 && (s > 512 ? size + size / 2 : size) <= (fine ? 5 : 2.5) * (1 << 20);
}

Plan make_plan(int type_g, int type_o, int L, int m, int n, int steps) {
  Plan p{};
  p.tall = m > n;
  p.s = p.tall ? n : m;
  p.t = p.tall ? m : n;
  p.sp = (int)round_up(std::max(p.s, fused::kMinRows), 64);
  p.tp = (int)round_up(std::max(p.t, fused::kMinRows), 64);
  p.fine = type_o != GEMM_TYPE_BF16;
  p.x0_lo = type_g == kF32 && (p.fine || steps > 1);
  p.x_lo = p.fine || steps > 2;
  const int64_t pieces = ((int64_t)m * n + 7) / 8;
  p.blocks = (int)std::min<int64_t>(kNormBlocks, (pieces + 4 * kThreads - 1) / (4 * kThreads));
  p.x = round256((size_t)L * p.sp * p.tp * 2);
  p.a = round256((size_t)L * p.sp * p.sp * 2);
  p.sums = round256((size_t)L * p.blocks * sizeof(double));
  p.coef = round256((size_t)L * 4 * sizeof(float));
  p.small = p.s <= kSmallSide;
  if (p.small) {
    p.few = plan_small(L, p.s, p.t);
    return p;
  }
  p.mid = by_mid(p.fine, L, p.s, p.t);
  if (p.mid) {
    p.between = plan_mid(L, p.s, p.t);
    return p;
  }
  p.x_count = 2 + (p.x_lo || p.x0_lo ? 2 : 0);
  p.a_count = p.fine ? 4 : 2;
  p.cut = plan_square(p, L).sum_bytes();
  for (bool lo : {false, true}) p.cut = std::max(p.cut, plan_gram(p, L, lo).sum_bytes());
  return p;
}

bool bad_types(int type_g, int type_o) {
  return (type_g != GEMM_TYPE_F16 && type_g != GEMM_TYPE_BF16 && type_g != GEMM_TYPE_F32) ||
         (type_o != GEMM_TYPE_F16 && type_o != GEMM_TYPE_BF16 && type_o != GEMM_TYPE_F32);
}
int inner_type(int type) { return type == GEMM_TYPE_F32 ? kF32 : type; }

// Sizes of one matrix below 2^16 keep every count of tiles and every leading
// dimension far inside the tile kernel's 32-bit ranges.
constexpr int kMaxSide = 1 << 16;
constexpr int kMaxSteps = 64;

int check(int type_g, int type_o, int L, int m, int n, int steps) {
  if (L < 0 || m < 0 || n < 0) return GEMM_ERR_NEGATIVE_DIM;
  if (bad_types(type_g, type_o) || steps < 1 || steps > kMaxSteps || m > kMaxSide || n > kMaxSide ||
      L > kMaxSide)
    return GEMM_ERR_BAD_ARG;
  return GEMM_OK;
}

}  // namespace
}  // namespace tune
}  // namespace mi355gemm

using namespace mi355gemm;
using namespace mi355gemm::tune;

extern "C" {

MI355TUNE_API unsigned long long gemm_ortho_workspace(int type_g, int type_o, int L, int m, int n,
                                                      int steps) {
  if (check(type_g, type_o, L, m, n, steps) != GEMM_OK || L == 0 || m == 0 || n == 0) return 0;
  return make_plan(inner_type(type_g), inner_type(type_o), L, m, n, steps).total();
}

MI355TUNE_API int gemm_ortho(int type_g, int type_o, int L, int m, int n, const void* G, int ldg,
                             long long stride_g, int steps, const float* coeffs, float eps, void* O,
                             int ldo, long long stride_o, void* workspace,
                             unsigned long long workspace_bytes, void* stream) {
  const int status = check(type_g, type_o, L, m, n, steps);
  if (status != GEMM_OK) return status;
  if (coeffs == nullptr) return GEMM_ERR_NULL_POINTER;
  if (!(eps >= 0.f)) return GEMM_ERR_BAD_ARG;
  if (L == 0 || m == 0 || n == 0) return GEMM_OK;
  if (fused::bad_ld(ldg, n) || fused::bad_ld(ldo, n) ||
      (L > 1 && (stride_g < 0 || stride_o < (long long)(m - 1) * ldo + n)))
    return GEMM_ERR_BAD_LD;
  if (G == nullptr || O == nullptr) return GEMM_ERR_NULL_POINTER;
  const int tg = inner_type(type_g), to = inner_type(type_o);
  const Plan p = make_plan(tg, to, L, m, n, steps);
  if (!workspace_ok(p.total(), workspace, workspace_bytes)) return GEMM_ERR_WORKSPACE;
  const int cus = check_device();
  if (cus < 0) return cus;
  hipStream_t s = static_cast<hipStream_t>(stream);

  char* ws = static_cast<char*>(workspace);
  const hgemm::Growth start = growth_of(nullptr, coeffs, 0, steps);
  StartArgs st{G, ldg, stride_g, tg, m, n, L, p.blocks, reinterpret_cast<double*>(ws),
               reinterpret_cast<float*>(ws + p.sums), (double)eps, start.next, start.next_most,
               nullptr, nullptr,
               (int64_t)p.sp * p.tp, (int64_t)(p.sp / 64) * (p.tp / 64), p.sp, p.tp};
  ws += p.sums + p.coef;
  hipError_t e = launch_tiles((const void*)norm_kernel, st, (int64_t)L * p.blocks, kThreads, 0, s);
  if (e != hipSuccess) return to_status(e);
  if (p.small)
    return to_status(launch_small(st, p.few, steps, coeffs, SmallOut{O, ldo, stride_o, to}, ws, s));
  if (p.mid)
    return to_status(launch_mid(st, p.between, steps, coeffs, SmallOut{O, ldo, stride_o, to}, ws, s));
  half_t* x[2][2];   // [iterate][hi, lo]
  for (int v = 0; v < 2; ++v)
    for (int i = 0; i < 2; ++i) {
      x[i][v] = 2 * v < p.x_count ? reinterpret_cast<half_t*>(ws) : nullptr;
      if (x[i][v]) ws += p.x;
    }
  half_t *a[2], *c[2];
  for (int v = 0; v < 2; ++v) {
    a[v] = 2 * v < p.a_count ? reinterpret_cast<half_t*>(ws) : nullptr;
    c[v] = a[v] ? reinterpret_cast<half_t*>(ws + p.a) : nullptr;
    if (a[v]) ws += 2 * p.a;
  }
  float* cut = reinterpret_cast<float*>(ws);
  st.hi = x[0][0];
  st.lo = p.x0_lo ? x[0][1] : nullptr;
  const int64_t per = ((int64_t)p.sp * (p.tp / 8) + kThreads - 1) / kThreads;
  e = p.tall ? launch_tiles((const void*)start_t_kernel, st, L * st.tiles, kThreads, 0, s)
             : launch_tiles((const void*)start_kernel, st, L * per, kThreads, 0, s);
  if (e != hipSuccess) return to_status(e);

  // hi hi (+ hi lo (+ lo hi)): the products of two values that count
  auto parts = [](OrthoExtra& y, half_t* const* u, half_t* const* v, bool u_lo, bool v_lo) {
    y.parts = 0;
    auto add = [&](const half_t* q, const half_t* r) {
      y.a[y.parts] = q;
      y.b[y.parts++] = r;
    };
    add(u[0], v[0]);
    if (v_lo) add(u[0], v[1]);
    if (u_lo) add(u[1], v[0]);
  };
  const int64_t stride_x = (int64_t)p.sp * p.tp, stride_a = (int64_t)p.sp * p.sp;
  int cur = 0;
  for (int k = 0; k < steps; ++k) {
    const float* f = coeffs + 3 * k;
    const bool last = k + 1 == steps;
    const bool lo = held(p, k, steps);
    Args16 g{nullptr, nullptr, nullptr, p.tp, p.tp, p.sp, p.sp, p.sp, p.tp};
    OrthoExtra y;
    parts(y, x[cur], x[cur], p.fine && lo, p.fine && lo);
    y.stride_a = y.stride_b = stride_x;
    y.stride_c = stride_a;
    y.hi = a[0];
    y.lo = a[1];
    y.alpha = ldexpf(1.f, kScaleA - 2 * kScaleX);
    y.sum = cut;
    e = launch_sym_tiles(g, y, plan_gram(p, L, lo), L, cus, s);
    if (e != hipSuccess) return to_status(e);

    g.lda = g.ldb = p.sp;
    g.K = p.sp;
    y = OrthoExtra();
    parts(y, a, a, p.fine, p.fine);
    y.stride_a = y.stride_b = y.stride_c = stride_a;
    y.hi = c[0];
    y.lo = c[1];
    y.q_hi = a[0];
    y.q_lo = a[1];
    y.alpha = ldexpf(f[2], -kScaleA);
    y.beta = f[1];
    y.gamma = ldexpf(f[0], kScaleA);
    y.growth = growth_of(st.coef, coeffs, k, steps);
    y.sum = cut;
    e = launch_sym_tiles(g, y, plan_square(p, L), L, cus, s);
    if (e != hipSuccess) return to_status(e);

    y = OrthoExtra();
    const bool turned = last && p.tall;
    if (turned) {   // X^T C
      g = Args16{nullptr, nullptr, nullptr, p.tp, p.sp, 0, p.tp, p.sp, p.sp};
      parts(y, x[cur], c, lo, p.fine);
      y.stride_a = stride_x;
      y.stride_b = stride_a;
    } else {
      g = Args16{nullptr, nullptr, nullptr, p.sp, p.tp, p.tp, p.sp, p.tp, p.sp};
      parts(y, c, x[cur], p.fine, lo);
      y.stride_a = stride_a;
      y.stride_b = stride_x;
    }
    if (last) {
      y.alpha = ldexpf(1.f, -kScaleX - kScaleA);
      y.growth = growth_of(st.coef, coeffs, steps, steps);
      y.out = O;
      y.out_type = to;
      y.ldo = ldo;
      y.stride_o = stride_o;
      y.m_end = m;
      y.n_end = n;
    } else {
      y.alpha = ldexpf(1.f, -kScaleA);
      y.hi = x[1 - cur][0];
      y.lo = held(p, k + 1, steps) ? x[1 - cur][1] : nullptr;
      y.stride_c = stride_x;
    }
    e = launch_mul_tiles(g, y, turned, L, cus, s);
    if (e != hipSuccess) return to_status(e);
    cur = 1 - cur;
  }
  return GEMM_OK;
}

}  // extern "C"

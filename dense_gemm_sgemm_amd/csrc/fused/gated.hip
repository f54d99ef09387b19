// The gated product H = act(X Wg^T) * (X Wu^T) and its gradients: C entry
// points, and the elementwise kernel of the backward pass.
#define MI355FUSED_BUILDING 1
#include "fused.hpp"

namespace mi355gemm {
namespace fused {
namespace {

typedef _Float16 h8 __attribute__((ext_vector_type(8)));
constexpr int kThreads = 256;

// dG and dU as the products of the backward pass read them: rows of ld
// elements, dG's Np columns, then dU's, zero in the columns past N and the
// rows past M; and, for N % 64 != 0, the last 64 columns of each once more in
// `tail` (128 to a row), zero where they lie in a slab of 64 before the last.
struct GradArgs {
  const half_t *G, *U, *dH;
  half_t *dg, *du, *tail;      // dg, du: null for a part that is not asked for
  float* factor;               // fp16: the largest values, then the factor (below), or null for 1
  int64_t ldg, ldu, lddh, ld;
  int M, N, Mp, Np, Nk, act;   // Nk: columns the products sum over (N, or 128 if less)
  int64_t blocks;              // of dG and dU; the ones after them transpose X
  Transpose x;
};

// binary16 holds dG and dU to half a step only between 2^-14 and 65504, which
// dH * U * act'(G) leaves at both ends while the sums over it stay inside (dH of
// 1e-4 and U of 0.02: 1.5 % off; loss-scaled dH of 6000 and U of 100: infinite).
// So in fp16 both are stored times a power of two that brings the largest of
// them to 2^14 .. 2^15, and the fp32 sums are divided by it; a power of two, so
// that values that fit either way are rounded the same.  What is infinite or
// NaN stays so and does not count for the factor.  The area it is passed in:
// kMaxBlocks maxima, one a workgroup of the kernel that looks for them, then
// the factor and its inverse.
constexpr int kMaxBlocks = 256, kMaxThreads = 1024;
constexpr size_t kFactorBytes = 2048;
static_assert((kMaxBlocks + 2) * sizeof(float) <= kFactorBytes, "the factor's area");

// Columns c .. c + 7 of a row of N at any 2-byte address, zero past it.
__device__ __forceinline__ h8 load_cols(const half_t* row, int c, int N) {
  h8 v = {};
  if (c + 8 <= N) {
    __builtin_memcpy(&v, row + c, 16);
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (c + e < N) v[e] = row[c + e];
  }
  return v;
}

// Eight columns of dG and dU from a row's pieces of G, U and dH, in fp32: with
// s = 1 / (1 + e^-g), silu = g s and its slope s (1 + g (1 - s)).
template <int FMT>
__device__ __forceinline__ void gradients(h8 g, h8 u, h8 dh, int act, float (&dg)[8],
                                          float (&du)[8]) {
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const float x = word_to_f32<FMT>(g[e]), y = word_to_f32<FMT>(dh[e]);
    float a = x, slope = 1.f;
    if (act == GEMM_ACT_SILU) {
      const float s = __builtin_amdgcn_rcpf(1.f + __expf(-x));
      a = x * s;
      slope = s * (1.f + x * (1.f - s));
    } else if (act == GEMM_ACT_RELU) {
      a = gate_relu(x);
      slope = x > 0.f ? 1.f : a;   // 0, or NaN for NaN
    }
    dg[e] = y * word_to_f32<FMT>(u[e]) * slope;
    du[e] = y * a;
  }
}

// The largest finite |dG| and |dU| of a workgroup's share (fp16 only).  Bound by
// HBM: 6 bytes read an element; with it the fp16 backward pass takes 2031 instead
// of 1958 us at 4096 x 16384 x 4096, 333 instead of 303 at 2048 x 8192 x 2048
// and 64 instead of 58 at 1000 x 3001 x 768 (two pieces in flight a thread, or
// four times the workgroups: even).
__global__ __launch_bounds__(kMaxThreads) void gated_max_kernel(GradArgs p, int64_t base) {
  __shared__ float part[kMaxThreads / 64];
  const int chunks = (p.N + 7) / 8;
  const int64_t block = base + blockIdx.x, pieces = (int64_t)p.M * chunks;
  float top = 0.f;
  for (int64_t t = block * kMaxThreads + threadIdx.x; t < pieces;
       t += (int64_t)kMaxBlocks * kMaxThreads) {
    const int64_t m = t / chunks;
    const int c = (int)(t % chunks) * 8;   // (past N: zeros)
    float dg[8], du[8];
    gradients<kFmtF16>(load_cols(p.G + m * p.ldg, c, p.N), load_cols(p.U + m * p.ldu, c, p.N),
                       load_cols(p.dH + m * p.lddh, c, p.N), p.act, dg, du);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float a = fabsf(dg[e]), b = fabsf(du[e]);
      top = fmaxf(top, a < __builtin_inff() ? a : 0.f);
      top = fmaxf(top, b < __builtin_inff() ? b : 0.f);
    }
  }
#pragma unroll
  for (int k = 32; k >= 1; k /= 2) top = fmaxf(top, __shfl_xor(top, k));
  if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = top;
  __syncthreads();
  if (threadIdx.x != 0) return;
  for (int w = 1; w < kMaxThreads / 64; ++w) top = fmaxf(top, part[w]);
  p.factor[block] = top;
}

// The factor, found by each wave from the workgroups' maxima: 2^(14 - floor(log2
// top)); 1 where all are 0.
__device__ __forceinline__ float find_factor(const float* maxima) {
  typedef float f4 __attribute__((ext_vector_type(4)));
  static_assert(kMaxBlocks == 4 * 64, "four a lane");
  const f4 v = *(const f4*)(maxima + 4 * (threadIdx.x & 63));
  float top = fmaxf(fmaxf(v[0], v[1]), fmaxf(v[2], v[3]));
#pragma unroll
  for (int k = 32; k >= 1; k /= 2) top = fmaxf(top, __shfl_xor(top, k));
  if (top == 0.f) return 1.f;
  top = fmaxf(top, 0x1p-100f);   // the factor stays finite
  const int exponent = (int)(__float_as_uint(top) >> 23) - 127;
  return __uint_as_float((uint32_t)(127 + 14 - exponent) << 23);
}

// One thread makes 8 columns of dG and dU.  Bound by HBM: 6 bytes read and 4
// written an element.
template <int FMT>
__global__ __launch_bounds__(kThreads) void gated_grad_kernel(GradArgs p, int64_t base) {
  if (base + blockIdx.x >= p.blocks) {
    transpose_tile(p.x, (base + blockIdx.x - p.blocks) * (kThreads / 64) + (threadIdx.x >> 6),
                   threadIdx.x & 63);
    return;
  }
  float f = 1.f;
  if constexpr (FMT == kFmtF16) {
    if (p.factor) {
      f = find_factor(p.factor);
      if (base + blockIdx.x == 0 && threadIdx.x == 0) {
        p.factor[kMaxBlocks] = f;
        p.factor[kMaxBlocks + 1] = 1.f / f;
      }
    }
  }
  const int main = p.Np / 8, chunks = main + (p.tail ? 8 : 0);
  const int64_t t = (base + blockIdx.x) * kThreads + threadIdx.x;
  if (t >= (int64_t)p.Mp * chunks) return;
  const int64_t m = t / chunks;
  const int q = (int)(t % chunks);
  const bool is_tail = q >= main;
  const int c = is_tail ? p.Nk - 64 + 8 * (q - main) : 8 * q;
  const int first = is_tail ? (p.Nk - 1) / 64 * 64 : 0;   // first column that counts
  h8 dg = {}, du = {};
  if (m < p.M && c < p.N) {
    float xg[8], xu[8];
    gradients<FMT>(load_cols(p.G + m * p.ldg, c, p.N), load_cols(p.U + m * p.ldu, c, p.N),
                   load_cols(p.dH + m * p.lddh, c, p.N), p.act, xg, xu);
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (c + e >= first && c + e < p.N) {
        dg[e] = f32_to_word<FMT>(FMT == kFmtF16 ? xg[e] * f : xg[e]);
        du[e] = f32_to_word<FMT>(FMT == kFmtF16 ? xu[e] * f : xu[e]);
      }
  }
  if (is_tail) {
    half_t* d = p.tail + m * 128 + 8 * (q - main);
    *(h8*)d = dg;
    *(h8*)(d + 64) = du;
  } else {
    if (p.dg) *(h8*)(p.dg + m * p.ld + c) = dg;
    if (p.du) *(h8*)(p.du + m * p.ld + c) = du;
  }
}

int check(int type, int act, int M, int N, int K) {
  const int status = check_sizes(M, N, K);
  if (status != GEMM_OK) return status;
  return bad_type(type) || bad_act(act) ? GEMM_ERR_BAD_ARG : GEMM_OK;
}

const half_t* in16(const void* p) { return static_cast<const half_t*>(p); }
half_t* out16(void* p) { return static_cast<half_t*>(p); }

// The workspace of the backward pass: dG | dU, their tails, X^T, padded copies
// of the weights, fp32 sums of dX, the factor's area (fp16).  That is one range
// more of the sums where there are any.  Without dX, fp16 makes dG and dU one
// after the other in the first half of their place, and the area is in the
// second.
struct BwdPlan {
  int Mp, Np, Nk;         // Mp: whole slabs of rows (they are summed over for dW)
  int64_t ld;
  bool tail;
  GradXPlan gx;
  bool lone;              // dG and dU in turn
  size_t bytes_d, bytes_tail, bytes_x = 0, bytes_g = 0, bytes_u = 0, bytes_sum = 0;
  size_t bytes_factor = 0;
  size_t total() const {
    return bytes_d + bytes_tail + bytes_x + bytes_g + bytes_u + bytes_sum + bytes_factor;
  }
};
BwdPlan plan_bwd(int type, int M, int N, int K, Mat Wg, Mat Wu, bool dx, bool dw) {
  BwdPlan p;
  p.Mp = pad_slabs(M);
  p.Nk = pad_rows(N);
  p.Np = (int)line_ld(p.Nk);
  p.lone = type == GEMM_TYPE_F16 && !dx;
  p.ld = (p.lone ? 1 : 2) * (int64_t)p.Np;
  p.tail = dx && p.Nk % 64 != 0;
  p.bytes_d = round256((size_t)p.Mp * p.Np * 4);
  p.bytes_tail = p.tail ? (size_t)p.Mp * 256 : 0;
  if (dw) p.bytes_x = round256((size_t)pad_k(K) * p.Mp * 2);
  // W as a K-major operand of dX: both at one leading dimension
  const bool copy = needs_copy(Wg.p, Wg.ld, N, K) || needs_copy(Wu.p, Wu.ld, N, K) ||
                    Wg.ld != Wu.ld;
  if (dx && copy) p.bytes_g = p.bytes_u = copy_bytes(N, K);
  if (dx) {
    p.gx = plan_grad_x(pad_rows(M), pad_k(K), 2 * ((p.Nk + 63) / 64), false);
    if (p.gx.splits > 1)
      p.bytes_sum = round256((size_t)p.gx.splits * pad_rows(M) * pad_k(K) * sizeof(float));
    if (type == GEMM_TYPE_F16)
      p.bytes_factor = p.bytes_sum ? p.bytes_sum / p.gx.splits : kFactorBytes;
  }
  return p;
}

// The kernel for few rows (gated_rows.hip) streams the weights once for 64 rows
// of X: at most as many rows, or tiles would be too few for the chip, each with
// all of K to walk, in 0.65 us a slab of 64.  With ceil(M / 64) passes over 4 N K
// bytes at 4.2 TB/s both take the same near ceil(M / 64) N = 10000 (tiles and
// rows, bf16: 128 x 4096 x 4096 45.9 and 31.6 us, 80 x 2048 x 8192 88 and 28,
// 500 x 1024 x 1024 15.7 and 13.1; 128 x 8192 x 2048 26.9 and 35.2, 111 x 7756 x
// 2608 47 and 52).  Rows at odd addresses are read at a third of the rate (102 x
// 3667 x 1591: 36.6 and 40.4; 100 x 1000 x 2047: 33.8 and 29.9).
bool by_rows(int M, int N, Mat x, Mat g, Mat u) {
  const int64_t work = ((int64_t)M + 63) / 64 * N;
  auto even = [](Mat m) { return m.ld % 2 == 0 && (reinterpret_cast<uintptr_t>(m.p) & 3) == 0; };
  return M <= 64 || work <= (even(x) && even(g) && even(u) ? 10000 : 4000);
}

}  // namespace
}  // namespace fused
}  // namespace mi355gemm

using namespace mi355gemm;
using namespace mi355gemm::fused;

extern "C" {

MI355FUSED_API unsigned long long gemm_gated_workspace(int type, int M, int N, int K,
                                                       const void* X, int ldx, const void* Wg,
                                                       int ldwg, const void* Wu, int ldwu) {
  if (check(type, 0, M, N, K) != GEMM_OK || N == 0 || bad_ld(ldx, K) || bad_ld(ldwg, K) ||
      bad_ld(ldwu, K) || by_rows(M, N, Mat{in16(X), ldx}, Mat{in16(Wg), ldwg}, Mat{in16(Wu), ldwu}))
    return 0;
  return (needs_copy(X, ldx, M, K) ? copy_bytes(M, K) : 0) +
         (needs_copy(Wg, ldwg, N, K) ? copy_bytes(N, K) : 0) +
         (needs_copy(Wu, ldwu, N, K) ? copy_bytes(N, K) : 0);
}

MI355FUSED_API int gemm_gated(int type, int act, int M, int N, int K, const void* X, int ldx,
                              const void* Wg, int ldwg, const void* Wu, int ldwu, void* H, int ldh,
                              void* G, int ldg, void* U, int ldu, void* workspace,
                              unsigned long long workspace_bytes, void* stream) {
  const int status = check(type, act, M, N, K);
  if (status != GEMM_OK) return status;
  if (M == 0 || N == 0) return GEMM_OK;
  if (bad_ld(ldx, K) || bad_ld(ldwg, K) || bad_ld(ldwu, K) || bad_ld(ldh, N) ||
      (G && bad_ld(ldg, N)) || (U && bad_ld(ldu, N)))
    return GEMM_ERR_BAD_LD;
  if (H == nullptr || (K > 0 && (X == nullptr || Wg == nullptr || Wu == nullptr)))
    return GEMM_ERR_NULL_POINTER;
  const size_t need = gemm_gated_workspace(type, M, N, K, X, ldx, Wg, ldwg, Wu, ldwu);
  if (!workspace_ok(need, workspace, workspace_bytes)) return GEMM_ERR_WORKSPACE;
  const int cus = check_device();
  if (cus < 0) return cus;
  hipStream_t s = static_cast<hipStream_t>(stream);
  Args16 a{in16(X), in16(Wg), out16(H), ldx, ldwg, ldh, M, N, K};
  a.act = act;
  a.fmt = type == GEMM_TYPE_BF16 ? kFmtBF16 : kFmtF16;
  FusedExtra f;
  f.m_end = M;
  f.n_end = N;
  f.B2 = in16(Wu);
  f.ldb2 = ldwu;
  f.C2 = out16(G);
  f.ldc2 = ldg;
  f.C3 = out16(U);
  f.ldc3 = ldu;
  if (by_rows(M, N, Mat{a.A, ldx}, Mat{a.B, ldwg}, Mat{f.B2, ldwu}))
    return to_status(launch_gated_rows(a, f, cus, s));
  PadJobs jobs;
  char* ws = static_cast<char*>(workspace);
  const Mat x = jobs.add(Mat{a.A, ldx}, M, K, ws);
  const Mat g = jobs.add(Mat{a.B, ldwg}, N, K, ws);
  const Mat u = jobs.add(Mat{f.B2, ldwu}, N, K, ws);
  const hipError_t e = launch_pad(jobs, s);
  if (e != hipSuccess) return to_status(e);
  a.A = x.p;
  a.lda = x.ld;
  a.B = g.p;
  a.ldb = g.ld;
  f.B2 = u.p;
  f.ldb2 = u.ld;
  a.M = pad_rows(M);
  a.N = pad_rows(N);
  a.K = pad_k(K);
  return to_status(launch_gated_tiles(a, f, cus, s));
}

MI355FUSED_API unsigned long long gemm_gated_bwd_workspace(int type, int M, int N, int K,
                                                           const void* X, int ldx, const void* Wg,
                                                           int ldwg, const void* Wu, int ldwu,
                                                           int want_dx, int want_dw) {
  if (check(type, 0, M, N, K) != GEMM_OK || K == 0) return 0;
  const bool dx = want_dx && M > 0, dw = want_dw && N > 0;
  if (!dx && !dw) return 0;
  if ((dw && bad_ld(ldx, K)) || (dx && (bad_ld(ldwg, K) || bad_ld(ldwu, K)))) return 0;
  return plan_bwd(type, M, N, K, Mat{in16(Wg), ldwg}, Mat{in16(Wu), ldwu}, dx, dw).total();
}

MI355FUSED_API int gemm_gated_bwd(int type, int act, int M, int N, int K, const void* X, int ldx,
                                  const void* Wg, int ldwg, const void* Wu, int ldwu,
                                  const void* G, int ldg, const void* U, int ldu, const void* dH,
                                  int lddh, void* dX, int lddx, void* dWg, int lddwg, void* dWu,
                                  int lddwu, void* workspace, unsigned long long workspace_bytes,
                                  void* stream) {
  const int status = check(type, act, M, N, K);
  if (status != GEMM_OK) return status;
  const bool dx = dX != nullptr && M > 0 && K > 0;
  const bool dw = (dWg != nullptr || dWu != nullptr) && N > 0 && K > 0;
  if (!dx && !dw) return GEMM_OK;
  if ((dw && bad_ld(ldx, K)) || (dx && (bad_ld(ldwg, K) || bad_ld(ldwu, K) || bad_ld(lddx, K))) ||
      bad_ld(ldg, N) || bad_ld(ldu, N) || bad_ld(lddh, N) || (dw && dWg && bad_ld(lddwg, K)) ||
      (dw && dWu && bad_ld(lddwu, K)))
    return GEMM_ERR_BAD_LD;
  if (M > 0 && N > 0 &&
      (G == nullptr || U == nullptr || dH == nullptr || (dw && X == nullptr) ||
       (dx && (Wg == nullptr || Wu == nullptr))))
    return GEMM_ERR_NULL_POINTER;
  const BwdPlan p = plan_bwd(type, M, N, K, Mat{in16(Wg), ldwg}, Mat{in16(Wu), ldwu}, dx, dw);
  if (!workspace_ok(p.total(), workspace, workspace_bytes)) return GEMM_ERR_WORKSPACE;
  const int cus = check_device();
  if (cus < 0) return cus;
  hipStream_t s = static_cast<hipStream_t>(stream);
  const int fmt = type == GEMM_TYPE_BF16 ? kFmtBF16 : kFmtF16;
  char* ws = static_cast<char*>(workspace);
  half_t* d = reinterpret_cast<half_t*>(ws);
  half_t* tail = p.tail ? reinterpret_cast<half_t*>(ws + p.bytes_d) : nullptr;
  // (no rows or columns: dG and dU are zeros and need no factor)
  float* factor = nullptr;
  if (fmt == kFmtF16 && M > 0 && N > 0)
    factor = reinterpret_cast<float*>(p.lone ? ws + p.bytes_d / 2
                                             : ws + p.total() - p.bytes_factor);
  const float* scale = factor ? factor + kMaxBlocks : nullptr;
  ws += p.bytes_d + p.bytes_tail;

  half_t* xt = reinterpret_cast<half_t*>(ws);
  ws += p.bytes_x;
  const int64_t pieces = (int64_t)p.Mp * (p.Np / 8 + (p.tail ? 8 : 0));
  GradArgs ga{in16(G), in16(U), in16(dH), nullptr, nullptr, tail, factor, ldg, ldu, lddh,
              p.ld,    M,       N,        p.Mp,    p.Np,    p.Nk, act,
              (pieces + kThreads - 1) / kThreads,
              Transpose{in16(X), xt, ldx, p.Mp, M, K, p.Mp, pad_k(K)}};
  hipError_t e = hipSuccess;
  if (factor)
    e = launch_tiles((const void*)gated_max_kernel, ga, kMaxBlocks, kMaxThreads, 0, s);
  if (e != hipSuccess) return to_status(e);
  // dG and dU to dg and du (a part that is null is left out); X^T once
  auto make = [&](half_t* dg, half_t* du, bool with_x) {
    ga.dg = dg;
    ga.du = du;
    const int64_t blocks_x = with_x ? (ga.x.tiles() + kThreads / 64 - 1) / (kThreads / 64) : 0;
    return launch_tiles(fmt == kFmtBF16 ? (const void*)gated_grad_kernel<kFmtBF16>
                                        : (const void*)gated_grad_kernel<kFmtF16>,
                        ga, ga.blocks + blocks_x, kThreads, 0, s);
  };
  if (!p.lone) e = make(d, d + p.Np, dw);
  if (e != hipSuccess) return to_status(e);
  PadJobs jobs;
  Mat wg{in16(Wg), ldwg}, wu{in16(Wu), ldwu};
  if (p.bytes_g) {
    wg = jobs.copy(wg, N, K, ws);
    wu = jobs.copy(wu, N, K, ws);
  }
  e = launch_pad(jobs, s);
  if (e != hipSuccess) return to_status(e);
  if (dx) {
    Args16 a{d, wg.p, out16(dX), p.ld, wg.ld, lddx, pad_rows(M), pad_k(K), p.Nk};
    a.fmt = fmt;
    FusedExtra f;
    f.m_end = M;
    f.n_end = K;
    f.parts = 2;
    f.partA = p.Np;
    f.B2 = wu.p;
    f.tail = tail;
    f.ldt = 128;
    f.scale = scale;
    if (p.bytes_sum) {
      f.sum = reinterpret_cast<float*>(ws);
      f.ld_sum = a.N;
      f.split_stride = (int64_t)a.M * a.N;
    }
    e = launch_grad_x(a, f, p.gx, cus, s);
    if (e == hipSuccess && f.sum)
      e = launch_sums(fmt, f, p.gx.splits, out16(dX), lddx, M, K, s);
    if (e != hipSuccess) return to_status(e);
  }
  // dW of the part at `from`, or of both as two parts of one product's rows
  auto products = [&](half_t* from, void* to, int ld, bool both) {
    Args16 a{from, xt, out16(to), p.ld, p.Mp, ld, (int)round_up(p.Nk, 8), pad_k(K), p.Mp};
    a.fmt = fmt;
    FusedExtra f;
    f.m_end = N;
    f.n_end = K;
    f.parts = both ? 2 : 1;
    f.partA = p.Np;
    f.C2 = out16(dWu);
    f.ldc2 = lddwu;
    f.scale = scale;
    return launch_grad_w(a, f, cus, s);
  };
  if (dw && p.lone) {
    if (dWg != nullptr) {
      e = make(d, nullptr, true);
      if (e == hipSuccess) e = products(d, dWg, lddwg, false);
      if (e != hipSuccess) return to_status(e);
    }
    if (dWu != nullptr) {
      e = make(nullptr, d, dWg == nullptr);
      if (e == hipSuccess) e = products(d, dWu, lddwu, false);
    }
  } else if (dw) {
    e = dWg != nullptr ? products(d, dWg, lddwg, dWu != nullptr)
                       : products(d + p.Np, dWu, lddwu, false);
  }
  return to_status(e);
}

}  // extern "C"
